"""kv_append with norms of the query and key heads, against the formula in 64 bits.

Tolerances. The normed row in fp32: the mean of D squares along a tree of at most 16 + 5 additions (each off by at most 2^-24
of the sum, as are the squares and the division by D), the sum with eps, the inverse root (two units, 2^-22) and two
products (2^-24 each): less than 24 * 2^-24 / 2 + 2^-22 + 2^-23 < 2^-19 relative. The rotation adds two products and a
difference: 3 * 2^-24 of |a c| + |b s|. So y is off by at most r = 2^-18 (|a| + |b|) with a, b the pair's normed values,
and then rounds once: by 2^-8 |y| to bf16; by 2^-4 |y / s|, or half a step 2^-10 below 2^-6, to E4M3 at scale s.
"""
import ctypes
import math

import pytest
import torch

E4M3 = torch.float8_e4m3fn
EPS = 1e-5


def rope_table(n, max_pos):
    f = 10000.0 ** (-torch.arange(0, n, 2, dtype=torch.float64) / n)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def formula(x, w, pos, table, off, inter):
    """x [T, H, D] -> the normed and rotated rows, and r, in doubles."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + EPS) * w.double()
    mag = 2.0 ** -18 * y.abs() if w is not None else 2.0 ** -22 * y.abs()
    if table is None:
        return y, mag
    n = table.shape[1]
    t = table[pos].double()[:, None]
    c, s = t[..., :n // 2], t[..., n // 2:]
    i, j = (slice(off, off + n, 2), slice(off + 1, off + n, 2)) if inter else (slice(off, off + n // 2), slice(off + n // 2, off + n))
    a, b = y[..., i], y[..., j]
    z, r = y.clone(), mag.clone()
    z[..., i], z[..., j] = a * c - b * s, b * c + a * s
    r[..., i] = r[..., j] = 2.0 ** -18 * (a.abs() + b.abs())
    return z, r


def close(got, want, r, u=2.0 ** -8, least=0.0):
    err = (got.double() - want).abs()
    tol = torch.clamp(u * want.abs(), min=least) + r * (1 + u)
    assert torch.all(err <= tol), float((err - tol).max())


def make(kind, T, Hq, Hkv, D, rot, off, inter, w32, seed, sides="qk", strided=False, skipped=()):
    g = torch.Generator().manual_seed(seed)
    size = torch.exp(torch.randn((1, Hq + 2 * Hkv, 1), generator=g))
    x = (torch.randn((T, Hq + 2 * Hkv, D), generator=g) * size).to(torch.bfloat16).cuda()
    if strided:
        x = torch.cat([x, x[:, :1]], 1)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:Hq + 2 * Hkv]
    if not strided:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    nb = (T + 15) // 16 + 2
    # one sequence from slot 5 of a block on, in shuffled blocks
    perm = torch.randperm(nb, generator=g)
    at = torch.arange(T) + 5
    slot = perm[at // 16] * 16 + at % 16
    for t in skipped:
        slot[t] = -1
    wt = torch.float32 if w32 else torch.bfloat16
    w = {s: (1 + 0.3 * torch.randn(D, generator=g)).to(wt).cuda() if s in sides else None for s in "qk"}
    pos = torch.randint(0, 5000, (T,), generator=g)
    st = dict(kind=kind, q=q, k=k, v=v, qw=w["q"], kw=w["k"], slot=slot.cuda(), pos=pos.cuda(),
              table=None if rot == 0 else rope_table(rot, 5000).cuda(), off=off, inter=inter, nb=nb)
    if kind == "bf16":
        st.update(kc=torch.randn((nb, 16, Hkv, D), generator=g).to(torch.bfloat16).cuda(),
                  vc=torch.randn((nb, 16, Hkv, D), generator=g).to(torch.bfloat16).cuda())
    else:
        st.update(kc=torch.randint(0, 120, (nb, 16, Hkv, D), generator=g, dtype=torch.uint8).cuda(),
                  vc=torch.randint(0, 120, (nb, 16, Hkv, D), generator=g, dtype=torch.uint8).cuda())
        st.update(ks=0.03, vs=0.02) if kind == "tensor" else st.update(
            ks=torch.full((nb, Hkv), 2.0 ** -9).cuda(), vs=torch.full((nb, Hkv), 2.0 ** -9).cuda())
    return st


def append(st, norms=True, **more):
    import paged_kv_attention_reshape_gb300 as pkv
    kw = dict(k_scale=st["ks"], v_scale=st["vs"]) if "ks" in st else {}
    if norms:
        kw.update(q_norm=st["qw"], k_norm=st["kw"], norm_eps=EPS)
    r = pkv.kv_append(st["q"], st["k"], st["v"], st["pos"], st["slot"], st["kc"], st["vc"], st["table"], rope_offset=st["off"],
                      interleaved=st["inter"], **kw, **more)
    assert pkv.device_errors() == 0
    return r


def verify(st):
    kind, slot = st["kind"], st["slot"]
    T, Hq, D = st["q"].shape
    Hkv = st["k"].shape[1]
    q_out, k_out = (torch.full((T, h, D), 7.0, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv))
    before = {n: st[n].clone() for n in ("kc", "vc", "ks", "vs") if isinstance(st.get(n), torch.Tensor)}
    append(st, q_out=q_out, k_out=k_out)
    live = slot >= 0
    q, rq = formula(st["q"], st["qw"], st["pos"], st["table"], st["off"], st["inter"])
    k, rk = formula(st["k"], st["kw"], st["pos"], st["table"], st["off"], st["inter"])
    close(q_out[live], q[live], rq[live])
    close(k_out[live], k[live], rk[live])
    assert torch.all(q_out[~live] == 7.0) and torch.all(k_out[~live] == 7.0)
    s = slot[live]
    rows = st["kc"].view(-1, Hkv, D)[s]
    untouched = torch.ones(st["nb"] * 16, dtype=torch.bool, device="cuda")
    untouched[s] = False
    if kind == "bf16":
        close(rows, k[live], rk[live])
        assert torch.equal(rows, k_out[live]) and torch.equal(st["vc"].view(-1, Hkv, D)[s], st["v"][live])
    elif kind == "tensor":
        x = (k[live] / float(torch.tensor(st["ks"], dtype=torch.float32))).clamp(-448, 448)
        close(rows.view(E4M3).float(), x, rk[live] / 0.03 + 2.0 ** -22 * x.abs(), 2.0 ** -4, 2.0 ** -10)
    else:
        blk = s // 16
        # each block's scale: the larger of what it was (rows were there before) and what its new rows need
        amax = torch.zeros((st["nb"], Hkv), dtype=torch.float64, device="cuda").index_reduce_(0, blk, k[live].abs().amax(-1), "amax")
        first = torch.full((st["nb"],), 16, device="cuda").index_reduce_(0, blk, s % 16, "amin")
        wrote = first < 16
        need = torch.exp2(torch.ceil(torch.log2(amax / 448.0)))
        clear = (amax / (448.0 * need) < 1 - 2.0 ** -17) & (amax / (224.0 * need) > 1 + 2.0 ** -17)
        want = torch.where((first > 0)[:, None], torch.maximum(need, before["ks"].double()), need)
        ok = clear & wrote[:, None]
        assert torch.equal(st["ks"].double()[ok], want[ok]) and torch.equal(st["ks"][~wrote], before["ks"][~wrote])
        sc = st["ks"].double()[blk][:, :, None]
        x = (k[live] / sc).clamp(-448, 448)
        close(rows.view(E4M3).float(), x, rk[live] / sc, 2.0 ** -4, 2.0 ** -10)
    if kind != "block":
        for n in ("kc", "vc"):
            assert torch.equal(st[n].view(-1, Hkv, D)[untouched], before[n].view(-1, Hkv, D)[untouched])


# ---- refusals (no GPU) -------------------------------------------------------------------------------

def test_refusals():
    from paged_kv_attention_reshape_gb300 import _lib
    lib = _lib.load()
    fake = ctypes.c_void_p(1 << 20)
    other = ctypes.c_void_p(1 << 21)
    odd = ctypes.c_void_p((1 << 20) + 4)

    def run(norm, D=128, cache=None, latent=False):
        c = cache or _lib.PkvCache(fake, None if latent else other, 10, 16, 1, D, 16 * D)
        return lib.pkv_kv_append_norm(fake, 4 * D, fake, D, None if latent else fake, 0 if latent else D, fake, fake, 3, 4,
                                      _lib.PkvRope(None, 0, 0, 0, 0), norm, c, fake, fake, None)

    N = _lib.PkvHeadNorm
    assert run(N(None, None, 1e-6, 0)) == 1
    for eps in (0.0, -1.0, math.inf, math.nan):
        assert run(N(fake, fake, eps, 0)) == 1
    assert run(N(odd, fake, 1e-6, 0)) == 1 and run(N(fake, odd, 1e-6, 0)) == 1
    for D in (48, 96, 576, 1024):
        assert run(N(fake, fake, 1e-6, 0), D) == 2
    assert run(N(fake, fake, 1e-6, 0), 128, latent=True) == 2


# ---- the operator ----------------------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 3, 17, 300])
@pytest.mark.parametrize("kind,Hq,Hkv,D,rot,off,inter,w32", [
    ("bf16", 8, 2, 64, 64, 0, False, False), ("bf16", 5, 5, 128, 64, 32, True, True), ("bf16", 3, 1, 16, 16, 0, False, False),
    ("bf16", 4, 2, 512, 128, 256, False, True), ("bf16", 6, 3, 32, 0, 0, False, False), ("tensor", 16, 1, 128, 128, 0, True, False),
    ("tensor", 4, 4, 256, 32, 16, False, True), ("block", 8, 2, 128, 128, 0, False, False), ("block", 3, 3, 128, 32, 0, True, True)])
def test_norms(kind, Hq, Hkv, D, rot, off, inter, w32, T):
    verify(make(kind, T, Hq, Hkv, D, rot, off, inter, w32, 7 * T + D))


@pytest.mark.gpu
@pytest.mark.parametrize("kind,T", [("bf16", 700), ("tensor", 601), ("block", 2100), ("block", 3001), ("bf16", 1025)])
@pytest.mark.parametrize("Hq,Hkv,w32", [(8, 2, False), (24, 1, True)])
def test_long_batches(kind, T, Hq, Hkv, w32):
    """Rows through shared memory; skipped rows among them; slices of a fused projection."""
    verify(make(kind, T, Hq, Hkv, 128, 128, 0, False, w32, T + Hq, strided=True, skipped=(0, 5, 6, T - 1)))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,T", [(16, 1499), (16, 1500), (17, 1500), (17, 2299), (17, 2300)])
def test_both_sides_of_where_rows_beside_block_scales_change(Hq, T):
    verify(make("block", T, Hq, 1, 128, 128, 0, False, False, T + Hq, skipped=(0, 7, T - 1)))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "tensor", "block"])
@pytest.mark.parametrize("sides", ["q", "k"])
@pytest.mark.parametrize("T", [20, 800])
def test_one_side(kind, sides, T):
    verify(make(kind, T, 4, 2, 128, 64, 0, False, False, 40 + T, sides=sides))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [9, 900])
def test_in_place_without_queries_and_zero_rows(T):
    import paged_kv_attention_reshape_gb300 as pkv
    st = make("bf16", T, 4, 2, 128, 128, 0, False, False, 3)
    st["q"][T // 2] = 0  # a head of zeros stays one
    twin = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in st.items()}
    q, k = append(st)
    assert torch.all(q[T // 2] == 0) and torch.isfinite(q.float()).all()
    append(twin, q_out=twin["q"], k_out=twin["k"])
    assert torch.equal(q, twin["q"]) and torch.equal(k, twin["k"]) and torch.equal(st["kc"], twin["kc"])
    kc, vc = torch.zeros_like(st["kc"]), torch.zeros_like(st["vc"])
    none, k2 = pkv.kv_append(None, st["k"], st["v"], st["pos"], st["slot"], kc, vc, st["table"], k_norm=st["kw"], norm_eps=EPS)
    assert none is None and torch.equal(k2, k) and torch.equal(kc.view(-1, 2, 128)[st["slot"]], k)


@pytest.mark.gpu
def test_ends_of_the_range():
    """Rows of 2^59, and rows whose squares are far below eps, keep their precision; one NaN spoils its own head only."""
    st = make("bf16", 6, 2, 1, 128, 0, 0, False, False, 4)
    st["q"][0] *= 2.0 ** 55
    st["q"][1] *= 2.0 ** -40
    st["q"][2, 1, 3] = math.nan
    q, _ = append(st)
    want, r = formula(st["q"], st["qw"], st["pos"], None, 0, False)
    fine = torch.ones((6, 2), dtype=torch.bool, device="cuda")
    fine[2, 1] = False
    close(q[fine], want[fine], r[fine])
    assert torch.isnan(q[2, 1].float()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind,T", [("bf16", 3), ("block", 40), ("tensor", 700)])
def test_captured_and_on_another_stream(kind, T):
    import paged_kv_attention_reshape_gb300 as pkv
    a, b = (make(kind, T, 8, 2, 128, 128, 0, False, False, s) for s in (5, 6))
    names = ("q", "k", "v", "slot", "pos", "kc", "vc") + (("ks", "vs") if kind == "block" else ())
    copies = [{k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in x.items()} for x in (a, b)]
    want = [append(x) for x in copies]
    side = torch.cuda.Stream()
    other = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in a.items()}
    torch.cuda.synchronize()
    got = append(other, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want[0])) and torch.equal(other["kc"], copies[0]["kc"])
    g = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in a.items()}
    q_out, k_out = torch.zeros_like(want[0][0]), torch.zeros_like(want[0][1])
    kw = dict(k_scale=g["ks"], v_scale=g["vs"]) if "ks" in g else {}
    graph = torch.cuda.CUDAGraph()
    run = lambda: pkv.kv_append(g["q"], g["k"], g["v"], g["pos"], g["slot"], g["kc"], g["vc"], g["table"], q_norm=g["qw"],
                                k_norm=g["kw"], norm_eps=EPS, q_out=q_out, k_out=k_out, **kw)
    run()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run()
    for x, w, c in ((a, want[0], copies[0]), (b, want[1], copies[1])):
        for n in names:
            g[n].copy_(x[n])
        for n in ("qw", "kw"):
            g[n].copy_(x[n])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q_out, w[0]) and torch.equal(k_out, w[1])
        assert all(torch.equal(g[n], c[n]) for n in names)


@pytest.mark.gpu
def test_refused_by_the_binding():
    import paged_kv_attention_reshape_gb300 as pkv
    st = make("bf16", 4, 4, 2, 128, 0, 0, False, False, 4)
    args = (st["q"], st["k"], st["v"], st["pos"], st["slot"], st["kc"], st["vc"])
    w = st["qw"]
    for kw in (dict(q_norm=w.half(), k_norm=w), dict(q_norm=w.float(), k_norm=w), dict(q_norm=w[:64]), dict(k_norm=w.cpu()),
               dict(q_norm=w, norm_eps=0.0), dict(q_norm=torch.stack([w, w], 1)[:, 0])):
        with pytest.raises(pkv.PkvError):
            pkv.kv_append(*args, **kw)
    lat = torch.zeros((4, 16, 1, 576), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pkv.PkvError):
        pkv.kv_append(None, torch.zeros((4, 1, 576), dtype=torch.bfloat16, device="cuda"), None, st["pos"], st["slot"], lat, None,
                      k_norm=torch.ones(576, dtype=torch.bfloat16, device="cuda"))
