"""The block-scaled E4M3 cache: kv_append (rotation and append), paged_decode_attn and extend_attn
over it, and a run of them together, against plain implementations.

kv_append is compared bit for bit with the same fp32 steps in plain torch operations on the CPU (each
product and sum rounded by itself, one rounding to the stored type) and, for the rotation, with
64 bits. The attentions are compared with dense softmax in 64 bits over the cache's values.

Tolerances of the attentions (u = 2^-8, half a step of bf16 relative to the value):
  * out: u |o| for its own rounding; P is rounded to 8 bits or better before the product with V (u A,
    A = sum_j p_j |v_j|); the exponent's error e (below) moves p and the sum by e each. So
    u |o| + u A + 2 e A.
    A P that is far below the largest, P_top, is rounded to a fixed step instead: fp16 in the extend kernel
    (steps of 2^-24, P_top >= 2^7: half a step is 2^-32 P_top), E4M3 hi + lo / 16 in the decode (at most
    2^-22 P_top). With the codes c of V, P_j = 2^(u_j - m), out = sum_j P_j c_j / l and l >= P_top / vs_top,
    that adds at most f vs_top sum_j |c_j| (f = 2^-32 or 2^-22; vs_top: the value scale of the row's largest u).
  * lse: e = the error of a score: 128 fp32 additions of products that are exact, each off by at
    most 2^-23 of the sum of magnitudes M = scale sum_d |q_d k_d| (a truncating adder): 2^-16 M,
    and 2^-20 (1 + |lse|) for the rounding of s * scale * log2(e) - m, of 2^x and of the logarithm
    (each within 2^-22 of a number of that size).
"""
import ctypes
import math

import numpy as np
import pytest
import torch

E4M3 = torch.float8_e4m3fn
U = 2.0 ** -8


# ---- plain forms ---------------------------------------------------------------------------------

def values(codes):
    """E4M3 codes (uint8) as doubles."""
    return codes.view(E4M3).float().double()


def to_codes(x):
    """fp32 -> E4M3 codes, nearest even, saturated; a NaN stays one."""
    return x.clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)


def rope_table(n, max_pos):
    f = 10000.0 ** (-torch.arange(0, n, 2, dtype=torch.float64) / n)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def rotate(x, pos, table, off, inter):
    """x [T, H, d] (fp32 or fp64) rotated at pos [T], each operation by itself."""
    if table is None:
        return x.clone()
    n = table.shape[1]
    t = table[pos].to(x.dtype)[:, None]
    c, s = t[..., :n // 2], t[..., n // 2:]
    y = x.clone()
    if inter:
        i, j = slice(off, off + n, 2), slice(off + 1, off + n, 2)
    else:
        i, j = slice(off, off + n // 2), slice(off + n // 2, off + n)
    a, b = x[..., i], x[..., j]
    y[..., i] = a * c - b * s
    y[..., j] = b * c + a * s
    return y


def scale_for(amax):
    """The smallest power of two s with amax <= 448 s, within [2^-64, 2^120]."""
    if not amax > 0:
        return 2.0 ** -64
    e = math.floor(math.log2(amax)) - 9
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** min(max(e, -64), 120)


def plain_append(st):
    """What kv_append leaves, on CPU copies of st's tensors: (q_out, k_out, kc, vc, ks, vs)."""
    kind, table = st["kind"], st["table"]
    q, k, v = st["q"], st["k"], st["v"]
    kc = st["kc"].clone()
    vc = kc if st["vc"] is None else st["vc"].clone()
    ks, vs = (st["ks"].clone(), st["vs"].clone()) if kind == "block" else (st.get("ks"), st.get("vs"))
    q_out = None if q is None else st["q_out"].clone()
    k_out = st["k_out"].clone()
    nb, bs, H, d = kc.shape
    slot, pos = st["slot"], st["pos"]
    ok = (slot >= 0) & (slot < nb * bs)
    if table is not None:
        ok &= (pos >= 0) & (pos < table.shape[0])
    p = torch.where(ok, pos, 0)
    if q is not None:
        q_out[ok] = rotate(q.float(), p, table, st["off"], st["inter"]).to(torch.bfloat16)[ok]
    kr = rotate(k.float(), p, table, st["off"], st["inter"])
    k_out[ok] = kr.to(torch.bfloat16)[ok]
    rows = [(kr, kc, ks)] + ([] if v is None else [(v.float(), vc, vs)])
    for x, cache, sc in rows:
        flat = cache.view(nb * bs, H, d)
        if kind in ("bf16", "latent"):
            flat[slot[ok]] = x.to(torch.bfloat16)[ok]
        elif kind == "tensor":
            flat[slot[ok]] = to_codes(x * float(np.float32(1.0) / np.float32(sc)))[ok]
        else:
            runs = {}  # by block: its tokens, those that are skipped for their position included
            for t, n in enumerate(slot.tolist()):
                if 0 <= n < nb * bs:
                    runs.setdefault(n // bs, []).append(t)
            for b, run in runs.items():
                a = int(slot[run[0]]) % bs
                run = [t for t in run if bool(ok[t])]
                if not run:
                    continue
                for h in range(H):
                    mag = x[run, h].abs()
                    mag = torch.where(torch.isfinite(mag), mag, torch.zeros(()))
                    need = torch.tensor(scale_for(float(mag.max())), dtype=torch.float32)
                    s0 = sc[b, h].clone()
                    s1 = need if a == 0 else torch.maximum(s0, need)
                    if a > 0 and s1 != s0:
                        cache[b, :a, h] = to_codes(values(cache[b, :a, h]).float() * (s0 / s1))
                    sc[b, h] = s1
                    cache[b, slot[run] % bs, h] = to_codes(x[run, h] * (torch.tensor(1.0) / s1))
    return q_out, k_out, kc, vc, ks, vs


def dense(q, k, v, scale, causal_from=None):
    """q [n, G, d], k, v [c, d] doubles -> out, lse, A = sum p |v|, M = max scale sum |q k|.
    causal_from: token i of q sees keys 0 .. causal_from + i."""
    s = torch.einsum("tgd,jd->tgj", q, k) * scale
    mag = torch.einsum("tgd,jd->tgj", q.abs(), k.abs()) * scale
    if causal_from is not None:
        i = torch.arange(q.shape[0])[:, None, None]
        hide = torch.arange(k.shape[0])[None, None] > causal_from + i
        s = s.masked_fill(hide, -math.inf)
        mag = mag.masked_fill(hide, 0.0)
    z = torch.logsumexp(s, -1)
    p = torch.exp(s - z[..., None])
    return (torch.einsum("tgj,jd->tgd", p, v), z, torch.einsum("tgj,jd->tgd", p, v.abs()), mag.amax(-1))


def fixed_steps(st, r, h, c, q, k, scale, causal_from, f):
    """f vs_top sum_j |c_j| of the rows q [n, G, d] over the context's c keys and the new ones (vs = 1) behind them."""
    blocks = st["table"][r].long()[torch.arange(c) // 16]
    vs = torch.cat([st["vs"][blocks, h].double(), torch.ones(len(k) - c, dtype=torch.float64)])
    u = torch.einsum("tgd,jd->tgj", q, k) * scale + vs.log()
    if causal_from is not None:
        u = u.masked_fill(torch.arange(len(k))[None, None] > causal_from + torch.arange(len(q))[:, None, None], -math.inf)
    codes = (context(st, r, h, c)[1] / vs[:c, None]).abs().sum(0)
    return f * vs[u.argmax(-1)][..., None] * codes


def check(out, lse, ref, what="", more=0.0):
    """out, lse of some rows against dense()'s."""
    o, z, A, M = ref
    e = 2.0 ** -16 * M + 2.0 ** -20 * (1 + z.abs())
    d = (lse.double() - z).abs()
    assert bool((d <= e).all()), f"{what}: lse off by {float((d / e).max()):.2f} of its bound"
    tol = U * o.abs() + (U + 2 * e[..., None]) * A + more + 1e-37
    d = (out.double() - o).abs()
    assert bool(torch.isfinite(out.float()).all()) and bool((d <= tol).all()), \
        f"{what}: out off by {float((d / tol).max()):.2f} of its bound"


# ---- inputs --------------------------------------------------------------------------------------

def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def block_cache(nb, H, g, spread=0.5, pow2=False, gap=0):
    """Codes and scales of normal values whose size varies by block and head; `gap` extra blocks' worth of
    elements between blocks (a cache that shares its allocation)."""
    x = torch.randn((nb, 16, H, 128), generator=g) * torch.exp(spread * torch.randn((nb, 1, H, 1), generator=g))
    s = x.abs().amax((1, 3)) / 448.0
    if pow2:
        s = torch.exp2(torch.ceil(torch.log2(s)))
    c = to_codes(x / s[:, None, :, None])
    if gap:
        whole = torch.full((nb, 1 + gap, 16, H, 128), 0x7F, dtype=torch.uint8)  # NaN codes between the blocks
        whole[:, 0] = c
        c = whole
    return c, s


def tables(need, g, extra=3):
    nb = sum(need) + extra
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    t = torch.zeros((len(need), max([1] + need)), dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        t[r, :n] = perm[at:at + n]
        at += n
    return t, nb


def on(t, dev="cuda"):
    return None if t is None else t.to(dev)


def append_state(kind, ctx, new, Hq, Hkv, d, rot, off=0, inter=False, pad=0, seed=0, max_pos=600, size=1.0, bs=16):
    """A batch of appends: request r has ctx[r] tokens and gets new[r] more."""
    g = gen(seed)
    table, nb = tables([(c + n + bs - 1) // bs for c, n in zip(ctx, new)], g)
    pos = torch.cat([torch.arange(c, c + n) for c, n in zip(ctx, new)])
    req = torch.arange(len(ctx)).repeat_interleave(torch.tensor(new))
    slot = table[req, pos // bs].long() * bs + pos % bs
    slot, pos = torch.cat([slot, torch.full((pad,), -1)]), torch.cat([pos, torch.full((pad,), 1 << 40)])
    T = len(slot)
    # heads and tokens of very different sizes, so that scales grow often
    amp = size * torch.exp(torch.randn((T, Hkv, 1), generator=g))
    st = dict(kind=kind, off=off, inter=inter, pos=pos, slot=slot, table=rope_table(rot, max_pos) if rot else None,
              blocks=table, nb=nb,
              q=torch.randn((T, Hq, d), generator=g).to(torch.bfloat16) if Hq else None,
              k=(torch.randn((T, Hkv, d), generator=g) * amp).to(torch.bfloat16),
              v=None if kind == "latent" else (torch.randn((T, Hkv, d), generator=g) * amp).to(torch.bfloat16),
              q_out=torch.full((T, Hq, d), 7.0, dtype=torch.bfloat16), k_out=torch.full((T, Hkv, d), 7.0, dtype=torch.bfloat16))
    if kind == "block":
        (st["kc"], st["ks"]), (st["vc"], st["vs"]) = (block_cache(nb, Hkv, g, pow2=True) for _ in "kv")
    elif kind == "tensor":
        st["kc"], st["vc"] = (torch.randint(0, 256, (nb, bs, Hkv, d), generator=g, dtype=torch.uint8) for _ in "kv")
        st["ks"], st["vs"] = 5.0 / 448.0, 0.011
    else:
        st["kc"] = torch.randn((nb, bs, Hkv, d), generator=g).to(torch.bfloat16)
        st["vc"] = None if kind == "latent" else torch.randn((nb, bs, Hkv, d), generator=g).to(torch.bfloat16)
    return st


def gpu_append(st, **more):
    """kv_append on GPU copies; returns what plain_append returns, on the CPU, and the error word."""
    import paged_kv_attention_reshape_gb300 as pkv
    dev = {n: on(st[n]) for n in ("q", "k", "v", "kc", "vc", "pos", "slot", "table", "q_out", "k_out")}
    sc = {}
    if "ks" in st:
        sc = dict(k_scale=on(st["ks"]) if st["kind"] == "block" else st["ks"],
                  v_scale=on(st["vs"]) if st["kind"] == "block" else st["vs"])
    dev.update(more)
    q_out, k_out = pkv.kv_append(dev["q"], dev["k"], dev["v"], dev["pos"], dev["slot"], dev["kc"], dev["vc"], dev["table"],
                                 rope_offset=st["off"], interleaved=st["inter"],
                                 q_out=dev["q_out"] if st["q"] is not None else None, k_out=dev["k_out"], **sc)
    err = pkv.device_errors()
    c = lambda t: t.cpu() if isinstance(t, torch.Tensor) else t  # noqa: E731
    return (c(q_out), c(k_out), c(dev["kc"]), c(dev["kc"] if dev["vc"] is None else dev["vc"]), c(sc.get("k_scale")),
            c(sc.get("v_scale"))), err


def same(a, b):
    """The same bits (any NaN is as good as another)."""
    if isinstance(a, torch.Tensor) and a.dtype == torch.bfloat16:
        a, b = (torch.where(x.isnan(), torch.tensor(0x7FC0, dtype=torch.int16), x.view(torch.int16)) for x in (a, b))
    return a is b or (torch.equal(a, b) if isinstance(a, torch.Tensor) else a == b)


def assert_append(got, want):
    for x, y, n in zip(got, want, ("q_out", "k_out", "k_cache", "v_cache", "k_scale", "v_scale")):
        if not same(x, y):
            pytest.fail(f"{n} differs")


# ---- kv_append -----------------------------------------------------------------------------------

CTX = [0, 3, 16, 31, 40, 200]
NEW = [1, 13, 16, 2, 37, 5]


@pytest.mark.gpu
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("kind,Hq,Hkv,d,rot,off", [
    ("bf16", 8, 2, 64, 64, 0), ("bf16", 5, 3, 128, 32, 16), ("tensor", 4, 4, 128, 128, 0), ("tensor", 16, 1, 64, 32, 32),
    ("latent", 16, 1, 576, 64, 512), ("block", 8, 2, 128, 128, 0), ("block", 3, 3, 128, 64, 32), ("block", 16, 1, 128, 16, 112)])
def test_append_is_the_plain_form(kind, Hq, Hkv, d, rot, off, inter):
    st = append_state(kind, CTX, NEW, Hq, Hkv, d, rot, off, inter, pad=3, seed=d + rot)
    got, err = gpu_append(st)
    assert err == 0
    assert_append(got, plain_append(st))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "tensor", "block"])
def test_append_without_rotation_or_queries(kind):
    st = append_state(kind, [5, 0, 33], [20, 1, 4], 0, 2, 128, 0, seed=3)
    got, err = gpu_append(st)
    assert err == 0
    assert_append(got, plain_append(st))


@pytest.mark.gpu
def test_append_rotation_in_64_bits_at_far_positions():
    """|y - exact| <= u |exact| + 2^-22 (|x_i| + |x_j|): one bf16 rounding, three fp32 ones (the table is an input)."""
    st = append_state("bf16", [131000], [72], 4, 2, 128, 128, max_pos=131072, seed=5)
    got, err = gpu_append(st)
    assert err == 0
    for x, y in ((st["q"], got[0]), (st["k"], got[1])):
        ref = rotate(x.double(), st["pos"], st["table"], 0, False)
        room = x.double().abs()
        room = room + torch.cat([room[..., 64:], room[..., :64]], -1)
        assert bool(((y.double() - ref).abs() <= U * ref.abs() + 2.0 ** -22 * room).all())


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 1025, 4097])
def test_append_block_scaled_batch_sizes(T):
    """Each way of dealing the runs (one, four or sixteen tokens a CTA): one prompt, and one token a request."""
    for ctx, new in (([7], [T]), ([3 + 5 * i % 60 for i in range(T)], [1] * T)):
        st = append_state("block", ctx, new, 1, 1, 128, 32, max_pos=8192, seed=T)
        got, err = gpu_append(st)
        assert err == 0
        assert_append(got, plain_append(st))


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,T", [(16, 2047), (16, 2048), (17, 2048), (17, 2899), (17, 2900)])
def test_append_block_scaled_where_the_launch_changes(Hq, T):
    """Batches on both sides of the sizes from which rows go through shared memory."""
    ctx = [5, 16, 0, 31]
    new = [T - 700, 600, 1, 99]
    st = append_state("block", ctx, new, Hq, 1, 128, 128, seed=T + Hq, max_pos=T)
    got, err = gpu_append(st)
    assert err == 0
    assert_append(got, plain_append(st))


@pytest.mark.gpu
def test_append_slices_of_a_fused_projection_in_place_and_a_shared_allocation():
    """q, k, v as slices of one [T, (Hq + 2 Hkv) d] tensor; K and V blocks interleaved in one allocation."""
    Hq, Hkv, d = 6, 2, 128
    st = append_state("block", [2, 40], [17, 9], Hq, Hkv, d, 128, seed=11)
    want = plain_append(st)
    T = len(st["slot"])
    fused = torch.cat([st["q"].reshape(T, -1), st["k"].reshape(T, -1), st["v"].reshape(T, -1)], 1).cuda()
    q = fused[:, :Hq * d].view(T, Hq, d)
    k = fused[:, Hq * d:(Hq + Hkv) * d].view(T, Hkv, d)
    v = fused[:, (Hq + Hkv) * d:].view(T, Hkv, d)
    both = torch.stack([st["kc"], st["vc"]], 1).cuda()
    got, err = gpu_append(st, q=q, k=k, v=v, kc=both[:, 0], vc=both[:, 1])
    assert err == 0
    assert_append(got, want)
    # contiguous inputs, outputs over them
    qi, ki = st["q"].cuda(), st["k"].cuda()
    got, err = gpu_append(st, q=qi, k=ki, q_out=qi, k_out=ki)
    assert err == 0
    assert_append(got, want)


@pytest.mark.gpu
def test_append_of_zeros_infinities_and_nans():
    """A run of zeros gets the smallest scale; what is not finite takes no part in a scale and saturates (or stays NaN)."""
    st = append_state("block", [0, 4, 30], [3, 2, 1], 2, 2, 128, 0, seed=2)
    st["k"][0:3] = 0.0
    st["v"][3, 1, 5] = math.inf
    st["v"][4, 0, 6] = -math.inf
    st["k"][5, 0, 0] = math.nan
    st["k"][5, 1] = 3.0e38  # the largest sizes bf16 has
    got, err = gpu_append(st)
    assert err == 0
    want = plain_append(st)
    assert float(want[4][int(st["slot"][0]) // 16, 0]) == 2.0 ** -64
    assert_append(got, want)


@pytest.mark.gpu
def test_append_skips_and_flags_bad_slots_and_positions():
    for kind in ("bf16", "block"):
        st = append_state(kind, [4, 20, 9], [6, 3, 1], 2, 1, 128, 64, seed=4, max_pos=64)
        st["pos"][1] = 64            # past the table
        st["pos"][7] = -1
        st["slot"][9] = st["nb"] * 16  # past the pool
        got, err = gpu_append(st)
        assert err == 0x1 | 0x8
        assert_append(got, plain_append(st))


@pytest.mark.gpu
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("kind,Hq,Hkv,d,rot,off,inter", [
    ("bf16", 3, 1, 128, 64, 32, False), ("bf16", 0, 2, 64, 0, 0, False), ("bf16", 5, 2, 128, 0, 0, False),
    ("tensor", 2, 1, 64, 64, 0, True), ("tensor", 9, 3, 128, 32, 96, False), ("latent", 4, 1, 576, 64, 512, True),
    ("block", 5, 1, 128, 128, 0, False), ("block", 2, 3, 128, 16, 0, True),
    # rows of which two CTAs do not hold enough in shared memory
    ("bf16", 100, 8, 128, 128, 0, False), ("latent", 25, 1, 576, 64, 512, False), ("block", 150, 1, 128, 128, 0, False)])
def test_append_of_many_tokens(kind, Hq, Hkv, d, rot, off, inter, fused):
    """Long batches: a long chunk, short ones, padding, bad slots and positions in between. fused: q, k
    and v are slices of one tensor, and the rotated q and k of contiguous ones replace them."""
    ctx, new = [5, 0, 77, 300], [2011, 1, 16, 100]
    st = append_state(kind, ctx, new, Hq, Hkv, d, rot, off, inter, pad=29, seed=Hq + d, max_pos=2100)
    st["slot"][700], st["slot"][2050], want_err = -1, st["nb"] * 16 + 5, 1
    if rot:
        st["pos"][3], st["pos"][2100], want_err = 2100, -7, 1 | 8
    want = plain_append(st)
    T = len(st["slot"])
    more = {}
    if fused:
        parts = [st[n].reshape(T, -1) for n in "qkv" if st[n] is not None]
        one = torch.cat(parts, 1).cuda()
        at = 0
        for n in "qkv":
            if st[n] is not None:
                h = st[n].shape[1]
                more[n] = one[:, at:at + h * d].view(T, h, d)
                at += h * d
    got, err = gpu_append(st, **more)
    assert err == want_err
    assert_append(got, want)
    if fused:
        qi, ki = on(st["q"]), on(st["k"])
        skip = torch.ones(T, dtype=torch.bool)  # the tokens that are skipped keep what q and k held
        skip[st["slot"] >= 0] = False
        skip[2050] = True
        if rot:
            skip[[3, 2100]] = True
        for n, x in (("q_out", st["q"]), ("k_out", st["k"])):
            if x is not None:
                i = 0 if n == "q_out" else 1
                want = tuple(torch.where(skip[:, None, None], x, w) if j == i else w for j, w in enumerate(want))
        got, err = gpu_append(st, q=qi, k=ki, q_out=qi, k_out=ki)
        assert err == want_err
        assert_append(got, want)


@pytest.mark.gpu
def test_append_twice_is_append_once():
    """Appending the same rows again changes nothing: the scales already hold them."""
    st = append_state("block", [3, 0, 50], [30, 2, 1], 2, 2, 128, 128, seed=8)
    got, _ = gpu_append(st)
    st2 = dict(st, kc=got[2], vc=got[3], ks=got[4], vs=got[5])
    assert_append(gpu_append(st2)[0], got)


# ---- decode --------------------------------------------------------------------------------------

def decode_state(lens, Hq, Hkv, seed=0, qs=1.0, spread=0.5, gap=0, pow2=False):
    g = gen(seed)
    t, nb = tables([(c + 15) // 16 for c in lens], g)
    (kc, ks), (vc, vs) = (block_cache(nb, Hkv, g, spread, pow2, gap) for _ in "kv")
    q = (torch.randn((len(lens), Hq, 128), generator=g) * qs).to(torch.bfloat16)
    st = dict(lens=lens, q=q, table=t, kc=kc, ks=ks, vc=vc, vs=vs, gap=gap)
    # NaN codes behind every sequence's last token
    for r, c in enumerate(lens):
        if c % 16:
            b = int(t[r, c // 16])
            for x in (kc, vc):
                (x[:, 0] if gap else x)[b, c % 16:] = 0x7F
    return st


def pools(st):
    """The caches on the GPU as [nb, 16, Hkv, 128] (blocks apart when the state has gaps)."""
    return tuple(on(st[n])[:, 0] if st["gap"] else on(st[n]) for n in ("kc", "vc"))


def context(st, r, h, c):
    j = torch.arange(c)
    b = st["table"][r].long()[j // 16]
    kc, vc = ((st[n][:, 0] if st["gap"] else st[n]) for n in ("kc", "vc"))
    return (values(kc[b, j % 16, h]) * st["ks"][b, h].double()[:, None],
            values(vc[b, j % 16, h]) * st["vs"][b, h].double()[:, None])


def check_decode(st, out, lse, scale, rows=None, reqs=None):
    Hkv = st["ks"].shape[1]
    G = st["q"].shape[1] // Hkv
    out, lse = out.cpu(), lse.cpu()
    for r in range(len(st["lens"])) if reqs is None else reqs:
        row, c = (r if rows is None else rows[r]), st["lens"][r]
        if c == 0:
            assert bool((out[row] == 0).all()) and bool((lse[row] == -math.inf).all())
            continue
        for h in range(Hkv):
            hq = slice(h * G, (h + 1) * G)
            q, (k, v) = st["q"][row:row + 1, hq].double(), context(st, r, h, c)
            check(out[row:row + 1, hq], lse[row:row + 1, hq], dense(q, k, v, scale), f"request {r} head {h}",
                  fixed_steps(st, r, h, c, q, k, scale, None, 2.0 ** -22))


def gpu_decode(st, scale=None, **more):
    import paged_kv_attention_reshape_gb300 as pkv
    kc, vc = pools(st)
    out, lse = pkv.paged_decode_attn(on(st["q"]), kc, vc, on(st["table"]), torch.tensor(st["lens"], dtype=torch.int32).cuda(),
                                     max(st["lens"] + [1]), k_scale=on(st["ks"]), v_scale=on(st["vs"]), scale=scale, **more)
    assert pkv.device_errors() == 0
    return out, lse


SCALE = 1.0 / math.sqrt(128)
EDGES = [0, 1, 2, 15, 16, 17, 31, 33, 127, 128, 129, 143, 145, 255, 256, 257, 400, 1]


@pytest.mark.gpu
@pytest.mark.parametrize("G,Hkv", [(1, 2), (2, 3), (4, 1), (8, 8), (16, 4), (16, 1), (1, 1), (8, 5)])
def test_decode_edge_lengths(G, Hkv):
    st = decode_state(EDGES, G * Hkv, Hkv, seed=G * 10 + Hkv)
    check_decode(st, *gpu_decode(st), SCALE)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,G,Hkv,qs", [
    ([5000], 8, 2, 1.0), ([20011], 16, 1, 3.0), ([40003], 2, 8, 1.0), ([100 + i % 37 for i in range(300)], 1, 8, 2.0), ([3000, 1, 2500, 17, 2900] * 3, 4, 4, 1.0), ([777] * 40, 2, 2, 6.0),
    ([9000, 40], 1, 3, 2.0)])
def test_decode_long_and_cut_sequences(lens, G, Hkv, qs):
    st = decode_state(lens, G * Hkv, Hkv, seed=len(lens), qs=qs)
    check_decode(st, *gpu_decode(st), SCALE)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,G", [([1500, 1, 1900, 130], 1), ([4003, 2500], 2), ([700, 650, 3001], 16)])
def test_decode_many_tiles_a_share(lens, G):
    """Many KV heads, so that each of them has few shares and a share holds tens of 128-token tiles."""
    Hkv = 64
    g = gen(len(lens))
    t, nb = tables([(c + 15) // 16 for c in lens], g)
    any_codes = lambda: torch.randint(0, 120, (nb, 16, Hkv, 128), generator=g, dtype=torch.uint8) + \
        128 * torch.randint(0, 2, (nb, 16, Hkv, 128), generator=g, dtype=torch.uint8)  # noqa: E731
    st = dict(lens=lens, table=t, kc=any_codes(), vc=any_codes(), gap=0, ks=0.01 * torch.rand((nb, Hkv), generator=g) + 0.001,
              vs=0.01 * torch.rand((nb, Hkv), generator=g) + 0.001,
              q=torch.randn((len(lens), G * Hkv, 128), generator=g).to(torch.bfloat16))
    for _ in range(3):
        out = gpu_decode(st)
    check_decode(st, *out, SCALE)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["wide_v", "wide_k", "tiny", "sink", "zero", "scale"])
def test_decode_extreme_scales_and_scores(what):
    """Values whose size changes from block to block by many powers of two, scores that one token dominates."""
    st = decode_state([700, 130, 16], 16, 2, seed=9, qs=1.0 if what != "sink" else 4.0)
    g = gen(1)
    scale = SCALE
    if what == "wide_v":
        st["vs"] = st["vs"] * torch.exp2(torch.randint(-30, 31, st["vs"].shape, generator=g).float())
    elif what == "wide_k":
        st["ks"] = st["ks"] * torch.exp2(torch.randint(-12, 3, st["ks"].shape, generator=g).float())
    elif what == "tiny":
        st["vs"], st["ks"] = st["vs"] * 2.0 ** -80, st["ks"] * 2.0 ** -20
        scale = 2.0 ** 20 * SCALE
    elif what == "sink":
        b = int(st["table"][0, 0])
        st["ks"][b] *= 12.0  # the first block's scores stand far above the others'
    elif what == "zero":
        st["q"][1] = 0
        st["kc"][int(st["table"][0, 3])] = 0
        st["vc"][int(st["table"][0, 4])] = 0x80  # -0
    elif what == "scale":
        scale = 3.7e-3
    check_decode(st, *gpu_decode(st, scale=scale), scale)


@pytest.mark.gpu
@pytest.mark.parametrize("G,Hkv", [(8, 8), (16, 4), (1, 2)])
def test_decode_gives_the_same_bits_every_time(G, Hkv):
    """Shares that end in a piece of one tile, whose sums follow those of the piece before without another tile in
    between: 300 calls with the cache now in L2 and now not."""
    import paged_kv_attention_reshape_gb300 as pkv
    g = gen(80 + G)
    lens = torch.randint(1, 260, (400,), generator=g).tolist()
    st = decode_state(lens, G * Hkv, Hkv, seed=80 + G, qs=2.0)
    kc, vc = pools(st)
    q, table, ks, vs = (on(st[n]) for n in ("q", "table", "ks", "vs"))
    dev = torch.tensor(lens, dtype=torch.int32).cuda()
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    first, differ = None, torch.zeros((), dtype=torch.bool, device="cuda")
    for i in range(300):
        if i % 3 == 0:
            flush.fill_(i & 127)
        out, lse = pkv.paged_decode_attn(q, kc, vc, table, dev, 260, k_scale=ks, v_scale=vs)
        if first is None:
            first = out, lse
        else:
            differ |= (out != first[0]).any() | (lse != first[1]).any()
    assert not bool(differ) and pkv.device_errors() == 0
    check_decode(st, *first, SCALE)


@pytest.mark.gpu
@pytest.mark.parametrize("G,Hkv", [(16, 1), (8, 2), (4, 3), (2, 2)])
def test_decode_heads_of_very_different_size(G, Hkv):
    """Heads 2^20 apart in one group: each keeps its own bits (the scores of the small ones are of ordinary size)."""
    st = decode_state([300, 5, 2500, 129, 1000], G * Hkv, Hkv, seed=7 + G)
    size = torch.exp2(torch.tensor([10.0, -10.0] * (G * Hkv // 2)))
    st["q"] = (st["q"].float() * size[None, :, None]).to(torch.bfloat16)
    st["q"][1, 0], st["q"][1, 1] = 0, st["q"][0, 1]
    st["ks"] = st["ks"] * 2.0 ** 10
    check_decode(st, *gpu_decode(st), SCALE)
    # the largest and the smallest numbers of bf16
    st["ks"] = st["ks"] * 2.0 ** -10
    scale = 2.0 ** -30
    st["q"] = (st["q"].float() * torch.exp2(torch.tensor([105.0, -100.0] * (G * Hkv // 2)))[None, :, None]).to(torch.bfloat16)
    st["ks"] = st["ks"] * 2.0 ** -85
    check_decode(st, *gpu_decode(st, scale=scale), scale)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["q", "k", "v", "inf"])
@pytest.mark.parametrize("lens,G,Hkv", [([300, 40, 7], 8, 2), ([9001, 20], 16, 1), ([777] * 60, 4, 8)])
def test_decode_of_what_is_no_number(lens, G, Hkv, what):
    """A NaN in a query, a cached key or a cached value: NaN in out and lse of the rows (or dims) that attend to it, whole
    or cut; the other rows as they are."""
    st = decode_state(lens, G * Hkv, Hkv, seed=90 + G)
    if what == "q":
        st["q"][0, 1, 77] = math.nan
        st["q"][1, G * Hkv - 1] = math.nan
    elif what == "inf":
        st["q"][0, 1, 77] = math.inf
    else:
        st[what + "c"][int(st["table"][0, lens[0] // 32]), 5, 0, 9] = 0x7F
    out, lse = gpu_decode(st)
    out, lse = out.cpu().double(), lse.cpu().double()
    for r, c in enumerate(lens):
        for h in range(Hkv):
            hq = slice(h * G, (h + 1) * G)
            q, (k, v) = st["q"][r:r + 1, hq].double(), context(st, r, h, c)
            o, z, A, M = dense(q, k, v, SCALE)
            a, b = out[r:r + 1, hq], lse[r:r + 1, hq]
            if what == "inf" and r == 0 and h == 0:  # (scores that are infinite: no number, in 64 bits or here)
                o[0, 1], z[0, 1] = math.nan, math.nan
            assert torch.equal(o.isnan(), a.isnan()) and torch.equal(z.isnan(), b.isnan()), f"request {r} head {h}"
            e = 2.0 ** -16 * M + 2.0 ** -20 * (1 + z.abs())
            assert bool(((b - z).abs() <= e)[z.isfinite()].all()), f"request {r} head {h}"
            tol = U * o.abs() + (U + 2 * e[..., None]) * A + fixed_steps(st, r, h, c, q, k, SCALE, None, 2.0 ** -22) + 1e-37
            assert bool(((a - o).abs() <= tol)[o.isfinite()].all()), f"request {r} head {h}"


@pytest.mark.gpu
def test_decode_request_sets_rows_and_block_strides():
    """A reordered set of the batch with query rows from cu_q; rows outside it are left as they were."""
    import paged_kv_attention_reshape_gb300 as pkv
    st = decode_state([300, 20, 1, 77, 500], 8, 2, seed=21, gap=1)
    rows = [3, 0, 9, 5, 7]
    q = torch.full((11, 8, 128), math.nan, dtype=torch.bfloat16)
    q[rows] = st["q"]
    st["q"] = q
    out = torch.full((11, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((11, 8), 5.0, device="cuda")
    cu = torch.tensor(rows + [11], dtype=torch.int32).cuda()
    order = torch.tensor([4, 0, 2, 1, 3], dtype=torch.int32).cuda()
    bounds = torch.tensor([0, 3, 3, 5], dtype=torch.int32).cuda()
    kc, vc = pools(st)
    pkv.paged_decode_attn(q.cuda(), kc, vc, on(st["table"]), torch.tensor(st["lens"], dtype=torch.int32).cuda(), 500, cu_q=cu,
                          reqs=pkv.Reqs(5, 5, order, bounds, 0), k_scale=on(st["ks"]), v_scale=on(st["vs"]), out=out, lse=lse)
    assert pkv.device_errors() == 0
    check_decode(st, out, lse, SCALE, rows, reqs=[4, 0, 2])
    rest = [r for r in range(11) if r not in (rows[4], rows[0], rows[2])]
    assert bool((out[rest] == 5).all()) and bool((lse[rest] == 5).all())


@pytest.mark.gpu
def test_decode_more_requests_than_a_launch_holds():
    lens = [(7 * i) % 50 for i in range(1100)]
    st = decode_state(lens, 2, 1, seed=6)
    check_decode(st, *gpu_decode(st), SCALE)


@pytest.mark.gpu
def test_decode_flags_bad_blocks_lengths_and_requests():
    """Bad ids and lengths are flagged; the other requests' rows are right."""
    import paged_kv_attention_reshape_gb300 as pkv
    st = decode_state([100, 200, 50, 64], 8, 2, seed=30)
    t = st["table"].clone()
    t[0, 3], t[0, 5] = -5, 1 << 30
    kc, vc = pools(st)
    args = dict(k_scale=on(st["ks"]), v_scale=on(st["vs"]))
    lens = torch.tensor(st["lens"], dtype=torch.int32).cuda()
    out, lse = pkv.paged_decode_attn(on(st["q"]), kc, vc, t.cuda(), lens, 200, **args)
    assert pkv.device_errors() == 0x2
    check_decode(st, out, lse, SCALE, reqs=[1, 2, 3])
    # a length past the host's bound is cut to it
    out, lse = pkv.paged_decode_attn(on(st["q"]), kc, vc, on(st["table"]), lens, 128, **args)
    assert pkv.device_errors() == 0x8
    check_decode(dict(st, lens=[100, 128, 50, 64]), out, lse, SCALE)
    # a request id outside the batch
    order = torch.tensor([2, 4, -1, 0], dtype=torch.int32).cuda()
    out, lse = pkv.paged_decode_attn(on(st["q"]), kc, vc, on(st["table"]), lens, 200, reqs=pkv.Reqs(4, 4, order), **args)
    assert pkv.device_errors() == 0x4
    check_decode(st, out, lse, SCALE, reqs=[2, 0])


@pytest.mark.gpu
def test_decode_in_a_graph_on_two_streams_and_without_a_workspace():
    """Captured once and replayed over changing lengths; two streams with a workspace each; the no-alloc form; a
    workspace full of anything."""
    import paged_kv_attention_reshape_gb300 as pkv
    st = decode_state([4000, 900, 60], 16, 2, seed=41)
    kc, vc = pools(st)
    q, t, ks, vs = (on(st[n]) for n in ("q", "table", "ks", "vs"))
    lens = torch.tensor(st["lens"], dtype=torch.int32).cuda()
    need = pkv.paged_decode_workspace_size(3, 16, 2, 128, 4000)
    ws = [torch.randint(0, 256, (need,), dtype=torch.uint8).cuda() for _ in range(2)]
    bufs = [(torch.empty_like(q), torch.empty((3, 16), device="cuda")) for _ in range(2)]
    call = lambda i: pkv.paged_decode_attn(q, kc, vc, t, lens, 4000, k_scale=ks, v_scale=vs, workspace=ws[i],  # noqa: E731
                                           out=bufs[i][0], lse=bufs[i][1])
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(side[i]):
                call(i)
    torch.cuda.synchronize()
    for i in range(2):
        check_decode(st, *bufs[i], SCALE)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0)
    for new in ([4000, 900, 60], [1, 3999, 17], [2222, 0, 512]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        # lengths inside what the tables hold: request 1 and 2 have fewer blocks
        n = [min(a, b) for a, b in zip(new, st["lens"])]
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        ok = dict(st, lens=n)
        check_decode(ok, *bufs[0], SCALE)
        out, lse = torch.empty_like(q), torch.empty((3, 16), device="cuda")
        pkv.paged_decode_attn_noalloc(q, kc, vc, t, lens, 4000, out, lse, k_scale=ks, v_scale=vs)
        check_decode(ok, out, lse, SCALE)
    assert pkv.device_errors() == 0


# ---- extend --------------------------------------------------------------------------------------

def extend_state(ctx, new, Hq, Hkv, seed=0, qs=1.0, spread=0.5, gap=0, pow2=False):
    st = decode_state(ctx, Hq, Hkv, seed, qs, spread, gap, pow2)
    g = gen(seed + 100)
    T = sum(new)
    st.update(ctx=ctx, new=new, cu=torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32),
              q=(torch.randn((T, Hq, 128), generator=g) * qs).to(torch.bfloat16),
              k_new=torch.randn((T, Hkv, 128), generator=g).to(torch.bfloat16),
              v_new=torch.randn((T, Hkv, 128), generator=g).to(torch.bfloat16))
    return st


def gpu_extend(st, errors=0, **more):
    import paged_kv_attention_reshape_gb300 as pkv
    kc, vc = pools(st)
    total = [c + n for c, n in zip(st["ctx"], st["new"])]
    out, lse = pkv.extend_attn(on(st["q"]), on(st["k_new"]), on(st["v_new"]), on(st["cu"]),
                               torch.tensor(total, dtype=torch.int32).cuda(), kc, vc, on(st["table"]), max(st["new"]), max(total),
                               k_scale=on(st["ks"]), v_scale=on(st["vs"]), **more)
    assert pkv.device_errors() == errors
    return out, lse


def check_extend(st, out, lse, scale, reqs=None):
    Hkv = st["ks"].shape[1]
    G = st["q"].shape[1] // Hkv
    out, lse = out.cpu(), lse.cpu()
    for r in range(len(st["ctx"])) if reqs is None else reqs:
        rows = slice(int(st["cu"][r]), int(st["cu"][r + 1]))
        c = st["ctx"][r]
        if rows.start == rows.stop:
            continue
        for h in range(Hkv):
            hq = slice(h * G, (h + 1) * G)
            k, v = context(st, r, h, c)
            k, v = torch.cat([k, st["k_new"][rows, h].double()]), torch.cat([v, st["v_new"][rows, h].double()])
            q = st["q"][rows, hq].double()
            check(out[rows, hq], lse[rows, hq], dense(q, k, v, scale, c), f"request {r} head {h}",
                  fixed_steps(st, r, h, c, q, k, scale, c, 2.0 ** -32))


@pytest.mark.gpu
@pytest.mark.parametrize("G,Hkv", [(1, 2), (2, 3), (4, 1), (8, 2), (16, 1)])
def test_extend_edge_lengths(G, Hkv):
    st = extend_state([0, 1, 15, 16, 17, 127, 128, 129, 300, 5, 0], [1, 2, 4, 1, 5, 3, 130, 128, 40, 0, 150], G * Hkv, Hkv,
                      seed=G + Hkv)
    check_extend(st, *gpu_extend(st), SCALE)


@pytest.mark.gpu
@pytest.mark.parametrize("G,Hkv,most", [(1, 2, 128), (1, 1, 32), (2, 3, 32), (4, 2, 16), (4, 1, 32), (8, 2, 4), (8, 1, 9), (16, 1, 8),
                                         (16, 2, 1)])
def test_extend_of_a_few_tokens(G, Hkv, most):
    """Sets whose requests have up to 128 rows for a KV head (up to 32, 64 and 128: four, two and one copies)."""
    ctx = [0, 1, 15, 16, 17, 127, 128, 129, 300, 5, 0, 1000, 2500]
    new = [1, most, 1 + most // 2, most, 1, 1 + most // 3, most, max(1, most - 1), most, 0, most, 1 + most // 4, most]
    st = extend_state(ctx, new, G * Hkv, Hkv, seed=G + most, qs=1.5, gap=1)
    check_extend(st, *gpu_extend(st), SCALE)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["wide_v", "wide_k", "tiny", "sink"])
def test_extend_of_a_few_tokens_extreme_scales(what):
    st = extend_state([700, 130, 1300], [3, 4, 2], 16, 2, seed=19, qs=1.0 if what != "sink" else 4.0)
    g = gen(3)
    if what == "wide_v":
        st["vs"] = st["vs"] * torch.exp2(torch.randint(-30, 31, st["vs"].shape, generator=g).float())
    elif what == "wide_k":
        st["ks"] = st["ks"] * torch.exp2(torch.randint(-12, 3, st["ks"].shape, generator=g).float())
    elif what == "tiny":
        st["vs"] = st["vs"] * 2.0 ** -80
        st["v_new"] = (st["v_new"].float() * 2.0 ** -80).to(torch.bfloat16)
    elif what == "sink":
        st["ks"][int(st["table"][0, 0])] *= 12.0
    check_extend(st, *gpu_extend(st), SCALE)


@pytest.mark.gpu
@pytest.mark.parametrize("ctx,new,G,Hkv", [
    ([9001], [4], 8, 1), ([5000, 17, 700], [1, 16, 3], 8, 2), ([1100], [64], 2, 1),     # up to 128 rows
    ([4000, 3000, 5], [200, 90, 1], 4, 2), ([2047], [700], 16, 1), ([6001], [130], 1, 3), ([900, 0], [300, 1000], 2, 1)])
def test_extend_of_few_long_contexts(ctx, new, G, Hkv):
    """Contexts that are cut into pieces; without a workspace they are not."""
    import paged_kv_attention_reshape_gb300 as pkv
    st = extend_state(ctx, new, G * Hkv, Hkv, seed=len(ctx) + G, qs=1.5, gap=1)
    n = pkv.launch_count()
    out, lse = gpu_extend(st)
    assert pkv.launch_count() == n + 2
    check_extend(st, out, lse, SCALE)
    kc, vc = pools(st)
    total = torch.tensor([c + m for c, m in zip(ctx, new)], dtype=torch.int32)
    args = [on(st[n]) for n in ("q", "k_new", "v_new", "cu", "table", "ks", "vs")]
    q, k, v, cu, table, ks, vs = args
    total = total.cuda()
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
    lib = pkv._lib.load()
    status = lib.pkv_extend_attn(q.data_ptr(), k.data_ptr(), v.data_ptr(), len(q), cu.data_ptr(), total.data_ptr(),
                                 pkv.make_cache(kc, vc, ks, vs), table.data_ptr(), table.shape[1],
                                 pkv.Reqs(max_reqs=len(ctx), batch_reqs=len(ctx)).c(), G * Hkv, max(new), int(total.max()),
                                 0, SCALE, out.data_ptr(), lse.data_ptr(), None, 0, torch.cuda.current_stream().cuda_stream)
    assert status == 0 and pkv.device_errors() == 0
    check_extend(st, out, lse, SCALE)


@pytest.mark.gpu
@pytest.mark.parametrize("new,G,Hkv", [([13, 1, 0, 8, 1], 4, 2), ([4] * 24, 8, 8), ([200, 90, 1, 300], 4, 3)])
def test_extend_gives_the_same_bits_every_time(new, G, Hkv):
    """300 calls with the cache now in L2 and now not: the order in which loads land must not matter."""
    import paged_kv_attention_reshape_gb300 as pkv
    g = gen(70 + G)
    ctx = [4491, 36, 2157, 1419, 61] if len(new) == 5 else torch.randint(30, 2600, (len(new),), generator=g).tolist()
    st = extend_state(ctx, new, G * Hkv, Hkv, seed=70 + G, qs=3.0)
    kc, vc = pools(st)
    q, k, v, cu, table, ks, vs = (on(st[n]) for n in ("q", "k_new", "v_new", "cu", "table", "ks", "vs"))
    total = torch.tensor([c + m for c, m in zip(ctx, new)], dtype=torch.int32).cuda()
    flush = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    first, differ = None, torch.zeros((), dtype=torch.bool, device="cuda")
    for i in range(300):
        if i % 3 == 0:
            flush.fill_(i & 127)
        out, lse = pkv.extend_attn(q, k, v, cu, total, kc, vc, table, max(new), int(total.max()) if i == 0 else 8000,
                                   k_scale=ks, v_scale=vs)
        if first is None:
            first = out, lse
        else:
            differ |= (out != first[0]).any() | (lse != first[1]).any()
    assert not bool(differ) and pkv.device_errors() == 0
    check_extend(st, *first, SCALE)


@pytest.mark.gpu
@pytest.mark.parametrize("new,G,Hkv", [([4, 2], 8, 1), ([200, 90], 4, 2)])
def test_extend_in_a_graph_with_other_lengths_and_beside_another_stream(new, G, Hkv):
    """A captured call replayed for other contexts (cut otherwise, then not at all), and two calls at once."""
    import paged_kv_attention_reshape_gb300 as pkv
    st = extend_state([6000, 1500], new, G * Hkv, Hkv, seed=40 + G)
    kc, vc = pools(st)
    q, k, v, cu, table, ks, vs = (on(st[n]) for n in ("q", "k_new", "v_new", "cu", "table", "ks", "vs"))
    lens = torch.tensor([c + m for c, m in zip(st["ctx"], new)], dtype=torch.int32).cuda()
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
    need = pkv.extend_block_workspace_size(max(new), 6300, G * Hkv, Hkv)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")

    def call(out, lse, ws):
        pkv.extend_attn(q, k, v, cu, lens, kc, vc, table, max(new), 6300, out=out, lse=lse, workspace=ws, k_scale=ks, v_scale=vs)

    call(out, lse, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out, lse, ws)
    for ctx in ([6000, 1500], [5, 700], [4001, 0], [0, 3], [6000, 1500]):
        lens.copy_(torch.tensor([c + m for c, m in zip(ctx, new)], dtype=torch.int32))
        out.zero_(), lse.zero_()
        graph.replay()
        check_extend(dict(st, ctx=ctx), out, lse, SCALE)
    other = torch.cuda.Stream()
    out2, lse2, ws2 = torch.zeros_like(out), torch.zeros_like(lse), torch.zeros_like(ws)
    other.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        call(out, lse, ws)
        with torch.cuda.stream(other):
            call(out2, lse2, ws2)
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    check_extend(st, out2, lse2, SCALE)
    assert pkv.device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("G,longest", [(8, 4), (2, 90)])
def test_extend_of_many_requests_beside_a_long_context(G, longest):
    """More requests than a launch holds, one of the first and one of the last far longer than the others: short
    items in shares whole, long ones cut over many of them."""
    n = 290
    ctx, new = [(13 * i) % 90 for i in range(n)], [1 + i % 3 for i in range(n)]
    ctx[3], ctx[280], new[3] = 12000, 5000, longest
    st = extend_state(ctx, new, G, 1, seed=50 + G)
    check_extend(st, *gpu_extend(st), SCALE)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["extend", "decode"])
def test_a_workspace_of_the_binding_on_another_stream(what):
    """The scratch that the binding allocates is not given to the current stream's tensors while the other's call runs."""
    import paged_kv_attention_reshape_gb300 as pkv
    st = extend_state([20000, 9000], [4, 4] if what == "extend" else [1, 1], 8, 1, seed=60)
    kc, vc = pools(st)
    q, k, v, cu, table, ks, vs = (on(st[n]) for n in ("q", "k_new", "v_new", "cu", "table", "ks", "vs"))
    lens = torch.tensor([c + (m if what == "extend" else 0) for c, m in zip(st["ctx"], st["new"])], dtype=torch.int32).cuda()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    outs = []
    for handle in (other, other.cuda_stream):
        for _ in range(4):
            if what == "extend":
                outs.append(pkv.extend_attn(q, k, v, cu, lens, kc, vc, table, 4, 20100, stream=handle, k_scale=ks, v_scale=vs))
                need = pkv.extend_block_workspace_size(4, 20100, 8, 1)
            else:
                outs.append(pkv.paged_decode_attn(q, kc, vc, table, lens, 20100, stream=handle, k_scale=ks, v_scale=vs))
                need = pkv.paged_decode_workspace_size(2, 8, 1, 128, 20100)
            torch.empty(need, dtype=torch.uint8, device="cuda").fill_(0x7F)
    torch.cuda.synchronize()
    assert pkv.device_errors() == 0
    for out, lse in outs:
        assert torch.equal(out, outs[0][0]) and torch.equal(lse, outs[0][1])
    if what == "extend":
        check_extend(st, *outs[0], SCALE)


@pytest.mark.gpu
@pytest.mark.parametrize("most", [3, 200])
def test_extend_cuts_and_flags_more_tokens_than_its_bound(most):
    """A request with more new tokens than max_q_len: its first max_q_len rows are right, the others stay as they were."""
    import paged_kv_attention_reshape_gb300 as pkv
    st = extend_state([100, 40, 7], [most, most + 2, 1], 8, 2, seed=23)
    kc, vc = pools(st)
    out = torch.full(st["q"].shape, 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(st["q"].shape[:2], 5.0, device="cuda")
    total = torch.tensor([c + n for c, n in zip(st["ctx"], st["new"])], dtype=torch.int32)
    pkv.extend_attn(on(st["q"]), on(st["k_new"]), on(st["v_new"]), on(st["cu"]), on(total), kc, vc, on(st["table"]), most,
                    int(total.max()), out=out, lse=lse, k_scale=on(st["ks"]), v_scale=on(st["vs"]))
    assert pkv.device_errors() == 0x8
    cut = slice(int(st["cu"][1]) + most, int(st["cu"][2]))
    assert bool((out[cut] == 5.0).all()) and bool((lse[cut] == 5.0).all())
    check_extend(st, out, lse, SCALE, reqs=[0, 2])
    few = dict(st, new=[most] * 2 + [1], cu=torch.tensor([0, most, 2 * most, 2 * most + 1], dtype=torch.int32))
    keep = torch.ones(len(st["q"]), dtype=torch.bool)
    keep[cut] = False
    few.update(q=st["q"][keep], k_new=st["k_new"][keep], v_new=st["v_new"][keep])
    check_extend(few, out.cpu()[keep], lse.cpu()[keep], SCALE)


@pytest.mark.gpu
@pytest.mark.parametrize("ctx,new,G,Hkv,qs", [([5000, 40], [20, 300], 8, 2, 1.0), ([1037] * 6, [4] * 6, 4, 2, 3.0),
                                              ([2500], [1], 16, 2, 1.0), ([800, 900], [200, 1], 1, 4, 2.0)])
def test_extend_longer_contexts(ctx, new, G, Hkv, qs):
    st = extend_state(ctx, new, G * Hkv, Hkv, seed=len(ctx), qs=qs, gap=1)
    check_extend(st, *gpu_extend(st), SCALE)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["wide_v", "wide_k", "tiny", "sink", "pow2"])
def test_extend_extreme_scales(what):
    st = extend_state([700, 130], [9, 140], 8, 2, seed=9, qs=1.0 if what != "sink" else 4.0, pow2=what == "pow2")
    g = gen(1)
    if what == "wide_v":
        st["vs"] = st["vs"] * torch.exp2(torch.randint(-30, 31, st["vs"].shape, generator=g).float())
    elif what == "wide_k":
        st["ks"] = st["ks"] * torch.exp2(torch.randint(-12, 3, st["ks"].shape, generator=g).float())
    elif what == "tiny":
        st["vs"] = st["vs"] * 2.0 ** -80
        st["v_new"] = (st["v_new"].float() * 2.0 ** -80).to(torch.bfloat16)
    elif what == "sink":
        st["ks"][int(st["table"][0, 0])] *= 12.0
    check_extend(st, *gpu_extend(st), SCALE)


@pytest.mark.gpu
def test_extend_of_many_requests_and_neighbours_that_are_not_finite():
    """More requests than a launch holds; a request whose new tokens are NaN beside others."""
    n = 300
    ctx, new = [(11 * i) % 70 for i in range(n)], [1 + i % 3 for i in range(n)]
    st = extend_state(ctx, new, 4, 2, seed=12)
    bad = slice(int(st["cu"][7]), int(st["cu"][8]))
    st["v_new"][bad] = math.nan
    out, lse = gpu_extend(st)
    check_extend(st, out, lse, SCALE, reqs=[r for r in range(n) if r != 7])


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["decode", "few", "many", "pieces"])
def test_value_scales_a_factor_2_to_the_100_apart(what):
    """Blocks of zeros at the smallest scale that kv_append writes beside blocks 2^100 larger: every block counts in the
    sum of weights."""
    ctx = [700, 130, 33] if what != "pieces" else [5000, 130, 33]
    new = {"few": [3, 4, 2], "many": [9, 140, 33], "pieces": [4, 2, 1]}.get(what)
    st = decode_state(ctx, 16, 2, seed=29) if what == "decode" else extend_state(ctx, new, 16, 2, seed=29)
    g = gen(4)
    zero = torch.rand(st["vs"].shape, generator=g) < 0.5
    st["vc"] = torch.where(zero[:, None, :, None] & (st["vc"] != 0x7F), torch.zeros((), dtype=torch.uint8), st["vc"])
    if what == "decode":
        st["vs"] = torch.where(zero, torch.tensor(2.0 ** -64), torch.tensor(2.0 ** 36))
        check_decode(st, *gpu_decode(st), SCALE)
    else:  # (the new tokens' values are 1 times themselves: 2^50 of the smallest and of the largest scale)
        st["vs"] = torch.where(zero, torch.tensor(2.0 ** -50), torch.tensor(2.0 ** 50))
        check_extend(st, *gpu_extend(st), SCALE)


@pytest.mark.gpu
@pytest.mark.parametrize("most,G", [(4, 8), (90, 4)])
def test_extend_request_sets(most, G):
    """The extend part of a reordered batch, its requests in any order; rows outside it are left as they were, also with
    a set bound far above the set's size."""
    import paged_kv_attention_reshape_gb300 as pkv
    ctx, new = [300, 20, 1, 1500, 77, 0, 900], [most, 1, 2, most - 1, 3, most, 1]
    st = extend_state(ctx, new, 2 * G, 2, seed=31 + G, gap=1)
    kc, vc = pools(st)
    total = torch.tensor([c + n for c, n in zip(ctx, new)], dtype=torch.int32)
    order = torch.tensor([1, 6, 5, 0, 3, 2, 4], dtype=torch.int32).cuda()
    bounds = torch.tensor([0, 2, 5, 7], dtype=torch.int32).cuda()
    q, k, v, cu, table, ks, vs = (on(st[n]) for n in ("q", "k_new", "v_new", "cu", "table", "ks", "vs"))
    for bound in (7, 3, 5000):
        for cls, reqs in enumerate(([1, 6], [5, 0, 3], [2, 4])):
            if bound < len(reqs):
                continue
            out, lse = torch.full_like(q, 5.0), torch.full(q.shape[:2], 5.0, device="cuda")
            pkv.extend_attn(q, k, v, cu, on(total), kc, vc, table, most, int(total.max()), out=out, lse=lse, k_scale=ks, v_scale=vs,
                            reqs=pkv.Reqs(bound, 7, order, bounds, cls))
            assert pkv.device_errors() == 0
            check_extend(st, out, lse, SCALE, reqs=reqs)
            rest = torch.cat([torch.arange(int(st["cu"][r]), int(st["cu"][r + 1])) for r in range(7) if r not in reqs]).cuda()
            assert bool((out[rest] == 5).all()) and bool((lse[rest] == 5).all())


def check_rows_that_are_no_numbers(st, out, lse, infinite=False):
    """out and lse are NaN where the definition in 64 bits says so, and within their bounds elsewhere."""
    Hkv = st["ks"].shape[1]
    G = st["q"].shape[1] // Hkv
    out, lse = out.cpu(), lse.cpu()
    for r, c in enumerate(st["ctx"]):
        rows = slice(int(st["cu"][r]), int(st["cu"][r + 1]))
        for h in range(Hkv):
            hq = slice(h * G, (h + 1) * G)
            k, v = context(st, r, h, c)
            k, v = torch.cat([k, st["k_new"][rows, h].double()]), torch.cat([v, st["v_new"][rows, h].double()])
            q = st["q"][rows, hq].double()
            o, z, A, M = dense(q, k, v, SCALE, c)
            a, b = out[rows, hq].double(), lse[rows, hq].double()
            if infinite:
                z = torch.where(q.isinf().any(-1), math.nan, z)
            assert torch.equal(o.isnan(), a.isnan()), f"request {r} head {h}"
            assert torch.equal(z.isnan(), b.isnan()) and not bool(b.isinf().any()), f"request {r} head {h}"
            e = 2.0 ** -16 * M + 2.0 ** -20 * (1 + z.abs())
            fixed = fixed_steps(st, r, h, c, q, k, SCALE, c, 2.0 ** -32)
            assert bool(((b - z).abs() <= e)[z.isfinite()].all()), f"request {r} head {h}"
            tol = U * o.abs() + (U + 2 * e[..., None]) * A + fixed + 1e-37
            assert bool(((a - o).abs() <= tol)[o.isfinite()].all()), f"request {r} head {h}"


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["q", "k", "v", "new_k", "all", "below"])
@pytest.mark.parametrize("ctx,new,G,Hkv", [
    ([300, 40], [4, 2], 8, 2), ([257, 3], [8, 8], 16, 1), ([9001, 20], [4, 3], 8, 1),          # up to 128 rows; the last in pieces
    ([130, 20], [200, 9], 4, 2), ([700, 33], [40, 100], 2, 1), ([4000, 3000, 5], [200, 90, 1], 4, 2)])
def test_extend_of_what_is_no_number(ctx, new, G, Hkv, what):
    """A NaN in a query, in a cached key or value, in a new key: NaN in the rows (or dims) that attend to it, in out and
    lse, whatever the launch and the plan; the other rows as they are. An infinite query counts as NaN."""
    st = extend_state(ctx, new, G * Hkv, Hkv, seed=90 + G, qs=1.0)
    if what == "q":
        st["q"][1, 0, 77] = math.nan
        st["q"][int(st["cu"][1]), G * Hkv - 1] = math.nan
    elif what in ("k", "v"):
        st[what + "c"][int(st["table"][0, ctx[0] // 32]), 5, 0, 9] = 0x7F
    elif what == "new_k":  # the second token's key: every row of the request but the first
        st["k_new"][int(st["cu"][1]) + 1, Hkv - 1, 100] = math.nan
    elif what == "all":
        st["q"][0] = math.nan
        for r in range(len(ctx)):
            st["kc"][st["table"][r, :(ctx[r] + 15) // 16].long()] = 0xFF
    else:  # a token without context, its one score -inf in 64 bits: no weights
        st["ctx"] = [ctx[0], 0] + ctx[2:]
        t = int(st["cu"][1])
        st["q"][t, 0], st["k_new"][t, 0] = 0.5, 0.5
        st["q"][t, 0, 3], st["k_new"][t, 0, 3] = math.inf, -1.0
    check_rows_that_are_no_numbers(st, *gpu_extend(st), infinite=what == "below")


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["q", "new_k"])
@pytest.mark.parametrize("ctx,new,G,Hkv", [([300, 40], [4, 3], 8, 2), ([130, 20], [200, 9], 4, 2), ([9001, 20], [4, 3], 8, 1)])
def test_extend_of_numbers_beyond_fp16(ctx, new, G, Hkv, what):
    """A query or new key that fp16 does not hold is seen in the rows that attend to it, also where its score is far
    below the others'; the largest that it holds are multiplied as they are."""
    st = extend_state(ctx, new, G * Hkv, Hkv, seed=95 + G)
    t = int(st["cu"][1]) + 1
    st["q"][0, 0, 3] = 65280.0
    st["ks"], st["k_new"] = st["ks"] * 2.0 ** -10, (st["k_new"].float() * 2.0 ** -10).to(torch.bfloat16)
    if what == "q":
        st["q"][t, 0, 9] = -70000.0
        rows = slice(t, t + 1)
    else:
        st["k_new"][t, 0, 9] = -70000.0
        st["q"][:, :, 9] = st["q"][:, :, 9].abs() + 0.01
        rows = slice(t, int(st["cu"][2]))
    out, lse = gpu_extend(st)
    heads = slice(0, 1) if what == "q" else slice(0, G)
    assert bool(out[rows, heads].isnan().all()) and bool(lse[rows, heads].isnan().all())
    for r in range(2):
        for h in range(Hkv):
            at, hq = slice(int(st["cu"][r]), int(st["cu"][r + 1])), slice(h * G, (h + 1) * G)
            k, v = context(st, r, h, ctx[r])
            k, v = torch.cat([k, st["k_new"][at, h].double()]), torch.cat([v, st["v_new"][at, h].double()])
            q = st["q"][at, hq].double()
            o, z, A, M = dense(q, k, v, SCALE, ctx[r])
            a, b = out.cpu()[at, hq].double(), lse.cpu()[at, hq].double()
            fine = ~b.isnan()
            assert int((~fine).sum()) == (0 if h or not r else 1 if what == "q" else G * (rows.stop - rows.start))
            e = 2.0 ** -16 * M + 2.0 ** -20 * (1 + z.abs())
            tol = U * o.abs() + (U + 2 * e[..., None]) * A + fixed_steps(st, r, h, ctx[r], q, k, SCALE, ctx[r], 2.0 ** -32) + 1e-37
            assert bool(((b - z).abs() <= e)[fine].all()) and bool(((a - o).abs() <= tol)[fine].all()), f"request {r} head {h}"


@pytest.mark.gpu
def test_extend_flags_bad_blocks():
    st = extend_state([100, 200], [5, 6], 8, 2, seed=30)
    good = st["table"].clone()
    st["table"][0, 3], st["table"][0, 5] = -5, 1 << 30
    out, lse = gpu_extend(st, errors=0x2)
    st["table"] = good
    check_extend(st, out, lse, SCALE, reqs=[1])


# ---- the run of them -----------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
def test_prompt_chunks_then_decode_steps(captured):
    """Two sequences: a prompt in two chunks, then decode steps, every step appended and attended; each step's cache is
    the plain form's bit for bit and each output is dense softmax over it. Captured: the decode step is one graph,
    replayed, in a batch padded to four rows."""
    import paged_kv_attention_reshape_gb300 as pkv
    Hq, Hkv, d, R, B = 8, 2, 128, 2, 4
    g = gen(77)
    t, nb = tables([5, 9], g)
    table = rope_table(d, 256)
    kc, vc = (torch.randint(0, 256, (nb, 16, Hkv, d), generator=g, dtype=torch.uint8) for _ in "kv")
    ks, vs = (torch.full((nb, Hkv), 1e30) for _ in "kv")  # stale: every block starts afresh
    dev = dict(kc=kc.cuda(), vc=vc.cuda(), ks=ks.cuda(), vs=vs.cuda(), t=t.cuda(), table=table.cuda())
    host = dict(kind="block", table=table, off=0, inter=False, kc=kc, vc=vc, ks=ks, vs=vs)

    def batch(have, new, rows):
        """Token rows of a step: `new[r]` tokens of each sequence, padded to `rows`."""
        pos = torch.cat([torch.arange(have[r], have[r] + new[r]) for r in range(R)])
        req = torch.arange(R).repeat_interleave(torch.tensor(new))
        slot = t[req, pos // 16].long() * 16 + pos % 16
        T = len(pos)
        full = lambda x, v: torch.cat([x, torch.full((rows - T,), v, dtype=x.dtype)])  # noqa: E731
        mk = lambda h: (torch.randn((rows, h, d), generator=g) * torch.exp(torch.randn((rows, h, 1), generator=g))).to(torch.bfloat16)  # noqa: E731
        return dict(pos=full(pos, 0), slot=full(slot, -1), q=mk(Hq), k=mk(Hkv), v=mk(Hkv),
                    q_out=torch.zeros((rows, Hq, d), dtype=torch.bfloat16), k_out=torch.zeros((rows, Hkv, d), dtype=torch.bfloat16))

    def check_cache(b):
        want = plain_append(dict(host, **b))
        host.update(kc=want[2], vc=want[3], ks=want[4], vs=want[5])
        for n in ("kc", "vc", "ks", "vs"):
            assert torch.equal(dev[n].cpu(), host[n]), n
        return want

    have = [0, 0]
    for new in ([20, 61], [33, 40]):
        b = batch(have, new, sum(new))
        qr, kr = pkv.kv_append(on(b["q"]), on(b["k"]), on(b["v"]), on(b["pos"]), on(b["slot"]), dev["kc"], dev["vc"], dev["table"],
                               k_scale=dev["ks"], v_scale=dev["vs"])
        want = check_cache(b)
        assert same(qr.cpu(), want[0]) and same(kr.cpu(), want[1])
        total = [h + n for h, n in zip(have, new)]
        cu = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
        out, lse = pkv.extend_attn(qr, kr, on(b["v"]), cu.cuda(), torch.tensor(total, dtype=torch.int32).cuda(), dev["kc"],
                                   dev["vc"], dev["t"], max(new), max(total), k_scale=dev["ks"], v_scale=dev["vs"])
        check_extend(dict(ctx=have, new=new, cu=cu, q=want[0], k_new=want[1], v_new=b["v"], table=t, gap=0, kc=host["kc"],
                          vc=host["vc"], ks=host["ks"], vs=host["vs"]), out, lse, SCALE)
        have = total
    b = batch(have, [1, 1], B)
    live = {n: on(b[n]) for n in ("pos", "slot", "q", "k", "v", "q_out", "k_out")}
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    tabs = torch.zeros((B, t.shape[1]), dtype=torch.int32, device="cuda")
    tabs[:R] = dev["t"]
    out, lse = torch.empty((B, Hq, d), dtype=torch.bfloat16, device="cuda"), torch.empty((B, Hq), device="cuda")
    ws = torch.empty(pkv.paged_decode_workspace_size(B, Hq, Hkv, d, 144), dtype=torch.uint8, device="cuda")

    def step():
        pkv.kv_append(live["q"], live["k"], live["v"], live["pos"], live["slot"], dev["kc"], dev["vc"], dev["table"],
                      q_out=live["q_out"], k_out=live["k_out"], k_scale=dev["ks"], v_scale=dev["vs"])
        pkv.paged_decode_attn(live["q_out"], dev["kc"], dev["vc"], tabs, lens, 144, out=out, lse=lse, workspace=ws,
                              k_scale=dev["ks"], v_scale=dev["vs"])

    graph = None
    for _ in range(20):
        b = batch(have, [1, 1], B)
        for n in live:
            live[n].copy_(b[n])
        have = [h + 1 for h in have]
        lens.copy_(torch.tensor(have + [0, 0], dtype=torch.int32))
        if captured and graph is None:
            saved = {n: dev[n].clone() for n in ("kc", "vc", "ks", "vs")}
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for n, x in saved.items():
                assert torch.equal(x, dev[n])  # capturing runs nothing
        if captured:
            graph.replay()
        else:
            step()
        assert pkv.device_errors() == 0
        want = check_cache(b)
        check_decode(dict(lens=have + [0, 0], q=want[0], table=tabs.cpu(), gap=0, kc=host["kc"], vc=host["vc"], ks=host["ks"],
                          vs=host["vs"]), out, lse, SCALE)


# ---- refusals (no GPU) ---------------------------------------------------------------------------

def _refusals():
    import paged_kv_attention_reshape_gb300 as pkv
    from paged_kv_attention_reshape_gb300 import _lib
    P = ctypes.c_void_p
    fake = P(1 << 20)  # never dereferenced: each call fails its host checks
    return pkv.load(), _lib, P, fake


def test_append_refusals():
    lib, L, P, fake = _refusals()
    bf = L.PkvCache(fake, P(1 << 21), 10, 16, 2, 128, 16 * 2 * 128)
    blk = L.PkvCache(fake, P(1 << 21), 10, 16, 2, 128, 16 * 2 * 128, L.KV_FP8_E4M3_BLOCK, 1.0, 1.0, fake, fake)
    lat = L.PkvCache(fake, None, 10, 16, 1, 576, 16 * 576)
    rope = L.PkvRope(fake, 100, 128, 0, 0)

    def call(q=fake, qs=8 * 128, k=fake, kstr=256, v=fake, vstr=256, pos=fake, slot=fake, T=4, Hq=8, rope=rope, cache=bf,
             qo=P(1 << 22), ko=P(1 << 22)):
        return lib.pkv_kv_append(q, qs, k, kstr, v, vstr, pos, slot, T, Hq, rope, cache, qo, ko, None)

    assert call(T=0) == 0
    assert call(T=-1) == 1 and call(Hq=-1) == 1
    assert call(k=None) == 1 and call(v=None) == 1 and call(slot=None) == 1 and call(pos=None) == 1
    assert call(q=None) == 1 and call(qo=None) == 1 and call(Hq=0) == 1
    assert call(k=P((1 << 20) + 2)) == 1 and call(qo=P((1 << 20) + 8)) == 1 and call(rope=L.PkvRope(P(4), 9, 16, 0, 0)) == 1
    assert call(qs=8 * 128 - 8) == 1 and call(kstr=260) == 1 and call(vstr=128) == 1
    assert call(qo=fake, qs=2048) == 1 and call(ko=fake, kstr=512) == 1  # in place over strided rows
    assert call(rope=L.PkvRope(None, 100, 128, 0, 0)) == 1 and call(rope=L.PkvRope(fake, 0, 128, 0, 0)) == 1
    assert call(rope=L.PkvRope(fake, 100, -16, 0, 0)) == 1 and call(rope=L.PkvRope(fake, 100, 16, -16, 0)) == 1
    assert call(rope=L.PkvRope(fake, 100, 8, 0, 0)) == 2 and call(rope=L.PkvRope(fake, 100, 64, 8, 0)) == 2
    assert call(rope=L.PkvRope(fake, 100, 128, 16, 0)) == 2
    assert call(cache=L.PkvCache(fake, fake, 10, 16, 2, 72, 16 * 2 * 72), kstr=144, vstr=144, qs=576) == 2
    assert call(T=1 << 31) == 2
    # a latent cache has no values; any other has
    assert call(cache=lat, Hq=1, qs=576, kstr=576, v=fake, rope=L.PkvRope(fake, 9, 64, 512, 0)) == 1
    # block scales: their pointers, the head width, the block size
    assert call(cache=L.PkvCache(fake, fake, 10, 16, 2, 128, 4096, L.KV_FP8_E4M3_BLOCK, 1.0, 1.0, None, fake)) == 1
    assert call(cache=L.PkvCache(fake, fake, 10, 16, 2, 128, 4096, L.KV_FP8_E4M3_BLOCK, 1.0, 1.0, P((1 << 20) + 2), fake)) == 1
    assert call(cache=L.PkvCache(fake, fake, 10, 16, 2, 64, 2048, L.KV_FP8_E4M3_BLOCK, 1.0, 1.0, fake, fake), kstr=128, vstr=128,
                qs=512, rope=L.PkvRope(fake, 9, 64, 0, 0)) == 2
    assert call(cache=L.PkvCache(fake, fake, 10, 32, 2, 128, 8192, L.KV_FP8_E4M3_BLOCK, 1.0, 1.0, fake, fake)) == 2
    assert call(cache=L.PkvCache(fake, fake, 10, 16, 2, 128, 4096, 7)) == 1
    assert call(cache=blk, T=0) == 0


def test_block_scaled_cache_is_refused_where_it_is_not_known():
    lib, L, P, fake = _refusals()
    blk = L.PkvCache(fake, fake, 10, 16, 2, 128, 4096, L.KV_FP8_E4M3_BLOCK, 1.0, 1.0, fake, fake)
    none = L.PkvCache(fake, fake, 10, 16, 2, 128, 4096, L.KV_FP8_E4M3_BLOCK, 1.0, 1.0, fake, None)
    reqs = L.PkvReqs(None, None, 0, 4, 4)
    assert lib.pkv_kv_cache_write(fake, fake, fake, 1, blk, None) == 2
    assert lib.pkv_kv_block_pack(blk, fake, 3, fake, None) == 2
    assert lib.pkv_kv_block_unpack(fake, fake, 3, blk, None) == 2
    ws = P(1 << 21)
    n = lib.pkv_paged_decode_workspace_size(4, 8, 2, 128, 100)
    dec = lambda c, hq=8, ws=ws, n=n, scale=1.0: lib.pkv_paged_decode_attn(fake, c, fake, 4, fake, None, reqs, hq, 100, scale, fake,  # noqa: E731
                                                                           None, ws, n, None)
    ext = lambda c, hq=8, scale=1.0: lib.pkv_extend_attn(fake, fake, fake, 8, fake, fake, c, fake, 4, reqs, hq, 8, 100, 0, scale,  # noqa: E731
                                                         fake, None, None, 0, None)
    assert dec(none) == 1 and ext(none) == 1
    assert dec(blk, hq=6) == 2 and ext(blk, hq=6) == 2 and dec(blk, hq=64) == 2 and ext(blk, hq=64) == 2
    for bad in (0.0, -1.0, math.inf, math.nan):
        assert dec(blk, scale=bad) == 1 and ext(blk, scale=bad) == 1
    d64 = L.PkvCache(fake, fake, 10, 16, 2, 64, 2048, L.KV_FP8_E4M3_BLOCK, 1.0, 1.0, fake, fake)
    b32 = L.PkvCache(fake, fake, 10, 32, 2, 128, 8192, L.KV_FP8_E4M3_BLOCK, 1.0, 1.0, fake, fake)
    assert dec(d64) == 2 and ext(d64) == 2 and dec(b32) == 2 and ext(b32) == 2
    # a workspace that is too small, or not aligned; contexts that no call can cut need none
    need = lib.pkv_extend_block_workspace_size(8, 5000, 8, 2)
    # (896 tokens are at most 7 key tiles of context and one of new tokens, the 8 that a share has at least)
    assert lib.pkv_extend_block_workspace_size(8, 897, 8, 2) == need > lib.pkv_extend_block_workspace_size(8, 896, 8, 2) == 0
    assert lib.pkv_extend_block_workspace_size(33, 5000, 8, 2) > need and lib.pkv_extend_block_workspace_size(8, 5000, 8, 0) == 0
    for w, size in ((ws, need - 1), (P((1 << 21) + 8), need)):
        assert lib.pkv_extend_attn(fake, fake, fake, 8, fake, fake, blk, fake, 4, reqs, 8, 8, 5000, 0, 1.0, fake, None, w, size,
                                   None) == 3
    # more KV heads than the decode's tables hold
    wide = L.PkvCache(fake, fake, 10, 16, 257, 128, 257 * 2048, L.KV_FP8_E4M3_BLOCK, 1.0, 1.0, fake, fake)
    assert dec(wide, hq=257) == 2
    empty = L.PkvReqs(None, None, 0, 0, 4)
    assert lib.pkv_paged_decode_attn(fake, blk, fake, 4, fake, None, empty, 8, 100, 1.0, fake, None, None, 0, None) == 0


@pytest.mark.gpu
def test_binding_checks_its_tensors():
    import paged_kv_attention_reshape_gb300 as pkv
    st = append_state("block", [3], [2], 2, 2, 128, 64, seed=1)
    d = {n: on(st[n]) for n in ("q", "k", "v", "pos", "slot", "kc", "vc", "ks", "vs", "table")}
    args = lambda **m: [dict(d, **m)[n] for n in ("q", "k", "v", "pos", "slot", "kc", "vc", "table")]  # noqa: E731
    sc = dict(k_scale=d["ks"], v_scale=d["vs"])
    for bad in (dict(q=d["q"].float()), dict(q=st["q"]), dict(k=d["k"][:1]), dict(v=d["v"][:, :1]), dict(pos=d["pos"].int()),
                dict(slot=d["slot"][:1]), dict(v=None), dict(table=d["table"].double()), dict(q=d["q"].transpose(1, 2)),
                dict(kc=d["kc"][:, :8])):
        with pytest.raises(pkv.PkvError):
            pkv.kv_append(*args(**bad), **sc)
    for bad in (dict(k_scale=d["ks"], v_scale=1.0), dict(k_scale=d["ks"][:1], v_scale=d["vs"]),
                dict(k_scale=d["ks"].double(), v_scale=d["vs"]), dict(k_scale=st["ks"], v_scale=d["vs"]),
                dict(k_scale=d["ks"].t(), v_scale=d["vs"])):
        with pytest.raises(pkv.PkvError):
            pkv.kv_append(*args(), **bad)
    with pytest.raises(pkv.PkvError):
        pkv.kv_append(*args(), q_out=torch.empty_like(d["q"])[:1], **sc)
    with pytest.raises(pkv.PkvError):
        pkv.kv_cache_write(d["k"], d["v"], d["slot"], d["kc"], d["vc"], **sc)
