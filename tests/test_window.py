"""Attention with a sliding window and sinks: decode, extend and prefill, and a run of them together, against a
dense softmax in 64 bits over the keys that each row sees.

Tolerances (u = 2^-8, half a step of bf16 relative to the value; A = sum_j p_j |v_j|, n the number of keys):
  * a score: D <= 128 fp32 additions of exact products, each off by at most 2^-23 of the sum of magnitudes
    M = scale sum_d |q_d k_d| (a truncating adder): 2^-16 M; 2^-20 (1 + |lse|) for the rounding of
    s * scale * log2(e) - m, of 2^x and of the logarithm (each within 2^-22 of a number of that size). Over an
    8-bit cache the extend's q becomes fp16, which is exact from 2^-14 on and off by at most 2^-25 below: 2^-25 scale
    sum_d |k_d|, and the new keys likewise. The decode's q is two E4M3 parts, exact down to 2^-14 of the head's largest
    |q| and off by at most 2^-21 of that below: 2^-21 scale q_top sum_d |k_d|. e is the sum of these.
  * lse: e.
  * out: u |o| for its own rounding; P is rounded to bf16 (u A; fp16 over an 8-bit cache, finer); the exponent's
    error moves p and the sum by e each (2 e A); n fp32 additions of P V (n 2^-23 A). The extend over an 8-bit
    cache rounds new values / v_scale to fp16 (2^-11 A) and P below 2^-14 to steps of 2^-24, where the largest P of the row
    is 1 at least: 2^-25 sum_j |v_j|. The decode over codes rounds P to two E4M3 parts in a frame a tile, off by at most
    2^-9 P, or 2^-22 of the tile's largest P' = P vs below 2^-14 of it. With values v = vs c and P' <= l vs_top (vs_top: the
    value scale of the row's largest P'): 2^-22 vs_top sum_j |c_j|, which is 2^-22 sum_j |v_j| where all vs are one.
"""
import ctypes
import math

import pytest
import torch

E4M3 = torch.float8_e4m3fn
U = 2.0 ** -8
BS = 16


def seen_mask(at, keys, window, sinks):
    """Which of the keys at positions `keys` the rows at positions `at` see."""
    i, j = at[:, None], keys[None]
    return (j <= i) & ((j > i - window) | (j < sinks))


def make(reqs, Hq, Hkv, D, kind, window, sinks, seed, cached_all=False, pad=3):
    """reqs: (cached, new) of each request. A pool whose unused pages, and whose tokens that no row sees, hold NaN; table
    entries of pages that no row sees are far out of range. cached_all: the new tokens are in the cache too (decode)."""
    g = torch.Generator().manual_seed(seed)
    new = [n for _, n in reqs]
    T = sum(new)
    normal = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)
    st = dict(reqs=reqs, Hq=Hq, Hkv=Hkv, D=D, kind=kind, window=window, sinks=sinks, T=T, q=normal(T + pad, Hq, D),
              k_new=normal(T + pad, Hkv, D), v_new=normal(T + pad, Hkv, D))
    st["k_new"][T:] = math.nan  # rows behind the last sequence
    st["v_new"][T:] = math.nan
    held = [c + (n if cached_all else 0) for c, n in reqs]
    most = max(1, max((h + BS - 1) // BS for h in held))
    nb = sum((h + BS - 1) // BS for h in held) + 3
    perm = torch.randperm(nb, generator=g)
    if kind == "block":
        st.update(ks=torch.exp(torch.randn((nb, Hkv), generator=g)) * 0.02, vs=torch.exp(torch.randn((nb, Hkv), generator=g)) * 0.03)
    if kind == "tensor":
        st.update(ks=0.02, vs=0.03)
    if kind in ("tensor", "block"):
        kc, vc = (torch.randint(0, 127, (nb, BS, Hkv, D), generator=g, dtype=torch.uint8) + 128 *
                  torch.randint(0, 2, (nb, BS, Hkv, D), generator=g, dtype=torch.uint8) for _ in "kv")
        # (magnitudes up to 448: as normal values at these scales would not be larger than 4)
        kc, vc = ((c.view(E4M3).float() / 3.0).to(E4M3).view(torch.uint8) for c in (kc, vc))
        hole = 0x7F
    else:
        kc, vc = (torch.randn((nb, BS, Hkv, D), generator=g).to(torch.bfloat16) for _ in "kv")
        hole = math.nan
    table = torch.full((len(reqs), most), 10 ** 9, dtype=torch.int32)
    live = torch.zeros((nb, BS), dtype=torch.bool)
    at = 0
    for r, ((c, n), h) in enumerate(zip(reqs, held)):
        rows = torch.arange(c, c + n)
        keys = torch.arange(h)
        any_row = seen_mask(rows, keys, window, sinks).any(0) if n else torch.zeros(h, dtype=torch.bool)
        for b in range((h + BS - 1) // BS):
            s = any_row[b * BS:(b + 1) * BS]
            if s.any():
                table[r, b] = perm[at]
                live[perm[at], :len(s)] = s
                at += 1
    for x in (kc, vc):
        x[~live] = hole
    st.update(kc=kc, vc=vc, table=table, lens=torch.tensor([c + n for c, n in reqs], dtype=torch.int32),
              cu=torch.tensor([0] + new).cumsum(0).to(torch.int32))
    return st


def cached(st, r, n):
    """The first n cached keys and values of request r as doubles [n, Hkv, D] (unseen ones 0)."""
    j = torch.arange(n)
    page = st["table"][r].long()[j // BS]
    ok = page < st["kc"].shape[0]
    out = []
    for c, s in (("kc", "ks"), ("vc", "vs")):
        x = st[c][torch.where(ok, page, 0), j % BS]
        if st["kind"] == "tensor":
            x = x.view(E4M3).float().double() * float(torch.tensor(st[s], dtype=torch.float32))
        elif st["kind"] == "block":
            x = x.view(E4M3).float().double() * st[s][torch.where(ok, page, 0)].double()[:, :, None]
        else:
            x = x.double()
        x[~ok] = 0
        out.append(torch.nan_to_num(x))
    return out


def reference(st, decode=False):
    """out, lse and their tolerances, rows [T]."""
    T, Hq, Hkv, D = st["T"], st["Hq"], st["Hkv"], st["D"]
    G, scale = Hq // Hkv, 1.0 / math.sqrt(D)
    out, tol = torch.zeros((T, Hq, D), dtype=torch.float64), torch.zeros((T, Hq, D), dtype=torch.float64)
    lse, ltol = torch.full((T, Hq), -math.inf, dtype=torch.float64), torch.zeros((T, Hq), dtype=torch.float64)
    row = 0
    for r, (c, n) in enumerate(st["reqs"]):
        if n == 0 or c + n == 0:
            row += n
            continue
        kv = []
        if st["kind"] != "none":
            kv.append(cached(st, r, c + n if decode else c))
        if not decode:
            kv.append((st["k_new"][row:row + n].double(), st["v_new"][row:row + n].double()))
        k, v = (torch.cat([x[i] for x in kv]) for i in (0, 1))
        seen = seen_mask(torch.arange(c, c + n), torch.arange(c + n), st["window"], st["sinks"])
        for h in range(Hq):
            q = st["q"][row:row + n, h].double()
            kh, vh = k[:, h // G], v[:, h // G]
            s = (q @ kh.T * scale).masked_fill(~seen, -math.inf)
            mag = (q.abs() @ kh.abs().T * scale).masked_fill(~seen, 0).amax(-1)
            z = torch.logsumexp(s, -1)
            p = torch.exp(s - z[:, None])
            o, A = p @ vh, p @ vh.abs()
            e = 2.0 ** -16 * mag + 2.0 ** -20 * (1 + z.abs())
            sumv = 0.0
            if st["kind"] in ("tensor", "block") and decode:
                e = e + 2.0 ** -21 * scale * q.abs().max() * kh.abs().sum(-1).max()
                codes = vh.abs() / (st["vs"] if st["kind"] == "tensor" else torch.ones(()))
                if st["kind"] == "block":
                    j = torch.arange(c + n)
                    page = st["table"][r].long()[j // BS]
                    vs = st["vs"][torch.where(page < st["vs"].shape[0], page, 0), h // G].double()
                    codes = vh.abs() / vs[:, None]
                    top = vs[(s + torch.log(vs)).argmax(-1)][:, None]
                else:
                    top = st["vs"]
                sumv = 2.0 ** -22 * top * (seen.double() @ codes)
            elif st["kind"] == "tensor":
                e = e + 2.0 ** -25 * scale * (kh.abs().sum(-1).max() + q.abs().sum(-1))
                sumv = 2.0 ** -25 * (seen.double() @ vh.abs())
            rows = slice(row, row + n)
            out[rows, h], lse[rows, h], ltol[rows, h] = o, z, e
            more = (c + n) * 2.0 ** -23 + (2.0 ** -11 if st["kind"] == "tensor" else 0.0)
            tol[rows, h] = U * o.abs() + (U + 2 * e[:, None] + more) * A + sumv
        row += n
    return out, lse, tol, ltol


def on_gpu(st):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in st.items()}


def call(st, which, **more):
    """One call; out and lse start at a pattern that rows no request owns have to keep."""
    import paged_kv_attention_reshape_gb300 as pkv
    g = on_gpu(st)
    out = torch.full_like(g["q"], 7.0)
    lse = torch.full(g["q"].shape[:2], 7.0, dtype=torch.float32, device="cuda")
    kw = dict(window=st["window"], sinks=st["sinks"], out=out, lse=lse, **more)
    if st["kind"] in ("tensor", "block"):
        kw.update(k_scale=g["ks"], v_scale=g["vs"])
    max_len, max_new = max(1, int(st["lens"].max())), max(1, max(n for _, n in st["reqs"]))
    if which == "decode":
        pkv.paged_decode_attn(g["q"], g["kc"], g["vc"], g["table"], g["lens"], max_len, cu_q=g["cu"], **kw)
    elif which == "extend":
        pkv.extend_attn(g["q"], g["k_new"], g["v_new"], g["cu"], g["lens"], g["kc"], g["vc"], g["table"], max_new, max_len, **kw)
    else:
        pkv.varlen_prefill_attn(g["q"], g["k_new"], g["v_new"], g["cu"], max_new, **kw)
    assert pkv.device_errors() == 0
    return out.cpu(), lse.cpu()


def check(got, ref, T):
    (out, lse), (o, z, tol, ltol) = got, ref
    assert torch.all(out[T:] == 7.0) and torch.all(lse[T:] == 7.0), "rows behind the last sequence"
    out, lse = out[:T].double(), lse[:T].double()
    none = torch.isneginf(z)
    assert torch.equal(none, torch.isneginf(lse)), "rows that see nothing"
    assert torch.all(out[none] == 0)
    bad = ~((out - o).abs() <= tol)
    bad[none] = False
    assert not bad.any(), (int(bad.sum()), float(((out - o).abs() / tol)[bad].nan_to_num(1e9).max()), bad.nonzero()[:4].tolist())
    lbad = ~((lse - z).abs() <= ltol) & ~none
    assert not lbad.any(), (float(((lse - z).abs() / ltol)[lbad].nan_to_num(1e9).max()), lbad.nonzero()[:4].tolist())


# ---- refusals (no GPU) ----------------------------------------------------------------------------

def test_refusals():
    from paged_kv_attention_reshape_gb300 import _lib, binding
    lib = _lib.load()
    fake = ctypes.c_void_p(1 << 20)  # never read: every call fails its host checks first
    c = _lib.PkvCache(fake, fake, 10, 16, 2, 128, 16 * 2 * 128)
    reqs = _lib.PkvReqs(None, None, 0, 4, 4)

    def decode(window, sinks, cache=c, Hq=4, ws=None, n=0):
        return lib.pkv_window_decode_attn(fake, cache, fake, 4, fake, None, reqs, Hq, 64, window, sinks, 1.0, fake, None, ws, n, None)

    def extend(window, sinks, cache=c, Hq=4):
        return lib.pkv_window_extend_attn(fake, fake, fake, 8, fake, fake, cache, fake, 4, reqs, Hq, 8, 64, window, sinks, 1.0, fake,
                                          None, None, 0, None)

    def prefill(window, sinks, D=128, Hq=4):
        return lib.pkv_window_prefill_attn(fake, fake, fake, 8, fake, reqs, Hq, 2, D, 8, window, sinks, 1.0, fake, None, None)

    for f in (decode, extend, prefill):
        assert f(0, 0) == 1 and f(-3, 0) == 1 and f(5, -1) == 1
        assert f(5, 0, Hq=6) == 2
    assert prefill(5, 0, D=96) == 2
    assert decode(5, 0) == 3  # no workspace
    # caches that windowed calls do not read
    scaled = _lib.PkvCache(fake, fake, 10, 16, 2, 128, 16 * 2 * 128, _lib.KV_FP8_E4M3_BLOCK, 1.0, 1.0, fake, fake)
    fp8_64 = _lib.PkvCache(fake, fake, 10, 16, 2, 64, 16 * 2 * 64, _lib.KV_FP8_E4M3, 1.0, 1.0)
    block32 = _lib.PkvCache(fake, fake, 10, 32, 2, 128, 32 * 2 * 128)
    for cache in (fp8_64, block32):
        assert decode(5, 0, cache) == 2 and extend(5, 0, cache) == 2
    assert decode(5, 0, scaled) == 3 and extend(5, 0, scaled) == 2
    # the binding's arguments
    with pytest.raises(binding.PkvError):
        binding._window(None, 4)
    assert binding._window(None, 0) is None and binding._window(7, 2) == (7, 2) and binding._window(1 << 40, 0) == (2 ** 31 - 1, 0)


def test_the_plain_form_by_hand():
    """The mask of a row: the window, the sinks, both, neither beyond the row."""
    m = seen_mask(torch.tensor([0, 5, 9]), torch.arange(10), 3, 2)
    assert m.int().tolist() == [[1, 0, 0, 0, 0, 0, 0, 0, 0, 0], [1, 1, 0, 1, 1, 1, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0, 0, 1, 1, 1]]


# ---- decode --------------------------------------------------------------------------------------------

LENS = [0, 1, 2, 15, 16, 17, 31, 33, 100, 127, 129, 260, 300]


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (16, 0), (17, 16), (64, 4), (100, 17), (128, 130), (260, 0), (5000, 3)])
@pytest.mark.parametrize("kind,D,Hq,Hkv", [("bf16", 64, 8, 2), ("bf16", 128, 16, 1), ("tensor", 128, 6, 3), ("bf16", 128, 5, 5),
                                           ("tensor", 128, 32, 2), ("block", 128, 16, 2), ("block", 128, 16, 1)])
def test_decode(kind, D, Hq, Hkv, window, sinks):
    st = make([(n - 1, 1) if n else (-1, 1) for n in LENS], Hq, Hkv, D, kind, window, sinks, 3, cached_all=True)
    check(call(st, "decode"), reference(st, decode=True), st["T"])


@pytest.mark.gpu
@pytest.mark.parametrize("kind,D,Hq,Hkv", [("bf16", 128, 64, 8), ("tensor", 128, 64, 8), ("bf16", 64, 16, 4), ("block", 128, 32, 8)])
@pytest.mark.parametrize("lens,window,sinks", [([9000], 4096, 64), ([5000, 40, 7001], 3001, 5), ([700] * 40, 500, 0)])
def test_decode_cut_sequences(kind, D, Hq, Hkv, lens, window, sinks):
    """Few long windows: their blocks are cut into shares and merged."""
    st = make([(n - 1, 1) for n in lens], Hq, Hkv, D, kind, window, sinks, 5, cached_all=True)
    check(call(st, "decode"), reference(st, decode=True), st["T"])


@pytest.mark.gpu
def test_decode_many_requests():
    """More requests than a launch holds."""
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(1, 60, (1500,), generator=g).tolist()
    st = make([(n - 1, 1) for n in lens], 2, 1, 64, "bf16", 20, 3, 6, cached_all=True)
    check(call(st, "decode"), reference(st, decode=True), st["T"])


@pytest.mark.gpu
def test_a_wide_window_is_the_decode_without_one():
    import paged_kv_attention_reshape_gb300 as pkv
    st = make([(n, 1) for n in (0, 15, 16, 511, 2000)], 16, 2, 128, "bf16", 1 << 40, 0, 8, cached_all=True)
    out, lse = call(st, "decode")
    g = on_gpu(st)
    o, z = pkv.paged_decode_attn(g["q"][:st["T"]], g["kc"], g["vc"], g["table"], g["lens"], 2001)
    assert torch.equal(out[:st["T"]], o.cpu()) and torch.equal(lse[:st["T"]], z.cpu())


# ---- extend and prefill ---------------------------------------------------------------------------------

MIXES = {
    "short": [(0, 1), (0, 2), (15, 1), (16, 3), (17, 16), (1, 17), (0, 0), (40, 5)],
    "tiles": [(0, 127), (100, 129), (128, 128), (130, 64), (300, 1), (5, 300)],
    "long": [(1000, 40), (513, 260), (0, 700)],
}


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(1, 0), (2, 1), (16, 4), (33, 17), (100, 0), (128, 130), (129, 300), (400, 16), (100000, 0)])
@pytest.mark.parametrize("kind,D,Hq,Hkv", [("bf16", 64, 8, 2), ("bf16", 128, 16, 1), ("bf16", 128, 3, 3), ("tensor", 128, 16, 2),
                                           ("tensor", 128, 2, 1)])
@pytest.mark.parametrize("mix", list(MIXES))
def test_extend(mix, kind, D, Hq, Hkv, window, sinks):
    st = make(MIXES[mix], Hq, Hkv, D, kind, window, sinks, 11)
    check(call(st, "extend"), reference(st), st["T"])


def extend_with(st, workspace, nbytes):
    """A windowed extend over codes through the C call, with that much of a workspace."""
    import paged_kv_attention_reshape_gb300 as pkv
    from paged_kv_attention_reshape_gb300 import binding
    g = on_gpu(st)
    out, lse = torch.full_like(g["q"], 7.0), torch.full(g["q"].shape[:2], 7.0, device="cuda")
    p, R = (lambda t: t.data_ptr()), len(st["reqs"])
    cache = binding.make_cache(g["kc"], g["vc"], st["ks"], st["vs"])
    rc = pkv.load().pkv_window_extend_attn(
        p(g["q"]), p(g["k_new"]), p(g["v_new"]), g["q"].shape[0], p(g["cu"]), p(g["lens"]), cache, p(g["table"]), g["table"].shape[1],
        pkv.Reqs(R, R).c(), st["Hq"], max(n for _, n in st["reqs"]), int(st["lens"].max()), st["window"], st["sinks"],
        1.0 / math.sqrt(st["D"]), p(out), p(lse), workspace.data_ptr() if workspace is not None else None, nbytes,
        torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and pkv.device_errors() == 0
    return out.cpu(), lse.cpu()


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(1800, 0), (1750, 130), (2000, 1000), (1700, 40), (100000, 0), (1, 2400)])
@pytest.mark.parametrize("Hq,Hkv,reqs", [(32, 2, [(0, 64), (100, 63), (33, 730), (2500, 1), (2016, 300), (0, 0), (1700, 80), (5, 600)]),
                                         (32, 4, [(2311, 1999)]), (48, 3, [(1000, 700), (31, 3), (0, 127), (2400, 600)])])
def test_extend_converted_ahead(Hq, Hkv, reqs, window, sinks):
    """Requests of many new tokens from rows that were converted once, the others beside them: with room for all of them, for a
    part and for none, whatever the workspace held."""
    import paged_kv_attention_reshape_gb300 as pkv
    st = make(reqs, Hq, Hkv, 128, "tensor", window, sinks, 17)
    need = pkv.window_extend_workspace_size(st["q"].shape[0], len(reqs), max(n for _, n in reqs), int(st["lens"].max()), Hq, Hkv, 128,
                                            window, sinks)
    assert need > 0 and need % (2 * 16 * Hkv * 128 * 2) == 0
    ref = reference(st)
    check(extend_with(st, None, 0), ref, st["T"])
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for n in (need, need // 2, 5):
        ws.fill_(0xFF)  # NaN
        check(extend_with(st, ws, min(n, need)), ref, st["T"])
    check(call(st, "extend"), ref, st["T"])


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (65, 0), (128, 130), (300, 16), (100000, 0)])
@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 4), (128, 8, 1), (64, 32, 2), (128, 4, 2)])
@pytest.mark.parametrize("lens", [[1, 2, 16, 0, 17], [127, 129, 300], [900]])
def test_prefill(lens, D, Hq, Hkv, window, sinks):
    st = make([(0, n) for n in lens], Hq, Hkv, D, "none", window, sinks, 12)
    check(call(st, "prefill"), reference(st), st["T"])


@pytest.mark.gpu
def test_extend_many_requests():
    """More requests than a launch holds, in a set of its own order."""
    import paged_kv_attention_reshape_gb300 as pkv
    g = torch.Generator().manual_seed(2)
    reqs = [(int(c), int(n)) for c, n in zip(torch.randint(0, 90, (600,), generator=g), torch.randint(1, 9, (600,), generator=g))]
    st = make(reqs, 4, 1, 64, "bf16", 20, 3, 6)
    order = torch.randperm(600, generator=g).to(torch.int32).cuda()
    check(call(st, "extend", reqs=pkv.Reqs(600, 600, order=order)), reference(st), st["T"])


@pytest.mark.gpu
def test_large_scores():
    """Scores whose maximum grows far along the keys (sums are rescaled), and far below it."""
    st = make([(400, 60), (0, 500)], 8, 2, 128, "bf16", 300, 20, 13)
    st["q"] *= 6
    check(call(st, "extend"), reference(st), st["T"])
    st = make([(n - 1, 1) for n in (500, 30, 900)], 8, 2, 128, "bf16", 300, 20, 14, cached_all=True)
    st["q"] *= 6
    check(call(st, "decode"), reference(st, decode=True), st["T"])


# ---- used together -------------------------------------------------------------------------------------

@pytest.mark.gpu
def test_chunks_then_decode():
    """A prompt in chunks, each appended to the cache, then decoded: every row as in one prefill of all tokens; pages
    that slide out of the window are given back (their table entries go out of range) between the calls."""
    import paged_kv_attention_reshape_gb300 as pkv
    window, sinks, Hq, Hkv, D = 70, 5, 8, 2, 128
    n, steps = 333, [100, 100, 100, 1, 30, 1, 1]
    st = make([(0, n)], Hq, Hkv, D, "none", window, sinks, 21, pad=0)
    whole = call(st, "prefill")
    ref = reference(st)
    check(whole, ref, n)
    g = on_gpu(st)
    nb = (n + BS - 1) // BS
    kc, vc = (torch.full((nb + 2, BS, Hkv, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(4)).to(torch.int32)
    full = perm[None].cuda()
    at = 0
    outs, lses = [], []
    for m in steps:
        q, k, v = (g[x][at:at + m].contiguous() for x in ("q", "k_new", "v_new"))
        pos = torch.arange(at, at + m, device="cuda")
        slot = full[0].long()[pos // BS] * BS + pos % BS
        pkv.kv_cache_write(k, v, slot, kc, vc)
        b = torch.arange(nb, device="cuda")
        first = max(0, at - window + 1)
        table = torch.where((b * BS < sinks) | (b * BS + BS - 1 >= first), full, torch.full_like(full, -7))
        lens = torch.tensor([at + m], dtype=torch.int32, device="cuda")
        if m == 1:
            o, z = pkv.paged_decode_attn(q, kc, vc, table, lens, at + 1, window=window, sinks=sinks)
        else:
            cu = torch.tensor([0, m], dtype=torch.int32, device="cuda")
            o, z = pkv.extend_attn(q, k, v, cu, lens, kc, vc, table, m, at + m, window=window, sinks=sinks)
        outs.append(o)
        lses.append(z)
        at += m
    assert at == n and pkv.device_errors() == 0
    check((torch.cat(outs).cpu(), torch.cat(lses).cpu()), ref, n)


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["decode", "extend", "prefill"])
def test_captured_and_on_another_stream(which):
    """Captured into a graph and replayed for other inputs; and on a stream of its own: the bits of a direct call."""
    import paged_kv_attention_reshape_gb300 as pkv
    kind = "none" if which == "prefill" else "bf16"
    mix = [(0, 200), (0, 77)] if which == "prefill" else [(3000, 1), (90, 1)] if which == "decode" else [(500, 40), (30, 300)]
    a, b = (make(mix, 8, 2, 128, kind, 150, 9, s, cached_all=which == "decode", pad=0) for s in (31, 32))
    want = [call(x, which) for x in (a, b)]
    side = torch.cuda.Stream()
    got = call(a, which, stream=side)
    assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[0][1])
    g = on_gpu(a)
    out, lse = torch.zeros_like(g["q"]), torch.zeros(g["q"].shape[:2], dtype=torch.float32, device="cuda")
    kw = dict(window=150, sinks=9, out=out, lse=lse)
    max_len, max_new = int(a["lens"].max()), max(n for _, n in mix)
    if which == "decode":
        ws = torch.empty(pkv.paged_decode_workspace_size(2, 8, 2, 128, max_len), dtype=torch.uint8, device="cuda")
        run = lambda: pkv.paged_decode_attn(g["q"], g["kc"], g["vc"], g["table"], g["lens"], max_len, workspace=ws, **kw)
    elif which == "extend":
        run = lambda: pkv.extend_attn(g["q"], g["k_new"], g["v_new"], g["cu"], g["lens"], g["kc"], g["vc"], g["table"], max_new,
                                      max_len, **kw)
    else:
        run = lambda: pkv.varlen_prefill_attn(g["q"], g["k_new"], g["v_new"], g["cu"], max_new, **kw)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for x, w in ((b, want[1]), (a, want[0]), (b, want[1])):
        for k in ("q", "k_new", "v_new", "kc", "vc", "table", "lens", "cu"):
            g[k].copy_(x[k])
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), w[0]) and torch.equal(lse.cpu(), w[1])
    assert pkv.device_errors() == 0


@pytest.mark.gpu
def test_bad_pages_and_lengths_are_flagged():
    """A page out of range among those that are read, and a length beyond the table, set their bits and touch nothing else."""
    import paged_kv_attention_reshape_gb300 as pkv
    st = on_gpu(make([(60, 1), (40, 1)], 4, 2, 128, "bf16", 40, 0, 3, cached_all=True, pad=0))
    table = st["table"].clone()
    table[0, 3] = 10 ** 6
    pkv.paged_decode_attn(st["q"], st["kc"], st["vc"], table, st["lens"], 64, window=40)
    assert pkv.device_errors() == 2
    long = st["lens"].clone()
    long[1] = 10 ** 6
    full = torch.zeros_like(table)
    pkv.paged_decode_attn(st["q"], st["kc"], st["vc"], full, long, 64, window=40)
    assert pkv.device_errors() == 8
    ex = on_gpu(make([(60, 3), (40, 2)], 4, 2, 128, "bf16", 40, 0, 3, pad=0))
    table = ex["table"].clone()
    table[0, 3] = -5
    pkv.extend_attn(ex["q"], ex["k_new"], ex["v_new"], ex["cu"], ex["lens"], ex["kc"], ex["vc"], table, 3, 64, window=40)
    assert pkv.device_errors() == 2


@pytest.mark.gpu
def test_refused_by_the_binding():
    import paged_kv_attention_reshape_gb300 as pkv
    st = on_gpu(make([(60, 1)], 4, 2, 128, "tensor", 40, 0, 3, cached_all=True, pad=0))
    s = torch.ones((st["kc"].shape[0], 2), device="cuda")
    a = (st["q"], st["kc"], st["vc"], st["table"], st["lens"], 64)
    for kw in (dict(window=0), dict(window=-1), dict(window=4, sinks=-1), dict(sinks=3)):
        with pytest.raises(pkv.PkvError):
            pkv.paged_decode_attn(*a, **kw)
    with pytest.raises(pkv.PkvError):  # extend over block scales has no window
        cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        pkv.extend_attn(st["q"], st["k_new"], st["v_new"], cu, st["lens"], st["kc"], st["vc"], st["table"], 1, 64, window=4,
                        k_scale=s, v_scale=s)


@pytest.mark.gpu
def test_tensors_of_other_shapes_are_refused():
    import paged_kv_attention_reshape_gb300 as pkv
    st = on_gpu(make([(60, 3), (40, 2)], 4, 2, 128, "bf16", 40, 0, 3, pad=0))
    a = dict(q=st["q"], k=st["k_new"], v=st["v_new"], cu=st["cu"], lens=st["lens"], table=st["table"])

    def extend(out=None, lse=None, **x):
        t = {**a, **x}
        pkv.extend_attn(t["q"], t["k"], t["v"], t["cu"], t["lens"], st["kc"], st["vc"], t["table"], 3, 64, window=9, out=out, lse=lse)

    def decode(out=None, lse=None, **x):
        t = {**a, **x}
        pkv.paged_decode_attn(t["q"][:2], st["kc"], st["vc"], t["table"], t["lens"], 64, window=9, out=out, lse=lse)

    def prefill(out=None, lse=None, **x):
        t = {**a, **x}
        pkv.varlen_prefill_attn(t["q"], t["k"], t["v"], t["cu"], 3, window=9, out=out, lse=lse)

    bad = dict(q=st["q"][:, :, :64].contiguous(), k=st["k_new"][:3], v=st["v_new"][:, :1], cu=st["cu"][:2], lens=st["lens"].long(),
               table=st["table"][:1])
    for f, names in ((extend, bad), (decode, ("q", "lens", "table")), (prefill, ("k", "v"))):
        f()
        for n in names:
            with pytest.raises(pkv.PkvError):
                f(**{n: bad[n]})
        for o in (dict(out=torch.empty((1, 4, 128), dtype=torch.bfloat16, device="cuda")), dict(lse=torch.empty((9, 4), device="cuda"))):
            with pytest.raises(pkv.PkvError):
                f(**o)
    assert pkv.device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "tensor"])
def test_keys_and_values_in_one_allocation(kind):
    """[num_blocks, 2, ...]: K and V blocks alternate, and the pool's pages lie two blocks apart."""
    import paged_kv_attention_reshape_gb300 as pkv
    for which, mix in (("decode", [(300, 1), (17, 1)]), ("extend", [(300, 40), (17, 3)])):
        st = make(mix, 8, 2, 128, kind, 150, 9, 41, cached_all=which == "decode")
        want = call(st, which)
        both = torch.stack([st["kc"], st["vc"]], 1)
        st["kc"], st["vc"] = both[:, 0], both[:, 1]
        g = both.cuda()
        one = dict(st, kc=g[:, 0], vc=g[:, 1])
        got = call(one, which)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_two_calls_at_once():
    """Extends and decodes on two streams beside one another, each with what is its own: the bits of calls alone."""
    import paged_kv_attention_reshape_gb300 as pkv
    cases = [make([(700, 90), (30, 300), (0, 400)], 16, 2, 128, "bf16", 200, 9, s, pad=0) for s in (51, 52)]
    want = [call(c, "extend") for c in cases]
    g = [on_gpu(c) for c in cases]
    outs = [[torch.empty_like(x["q"]) for _ in range(20)] for x in g]
    streams = [torch.cuda.Stream() for _ in g]
    torch.cuda.synchronize()
    for i in range(20):
        for x, o, s in zip(g, outs, streams):
            with torch.cuda.stream(s):
                pkv.extend_attn(x["q"], x["k_new"], x["v_new"], x["cu"], x["lens"], x["kc"], x["vc"], x["table"], 400, 800,
                                window=200, sinks=9, out=o[i])
    torch.cuda.synchronize()
    assert pkv.device_errors() == 0
    for o, w in zip(outs, want):
        assert all(torch.equal(x.cpu(), w[0]) for x in o)
