"""Windowed calls at the ends of what their numbers may be: windows and sinks up to 2^31 - 1, beside caches whose last block is
partly filled. The reference and its tolerances are those of test_window.py."""
import math

import pytest
import torch

from test_window import call, check, extend_with, make, on_gpu, reference

MOST = 2 ** 31 - 1
# cached lengths that end inside a block, and new tokens that cross a group of 32 walk columns
PARTLY = [(1, 20), (17, 3), (22, 70), (2001, 45), (15, 300), (31, 1), (0, 33), (16, 40)]
ENDS = [(MOST, 0), (1 << 40, 0), (MOST, 5), (MOST - 7, 0), (MOST - 15, 18), (MOST - 16, 0), (MOST - 40, 0), (MOST, MOST), (9, MOST),
        (1, 1 << 40)]


def test_numbers_beyond_32_bits():
    """Larger windows and sinks are the largest there are; numbers far below zero stay below it (none may wrap around)."""
    import paged_kv_attention_reshape_gb300 as pkv
    from paged_kv_attention_reshape_gb300 import binding
    assert binding._window(1 << 40, (1 << 32) + 5) == (MOST, MOST) and binding._window(MOST, 0) == (MOST, 0)
    for x in (5 - (1 << 32), -(1 << 40), -1):
        window, sinks = binding._window(x, x)
        assert -2 ** 31 <= window < 1 and -2 ** 31 <= sinks < 0
    size = lambda window, sinks: pkv.window_extend_workspace_size(2048, 1, 2048, 100000, 64, 8, 128, window, sinks)
    assert size(1 << 40, 0) == size(MOST, 0) > 0 and size((1 << 32) + 1, 4) == size(MOST, 4) > 0
    assert size(4096, 1 << 40) == size(4096, MOST) > 0
    assert size(5 - (1 << 32), 0) == 0 and size(4096, 4 - (1 << 32)) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", ENDS)
@pytest.mark.parametrize("kind,D,Hq,Hkv", [("bf16", 64, 8, 2), ("bf16", 128, 16, 1), ("bf16", 128, 2, 2), ("tensor", 128, 16, 2)])
def test_extend_under_the_widest_windows(kind, D, Hq, Hkv, window, sinks):
    st = make(PARTLY, Hq, Hkv, D, kind, window, sinks, 91)
    check(call(st, "extend"), reference(st), st["T"])


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [e for e in ENDS if max(e) <= MOST])
def test_extend_converted_ahead_under_the_widest_windows(window, sinks):
    """A request of the rows that were converted once, beside short ones that are read as codes."""
    import paged_kv_attention_reshape_gb300 as pkv
    st = make([(2001, 700), (17, 600), (1, 20), (22, 70)], 48, 3, 128, "tensor", window, sinks, 92)
    need = pkv.window_extend_workspace_size(st["q"].shape[0], 4, 700, int(st["lens"].max()), 48, 3, 128, window, sinks)
    assert need > 0
    ref = reference(st)
    check(extend_with(st, torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda"), need), ref, st["T"])
    check(extend_with(st, None, 0), ref, st["T"])


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", ENDS)
def test_prefill_and_decode_under_the_widest_windows(window, sinks):
    st = make([(0, n) for n in (1, 17, 300, 45)], 16, 2, 128, "none", window, sinks, 93)
    check(call(st, "prefill"), reference(st), st["T"])
    for kind in ("bf16", "tensor", "block"):
        st = make([(c, 1) for c in (0, 1, 16, 22, 2001)], 16, 2, 128, kind, window, sinks, 94, cached_all=True)
        check(call(st, "decode"), reference(st, decode=True), st["T"])


@pytest.mark.gpu
@pytest.mark.parametrize("kind,D", [("bf16", 64), ("bf16", 128), ("tensor", 128)])
def test_the_widest_window_is_the_widest_but_one(kind, D):
    """Windows that no row reaches the end of are alike to the bit, whatever their number."""
    st = make(PARTLY, 16, 2, D, kind, 100000, 0, 95)
    want = call(st, "extend")
    for window in (MOST, MOST - 9, 1 << 40):
        st["window"] = window
        got = call(st, "extend")
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("ahead", [False, True])
@pytest.mark.parametrize("reqs,Hq,Hkv", [([(2400, 600)], 48, 3), ([(3001, 700), (2990, 5)], 32, 2)])
def test_small_terms_add_up(reqs, Hq, Hkv, ahead):
    """Over an 8-bit cache P is fp16, with steps of 2^-24 below 2^-14. One key 2^26 times the others' weight, with value 0, and
    thousands of others: out is theirs alone. The row's largest P is 2^8 at least, so each p is off by 2^-33 at most from the steps:
    2^-33 sum |v| in the place of the 2^-25 sum |v| that test_window.py allows."""
    import paged_kv_attention_reshape_gb300 as pkv
    st = make(reqs, Hq, Hkv, 128, "tensor", 5000, 0, 96)
    for n in ("q", "k_new", "v_new"):
        st[n][:st["T"]] = 0
    st["q"][:st["T"], :, 0] = 10240.0  # times 0.02 / sqrt(128): 18.1, or 2^26.1
    st["v_new"][:st["T"]] = 0.03
    held = st["kc"] != 0x7F  # (NaN: tokens that no row sees)
    st["kc"][held] = 0x00
    st["vc"][held] = 0x38  # 1.0
    for r in range(len(reqs)):
        page = int(st["table"][r, 0])
        st["kc"][page, 0, :, 0] = 0x38
        st["vc"][page, 0] = 0x00
    if ahead:
        need = pkv.window_extend_workspace_size(st["q"].shape[0], len(reqs), max(n for _, n in reqs), int(st["lens"].max()), Hq, Hkv,
                                                128, 5000)
        assert need > 0
        got = extend_with(st, torch.empty(need, dtype=torch.uint8, device="cuda"), need)
    else:
        got = extend_with(st, None, 0)
    o, z, tol, ltol = reference(st)
    row = 0
    code, new = float(torch.tensor(st["vs"])), float(st["v_new"][0, 0, 0])
    for c, n in reqs:
        sumv = (c - 1) * code + new * torch.arange(1, n + 1, dtype=torch.float64)[:, None, None]
        tol[row:row + n] -= (2.0 ** -25 - 2.0 ** -33) * sumv
        row += n
    assert (tol[:st["T"]] > 0).all() and (tol < 0.05 * o)[:st["T"]].all()
    check(got, (o, z, tol, ltol), st["T"])


@pytest.mark.gpu
@pytest.mark.parametrize("which,D", [("extend", 128), ("extend", 64), ("prefill", 128)])
def test_the_largest_values(which, D):
    """Scores that rise by nearly 2^20 after the first key tile, which a row's m does not follow, over values of 2^108 by the
    number of keys: 2^99 for up to 400 of them."""
    mix = [(0, 400)] if which == "prefill" else [(300, 100), (0, 390)]
    st = make(mix, 16, 2, D, "none" if which == "prefill" else "bf16", 1000, 0, 97)
    T = st["T"]
    st["q"][:T] = 0
    st["q"][:T, :, 0] = 19.9 * math.sqrt(D) / math.log2(math.e)
    assert float(st["q"][0, 0, 0]) / math.sqrt(D) * math.log2(math.e) < 20
    st["k_new"][:T] = 0
    st["v_new"][:T] = 2.0 ** 99
    row = 0
    for r, (c, n) in enumerate(mix):
        at = torch.arange(c, c + n)
        st["k_new"][row:row + n, :, 0] = (at >= 128).to(torch.bfloat16)[:, None]
        for j in range(c):
            page = st["table"][r, j // 16]
            st["kc"][page, j % 16] = 0
            st["kc"][page, j % 16, :, 0] = float(j >= 128)
            st["vc"][page, j % 16] = 2.0 ** 99
        row += n
    check(call(st, which), reference(st), T)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv", [(48, 3), (64, 8)])
def test_requests_of_an_item_of_rows(Hq, Hkv):
    """Requests of one row less than an item of 256 rows a KV head, of an item, of one more: the former are read as codes."""
    import paged_kv_attention_reshape_gb300 as pkv
    t = 256 * Hkv // Hq
    reqs = [(300, t - 1), (2400, 900), (300, t), (317, t + 1), (5, t), (0, t), (40, 1)]
    st = make(reqs, Hq, Hkv, 128, "tensor", 3000, 5, 98)
    need = pkv.window_extend_workspace_size(st["q"].shape[0], len(reqs), 900, 3300, Hq, Hkv, 128, 3000, 5)
    assert need > 0
    ref = reference(st)
    for n in (need, need // 3):
        check(extend_with(st, torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda"), n), ref, st["T"])
    check(extend_with(st, None, 0), ref, st["T"])


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["key", "value"])
@pytest.mark.parametrize("kind,D,Hq,Hkv", [("bf16", 64, 8, 2), ("bf16", 128, 32, 2), ("tensor", 128, 16, 2), ("block", 128, 16, 2)])
@pytest.mark.parametrize("lens", [[40, 200, 33], [9000, 40, 9000]])
def test_decode_over_what_is_no_number(lens, kind, D, Hq, Hkv, which):
    """A key that the token sees and that is no number makes its KV head's rows of that request none, out and lse; a value makes its
    column of out one, and nothing else. Sequences of one piece, and cut ones."""
    st = make([(n - 1, 1) for n in lens], Hq, Hkv, D, kind, 5000, 3, 99, cached_all=True)
    ref = reference(st, decode=True)
    at = lens[0] - 30  # a key in the window
    page = int(st["table"][0, at // 16])
    (st["kc"] if which == "key" else st["vc"])[page, at % 16, 1, 5] = 0x7F if kind in ("tensor", "block") else math.nan
    out, lse = call(st, "decode")
    G = Hq // Hkv
    if which == "key":
        assert torch.isnan(out[0, G:]).all() and torch.isnan(lse[0, G:]).all()
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[0, G:] = True
        lse[0, G:] = ref[1][0, G:].float()
    else:
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[0, G:, 5] = True
        assert torch.isnan(out[hit]).all()
    assert not torch.isnan(out[~hit]).any()
    out = torch.where(hit, torch.cat([ref[0], torch.full_like(out[len(lens):], 7.0).double()]).to(out.dtype), out)
    check((out, lse), ref, st["T"])


@pytest.mark.gpu
@pytest.mark.parametrize("kind,D", [("none", 64), ("bf16", 128), ("tensor", 128)])
@pytest.mark.parametrize("n", [20, 200])
def test_new_keys_that_are_no_number(n, kind, D):
    """Extend and prefill: the rows that see such a key are none (others of the request may be), other KV heads and requests are as
    without it."""
    c = 0 if kind == "none" else 70
    st = make([(c, n), (0, 33)], 16, 2, D, kind, 100, 3, 100)
    ref = reference(st)
    st["k_new"][n // 2, 1, 7] = math.nan
    out, lse = call(st, "prefill" if kind == "none" else "extend")
    see = [i for i in range(n) if i >= n // 2 and i - n // 2 < 100]
    assert torch.isnan(out[see, 8:]).all() and torch.isnan(lse[see, 8:]).all()
    out[:n, 8:], lse[:n, 8:] = ref[0][:n, 8:].to(out.dtype), ref[1][:n, 8:].float()
    check((out, lse), ref, st["T"])


@pytest.mark.gpu
def test_converted_ahead_from_one_allocation_in_a_set_of_its_own():
    """Rows converted once from a pool whose K and V blocks alternate, for requests named by the device, one of them twice."""
    import paged_kv_attention_reshape_gb300 as pkv
    reqs = [(2001, 700), (17, 600), (1, 20), (300, 16), (900, 1)]
    st = make(reqs, 48, 3, 128, "tensor", 1900, 9, 101)
    T = st["q"].shape[0]
    assert pkv.window_extend_workspace_size(T, 6, 700, int(st["lens"].max()), 48, 3, 128, 1900, 9) > 0
    g = torch.stack([st["kc"], st["vc"]], 1).cuda()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ref = reference(st)
    check(call(dict(st, kc=g[:, 0], vc=g[:, 1]), "extend", reqs=pkv.Reqs(6, 5, order=i32(3, 1, 0, 4, 1, 2))), ref, st["T"])
    check(call(dict(st, kc=g[:, 0], vc=g[:, 1]), "extend", reqs=pkv.Reqs(6, 5, order=i32(4, 0, 3, 2, 1, 9), bounds=i32(0, 0, 5, 5), cls=1)),
          ref, st["T"])
