"""The calls of test_window.py, test_append_norm.py and test_kv_block_copy.py at the ends of what they allow: pages more than
2^32 bytes into a pool, request sets named by the device, sets that are empty or hold a request twice, nothing to do, graphs
that run beside one another, and launches that have no work-item counter of their own."""
import os
import subprocess
import sys

import pytest
import torch

from test_window import BS, call, check, make, on_gpu, reference

pytestmark = pytest.mark.gpu


def far(st, nb, at):
    """The state with its pages moved to ids `at` + their own of a pool of nb pages, all others unwritten."""
    g = on_gpu(st)
    held = g["kc"].shape[0]
    for n in ("kc", "vc"):
        pool = torch.empty((nb, *g[n].shape[1:]), dtype=g[n].dtype, device="cuda")
        pool[at:at + held] = g[n]
        g[n] = pool
    g["table"] = torch.where(g["table"] < held, g["table"] + at, g["table"])
    return g


@pytest.mark.parametrize("kind", ["bf16", "tensor"])
def test_pages_beyond_32_bits(kind):
    """8 KV heads of 128: a page is 2^15 bytes (codes: 2^14), so page 2^17 (2^18) is 2^32 bytes in, and 2^31 elements are
    passed at 2^17 in both."""
    first = 2 ** 18 + 5 if kind == "tensor" else 2 ** 17 + 5
    for which, mix in (("decode", [(300, 1), (17, 1), (4000, 1)]), ("extend", [(300, 40), (17, 3), (2000, 260)])):
        st = make(mix, 16, 8, 128, kind, 150, 9, 61, cached_all=which == "decode")
        ref = reference(st, decode=which == "decode")
        check(call(far(st, first + st["kc"].shape[0], first), which), ref, st["T"])


def test_pages_beyond_32_bits_appended_and_copied():
    import paged_kv_attention_reshape_gb300 as pkv
    Hq, Hkv, D, nb, first = 16, 8, 128, 2 ** 17 + 40, 2 ** 17 + 7
    kc, vc = (torch.empty((nb, BS, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in "kv")
    q, k, v = (torch.randn((100, h, D), device="cuda").to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    w = torch.rand(D, device="cuda") + 0.5
    near = [torch.zeros((10, BS, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    slot = torch.arange(100, device="cuda")
    for caches, off in ((near, 0), ((kc, vc), first * BS)):
        out = pkv.kv_append(q, k, v, None, slot + off, *caches, q_norm=w, k_norm=w)
    for c, n in zip((kc, vc), near):
        assert torch.equal(c[first:first + 6], n[:6]) and torch.equal(c[first + 6, :4], n[6, :4])
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    kc[first + 6, 4:], vc[first + 6, 4:] = 1, 2
    # (from far to near, from near to far, and far away in both)
    pkv.kv_block_copy(pkv.CacheLayers([kc], [vc]), i32(first, 3, first + 6), i32(3 + 1, first + 20, first + 30))
    assert torch.equal(kc[4], near[0][0]) and torch.equal(vc[4], near[1][0])
    for c in (kc, vc):
        assert torch.equal(c[first + 20].view(torch.int16), c[3].view(torch.int16)) and torch.equal(c[first + 30], c[first + 6])
    assert pkv.device_errors() == 0


def test_sets_named_by_the_device():
    """A mixed batch reordered on the device, each class through its windowed call: rows as if each request were alone."""
    import paged_kv_attention_reshape_gb300 as pkv
    Hq, Hkv, D, window, sinks = 16, 4, 128, 90, 7
    # prefills, extends and decodes in arrival order; decodes have their new token in the cache too
    reqs = [(0, 50), (200, 30), (77, 1), (0, 130), (300, 1), (16, 16), (511, 1)]
    R = len(reqs)
    ext = make(reqs, Hq, Hkv, D, "bf16", window, sinks, 71)
    ref = reference(ext)
    g = on_gpu(ext)
    # the cache of the decodes: the same pages and one more token
    table = torch.cat([g["table"], torch.zeros((R, 1), dtype=torch.int32, device="cuda")], 1)
    nb = g["kc"].shape[0]
    kc, vc = (torch.cat([g[n], torch.full((R, *g[n].shape[1:]), float("nan"), dtype=torch.bfloat16, device="cuda")]) for n in ("kc", "vc"))
    row = 0
    for r, (c, n) in enumerate(reqs):
        if n == 1:
            if c % BS == 0:
                table[r, c // BS] = nb + r
            kc[table[r, c // BS].long(), c % BS], vc[table[r, c // BS].long(), c % BS] = g["k_new"][row], g["v_new"][row]
        row += n
    table = table.contiguous()
    out, lse = torch.full_like(g["q"], 7.0), torch.full(g["q"].shape[:2], 7.0, device="cuda")
    perm, bounds, _, _ = pkv.batch_classify_reorder(g["cu"], g["lens"])
    of = lambda c, most=R: pkv.Reqs(most, R, order=perm, bounds=bounds, cls=c)
    kw = dict(window=window, sinks=sinks, out=out, lse=lse)
    pkv.paged_decode_attn(g["q"], kc, vc, table, g["lens"], 600, cu_q=g["cu"], reqs=of(pkv.CLASS_DECODE), **kw)
    pkv.extend_attn(g["q"], g["k_new"], g["v_new"], g["cu"], g["lens"], kc, vc, table, 130, 600, reqs=of(pkv.CLASS_EXTEND), **kw)
    pkv.varlen_prefill_attn(g["q"], g["k_new"], g["v_new"], g["cu"], 130, reqs=of(pkv.CLASS_PREFILL), **kw)
    assert pkv.device_errors() == 0
    check((out.cpu(), lse.cpu()), ref, ext["T"])
    # a set larger than the call's bound is cut and flagged
    out.fill_(7.0)
    pkv.extend_attn(g["q"], g["k_new"], g["v_new"], g["cu"], g["lens"], kc, vc, table, 130, 600, reqs=of(pkv.CLASS_EXTEND, 1), **kw)
    assert pkv.device_errors() == 4
    assert int((out[:, 0, 0] != 7.0).sum()) in (30, 16)


def test_empty_sets_and_a_request_twice():
    import paged_kv_attention_reshape_gb300 as pkv
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    st = make([(100, 20), (40, 300), (0, 5)], 8, 2, 128, "bf16", 60, 5, 81)
    twice = pkv.Reqs(5, 3, order=i32(1, 0, 1, 2, 1))
    check(call(st, "extend", reqs=twice), reference(st), st["T"])
    dec = make([(100, 1), (40, 1), (0, 1)], 8, 2, 128, "bf16", 60, 5, 82, cached_all=True)
    check(call(dec, "decode", reqs=pkv.Reqs(5, 3, order=i32(1, 0, 1, 2, 1))), reference(dec, decode=True), 3)
    none = pkv.Reqs(3, 3, order=i32(0, 1, 2), bounds=i32(2, 2, 2, 2), cls=1)
    for s, which in ((st, "extend"), (dec, "decode"), (st, "prefill")):
        for reqs in (none, pkv.Reqs(0, 3)):
            out, lse = call(s, which, reqs=reqs)
            assert torch.all(out == 7.0) and torch.all(lse == 7.0)
    # nothing to append, nothing to copy
    g = on_gpu(st)
    before = g["kc"].clone()
    w = torch.ones(128, device="cuda")
    slot = torch.zeros(0, dtype=torch.int64, device="cuda")
    pkv.kv_append(g["q"][:0], g["k_new"][:0], g["v_new"][:0], None, slot, g["kc"], g["vc"], q_norm=w, k_norm=w)
    pkv.kv_block_copy(pkv.CacheLayers([g["kc"]], [g["vc"]]), i32(), i32())
    assert torch.equal(g["kc"].view(torch.int16), before.view(torch.int16)) and pkv.device_errors() == 0


def test_tokens_that_are_not_there():
    """cu_q that counts more tokens than q has rows: those that it has are as in the whole batch. Offsets below zero: flagged, and
    nothing written."""
    import paged_kv_attention_reshape_gb300 as pkv
    for kind in ("bf16", "tensor"):
        st = make([(40, 3), (300, 200)], 16, 2, 128, kind, 60, 5, 83, pad=0)
        ref = reference(st)
        g = on_gpu(st)
        kw = dict(window=60, sinks=5, **(dict(k_scale=st["ks"], v_scale=st["vs"]) if kind == "tensor" else {}))
        for T in (203, 202, 100, 40, 3, 2):
            out, lse = pkv.extend_attn(g["q"][:T], g["k_new"][:T], g["v_new"][:T], g["cu"], g["lens"], g["kc"], g["vc"], g["table"], 200,
                                       500, **kw)
            assert pkv.device_errors() == 0
            check((out.cpu(), lse.cpu()), [x[:T] for x in ref], T)
        cu = g["cu"].clone()
        cu[0] = -5
        out = torch.full_like(g["q"], 7.0)
        pkv.extend_attn(g["q"], g["k_new"], g["v_new"], cu, g["lens"], g["kc"], g["vc"], g["table"], 200, 500, out=out, **kw)
        assert pkv.device_errors() == 8
        assert torch.all(out[:3] == 7.0) and torch.all((out[3:].double().cpu() - ref[0][3:]).abs() <= ref[2][3:])


def test_workspaces_and_rows_that_are_refused():
    import paged_kv_attention_reshape_gb300 as pkv
    st = make([(60, 1), (40, 1)], 4, 2, 128, "bf16", 40, 0, 3, cached_all=True, pad=0)
    g = on_gpu(st)
    a = (g["kc"], g["vc"], g["table"], g["lens"], 64)
    need = pkv.paged_decode_workspace_size(2, 4, 2, 128, 64)
    for q, ws in ((g["q"], torch.empty(need, dtype=torch.uint8)), (g["q"], torch.empty((need, 2), dtype=torch.uint8, device="cuda")[:, 0]),
                  (g["q"][:1], None)):
        with pytest.raises(pkv.PkvError):
            pkv.paged_decode_attn(q, *a, window=9, workspace=ws)
    order = torch.tensor([1, 0], dtype=torch.int32)
    for reqs in (pkv.Reqs(2, 2, order=order), pkv.Reqs(2, 2, order=order.cuda().long()), pkv.Reqs(3, 2, order=order.cuda()),
                 pkv.Reqs(2, 2, order=order.cuda(), bounds=order.cuda(), cls=1)):
        with pytest.raises(pkv.PkvError):
            pkv.paged_decode_attn(g["q"], *a, window=9, reqs=reqs)
        with pytest.raises(pkv.PkvError):
            pkv.varlen_prefill_attn(g["q"], g["k_new"], g["v_new"], g["cu"], 1, window=9, reqs=reqs)
    with pytest.raises(pkv.PkvError):
        pkv.extend_attn(g["q"], g["k_new"], g["v_new"], g["cu"], g["lens"], *a[:3], 1, 64, window=9, workspace=torch.empty(5))


def test_graphs_beside_one_another():
    """Two captured steps (an append with norms, an extend or a decode, a copy of pages), each with its own tensors, replayed
    on two streams at once beside direct calls on a third: the bits of the steps alone."""
    import paged_kv_attention_reshape_gb300 as pkv
    w = torch.rand(128, device="cuda") + 0.5

    def step(which, seed):
        mix = [(700, 1), (90, 1), (3000, 1)] if which == "decode" else [(500, 40), (30, 300)]
        st = make(mix, 8, 2, 128, "bf16", 150, 9, seed, cached_all=which == "decode", pad=0)
        g = on_gpu(st)
        qn, lse = torch.empty_like(g["q"]), torch.empty(g["q"].shape[:2], device="cuda")
        out, kn = torch.empty_like(g["q"]), torch.empty_like(g["k_new"])
        pool = [torch.zeros((30, BS, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        layers = pkv.CacheLayers([pool[0]], [pool[1]])
        src, dst = (torch.arange(a, a + 15, dtype=torch.int32, device="cuda") for a in (0, 15))
        slot = torch.arange(st["T"], device="cuda") % 240
        max_len, max_new = int(st["lens"].max()), max(n for _, n in mix)
        ws = torch.empty(pkv.paged_decode_workspace_size(3, 8, 2, 128, max_len), dtype=torch.uint8, device="cuda")
        kw = dict(window=150, sinks=9, out=out, lse=lse)

        def run():
            pkv.kv_append(g["q"], g["k_new"], g["v_new"], None, slot[:st["T"]], *pool, q_out=qn, k_out=kn, q_norm=w, k_norm=w)
            if which == "decode":
                pkv.paged_decode_attn(qn, g["kc"], g["vc"], g["table"], g["lens"], max_len, workspace=ws, **kw)
            else:
                pkv.extend_attn(qn, kn, g["v_new"], g["cu"], g["lens"], g["kc"], g["vc"], g["table"], max_new, max_len, **kw)
            pkv.kv_block_copy(layers, src, dst)
        # (slots are unique below 240 tokens only: of an extend's longer batch the pool is left out)
        return run, (out, lse, qn, *(pool if which == "decode" else ()))

    steps = [step("extend", 91), step("decode", 92), step("extend", 93)]
    want = []
    for run, res in steps:
        run()
        torch.cuda.synchronize()
        want.append([x.clone() for x in res])
    streams = [torch.cuda.Stream() for _ in steps]
    graphs = []
    for (run, _), s in zip(steps[:2], streams):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            run()
    torch.cuda.synchronize()
    for _ in range(30):
        for _, res in steps:
            res[0].fill_(7.0)
        torch.cuda.synchronize()
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        with torch.cuda.stream(streams[2]):
            steps[2][0]()
        torch.cuda.synchronize()
        for (_, res), ws in zip(steps, want):
            assert all(torch.equal(x, y) for x, y in zip(res, ws))
    assert pkv.device_errors() == 0


def test_rows_converted_ahead_in_more_requests_than_a_launch_holds():
    """Long requests in both launches of a set, short ones between them, in a set of its own order; the launches share the pool."""
    import paged_kv_attention_reshape_gb300 as pkv
    reqs = [(3500 + i, 300) if i % 50 == 7 else (i % 50, 1 + i % 3) for i in range(300)]
    st = make(reqs, 32, 2, 128, "tensor", 4000, 30, 95)
    assert pkv.window_extend_workspace_size(st["q"].shape[0], 300, 300, int(st["lens"].max()), 32, 2, 128, 4000, 30) > 0
    order = torch.randperm(300, generator=torch.Generator().manual_seed(3)).to(torch.int32).cuda()
    check(call(st, "extend", reqs=pkv.Reqs(300, 300, order=order)), reference(st), st["T"])


def test_rows_converted_ahead_captured_on_two_streams_and_bad_pages():
    """An extend that converts rows ahead: captured and replayed for other inputs beside a direct call on another stream, the
    bits of calls alone; and a bad page among those that it converts sets its bit."""
    import paged_kv_attention_reshape_gb300 as pkv
    mix = [(2000, 1000), (40, 1000)]
    a, b = (make(mix, 32, 2, 128, "tensor", 1900, 20, s, pad=0) for s in (96, 97))
    assert pkv.window_extend_workspace_size(2000, 2, 1000, 3000, 32, 2, 128, 1900, 20) > 0
    want = [call(x, "extend") for x in (a, b)]
    g, h = on_gpu(a), on_gpu(b)
    bufs = [(torch.empty_like(g["q"]), torch.empty(g["q"].shape[:2], device="cuda")) for _ in "gh"]

    def run(x, out, lse, **kw):
        pkv.extend_attn(x["q"], x["k_new"], x["v_new"], x["cu"], x["lens"], x["kc"], x["vc"], x["table"], 1000, 3000, window=1900,
                        sinks=20, k_scale=0.02, v_scale=0.03, out=out, lse=lse, **kw)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(g, *bufs[0])
    side = torch.cuda.Stream()
    for x, w in ((b, want[1]), (a, want[0])):
        for k in ("q", "k_new", "v_new", "kc", "vc", "table", "lens", "cu"):
            g[k].copy_(x[k])
        torch.cuda.synchronize()
        for _ in range(5):
            graph.replay()
            run(h, *bufs[1], stream=side)
        torch.cuda.synchronize()
        for (o, l), y in zip(bufs, (w, want[1])):
            assert torch.equal(o.cpu(), y[0]) and torch.equal(l.cpu(), y[1])
    assert pkv.device_errors() == 0
    h["table"][0, 100] = -9
    run(h, *bufs[1])
    assert pkv.device_errors() == 2


_MANY = """
import sys, torch
sys.path[:0] = ["tests", "."]
import paged_kv_attention_reshape_gb300 as pkv
from test_window import call, check, make, on_gpu, reference
one, cu1 = torch.ones((1, 1, 128), dtype=torch.bfloat16, device="cuda"), torch.tensor([0, 1], dtype=torch.int32, device="cuda")
out1, lse1 = torch.empty_like(one), torch.empty((1, 1), device="cuda")
fill = lambda: pkv.varlen_prefill_attn(one, one, one, cu1, 1, out=out1, lse=lse1, window=5)
fill()
torch.cuda.synchronize()
with torch.cuda.stream(torch.cuda.Stream()):
    graph = torch.cuda.CUDAGraph()
    graph.capture_begin()
    for _ in range(8200):
        fill()
    graph.capture_end()
del graph
for kind in ("bf16", "tensor"):
    # more items than CTAs, of very different lengths, split ones among them
    st = make([(900, 300)] * 5 + [(37 * i, 1 + i % 40) for i in range(150)], 8, 2, 128, kind, 200, 9, 7)
    g = on_gpu(st)
    out, lse = torch.full_like(g["q"], 7.0), torch.full(g["q"].shape[:2], 7.0, device="cuda")
    kw = dict(k_scale=st["ks"], v_scale=st["vs"]) if kind == "tensor" else {}
    f = lambda: pkv.extend_attn(g["q"], g["k_new"], g["v_new"], g["cu"], g["lens"], g["kc"], g["vc"], g["table"], 300, 6000,
                                window=200, sinks=9, out=out, lse=lse, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f()
    ref = reference(st)
    for _ in range(3):
        out.fill_(7.0), lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        check((out.cpu(), lse.cpu()), ref, st["T"])
assert pkv.device_errors() == 0
print("as before")
"""


def test_captured_launches_without_a_counter():
    """A process that has captured more launches than have counters: windowed extends deal their items statically."""
    r = subprocess.run([sys.executable, "-c", _MANY], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "as before" in r.stdout, r.stdout + r.stderr
