"""Calls on another stream than the current one: what the binding allocates for them is neither written by what is
still queued on the current stream nor given away before the current stream has read it."""
import math

import pytest
import torch

from pkv_workloads import gen

pytestmark = pytest.mark.gpu


def _dev(*ts):
    return tuple(t.cuda() for t in ts)


def _calls(pkv):
    """name -> f(stream) -> the tensors that the call allocated. Each f can be called again for the same result."""
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    n, Hq, Hkv, nb = 40, 8, 2, 400
    kc, vc = rnd(nb, 16, Hkv, 128), rnd(nb, 16, Hkv, 128)
    codes = [torch.randint(0, 100, (nb, 16, Hkv, 128), generator=g, dtype=torch.uint8).cuda() for _ in "kv"]
    scales = [(torch.rand((nb, Hkv), generator=g) * 0.01 + 0.001).cuda() for _ in "kv"]
    block = dict(k_scale=scales[0], v_scale=scales[1])
    table = torch.randperm(nb, generator=g).to(torch.int32)[:4 * 100].view(4, 100).contiguous().cuda()
    lens, cu = _dev(torch.tensor([1590, 900, 33, 17], dtype=torch.int32), torch.tensor([0, 10, 20, 30, 40], dtype=torch.int32))
    q, k, v, q1 = rnd(n, Hq, 128), rnd(n, Hkv, 128), rnd(n, Hkv, 128), rnd(4, Hq, 128)
    pos, slot = torch.arange(n).cuda(), torch.randperm(nb * 16, generator=g)[:n].cuda()
    rope = torch.randn((64, 128), generator=g).cuda()
    app = rnd(nb, 16, Hkv, 128), rnd(nb, 16, Hkv, 128)
    latent, qm = rnd(nb, 16, 1, 576), rnd(4, 16, 576)
    ids = torch.randperm(nb, generator=g).to(torch.int32)[:50].cuda()
    return {
        "append": lambda s: pkv.kv_append(q, k, v, pos, slot, *app, rope, stream=s),
        "decode": lambda s: pkv.paged_decode_attn(q1, kc, vc, table, lens, 1600, stream=s),
        "decode_block": lambda s: pkv.paged_decode_attn(q1, *codes, table, lens, 1600, stream=s, **block),
        "mla": lambda s: pkv.mla_decode_attn(qm, latent, table, lens, 1600, gen.MLA_SCALE, stream=s),
        "extend": lambda s: pkv.extend_attn(q, k, v, cu, lens, kc, vc, table, 10, 1600, stream=s),
        "extend_block": lambda s: pkv.extend_attn(q, k, v, cu, lens, *codes, table, 10, 1600, stream=s, **block),
        "prefill": lambda s: pkv.varlen_prefill_attn(q, k, v, cu, 10, stream=s),
        "pack": lambda s: (pkv.kv_block_pack(kc, vc, ids, stream=s),),
        "reorder": lambda s: pkv.batch_classify_reorder(cu, lens, with_token_map=True, num_tokens=n, stream=s),
    }


NAMES = ["append", "decode", "decode_block", "mla", "extend", "extend_block", "prefill", "pack", "reorder"]


def _same(got, want):
    return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


@pytest.mark.parametrize("handle", ["stream", "integer"])
@pytest.mark.parametrize("name", NAMES)
def test_a_call_on_another_stream_shares_no_memory_with_the_current_one(name, handle, monkeypatch):
    import paged_kv_attention_reshape_gb300 as pkv
    from paged_kv_attention_reshape_gb300 import binding
    scratch = []
    plain = binding._scratch

    def spy(need, workspace, device, other):
        w = plain(need, workspace, device, other)
        if w is not None:
            scratch.append((w.data_ptr(), w.numel()))
        return w

    monkeypatch.setattr(binding, "_scratch", spy)
    call = _calls(pkv)[name]
    want = [t.clone() for t in call(None)]
    sizes = [t.numel() * t.element_size() for t in want] + [n for _, n in scratch]
    del scratch[:]
    other = torch.cuda.Stream()
    on = other if handle == "stream" else other.cuda_stream
    call(on)  # (what a first call loads is loaded)
    torch.cuda.synchronize()
    del scratch[:]
    # blocks of every size that the call allocates, given back to the current stream while their writes are queued
    torch.cuda._sleep(200_000_000)
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x7F) for n in sizes for _ in range(6)]
    held = [(b.data_ptr(), b.numel()) for b in blocks]
    del blocks
    got = call(on)
    for p, n in scratch:
        assert all(p + n <= a or a + m <= p for a, m in held), "the scratch lies in memory that is still written"
    torch.cuda.synchronize()
    assert _same(got, want)
    # the outputs given back while the current stream has yet to read them
    torch.cuda._sleep(200_000_000)
    copies = [t.clone() for t in got]
    del got
    with torch.cuda.stream(other):
        more = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x7F) for n in sizes for _ in range(6)]
    torch.cuda.synchronize()
    assert _same(copies, want)
    del more
    assert pkv.device_errors() == 0


def test_a_staged_layer_is_kept_until_the_current_stream_has_read_it():
    """LayerHandoff.stage without a buffer: what it allocates goes to no later pack while the current stream reads it."""
    import paged_kv_attention_reshape_gb300 as pkv
    kc, vc = (torch.randn((64, 16, 2, 128)).to(torch.bfloat16).cuda() for _ in "kv")
    ids = torch.randperm(64)[:40].to(torch.int32).cuda()
    want = torch.stack([kc[ids.long()], vc[ids.long()]])
    handoff = pkv.LayerHandoff(2)
    torch.cuda.synchronize()
    dst = handoff.stage(0, kc, vc, ids)
    handoff.ready(0)
    n = dst.numel() * dst.element_size()
    torch.cuda._sleep(200_000_000)
    copy = dst.clone()
    del dst
    with torch.cuda.stream(handoff.copy_stream):
        more = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0x7F) for _ in range(6)]
    torch.cuda.synchronize()
    assert torch.equal(copy, want)
    del more
    handoff.close()


def test_the_current_stream_by_name_and_the_default_stream():
    """The current stream given explicitly, and the default stream while another one is current."""
    import paged_kv_attention_reshape_gb300 as pkv
    from paged_kv_attention_reshape_gb300 import binding
    call = _calls(pkv)["extend_block"]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    default = torch.cuda.default_stream()
    assert binding._other(torch.cuda.current_stream()) is None and binding._other(torch.cuda.current_stream().cuda_stream) is None
    with torch.cuda.stream(side):
        assert binding._other(None) is None and binding._other(side.cuda_stream) is None
        assert binding._other(0) == default and binding._other(1) == default and binding._other(default) == default
        got = [call(side), call(0), call(default), call(side.cuda_stream)]
        torch.cuda.synchronize()
        assert all(_same(x, want) for x in got)
    assert pkv.device_errors() == 0 and math.isfinite(float(got[0][0].float().sum()))


@pytest.mark.parametrize("kind", ["prefill", "extend", "extend_block"])
def test_graphs_beside_direct_calls_and_beside_one_another(kind):
    """Two graphs of several launches and direct calls, each on a stream of its own and with buffers of its own, all at
    once: no launch takes another's work items."""
    import paged_kv_attention_reshape_gb300 as pkv
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    R, n, Hq, Hkv, nb = 24, 40, 16, 2, 24 * 40
    q, k, v = rnd(R * n, Hq, 128), rnd(R * n, Hkv, 128), rnd(R * n, Hkv, 128)
    cu, lens = _dev(torch.arange(0, R * n + 1, n, dtype=torch.int32), torch.randint(n, 600, (R,), generator=g).to(torch.int32))
    table = torch.randperm(nb, generator=g).to(torch.int32).view(R, 40).contiguous().cuda()
    if kind == "extend_block":
        cache = [torch.randint(0, 100, (nb, 16, Hkv, 128), generator=g, dtype=torch.uint8).cuda() for _ in "kv"]
        more = {x: (torch.rand((nb, Hkv), generator=g) * 0.01 + 0.001).cuda() for x in ("k_scale", "v_scale")}
    else:
        cache, more = [rnd(nb, 16, Hkv, 128) for _ in "kv"], {}

    def call(out, lse):
        if kind == "prefill":
            pkv.varlen_prefill_attn(q, k, v, cu, n, out=out, lse=lse)
        else:
            pkv.extend_attn(q, k, v, cu, lens, *cache, table, n, 600, out=out, lse=lse, **more)

    bufs = [(torch.zeros_like(q), torch.zeros((R * n, Hq), device="cuda")) for _ in range(4)]
    call(*bufs[3])
    torch.cuda.synchronize()
    want = [t.clone() for t in bufs[3]]
    bad = [torch.zeros((), dtype=torch.bool, device="cuda") for _ in range(3)]

    def checked(i):  # a call on cleared buffers, and whether it gave what it has to
        out, lse = bufs[i]
        out.fill_(7.0), lse.fill_(7.0)
        call(out, lse)
        bad[i] |= (out != want[0]).any() | (lse != want[1]).any()

    streams = [torch.cuda.Stream() for _ in range(3)]
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            for _ in range(6):
                checked(i)
    torch.cuda.synchronize()
    for _ in range(40):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
        with torch.cuda.stream(streams[2]):
            for _ in range(6):
                checked(2)
    torch.cuda.synchronize()
    assert not any(bool(b) for b in bad) and pkv.device_errors() == 0


_MANY = """
import sys, torch
sys.path[:0] = ["tests", "."]
import paged_kv_attention_reshape_gb300 as pkv
g = torch.Generator().manual_seed(6)
rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).cuda()
codes = [torch.randint(0, 100, (40, 16, 1, 128), generator=g, dtype=torch.uint8).cuda() for _ in "kv"]
more = {x: (torch.rand((40, 1), generator=g) * 0.01 + 0.001).cuda() for x in ("k_scale", "v_scale")}
table = torch.randperm(40, generator=g).to(torch.int32).view(2, 20).cuda()
one, cu1 = rnd(1, 1, 128), torch.tensor([0, 1], dtype=torch.int32).cuda()
out1, lse1 = torch.empty_like(one), torch.empty((1, 1), device="cuda")
fill = lambda: pkv.varlen_prefill_attn(one, one, one, cu1, 1, out=out1, lse=lse1)
R, n = 200, 9
q, k, v = rnd(R * n, 8, 128), rnd(R * n, 1, 128), rnd(R * n, 1, 128)
cu = torch.arange(0, R * n + 1, n, dtype=torch.int32).cuda()
lens = torch.randint(n, 310, (R,), generator=g).to(torch.int32).cuda()
tables = table[torch.arange(R) % 2].contiguous()
out, lse = torch.zeros_like(q), torch.zeros((R * n, 8), device="cuda")
calls = [lambda: pkv.varlen_prefill_attn(q, k, v, cu, n, out=out, lse=lse),
         lambda: pkv.extend_attn(q, k, v, cu, lens, *codes, tables, n, 310, out=out, lse=lse, **more),
         lambda: pkv.extend_attn(q, k, v, cu, lens, *codes, tables, 30, 2000, out=out, lse=lse, **more)]
want = []
for f in calls:
    f()
    want.append((out.clone(), lse.clone()))
fill()
s = torch.cuda.Stream()
torch.cuda.synchronize()
with torch.cuda.stream(s):
    graph = torch.cuda.CUDAGraph()
    graph.capture_begin()
    for _ in range(8200):
        fill()
    graph.capture_end()
del graph
for f, (o, l) in zip(calls, want):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f()
    for _ in range(3):
        out.zero_(), lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(lse, l)
assert pkv.device_errors() == 0
print("as before")
"""


def test_more_captured_launches_than_there_are_slots():
    """A process that has captured more extend/prefill launches than have a slot of their own: the later ones deal
    their items statically and give the same."""
    import os
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", _MANY], cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "as before" in r.stdout, r.stdout + r.stderr
