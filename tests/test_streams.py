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
