"""The decode calls captured into a graph and replayed for other queries and other lengths: a replay's sequences are cut
otherwise than the replay's before it, and nothing that one leaves in the workspace may pass for the next one's.

Bounds: u = 2^-8 (half a step of bf16 relative to the value) for the rounding of out and of each P before its product with
V; a score is a sum of D products that are exact in fp32, each addition off by at most 2^-23 of the sum of magnitudes M, and
2^-20 (1 + |lse|) covers the rounding of s - m, of 2^x, of the logarithm and of the merges' weights:
e = D 2^-23 M + 2^-20 (1 + |lse|), |out - o| <= u |o| + (u + 2 e) sum p |v|, |lse - z| <= e.
"""
import math

import pytest
import torch

from pkv_workloads import gen

pytestmark = pytest.mark.gpu

LENS = [[4000, 900, 60], [1300, 900, 60], [4000, 30, 2000], [200, 200, 200], [4000, 900, 60], [2500, 0, 2047], [31, 4000, 1],
        [3000, 3100, 4000], [4000, 900, 60]]
U = 2.0 ** -8


def _check(out, lse, q, k, v, scale, what):
    """One request: q [Hq, D], k [c, Hkv, D], v [c, Hkv, Dv] doubles."""
    Hkv = k.shape[1]
    q = q.view(Hkv, -1, q.shape[-1])
    s = torch.einsum("hgd,jhd->hgj", q, k) * scale
    M = (torch.einsum("hgd,jhd->hgj", q.abs(), k.abs()) * scale).amax(-1).flatten()
    z = torch.logsumexp(s, -1)
    p = torch.exp(s - z[..., None])
    o, A = (torch.einsum("hgj,jhd->hgd", p, x).flatten(0, 1) for x in (v, v.abs()))
    z = z.flatten()
    e = q.shape[-1] * 2.0 ** -23 * M + 2.0 ** -20 * (1 + z.abs())
    assert bool(((lse.double() - z).abs() <= e).all()), f"{what}: lse"
    assert bool(((out.double() - o).abs() <= U * o.abs() + (U + 2 * e[:, None]) * A + 1e-37).all()), f"{what}: out"


@pytest.mark.parametrize("what,Hq,Hkv,D", [
    ("bf16", 32, 4, 128), ("bf16", 8, 8, 64), ("fp8", 64, 4, 128), ("block", 16, 2, 128), ("noalloc", 32, 2, 128), ("mla", 16, 1, 576),
    ("mla", 32, 1, 576), ("mla", 128, 1, 576)])
def test_decode_replayed_for_other_queries_and_lengths(what, Hq, Hkv, D):
    import paged_kv_attention_reshape_gb300 as pkv
    g = torch.Generator(device="cuda").manual_seed(Hq + D)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    nb, scale, more = 3 * 250, gen.MLA_SCALE if what == "mla" else 1.0 / math.sqrt(D), {}
    table = torch.randperm(nb, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(3, 250).contiguous().cuda()
    if what in ("fp8", "block"):
        cache = [(rnd(nb, 16, Hkv, D) * 100).clamp(-448, 448).to(torch.float8_e4m3fn) for _ in "kv"]
        if what == "fp8":
            sc = [0.011, 0.017]
            values = [c.double() * s for c, s in zip(cache, sc)]
        else:
            sc = [torch.exp2(torch.randint(-9, -5, (nb, Hkv), generator=g, device="cuda").float()) for _ in "kv"]
            values = [c.double() * s[:, None, :, None].double() for c, s in zip(cache, sc)]
        more = dict(k_scale=sc[0], v_scale=sc[1])
    else:
        cache = [rnd(nb, 16, Hkv, D).to(torch.bfloat16) for _ in range(1 if what == "mla" else 2)]
        values = [c.double() for c in cache]
    dv = 512 if what == "mla" else D
    q = rnd(3, Hq, D).to(torch.bfloat16)
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros((3, Hq, dv), dtype=torch.bfloat16, device="cuda"), torch.zeros((3, Hq), device="cuda")
    if what == "mla":
        ws = torch.empty(pkv.mla_decode_workspace_size(3, Hq, 4000), dtype=torch.uint8, device="cuda")
        call = lambda: pkv.mla_decode_attn(q, cache[0], table, lens, 4000, scale, out=out, lse=lse, workspace=ws)  # noqa: E731
    elif what == "noalloc":
        call = lambda: pkv.paged_decode_attn_noalloc(q, *cache, table, lens, 4000, out, lse)  # noqa: E731
    else:
        ws = torch.empty(pkv.paged_decode_workspace_size(3, Hq, Hkv, D, 4000), dtype=torch.uint8, device="cuda")
        call = lambda: pkv.paged_decode_attn(q, *cache, table, lens, 4000, out=out, lse=lse, workspace=ws, **more)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i, new in enumerate(LENS * 2):
        q.copy_(rnd(3, Hq, D))
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        out.fill_(7.0), lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for r, c in enumerate(new):
            if c == 0:
                assert bool((out[r] == 0).all()) and bool((lse[r] == -math.inf).all())
                continue
            k, v = (x[table[r].long()].flatten(0, 1)[:c] for x in (values if len(values) == 2 else values * 2))
            _check(out[r], lse[r], q[r].double(), k, v[..., :dv], scale, f"replay {i} request {r}")
    assert pkv.device_errors() == 0
