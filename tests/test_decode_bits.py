"""Decodes whose sequences are cut into pieces: the pieces end in another order from call to call, the bits stay."""
import pytest
import torch

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def state(lens, Hq, Hkv, D, kind, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    blocks = [(n + 15) // 16 for n in lens]
    nb, most = sum(blocks), max(blocks)
    perm = torch.randperm(nb, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), most), dtype=torch.int32, device="cuda")
    at = 0
    for r, b in enumerate(blocks):
        table[r, :b] = perm[at:at + b]
        at += b
    shape = (nb, 16, 1, 576) if kind == "latent" else (nb, 16, Hkv, D)
    kc, vc = (torch.randn(shape, generator=g, device="cuda") for _ in "kv")
    kc, vc = (x.to(E4M3).view(torch.uint8) if kind in ("tensor", "block") else x.to(torch.bfloat16) for x in (kc, vc))
    q = torch.randn((len(lens), Hq, shape[3]), generator=g, device="cuda").to(torch.bfloat16)
    return q, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens)


@pytest.mark.parametrize("lens,Hq,Hkv,D,kind,kw", [
    ([8000] * 5, 64, 8, 128, "bf16", {}), ([700, 90, 3000], 8, 2, 128, "bf16", dict(window=150, sinks=9)),
    ([2500 + 9 * i for i in range(60)], 64, 4, 128, "bf16", dict(window=1024)), ([4000] * 7, 16, 4, 64, "bf16", {}),
    ([9000, 500, 12000], 32, 8, 128, "tensor", {}), ([9000, 500, 12000], 32, 8, 128, "tensor", dict(window=4096)),
    ([9000, 500, 12000], 32, 2, 128, "block", {}), ([3000, 777] * 4, 16, 1, 576, "latent", {})])
def test_the_same_bits_whatever_ends_first(lens, Hq, Hkv, D, kind, kw):
    import paged_kv_attention_reshape_gb300 as pkv
    q, kc, vc, table, n, most = state(lens, Hq, Hkv, D, kind, 7)
    if kind == "latent":
        call = lambda: pkv.mla_decode_attn(q, kc, table, n, most, 0.05)
    else:
        if kind == "tensor":
            kw = dict(kw, k_scale=0.5, v_scale=0.25)
        elif kind == "block":
            kw = dict(kw, **{x: torch.rand((kc.shape[0], Hkv), device="cuda") * 0.1 + 0.05 for x in ("k_scale", "v_scale")})
        call = lambda: pkv.paged_decode_attn(q, kc, vc, table, n, most, **kw)
    o, z = call()
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    side, a = torch.cuda.Stream(), torch.randn((3000, 3000), device="cuda")
    for i in range(300):
        with torch.cuda.stream(side):  # what takes SMs and memory beside the call, now less, now more
            a[:1 + 97 * (i % 31)].mul_(1.0)
        x, y = call()
        differ += (x != o).sum() + (y != z).sum()
    torch.cuda.synchronize()
    assert int(differ) == 0 and pkv.device_errors() == 0


@pytest.mark.parametrize("lens,Hq,Hkv,D,kind", [([8000] * 5, 16, 2, 128, "bf16"), ([8000] * 5, 8, 2, 64, "bf16"), ([40, 90], 16, 2, 128, "bf16"),
                                                ([9000, 500], 16, 2, 128, "tensor"), ([3000] * 4, 16, 1, 576, "latent"), ([50], 16, 1, 576, "latent")])
def test_a_key_that_is_no_number(lens, Hq, Hkv, D, kind):
    """It makes out and lse of its request and KV head none, in whichever piece of the sequence it lies, and of no other."""
    import paged_kv_attention_reshape_gb300 as pkv
    q, kc, vc, table, n, most = state(lens, Hq, Hkv, D, kind, 8)
    if kind == "latent":
        call = lambda: pkv.mla_decode_attn(q, kc, table, n, most, 0.05)
    else:
        kw = dict(k_scale=0.5, v_scale=0.25) if kind == "tensor" else {}
        call = lambda: pkv.paged_decode_attn(q, kc, vc, table, n, most, **kw)
    want = call()
    G = Hq // Hkv
    for at in (0, lens[0] // 2, lens[0] - 1):
        page = int(table[0, at // 16])
        was = kc[page, at % 16, Hkv - 1, 3].clone()
        kc[page, at % 16, Hkv - 1, 3] = 0x7F if kind == "tensor" else float("nan")
        o, z = call()
        kc[page, at % 16, Hkv - 1, 3] = was
        assert torch.isnan(o[0, Hq - G:]).all() and torch.isnan(z[0, Hq - G:]).all()
        assert torch.equal(o[1:], want[0][1:]) and torch.equal(z[1:], want[1][1:]) and torch.equal(o[0, :Hq - G], want[0][0, :Hq - G])
    assert pkv.device_errors() == 0
