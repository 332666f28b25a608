"""kv_block_copy: blocks of a pool onto other blocks of it, in every layer, bit for bit."""
import ctypes

import pytest
import torch

E4M3 = torch.float8_e4m3fn


def pools(L, nb, shape, kind, seed, gap=0):
    """L layers of (k, v, scales) on the GPU; gap: elements between blocks (they share one allocation then)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = 1
    for s in shape:
        n *= s
    made = []
    for _ in range(L):
        kv = []
        for _ in range(2):
            whole = torch.randint(0, 256, (nb, n + gap) if kind != "bf16" else (nb, 2 * (n + gap)), generator=g, dtype=torch.uint8,
                                  device="cuda")
            whole = whole if kind != "bf16" else whole.view(torch.int16).view(torch.bfloat16)
            kv.append(whole[:, :n].view((nb,) + shape) if gap == 0 else whole.as_strided((nb,) + shape, (n + gap,) + strides(shape)))
        sc = [torch.rand((nb, shape[1]), generator=g, device="cuda") for _ in range(2)] if kind == "block" else [None, None]
        made.append((*kv, *sc))
    return made


def strides(shape):
    st, k = [], 1
    for s in reversed(shape):
        st.insert(0, k)
        k *= s
    return tuple(st)


def raw(t):
    return t.contiguous().view(torch.uint8)


def layers_of(made, latent=False):
    import paged_kv_attention_reshape_gb300 as pkv
    cols = list(zip(*made))
    scaled = made[0][2] is not None
    return pkv.CacheLayers(cols[0], None if latent else cols[1], list(cols[2]) if scaled else None, list(cols[3]) if scaled else None)


def verify(made, src, dst, latent=False):
    import paged_kv_attention_reshape_gb300 as pkv
    nb = made[0][0].shape[0]
    want = []
    of = torch.arange(nb)
    for s, d in zip(src, dst):
        if 0 <= s < nb and 0 <= d < nb:
            of[d] = s
    of = of.cuda()
    for m in made:
        want.append([None if t is None else (t if latent and i else t[of].clone()) for i, t in enumerate(m)])
    i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()
    pkv.kv_block_copy(layers_of(made, latent), i32(src), i32(dst))
    for m, w in zip(made, want):
        for t, x in zip(m, w):
            assert t is None or torch.equal(raw(t), raw(x))


# ---- refusals (no GPU) --------------------------------------------------------------------------------

def test_refusals():
    from paged_kv_attention_reshape_gb300 import _lib
    lib = _lib.load()
    fake = ctypes.c_void_p(1 << 20)
    other = ctypes.c_void_p(1 << 21)
    C = _lib.PkvCache
    good = C(fake, other, 10, 16, 2, 128, 16 * 2 * 128)

    def run(*caches, n=3, src=fake, dst=fake):
        return lib.pkv_kv_block_copy((C * len(caches))(*caches), len(caches), src, dst, n, None)

    assert run(good, n=0) == 0 and run(good, n=0, src=None, dst=None) == 0
    assert run(good, n=-1) == 1 and run(good, src=None) == 1 and run(good, dst=None) == 1
    assert lib.pkv_kv_block_copy(None, 1, fake, fake, 0, None) == 1
    assert lib.pkv_kv_block_copy((C * 1)(good), 0, fake, fake, 0, None) == 1
    # layers that differ
    for differs in (C(fake, other, 11, 16, 2, 128, 16 * 2 * 128), C(fake, other, 10, 8, 2, 128, 16 * 2 * 128),
                  C(fake, other, 10, 16, 1, 128, 16 * 2 * 128), C(fake, other, 10, 16, 2, 64, 16 * 2 * 128),
                  C(fake, other, 10, 16, 2, 128, 16 * 2 * 128 + 8), C(fake, other, 10, 16, 2, 128, 16 * 2 * 128, 1, 1.0, 1.0),
                  C(fake, None, 10, 16, 2, 128, 16 * 2 * 128)):
        assert run(good, differs, n=0) == 1
    assert run(C(None, other, 10, 16, 2, 128, 16 * 2 * 128), n=0) == 1
    assert run(C(ctypes.c_void_p((1 << 20) + 2), other, 10, 16, 2, 128, 16 * 2 * 128), n=0) == 1
    # block-scaled: both scales, K and V
    blk = lambda v, ks: C(fake, v, 10, 16, 2, 128, 16 * 2 * 128, _lib.KV_FP8_E4M3_BLOCK, 1.0, 1.0, ks, fake)
    assert run(blk(other, fake), n=0) == 0 and run(blk(other, None), n=0) == 1 and run(blk(None, fake), n=0) == 2


# ---- the operator --------------------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "tensor", "block"])
@pytest.mark.parametrize("L,shape,gap", [(1, (16, 1, 128), 0), (3, (16, 8, 128), 0), (130, (16, 2, 128), 0), (2, (16, 3, 128), 64)])
def test_copies(kind, L, shape, gap):
    made = pools(L, 23, shape, kind, L, gap)
    verify(made, [0, 3, 5, 22, 3], [1, 2, 4, 21, 9])       # a source twice
    verify(made, [7, -1, 8, 11], [7, 12, -1, 10])          # itself, and padding
    verify(made, [], [])


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 1, 16), (5, 3, 8), (64, 1, 64), (128, 8, 128), (16, 1, 576)])
def test_any_block_size(shape):
    verify(pools(2, 40, shape, "bf16", 3), list(range(0, 19)), list(range(20, 39)))


@pytest.mark.gpu
def test_a_latent_cache():
    verify(pools(4, 12, (16, 1, 576), "bf16", 9), [0, 5], [3, 11], latent=True)


@pytest.mark.gpu
def test_one_allocation_for_k_and_v():
    """[num_blocks, 2, ...]: K and V blocks alternate."""
    import paged_kv_attention_reshape_gb300 as pkv
    whole = torch.randn((9, 2, 16, 2, 64), device="cuda").to(torch.bfloat16)
    want = whole.clone()
    want[4] = whole[7]
    layers = pkv.CacheLayers([whole[:, 0]], [whole[:, 1]])
    pkv.kv_block_copy(layers, torch.tensor([7], dtype=torch.int32).cuda(), torch.tensor([4], dtype=torch.int32).cuda())
    assert torch.equal(whole, want) and len(layers) == 1


@pytest.mark.gpu
def test_many_pairs():
    g = torch.Generator().manual_seed(1)
    perm = torch.randperm(4001, generator=g).tolist()
    verify(pools(2, 4001, (16, 2, 64), "bf16", 5), perm[:2000], perm[2000:4000])


@pytest.mark.gpu
def test_bad_ids_are_flagged():
    import paged_kv_attention_reshape_gb300 as pkv
    made = pools(2, 6, (16, 2, 128), "bf16", 5)
    verify(made, [0, 6, 1, 2 ** 31 - 1], [3, 4, 2 ** 30, 5])
    assert pkv.device_errors() == 2


@pytest.mark.gpu
def test_a_bad_id_onto_itself_is_flagged():
    import paged_kv_attention_reshape_gb300 as pkv
    for bad in (6, 2 ** 31 - 1):
        verify(pools(1, 6, (16, 2, 128), "bf16", 5), [0, bad, -1], [3, bad, bad])
        assert pkv.device_errors() == 2
    verify(pools(1, 6, (16, 2, 128), "bf16", 5), [5, -1, 6], [5, 6, -1])  # the last block onto itself, and padding
    assert pkv.device_errors() == 0


@pytest.mark.gpu
def test_captured_and_on_another_stream():
    import paged_kv_attention_reshape_gb300 as pkv
    made = pools(3, 20, (16, 4, 128), "block", 8)
    start = [[t.clone() for t in m] for m in made]
    layers = layers_of(made)
    src, dst = (torch.tensor(x, dtype=torch.int32).cuda() for x in ([1, 2, -1], [11, 12, -1]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pkv.kv_block_copy(layers, src, dst, stream=side)
    side.synchronize()
    for m, s in zip(made, start):
        assert all(torch.equal(t[[11, 12]], x[[1, 2]]) for t, x in zip(m, s))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.kv_block_copy(layers, src, dst)
    src.copy_(torch.tensor([4, 5, 4]))
    dst.copy_(torch.tensor([14, 15, 16]))
    graph.replay()
    torch.cuda.synchronize()
    for m, s in zip(made, start):
        assert all(torch.equal(t[[14, 15, 16]], x[[4, 5, 4]]) for t, x in zip(m, s))
    assert pkv.device_errors() == 0


@pytest.mark.gpu
def test_refused_by_the_binding():
    import paged_kv_attention_reshape_gb300 as pkv
    (k, v, _, _), (k2, v2, _, _) = pools(2, 6, (16, 2, 128), "bf16", 5)
    ids = torch.zeros(2, dtype=torch.int32, device="cuda")
    layers = pkv.CacheLayers([k, k2], [v, v2])
    for a, b in ((ids.long(), ids), (ids, ids[:1]), (ids.cpu(), ids), (torch.zeros((2, 2), dtype=torch.int32, device="cuda")[:, 0], ids)):
        with pytest.raises(pkv.PkvError):
            pkv.kv_block_copy(layers, a, b)
    for args in (([], []), ([k], [v, v2]), ([k, k2], [v, v2], [1.0])):
        with pytest.raises(pkv.PkvError):
            pkv.CacheLayers(*args)
    small = pools(1, 5, (16, 2, 128), "bf16", 5)[0]
    with pytest.raises(pkv.PkvError):
        pkv.kv_block_copy(pkv.CacheLayers([k, small[0]], [v, small[1]]), ids, ids)
