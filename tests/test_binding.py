"""What the binding makes of its arguments."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_scale_in_a_tensor_of_one_element():
    """One scale for the tensor, held in a tensor, is the number that it holds; a table of one block and head is a table."""
    import paged_kv_attention_reshape_gb300 as pkv
    k = torch.randn((3, 2, 128), dtype=torch.float32).to(torch.bfloat16).cuda()
    slot = torch.tensor([0, 5, 17]).cuda()
    got = []
    for ks, vs in ((0.01, 0.02), (torch.tensor(0.01), torch.tensor([0.02])), (torch.tensor([[0.01]]).cuda(), torch.tensor(0.02).cuda()),
                   (torch.tensor(0.01), 0.02)):
        kc, vc = (torch.zeros((2, 16, 2, 128), dtype=torch.uint8, device="cuda") for _ in "kv")
        pkv.kv_cache_write(k, k, slot, kc, vc, k_scale=ks, v_scale=vs)
        got.append((kc, vc))
    kb = torch.zeros((2, 16, 2, 128), dtype=torch.bfloat16, device="cuda")
    pkv.kv_cache_write(k, k, slot, kb, kb.clone(), k_scale=torch.tensor(1.0), v_scale=1.0)
    assert pkv.device_errors() == 0 and torch.equal(kb.view(32, 2, 128)[slot], k)
    assert all(torch.equal(a, b) for x in got for a, b in zip(x, got[0]))
    one = torch.zeros((1, 16, 1, 128), dtype=torch.uint8, device="cuda")
    table = torch.ones((1, 1), device="cuda")
    assert pkv.make_cache(one, one.clone(), table, table).kv_dtype == pkv._lib.KV_FP8_E4M3_BLOCK
    with pytest.raises(pkv.PkvError):
        pkv.make_cache(one, one.clone(), table, 1.0)
