"""Views that are dense although a stride that nothing uses says otherwise: one token's rows out of a wider buffer, one head.
Whichever way a call goes, it takes them."""
import pytest

from tests.test_kv4_gpu import pa  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,strides", [(8, (1029, 64, 1)), (8, (3, 64, 1)), (8, (1 << 41, 64, 1)), (1, (64, 7, 1)),
                                           (1, (1, 1, 1))])
def test_one_token(pa, heads, strides):
    import torch
    buffers = torch.randn((2, heads * 64), device="cuda").bfloat16()
    k, v = (torch.as_strided(b, (1, heads, 64), strides) for b in buffers)
    assert torch.equal(k.flatten(), buffers[0])
    slots = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    got, want = pa.kv4_pool(1, 16, heads, 64), pa.kv4_pool(1, 16, heads, 64)
    pa.paged_attn_append_kv4(buffers[0].view(1, heads, 64), buffers[1].view(1, heads, 64), slots, want)
    pa.paged_attn_append_kv4(k, v, slots, got)
    assert torch.equal(got, want) and want.any()
    # as queries
    table, lens = torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.full((1,), 6, dtype=torch.int32, device="cuda")
    q_start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    a = pa.attention_kv4(k, want, table, lens, q_start=q_start)
    b = pa.attention_kv4(buffers[0].view(1, heads, 64), want, table, lens, q_start=q_start)
    assert torch.equal(a, b)
    assert pa.paged_attn_last_error_word() == 0
