"""PagedAttention holds every call to the new tokens that it was made for."""
import pytest
import torch


@pytest.fixture(scope="module")
def pisa():
    from pyramid_top_block_mean_gb300 import build
    build.build()
    from pyramid_top_block_mean_gb300 import pisa as m
    return m


def test_appending_without_queries_is_held_to_the_tokens_asked_for(pisa):
    # two key heads of six tokens have the elements of four query heads of three
    p = pisa.make_params(2, 128, 4, 2, 64)
    layer = pisa.PagedAttention(p, n=3, device="cpu")
    pool = torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for q, n in ((None, 6), (None, 4), (torch.zeros(2, 4, 6, 64, dtype=torch.bfloat16), 6)):
        k = torch.zeros(2, 2, n, 64, dtype=torch.bfloat16)
        with pytest.raises(ValueError, match="more than the 3 new tokens"):
            layer.append(q, k, k, pool, pool, table, lens)
    k = torch.zeros(2, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="expected CUDA tensors"):  # the tokens are not the reason
        layer.append(None, k, k, pool, pool, table, lens)
