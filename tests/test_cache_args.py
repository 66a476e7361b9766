"""The selector's calls over 8-bit pages and PagedAttention look at every tensor
that they are given: shapes, types, devices and layouts that do not fit are
refused before anything reads them (on the CPU: no call gets as far as a GPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def pisa():
    from pyramid_top_block_mean_gb300 import build
    build.build()
    from pyramid_top_block_mean_gb300 import pisa as m
    return m


@pytest.fixture
def made(pisa):
    p = pisa.make_params(2, 500, 4, 2, 64, K=4)
    kp, _, scales = pisa.quantized_pages(p, 16, device="cpu")
    W = p.K + 3
    a = dict(k_pages=kp, page_table=torch.zeros(2, 8, dtype=torch.int32), scales=scales,
             seq_lens=torch.full((2,), 500, dtype=torch.int32),
             pyramid=torch.zeros(2, 2, pisa.pyramid_nodes(p), 64), ws=torch.zeros(1 << 16, dtype=torch.uint8))
    b = dict(q=torch.zeros(2, 4, 64, dtype=torch.bfloat16), out_idx=torch.zeros(2, 2, W, dtype=torch.int32),
             out_score=torch.zeros(2, 2, W),
             trace=torch.zeros(2, 2, pisa.pyramid_levels(p), p.K, dtype=torch.int32))
    return p, a, b


def bad_tensors(t):
    """The same tensor with another type, one element short, and not contiguous."""
    yield t.double() if t.dtype is not torch.float8_e4m3fn else t.float()
    yield t.flatten()[:-1]
    wide = torch.zeros(*t.shape, 2, dtype=torch.float32).to(t.dtype)
    yield wide[..., 0]


def test_build_over_8_bit_pages(pisa, made):
    p, a, _ = made
    with pytest.raises(ValueError, match="expected CUDA tensors"):
        pisa.build_pyramid_paged(p, **a)
    with pytest.raises(ValueError, match="expected CUDA tensors"):
        pisa.build_pyramid_paged(p, **(a | dict(seq_lens=None)))
    for name in set(a) - {"ws"}:
        for bad in bad_tensors(a[name]):
            with pytest.raises(ValueError, match=name):
                pisa.build_pyramid_paged(p, **(a | {name: bad}))
    for short in (a["page_table"][:, :7].contiguous(), a["page_table"][:1], a["page_table"].long()):
        with pytest.raises(ValueError, match="page_table"):
            pisa.build_pyramid_paged(p, **(a | dict(page_table=short)))


def test_step_over_8_bit_pages(pisa, made):
    p, a, b = made
    for some in (b, b | dict(out_score=None, trace=None), b | dict(q=b["q"][:, :, None])):
        with pytest.raises(ValueError, match="expected CUDA tensors"):
            pisa.select_decode_paged(p, **a, **some)
    for name in set(a | b) - {"ws"}:
        for bad in bad_tensors((a | b)[name]):
            with pytest.raises(ValueError, match=name):
                pisa.select_decode_paged(p, **(a | b | {name: bad}))


def test_8_bit_pages_without_their_scales(pisa, made):
    """Taken for pages of the model's type they would be read past their end."""
    p, a, b = made
    a = dict(a, scales=None)
    with pytest.raises(ValueError, match="8-bit pages"):
        pisa.build_pyramid_paged(p, **a)
    with pytest.raises(ValueError, match="8-bit pages"):
        pisa.select_decode_paged(p, **a, **b)


def test_a_scratch_of_too_few_bytes(pisa):
    p = pisa.make_params(1, 2048, 8, 2, 64)
    size = pisa.cache_scratch_bytes(p, 2048)
    assert size > 0
    for bad in (torch.zeros(size - 1, dtype=torch.uint8), torch.zeros(2, size, dtype=torch.uint8)[:, ::2]):
        with pytest.raises(ValueError):
            pisa.PagedAttention(p, n=2048, device="cpu", scratch=bad)
    pisa.PagedAttention(p, n=2048, device="cpu", scratch=torch.zeros(size, dtype=torch.uint8))
    pisa.PagedAttention(p, n=16, device="cpu", scratch=torch.zeros(1, dtype=torch.uint8))  # of no use to it
