"""GPU tests of decode over 8-bit pages where the rows' sizes, the weights or the
queries' dims spread far apart: a value row much larger than the others with
next to no weight, rows whose weights span fp32's range, queries with a dim
that no key answers.  Every element within the bound derived in paged_ref."""
import pytest
import torch

import cache_ref as C
import paged_ref as R
from test_gpu_paged_attention import i32, slopes_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pisa():
    from pyramid_top_block_mean_gb300 import pisa as m
    return m


def pages(k, v, lens, seed):
    kp, ks, table, k = C.paginate(k, lens, seed)
    vp, vs, _, v = C.paginate(v, lens, seed)
    return k.cuda(), v.cuda(), (kp.cuda(), vp.cuda(), table.cuda(), i32(lens)), torch.stack([ks, vs]).contiguous().cuda()


def check_dense(pisa, q, k, v, cache, scales, lens, N, **kw):
    B, Hq, d = q.shape
    layer = pisa.PagedAttention(pisa.make_params(B, N, Hq, k.shape[1], d))
    mask = pisa.AttentionMask(kw.get("softcap", 0.0), kw.get("window", 0), kw.get("slopes")) if kw else None
    out = layer.dense_decode(q, *cache, mask=mask, scales=scales)
    assert layer.device_status() == 0
    for b, n in enumerate(lens):
        want, tol = R.dense(q[b][:, None], k[b], v[b], n, torch.tensor([n - 1], device="cuda"), d ** -0.5, **kw)
        R.within(out[b], want[:, 0], tol[:, 0], f"sequence {b}")


def large_row(d, Hq, Hkv, N, lens, at, gap, nats, attended, seed=3):
    """Keys and values of which row at[b] of sequence b has values 2^gap times
    the others', none in half of its dims, and a score some `nats` below the
    others'; attended: with it, in the first head of each group, above them."""
    g = torch.Generator().manual_seed(seed)
    B, G = len(lens), Hq // Hkv
    k, v = (torch.randn(B, Hkv, N, d, generator=g) for _ in range(2))
    q = torch.randn(B, Hq, d, generator=g) * 2
    q[..., 0] = 4.0
    if attended:
        q[:, ::G, 0] = -4.0
    k[..., 0] = 0.0
    for b, j in enumerate(at):
        k[b, :, j, 0] = -nats / (4.0 * d ** -0.5)
        v[b, :, j, :d // 2] *= 2.0 ** gap
        v[b, :, j, d // 2:] = 0.0
    return q.to(torch.bfloat16).cuda(), *pages(k, v, lens, seed)


@pytest.mark.parametrize("attended", [False, True])
@pytest.mark.parametrize("gap,nats", [(24, 25), (33, 25), (40, 30), (60, 100), (100, 30), (100, 300), (5, 40), (119, 0), (119, 25),
                                      (119, 300)])
@pytest.mark.parametrize("d,Hq,Hkv", [(128, 2, 2), (128, 8, 2), (64, 2, 1), (64, 16, 2), (128, 8, 1)])
def test_a_large_row_without_weight(pisa, d, Hq, Hkv, gap, nats, attended):
    """Before, among and behind the rows that have the weight."""
    lens = [300, 290, 300, 280]
    q, *rest = large_row(d, Hq, Hkv, 300, lens, [0, 141, 299, 65], gap, nats, attended)
    check_dense(pisa, q, *rest, lens, 300)


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 2, 2), (128, 8, 2), (64, 16, 2)])
@pytest.mark.parametrize("gap,nats", [(112, 300), (112, 60), (80, 40)])
def test_small_values_beside_a_large_row(pisa, d, Hq, Hkv, gap, nats):
    """Rows of 2^-93, near the end of the bound's range, and one that is not small."""
    lens = [300, 290, 300, 280]
    q, k, v, cache, scales = large_row(d, Hq, Hkv, 300, lens, [0, 141, 299, 65], gap, nats, False)
    scales[1] = (scales[1].int() - 93).clamp_min(10).to(torch.uint8)
    v = v * 2.0 ** -93
    check_dense(pisa, q, k, v, cache, scales, lens, 300)


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 8, 2), (64, 8, 1)])
def test_a_large_row_in_a_cache_split_over_the_gpu(pisa, d, Hq, Hkv):
    lens = [9000, 8000]
    q, *rest = large_row(d, Hq, Hkv, 9000, lens, [4000, 70], 40, 30, True)
    check_dense(pisa, q, *rest, lens, 9000)


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 2, 2), (128, 8, 2), (64, 16, 2)])
def test_a_large_row_among_selected_blocks(pisa, d, Hq, Hkv):
    lens, K = [900, 900], 5
    for gap, nats in ((40, 30), (100, 300)):
        q, k, v, cache, scales = large_row(d, Hq, Hkv, 900, lens, [10, 500], gap, nats, False)
        layer = pisa.PagedAttention(pisa.make_params(2, 900, Hq, Hkv, d, K=K))
        idx = i32([0, 3, 7, 8, 13, 14, -1, -1])[None, None].expand(2, Hkv, -1).contiguous()
        idx[1, 0, :2] = i32([7, 2])
        out = layer.selected_decode(q, *cache, idx, scales=scales)
        assert layer.device_status() == 0
        for b, n in enumerate(lens):
            want, tol = R.selected(q[b], k[b], v[b], n, idx[b], d ** -0.5)
            R.within(out[b], want, tol, f"sequence {b}")


@pytest.mark.parametrize("kw", [dict(softcap=20.0), dict(window=100), dict(slopes=True)])
@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (16, 2)])
def test_a_large_row_and_masks(pisa, Hq, Hkv, kw):
    lens = [300, 290]
    kw = {**kw, "slopes": slopes_of(Hq)} if "slopes" in kw else kw
    q, *rest = large_row(128, Hq, Hkv, 300, lens, [260, 280], 40, 30, False)
    check_dense(pisa, q, *rest, lens, 300, **kw)


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 2, 2), (128, 8, 2), (64, 16, 2)])
def test_weights_over_all_of_fp32(pisa, d, Hq, Hkv):
    """Scores from 0 down to -90, and dims in which only the rows of one such size are not zero."""
    g = torch.Generator().manual_seed(8)
    lens, N = [640, 600], 640
    k, v = (torch.randn(2, Hkv, N, d, generator=g) for _ in range(2))
    q = torch.randn(2, Hq, d, generator=g)
    q[..., 0], k[..., 0] = 4.0, 0.0
    for b in range(2):  # within a page, and page by page
        size = torch.arange(N) % 10 if b == 0 else 9 - torch.arange(N) // 64
        k[b, :, :, 0] = -(10.0 * size) / (4.0 * d ** -0.5)
        v[b, :, :, 16:] = torch.where((torch.arange(d)[None, 16:] % 10) == size[:, None], v[b, :, :, 16:], 0.0)
    check_dense(pisa, q.to(torch.bfloat16).cuda(), *pages(k, v, lens, 8), lens, N)


@pytest.mark.parametrize("gap", [10, 14, 18, 24, 60, 120])
@pytest.mark.parametrize("d,Hq,Hkv", [(128, 2, 2), (128, 8, 2), (64, 4, 1), (64, 16, 2), (128, 8, 1)])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=20.0), dict(window=70)])
def test_a_query_dim_that_no_key_answers(pisa, d, Hq, Hkv, gap, kw):
    g = torch.Generator().manual_seed(gap)
    lens, N = [300, 290, 64], 300
    k, v = (torch.randn(3, Hkv, N, d, generator=g) for _ in range(2))
    q = torch.randn(3, Hq, d, generator=g) * 2
    q[..., 5] = 2.0 ** gap * 3
    q[0, 1, 5] = 1.0  # and a head without
    k[..., 5] = 0.0
    k[1, :, ::3] *= 2.0 ** -6
    check_dense(pisa, q.to(torch.bfloat16).cuda(), *pages(k, v, lens, 9), lens, N, **kw)


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 8, 2), (64, 16, 2)])
def test_query_dims_of_many_sizes(pisa, d, Hq, Hkv):
    """Dims from 2^-30 of a query's largest to it, and keys that make up for it: products of one size, large scores."""
    g = torch.Generator().manual_seed(4)
    lens, N = [300, 250], 300
    size = 2.0 ** -(torch.arange(d) % 31).float()
    k, v = (torch.randn(2, Hkv, N, d, generator=g) for _ in range(2))
    q = torch.randn(2, Hq, d, generator=g) * size * 2.0 ** 12
    k[..., :] *= torch.where(torch.arange(d) % 31 > 15, 1.0, 0.0)
    k[1] *= 2.0 ** 14
    check_dense(pisa, q.to(torch.bfloat16).cuda(), *pages(k, v, lens, 4), lens, N)
