"""GPU tests of the dense paged calls with scores of any finite size: with
integers times powers of two for queries and keys every dot is exact in fp32,
and scores that lie hundreds apart leave the largest alone (or the equal ones
together), so that the outcome is known: their values' mean, off by
  2^-8 A                 the weights are rounded to bf16 before P V,
  2^-8 |o|               the output is rounded to bf16,
  2^-16 A                sums and reciprocal in fp32
with A the mean of the values' magnitudes."""
import pytest
import torch

import paged_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pisa():
    from pyramid_top_block_mean_gb300 import pisa as m
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def setup(pisa, Hq, Hkv, d, N, n, seed, qs, ks):
    g = torch.Generator().manual_seed(seed)
    k = torch.randint(-3, 4, (1, Hkv, N, d), generator=g).float()
    q = torch.randint(-2, 3, (1, Hq, n, d), generator=g).float()
    v = torch.randn(1, Hkv, N, d, generator=g).to(torch.bfloat16)
    kp, table = R.paginate((k * ks).to(torch.bfloat16), [N], seed=seed)
    vp, _ = R.paginate(v, [N], seed=seed)
    layer = pisa.PagedAttention(pisa.make_params(1, N, Hq, Hkv, d), n=n)
    return q.cuda(), k.cuda(), v.cuda(), kp.cuda(), vp.cuda(), table.cuda(), layer, (q * qs).to(torch.bfloat16).cuda()


def check(out, q, k, v, pos, sign, window=0):
    """Rows [Hq, T, d] against the mean of the values at the largest dots (the smallest with a negative sign)."""
    N = k.shape[1]
    key = torch.arange(N, device="cuda")
    keep = key[None] <= pos[:, None]
    if window:
        keep &= key[None] > pos[:, None] - window
    G = q.shape[0] // k.shape[0]
    for h in range(q.shape[0]):
        x = (sign * (q[h].double() @ k[h // G].double().t())).masked_fill(~keep, -float("inf"))
        w = (x == x.amax(1, True)).double()
        w /= w.sum(1, True)
        vv = v[h // G].double()
        o, A = w @ vv, w @ vv.abs()
        R.within(out[h], o, 2.0 ** -8 * (A + o.abs()) + 2.0 ** -16 * A, f"head {h}")


SIZES = [(2.0 ** 6, 2.0 ** 6), (2.0 ** 10, 2.0 ** 8), (2.0 ** 14, 2.0 ** 10), (2.0 ** 15, 2.0 ** 15),
         (2.0 ** 30, 2.0 ** 30), (2.0 ** 60, 2.0 ** 50), (-2.0 ** 20, 2.0 ** 20)]


@pytest.mark.parametrize("qs,ks", SIZES)
@pytest.mark.parametrize("d,Hq,Hkv", [(64, 2, 2), (128, 8, 2)])
@pytest.mark.parametrize("N,n,window", [(700, 300, 0), (400, 400, 50), (6000, 30, 0)])
def test_prompt(pisa, qs, ks, d, Hq, Hkv, N, n, window):
    q, k, v, kp, vp, table, layer, big = setup(pisa, Hq, Hkv, d, N, n, 3, qs, ks)
    mask = pisa.AttentionMask(window=window) if window else None
    out = layer.dense_prefill(big, kp, vp, table, i32([N]), mask=mask)
    assert layer.device_status() == 0
    check(out[0], q[0], k[0], v[0], torch.arange(N - n, N, device="cuda"), 1 if qs > 0 else -1, window)


@pytest.mark.parametrize("qs,ks", SIZES)
@pytest.mark.parametrize("d,Hq,Hkv", [(64, 2, 2), (128, 8, 2)])
@pytest.mark.parametrize("N", [200, 9000])
def test_one_token(pisa, qs, ks, d, Hq, Hkv, N):
    q, k, v, kp, vp, table, layer, big = setup(pisa, Hq, Hkv, d, N, 1, 4, qs, ks)
    out = layer.dense_decode(big[:, :, 0].contiguous(), kp, vp, table, i32([N]))
    assert layer.device_status() == 0
    check(out[0][:, None], q[0], k[0], v[0], torch.tensor([N - 1], device="cuda"), 1 if qs > 0 else -1)


def test_a_row_whose_scores_grow_from_small_to_large(pisa):
    # the first keys' dots are ordinary, later ones' are not; and the other way round, for negative ones
    N, d = 600, 64
    q, k, v, kp, vp, table, layer, _ = setup(pisa, 2, 2, d, N, N, 5, 1.0, 1.0)
    q = q.clone()
    q[0, 0], q[0, 1] = 1.0, -1.0
    k = torch.zeros_like(k)
    k[:, :, :200] = 2.0 ** 4
    k[:, :, 200:400] = 2.0 ** 24
    k[:, :, 400:] = 2.0 ** 60
    kk, table = R.paginate(k.cpu().to(torch.bfloat16), [N], seed=5)
    vp, _ = R.paginate(v.cpu(), [N], seed=5)
    layer_out = layer.dense_prefill(q.to(torch.bfloat16), kk.cuda(), vp.cuda(), table.cuda(), i32([N]))
    check(layer_out[0], q[0], k[0], v[0], torch.arange(N, device="cuda"), 1)


def test_large_values_without_weight(pisa):
    # far keys' values are large, and their weights nothing: a prompt that is split over the keys
    N, n, d, H = 6000, 30, 64, 2
    g = torch.Generator().manual_seed(6)
    k, v, q = (torch.randn(1, H, x, d, generator=g) for x in (N, N, n))
    v[:, :, :4000] = 1e35
    k, v, q = (x.to(torch.bfloat16) for x in (k, v, q))
    kp, table = R.paginate(k, [N], seed=1)
    vp, _ = R.paginate(v, [N], seed=1)
    slopes = torch.full((H,), 0.5, device="cuda")
    layer = pisa.PagedAttention(pisa.make_params(1, N, H, H, d), n=n)
    pos = torch.arange(N - n, N, device="cuda")
    q, k, v, kp, vp, table = (x.cuda() for x in (q, k, v, kp, vp, table))
    out = layer.dense_prefill(q, kp, vp, table, i32([N]), mask=pisa.AttentionMask(slopes=slopes))
    want, tol = R.dense(q[0], k[0], v[0], N, pos, d ** -0.5, slopes=slopes)
    R.within(out[0], want, tol)
    one = layer.dense_decode(q[:, :, -1].contiguous(), kp, vp, table, i32([N]), mask=pisa.AttentionMask(slopes=slopes))
    R.within(one[0], want[:, -1], tol[:, -1])
