"""GPU tests of the tanh cap of the dense paged calls: a capped score is off by
a part of itself, not of the cap, so that a cap far above the scores is none.

The score's bound is paged_ref's without the cap's term, and in its place
2^-19 of the capped score: 2^-20.6 where the polynomial stands for tanh(u) / u
(|u| <= 1/2, 6.4e-7), with its six fp32 steps; 1 - 2 / (1 + e^2u) elsewhere:
an exponential off by 2^-22 + 2 |u| 2^-23 of itself, a sum and a reciprocal
(2^-23 each), at most 2^-20.4 of |tanh u| >= 0.46 (largest at u = -1/2)."""
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


def capped(q, k, v, length, pos, scale, softcap, slopes=None):
    """One sequence, causal: q [Hq, T, d] at pos [T], k and v [Hkv, >= length, d].  (out, bound) in 64 bits."""
    G, d = q.shape[0] // k.shape[0], q.shape[-1]
    key = torch.arange(length, device=q.device)
    keep = key[None] <= pos[:, None]
    outs, tols = [], []
    for h in range(q.shape[0]):
        kk, vv, qq = k[h // G, :length].double(), v[h // G, :length].double(), q[h].double()
        x = softcap * torch.tanh(scale * (qq @ kk.t()) / softcap)
        zero = torch.zeros_like(x)
        ds = ((d + 2) * 2.0 ** -23 * torch.where(keep, scale * (qq.abs() @ kk.abs().t()), zero).amax(1, True)
              + 2.0 ** -19 * torch.where(keep, x.abs(), zero).amax(1, True))
        if slopes is not None:
            bias = slopes[h].double() * (key[None] - pos[:, None]).double()
            x = x + bias
            ds = ds + 4 * 2.0 ** -24 * torch.where(keep, bias.abs(), zero).amax(1, True)
        w = torch.softmax(x.masked_fill(~keep, -float("inf")), dim=1)
        o, A = w @ vv, w @ vv.abs()
        outs.append(o)
        tols.append(A * (2.0 ** -8 + 2 * ds + (length + 64) * 2.0 ** -23) + 2.0 ** -8 * o.abs() + 1e-30)
    return torch.stack(outs), torch.stack(tols)


def setup(pisa, Hq, Hkv, d, N, n, seed, amp):
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(1, Hkv, N, d, generator=g).to(torch.bfloat16) for _ in range(2))
    kp, table = R.paginate(k, [N], seed=seed)
    vp, _ = R.paginate(v, [N], seed=seed)
    q = (torch.randn(1, Hq, n, d, generator=g) * amp).to(torch.bfloat16)
    layer = pisa.PagedAttention(pisa.make_params(1, N, Hq, Hkv, d), n=n)
    return q.cuda(), k.cuda(), v.cuda(), kp.cuda(), vp.cuda(), table.cuda(), layer


CAPS = [0.25, 5.0, 50.0, 3e4, 1e5, 1e6, 1e8, 1e12, 1e30]


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("d,Hq,Hkv,amp", [(128, 8, 2, 2.0), (64, 2, 2, 6.0)])
def test_decode(pisa, d, Hq, Hkv, amp, cap):
    q, k, v, kp, vp, table, layer = setup(pisa, Hq, Hkv, d, 700, 1, 3, amp)
    out = layer.dense_decode(q[:, :, 0].contiguous(), kp, vp, table, i32([700]), mask=pisa.AttentionMask(softcap=cap))
    want, tol = capped(q[0], k[0], v[0], 700, torch.tensor([699], device="cuda"), d ** -0.5, cap)
    R.within(out[0][:, None], want, tol)


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("d,Hq,Hkv,amp", [(128, 8, 2, 2.0), (64, 2, 2, 6.0)])
def test_prompt(pisa, d, Hq, Hkv, amp, cap, slopes):
    q, k, v, kp, vp, table, layer = setup(pisa, Hq, Hkv, d, 700, 300, 4, amp)
    sl = (2.0 ** (-8.0 * torch.arange(1, Hq + 1) / Hq)).float().cuda() if slopes else None
    out = layer.dense_prefill(q, kp, vp, table, i32([700]), mask=pisa.AttentionMask(softcap=cap, slopes=sl))
    pos = torch.arange(400, 700, device="cuda")
    want, tol = capped(q[0], k[0], v[0], 700, pos, d ** -0.5, cap, sl)
    R.within(out[0], want, tol)


@pytest.mark.parametrize("cap", [1e6, 1e8])
def test_scores_near_the_cap_beside_small_ones(pisa, cap):
    # one row whose scores reach the cap among rows whose scores are far below it
    q, k, v, kp, vp, table, layer = setup(pisa, 4, 2, 128, 700, 300, 5, 2.0)
    q[:, :, ::37] *= cap / 4
    pos = torch.arange(400, 700, device="cuda")
    want, tol = capped(q[0], k[0], v[0], 700, pos, 128 ** -0.5, cap)
    out = layer.dense_prefill(q, kp, vp, table, i32([700]), mask=pisa.AttentionMask(softcap=cap))
    R.within(out[0], want, tol)
    one = layer.dense_decode(q[:, :, 296].contiguous(), kp, vp, table, i32([697]), mask=pisa.AttentionMask(softcap=cap))
    R.within(one[0], want[:, 296], tol[:, 296])


def test_a_cap_far_above_the_scores_is_none(pisa):
    q, k, v, kp, vp, table, layer = setup(pisa, 8, 2, 128, 700, 300, 6, 2.0)
    pos = torch.arange(400, 700, device="cuda")
    none, tol = R.dense(q[0], k[0], v[0], 700, pos, 128 ** -0.5)
    out = layer.dense_prefill(q, kp, vp, table, i32([700]), mask=pisa.AttentionMask(softcap=1e9))
    R.within(out[0], none, tol)
    one = layer.dense_decode(q[:, :, 299].contiguous(), kp, vp, table, i32([700]), mask=pisa.AttentionMask(softcap=1e9))
    R.within(one[0], none[:, 299], tol[:, 299])


def test_a_row_computed_anew_is_capped_alike(pisa):
    # a value that is not finite at a key that the row does not see
    q, k, v, kp, vp, table, layer = setup(pisa, 4, 2, 64, 700, 300, 7, 2.0)
    vp[int(table[0, 550 // 64]), :, 550 % 64] = R.NAN
    out = layer.dense_prefill(q, kp, vp, table, i32([700]), mask=pisa.AttentionMask(softcap=1e8))
    pos = torch.arange(400, 700, device="cuda")
    want, tol = capped(q[0], k[0], v[0], 700, pos, 0.125, 1e8)
    R.within(out[0][:, :150], want[:, :150], tol[:, :150])
    assert bool(out[0][:, 150:].isnan().all())


@pytest.mark.parametrize("Hq,Hkv,d", [(16, 4, 64), (8, 8, 128), (16, 2, 128)])
@pytest.mark.parametrize("B,n,new,length", [(64, 64, 40, 40), (16, 100, 83, 700), (2, 30, 30, 5000), (70, 1, 1, 200)])
def test_what_no_row_sees_changes_no_bit(pisa, Hq, Hkv, d, B, n, new, length):
    # keys behind the end, in its page and in the page after it, and queries behind the new tokens
    N = length + 100
    g = torch.Generator().manual_seed(n)
    k, v = (torch.randn(B, Hkv, N, d, generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(B, Hq, n, d, generator=g).to(torch.bfloat16).cuda()
    vp, table = R.paginate(v, [N] * B, seed=1)
    vp, table = vp.cuda(), table.cuda()
    layer = pisa.PagedAttention(pisa.make_params(B, N, Hq, Hkv, d), n=n)
    lens, news = i32([length] * B), i32([new] * B)
    for kw in (dict(softcap=20.0), dict(softcap=20.0, slopes=torch.full((Hq,), 0.01, device="cuda"))):
        outs = []
        for keys, queries in ((0.0, 0.0), (1e4, 0.0), (0.0, 1e4), (float("inf"), 0.0), (R.NAN, R.NAN)):
            k[:, :, length:] = keys
            q[:, :, new:] = queries
            kp, _ = R.paginate(k, [N] * B, seed=1)
            out = layer.dense_prefill(q, kp.cuda(), vp, table, lens, new_lens=news, mask=pisa.AttentionMask(**kw))
            outs.append(out[:, :, :new].clone())
            assert layer.device_status() == 0
        for other in outs[1:]:
            assert torch.equal(other, outs[0]), f"{int((other != outs[0]).sum())} elements differ"
