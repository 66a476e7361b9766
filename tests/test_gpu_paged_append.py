"""GPU tests of pisa_append_paged: rotated keys and queries and plain values
against their 64-bit form, untouched positions left as they were, strided and
in-place calls, ragged lengths, faults in device data."""
import pytest
import torch

import paged_ref as R

pytestmark = pytest.mark.gpu
MARK = 77.0


@pytest.fixture(scope="module")
def pisa():
    from pyramid_top_block_mean_gb300 import pisa as m
    return m


def rope_table(N, rot, seed=0):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(N, dtype=torch.float64)[:, None] * f[None]
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


def setup(pisa, B, N, n, Hq, Hkv, d, dtype, seed, spare=2):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(seed)
    nb = -(-N // 64)
    qkv = torch.randn(B, n, Hq + 2 * Hkv, d, generator=g).to(dt).cuda()
    q, k, v = (x.transpose(1, 2) for x in (qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]))
    table = torch.randperm(B * nb + spare, generator=g)[:B * nb].reshape(B, nb).to(torch.int32).cuda()
    pools = [torch.full((B * nb + spare, Hkv, 64, d), MARK, dtype=dt, device="cuda") for _ in range(2)]
    p = pisa.make_params(B, N, Hq, Hkv, d, dtype=dtype)
    ws = torch.empty(pisa.paged_workspace_bytes(p, n), dtype=torch.uint8, device="cuda")
    return p, q, k, v, pools, table, ws


def check(p, q, k, v, pools, table, lens, new, rope, inter, q_out, k_out, marked=MARK):
    eps = torch.finfo(q.dtype).eps / 2
    kp, vp = pools
    want_k, want_v = torch.full_like(kp, MARK).double(), torch.full_like(vp, MARK)
    tol_k = torch.zeros_like(want_k)
    for b, (length, cnt) in enumerate(zip(lens, new)):
        pos = torch.arange(length - cnt, length, device="cuda")
        for x, got, in ((q, q_out), (k, k_out)):
            if got is None:
                continue
            y, t = R.rotate(x[b, :, :cnt], rope, pos, inter) if rope is not None else (x[b, :, :cnt].double(), 0.0)
            R.within(got[b, :, :cnt], y, t + eps * y.abs() + 1e-30, "rotated rows")
            if marked is not None:
                assert bool((got[b, :, cnt:] == marked).all()), "rows behind the new tokens were written"
        y, t = R.rotate(k[b, :, :cnt], rope, pos, inter) if rope is not None else (k[b, :, :cnt].double(),
                                                                                   torch.zeros_like(k[b, :, :cnt]).double())
        page, slot = table[b, pos // 64].long(), pos % 64
        want_k[page, :, slot] = y.transpose(0, 1)
        tol_k[page, :, slot] = (t + eps * y.abs() + 1e-30).transpose(0, 1)
        want_v[page, :, slot] = v[b, :, :cnt].transpose(0, 1)
    R.within(kp, want_k, tol_k, "key pages")
    assert torch.equal(vp, want_v), "value pages"


@pytest.mark.parametrize("dtype,d,Hq,Hkv,rot,inter", [
    ("bf16", 128, 16, 4, 128, False), ("bf16", 128, 8, 1, 64, False), ("bf16", 64, 4, 4, 64, True),
    ("bf16", 64, 2, 2, 16, True), ("fp32", 64, 4, 2, 64, False), ("fp32", 128, 8, 8, 48, True),
    ("fp32", 128, 1, 1, 16, False), ("bf16", 128, 5 * 8, 5, 0, False)])
@pytest.mark.parametrize("n,N,lens,new", [
    (1, 300, [300, 1, 65, 64], [1, 1, 1, 1]), (1, 1, [1, 1, 0, 1], [1, 0, 0, 1]),
    (70, 197, [197, 70, 64, 150], [70, 70, 0, 21]), (133, 1000, [1000, 500, 133, 3], [133, 1, 132, 3])])
def test_append(pisa, dtype, d, Hq, Hkv, rot, inter, n, N, lens, new):
    p, q, k, v, pools, table, ws = setup(pisa, 4, N, n, Hq, Hkv, d, dtype, seed=n + d + rot)
    rope = rope_table(N, rot).cuda() if rot else None
    lt, nt = torch.tensor(lens, dtype=torch.int32).cuda(), torch.tensor(new, dtype=torch.int32).cuda()
    q_out = torch.full((4, Hq, n, d), MARK, dtype=q.dtype, device="cuda")
    k_out = torch.full((4, Hkv, n, d), MARK, dtype=q.dtype, device="cuda")
    pisa.append_paged(p, k, v, *pools, table, lt, ws, rope, inter, q, q_out, k_out, nt)
    assert pisa.read_device_status(ws) == 0
    check(p, q, k, v, pools, table, lens, new, rope, inter, q_out, k_out)


@pytest.mark.parametrize("dtype,inter", [("bf16", False), ("fp32", True)])
def test_in_place_and_contiguous_inputs(pisa, dtype, inter):
    p, q, k, v, pools, table, ws = setup(pisa, 2, 150, 40, 8, 2, 64, dtype, seed=5)
    rope = rope_table(150, 64).cuda()
    lens, new = [150, 40], [40, 40]
    lt = torch.tensor(lens, dtype=torch.int32).cuda()
    q0, k0, v0 = (x.contiguous() for x in (q, k, v))
    q1, k1 = q0.clone(), k0.clone()
    pisa.append_paged(p, k1, v0, *pools, table, lt, ws, rope, inter, q1, q1, k1)  # new_lens null: n each
    check(p, q0, k0, v0, pools, table, lens, new, rope, inter, q1, k1, marked=None)


def test_broadcast_inputs(pisa):
    # one row for all heads, one for all tokens: strides of zero
    p, q, k, v, pools, table, ws = setup(pisa, 2, 150, 40, 8, 2, 64, "bf16", seed=11)
    rope = rope_table(150, 64).cuda()
    q, k, v = q[:, :1].expand(-1, 8, -1, -1), k[:, :, :1].expand(-1, -1, 40, -1), v[:1].expand(2, -1, -1, -1)
    q_out = torch.full((2, 8, 40, 64), MARK, dtype=q.dtype, device="cuda")
    lt = torch.tensor([150, 40], dtype=torch.int32).cuda()
    pisa.append_paged(p, k, v, *pools, table, lt, ws, rope, False, q, q_out)
    assert pisa.read_device_status(ws) == 0
    check(p, q, k, v, pools, table, [150, 40], [40, 40], rope, False, q_out, None)


def test_without_queries(pisa):
    p, _, k, v, pools, table, ws = setup(pisa, 2, 150, 40, 8, 2, 64, "bf16", seed=6)
    rope = rope_table(150, 64).cuda()
    lt = torch.tensor([150, 40], dtype=torch.int32).cuda()
    pisa.append_paged(p, k, v, *pools, table, lt, ws, rope)
    check(p, k, k, v, pools, table, [150, 40], [40, 40], rope, False, None, None)


def test_lengths_that_do_not_fit_and_pages_outside_the_pool(pisa):
    p, q, k, v, pools, table, ws = setup(pisa, 6, 200, 10, 4, 2, 64, "bf16", seed=7)
    rope = rope_table(200, 64).cuda()
    q_out = torch.full((6, 4, 10, 64), MARK, dtype=q.dtype, device="cuda")
    # sequences 1..4 do not fit: past N, new > n, new > length, negative
    lens, new = [100, 201, 100, 5, -1, 64], [10, 10, 11, 6, 0, 10]
    lt, nt = torch.tensor(lens, dtype=torch.int32).cuda(), torch.tensor(new, dtype=torch.int32).cuda()
    pisa.append_paged(p, k, v, *pools, table, lt, ws, rope, False, q, q_out, None, nt)
    assert pisa.read_device_status(ws) == pisa.DEV_BAD_SEQ_LEN
    check(p, q, k, v, pools, table, [100, 0, 0, 0, 0, 64], [10, 0, 0, 0, 0, 10], rope, False, q_out, None)
    for bad in (-1, pools[0].shape[0], 2 ** 31 - 1):
        p, q, k, v, pools, table, ws = setup(pisa, 2, 200, 10, 4, 2, 64, "bf16", seed=8)
        table[1, 1] = bad  # tokens 64..67 of sequence 1 go nowhere, 58..63 to page 0 of it
        q_out = torch.full((2, 4, 10, 64), MARK, dtype=q.dtype, device="cuda")
        lens = [100, 68]
        pisa.append_paged(p, k, v, *pools, table, torch.tensor(lens, dtype=torch.int32).cuda(), ws, rope, False, q,
                          q_out)
        assert pisa.read_device_status(ws) == pisa.DEV_BAD_INDEX
        y, t = R.rotate(q[1], rope, torch.arange(58, 68, device="cuda"), False)
        R.within(q_out[1], y, t + 2.0 ** -8 * y.abs() + 1e-30)
        kp = pools[0][table[1, 0].long(), :, 58:]
        y, t = R.rotate(k[1, :, :6], rope, torch.arange(58, 64, device="cuda"), False)
        R.within(kp, y, t + 2.0 ** -8 * y.abs() + 1e-30)
        written = sum(int((pools[1][i] != MARK).any(dim=-1).sum()) for i in range(pools[1].shape[0]))
        assert written == 2 * (10 + 6)


def test_offsets_past_32_bits(pisa):
    # 2^22 + pages of 1024 elements and more: the last page starts past 2^32 elements
    Hkv, d = 8, 128
    num = 2 ** 32 // (Hkv * 64 * d) + 3
    kp = torch.empty(num, Hkv, 64, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    kp[-1], vp[-1] = MARK, MARK
    p = pisa.make_params(1, 128, 8, Hkv, d)
    ws = torch.empty(pisa.paged_workspace_bytes(p, 2), dtype=torch.uint8, device="cuda")
    k = torch.randn(1, Hkv, 2, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    table = torch.tensor([[0, num - 1]], dtype=torch.int32, device="cuda")
    pisa.append_paged(p, k, -k, kp, vp, table, torch.tensor([67], dtype=torch.int32, device="cuda"), ws)
    assert pisa.read_device_status(ws) == 0
    assert torch.equal(kp[-1][:, 1:3], k[0]) and torch.equal(vp[-1][:, 1:3], -k[0])
    assert bool((kp[-1][:, 3:] == MARK).all()) and bool((kp[-1][:, :1] == MARK).all())


def test_more_sequences_than_a_grid_dimension(pisa):
    B = 70000
    p, q, k, v, pools, table, ws = setup(pisa, B, 1, 1, 1, 1, 64, "bf16", seed=9)
    lt = torch.ones(B, dtype=torch.int32, device="cuda")
    pisa.append_paged(p, k, v, *pools, table, lt, ws)
    assert pisa.read_device_status(ws) == 0
    assert torch.equal(pools[0][table[:, 0].long()][:, :, 0], k[:, :, 0])
    assert torch.equal(pools[1][table[:, 0].long()][:, :, 0], v[:, :, 0])
