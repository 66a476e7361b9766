"""GPU tests of appending with head norms and into 8-bit pages, and of reading
back: against 64-bit forms, at row edges, with faults in device data."""
import pytest
import torch

import cache_ref as C
import paged_ref as R
from test_gpu_paged_append import MARK, rope_table

pytestmark = pytest.mark.gpu
CODE, SCALE = 0x55, 99  # what untouched pages hold


@pytest.fixture(scope="module")
def pisa():
    from pyramid_top_block_mean_gb300 import pisa as m
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def setup(pisa, B, N, n, Hq, Hkv, d, dtype, in8, seed, spare=2):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(seed)
    nb = -(-N // 64)
    qkv = torch.randn(B, n, Hq + 2 * Hkv, d, generator=g).to(dt).cuda()
    q, k, v = (x.transpose(1, 2) for x in (qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]))
    table = torch.randperm(B * nb + spare, generator=g)[:B * nb].reshape(B, nb).to(torch.int32).cuda()
    shape = (B * nb + spare, Hkv, 64, d)
    scales = None
    if in8:
        pools = [torch.full(shape, CODE, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
        scales = torch.full((2,) + shape[:3], SCALE, dtype=torch.uint8, device="cuda")
    else:
        pools = [torch.full(shape, MARK, dtype=dt, device="cuda") for _ in range(2)]
    p = pisa.make_params(B, N, Hq, Hkv, d, dtype=dtype)
    ws = torch.empty(pisa.paged_workspace_bytes(p, n), dtype=torch.uint8, device="cuda")
    w = [(1 + 0.3 * torch.randn(d, generator=g)).cuda() for _ in range(2)]
    return p, q, k, v, pools, table, ws, scales, w


def check_rows(codes, scale, y, t):
    """Rows of codes with their scales against y, known to be within t of what was rounded."""
    top, top_t = y.abs().amax(-1), t.amax(-1)
    lo, hi = C.scale_of((top - top_t).clamp_min(0)), C.scale_of(top + top_t)
    s = scale.long()
    assert bool(((s == lo) | (s == hi)).all()), "scales"
    R.within(C.numbers(codes, scale), y, t + C.half_step(y.abs() + t, s[..., None]), "codes")


def check(q, k, v, pools, scales, table, lens, new, rope, inter, weights, eps, q_out, k_out):
    half_ulp = torch.finfo(q.dtype).eps / 2
    touched = torch.zeros(pools[0].shape[0], 64, dtype=torch.bool, device="cuda")
    for b, (length, cnt) in enumerate(zip(lens, new)):
        pos = torch.arange(length - cnt, length, device="cuda")
        page, slot = table[b, pos // 64].long(), pos % 64
        touched[page, slot] = True
        for x, w, got in ((q, weights[0], q_out), (k, weights[1], k_out)):
            y, t = C.norm_rotate(x[b, :, :cnt], w, eps, rope, pos, inter)
            R.within(got[b, :, :cnt], y, t + half_ulp * (y.abs() + t) + 1e-37, "normed and rotated rows")
            assert bool((got[b, :, cnt:] == MARK).all()), "rows behind the new tokens were written"
        for x, w, which in ((k, weights[1], 0), (v, None, 1)):
            y, t = C.norm_rotate(x[b, :, :cnt], w, eps, rope if which == 0 else None, pos, inter)
            got = pools[which].view(torch.uint8) if scales is not None else pools[which]
            got = got[page, :, slot].transpose(0, 1)
            if scales is None:
                R.within(got, y, t + half_ulp * (y.abs() + t) + 1e-37, "pages")
            else:
                check_rows(got.contiguous().view(torch.float8_e4m3fn), scales[which][page, :, slot].transpose(0, 1), y, t)
    rest = ~touched
    for which in range(2):
        if scales is None:
            assert bool((pools[which].transpose(1, 2)[rest] == MARK).all()), "other positions were written"
        else:
            assert bool((pools[which].view(torch.uint8).transpose(1, 2)[rest] == CODE).all())
            assert bool((scales[which].transpose(1, 2)[rest] == SCALE).all())


@pytest.mark.parametrize("in8,normed", [(False, "qk"), (True, ""), (True, "qk"), (False, "k"), (True, "q")])
@pytest.mark.parametrize("dtype,d,Hq,Hkv,rot,inter", [
    ("bf16", 128, 16, 4, 128, False), ("bf16", 128, 8, 1, 64, False), ("bf16", 64, 4, 4, 64, True),
    ("bf16", 64, 2, 2, 16, True), ("fp32", 64, 4, 2, 64, False), ("fp32", 128, 8, 8, 48, True),
    ("bf16", 128, 5 * 8, 5, 0, False)])
@pytest.mark.parametrize("n,N,lens,new", [
    (1, 300, [300, 1, 65, 64], [1, 1, 1, 1]), (1, 1, [1, 1, 0, 1], [1, 0, 0, 1]),
    (133, 1000, [1000, 500, 133, 3], [133, 1, 132, 3])])
def test_append(pisa, in8, normed, dtype, d, Hq, Hkv, rot, inter, n, N, lens, new):
    p, q, k, v, pools, table, ws, scales, w = setup(pisa, 4, N, n, Hq, Hkv, d, dtype, in8, seed=n + d + rot)
    rope = rope_table(N, rot).cuda() if rot else None
    w = [w[0] if "q" in normed else None, w[1] if "k" in normed else None]
    q_out = torch.full((4, Hq, n, d), MARK, dtype=q.dtype, device="cuda")
    k_out = torch.full((4, Hkv, n, d), MARK, dtype=q.dtype, device="cuda")
    pisa.append_paged(p, k, v, *pools, table, i32(lens), ws, rope, inter, q, q_out, k_out, i32(new), scales=scales,
                      q_norm=w[0], k_norm=w[1], norm_eps=1e-5)
    assert pisa.read_device_status(ws) == 0
    check(q, k, v, pools, scales, table, lens, new, rope, inter, w, 1e-5, q_out, k_out)
    # and read back: the numbers that the rows stand for, exactly
    outs = [torch.full((4, Hkv, n, d), MARK, dtype=q.dtype, device="cuda") for _ in range(2)]
    pisa.read_paged(p, *outs, *pools, table, i32(lens), ws, i32(new), scales)
    assert pisa.read_device_status(ws) == 0
    for out, which in zip(outs, range(2)):
        have = C.numbers(pools[which], scales[which]) if in8 else pools[which].double()
        for b, (length, cnt) in enumerate(zip(lens, new)):
            pos = torch.arange(length - cnt, length, device="cuda")
            assert torch.equal(out[b, :, :cnt].double(), have[table[b, pos // 64].long(), :, pos % 64].transpose(0, 1))
            assert bool((out[b, :, cnt:] == MARK).all())


def test_four_rows_a_thread(pisa):
    """Enough rows for the form of the kernel that takes four of them a thread."""
    for dtype, in8, normed in (("bf16", True, True), ("bf16", False, True), ("bf16", True, False), ("fp32", True, True)):
        B, n, N = 2, 2500, 2600
        p, q, k, v, pools, table, ws, scales, w = setup(pisa, B, N, n, 16, 4, 128, dtype, in8, seed=1)
        w = w if normed else [None, None]
        rope = rope_table(N, 128).cuda()
        q_out, k_out = (torch.full((B, h, n, 128), MARK, dtype=q.dtype, device="cuda") for h in (16, 4))
        lens, new = [2600, 2499], [2500, 2411]
        pisa.append_paged(p, k, v, *pools, table, i32(lens), ws, rope, False, q, q_out, k_out, i32(new), scales=scales,
                          q_norm=w[0], k_norm=w[1])
        check(q, k, v, pools, scales, table, lens, new, rope, False, w, 1e-6, q_out, k_out)


@pytest.mark.parametrize("dtype,Hq,Hkv,d,rot,inter,with_q", [
    ("bf16", 10, 5, 128, 64, True, True), ("bf16", 8, 1, 128, 128, False, True), ("bf16", 5, 5, 64, 48, False, False),
    ("fp32", 6, 3, 64, 64, False, True), ("fp32", 2, 2, 128, 0, False, False)])
@pytest.mark.parametrize("in8", [False, True])
def test_heads_that_are_no_multiple_of_four(pisa, dtype, Hq, Hkv, d, rot, inter, with_q, in8):
    """The same form with groups of fewer than four heads, with and without queries."""
    B, n, N = 4, 8000, 8100
    p, q, k, v, pools, table, ws, scales, w = setup(pisa, B, N, n, Hq, Hkv, d, dtype, in8, seed=2)
    rope = rope_table(N, rot).cuda() if rot else None
    lens, new = [8100, 7999, 8000, 31], [8000, 7911, 0, 30]
    q_out, k_out = (torch.full((B, h, n, d), MARK, dtype=q.dtype, device="cuda") for h in (Hq, Hkv))
    pisa.append_paged(p, k, v, *pools, table, i32(lens), ws, rope, inter, q if with_q else None,
                      q_out if with_q else None, k_out, i32(new), scales=scales, q_norm=w[0], k_norm=w[1])
    assert pisa.read_device_status(ws) == 0
    if not with_q:  # (what check() looks at besides)
        pisa.append_paged(p, k, v, *pools, table, i32(lens), ws, rope, inter, q, q_out, None, i32(new), scales=scales,
                          q_norm=w[0], k_norm=w[1])
    check(q, k, v, pools, scales, table, lens, new, rope, inter, w, 1e-6, q_out, k_out)


def edge_rows(d, dt):
    """Rows at the edges of the scales: zero, at and just over 448 times a power, large, small, not finite."""
    rows = []
    for top in (0.0, 448.0, 450.0, 447.0, 224.0, 1.75, 1.7578125, 7.0 * 2.0 ** 60, 2.9e38, 3.3e38, 448.0 * 2.0 ** -117,
                1.2e-38, 1e-40, float("inf"), -float("inf"), float("nan"), 57344.0, 57600.0, 3.0e5):
        x = torch.linspace(-1, 1, d) * (top if top == top and abs(top) < float("inf") else 1.0)
        x[5] = top
        rows.append(x)
    return torch.stack(rows).to(dt)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_at_the_edges(pisa, dtype, d):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rows = edge_rows(d, dt)
    n = rows.shape[0]
    p = pisa.make_params(1, n, 1, 1, d, dtype=dtype)
    kp, vp, scales = pisa.quantized_pages(p, 2)
    ws = torch.empty(pisa.paged_workspace_bytes(p, n), dtype=torch.uint8, device="cuda")
    k, v = rows[None, None].cuda(), rows.flip(0)[None, None].contiguous().cuda()
    table = i32([[1]])
    pisa.append_paged(p, k, v, kp, vp, table, i32([n]), ws, scales=scales)
    out = [torch.empty(1, 1, n, d, dtype=dt, device="cuda") for _ in range(2)]
    pisa.read_paged(p, *out, kp, vp, table, i32([n]), ws, scales=scales)
    for x, pages, s, y in ((k, kp, scales[0], out[0]), (v, vp, scales[1], out[1])):
        codes, want = C.quantize(x[0, 0].cpu())
        assert torch.equal(s[1, 0, :n].cpu(), want)
        assert torch.equal(pages[1, 0, :n].view(torch.uint8).cpu() & 0x7f, codes.view(torch.uint8) & 0x7f)
        back = C.numbers(codes, want)
        assert torch.allclose(y[0, 0].cpu().double(), back, rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_every_code_and_scale_is_read_exactly(pisa, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    p = pisa.make_params(1, 64 * 4, 1, 1, 64, dtype=dtype)
    ws = torch.empty(512, dtype=torch.uint8, device="cuda")
    codes = torch.arange(256, dtype=torch.uint8).view(4, 64)
    codes[(codes & 127) == 127] = 0
    pages = codes[:, None, None].expand(4, 1, 64, 64).contiguous().cuda()  # page j: codes 64 j .. 64 j + 63 in each row
    for first in (10, 71, 132, 183):
        row = torch.arange(first, first + 64)
        row[-1] = 255
        scales = row.to(torch.uint8).expand(2, 4, 1, 64).contiguous().cuda()
        out = torch.zeros(1, 1, 256, 64, dtype=dt, device="cuda")
        pisa.read_paged(p, out, None, pages.view(torch.float8_e4m3fn), pages.view(torch.float8_e4m3fn),
                        i32([[0, 1, 2, 3]]), i32([256]), ws, scales=scales)
        want = C.numbers(pages, scales[0])[:, 0].reshape(256, 64)
        assert torch.allclose(out[0, 0].double(), want, rtol=0, atol=0, equal_nan=True)


@pytest.mark.parametrize("size", [1e-30, 1e-12, 1.0, 1e15, 1e25, 3e37])
def test_norms_of_any_size(pisa, size):
    g = torch.Generator().manual_seed(3)
    for d, dtype in ((64, "fp32"), (128, "bf16")):
        dt = torch.bfloat16 if dtype == "bf16" else torch.float32
        p = pisa.make_params(1, 70, 2, 1, d, dtype=dtype)
        x = (torch.randn(1, 2, 70, d, generator=g) * size).clamp(-3.3e38, 3.3e38).to(dt).cuda()
        w = (1 + torch.rand(d, generator=g)).cuda()
        pool = torch.zeros(2, 1, 64, d, dtype=dt, device="cuda")
        ws = torch.empty(pisa.paged_workspace_bytes(p, 70), dtype=torch.uint8, device="cuda")
        out = torch.zeros_like(x)
        pisa.append_paged(p, x[:, :1], x[:, :1], pool, pool.clone(), i32([[0, 1]]), i32([70]), ws, q=x, q_out=out,
                          q_norm=w, norm_eps=1e-6)
        y, t = C.norm_rotate(x, w, 1e-6, None, None, False)
        # a product below fp32's normal range is off by 2^-149
        R.within(out, y, t + torch.finfo(dt).eps / 2 * (y.abs() + t) + 2e-38, "normed")


@pytest.mark.parametrize("n", [70, 6500])
@pytest.mark.parametrize("size,weight,eps", [(3e37, 1e-3, 1e-6), (1e-15, 1e30, 1e-30)])
def test_norms_whose_factor_times_the_weight_leaves_fp32(pisa, size, weight, eps, n):
    """The quotient x / rms is near one where 1 / rms and the weight are at the ends of fp32's range."""
    g = torch.Generator().manual_seed(4)
    p = pisa.make_params(1, n, 16, 4, 64, dtype="fp32")
    q, k = ((torch.randn(1, h, n, 64, generator=g) * size).clamp(-3.3e38, 3.3e38).cuda() for h in (16, 4))
    w = ((1 + torch.rand(64, generator=g)) * weight).cuda()
    pages = -(-n // 64)
    pool = torch.zeros(pages, 4, 64, 64, device="cuda")
    ws = torch.empty(pisa.paged_workspace_bytes(p, n), dtype=torch.uint8, device="cuda")
    q_out, k_out = torch.zeros_like(q), torch.zeros_like(k)
    pisa.append_paged(p, k, k, pool, pool.clone(), i32([list(range(pages))]), i32([n]), ws, q=q, q_out=q_out,
                      k_out=k_out, q_norm=w, k_norm=w, norm_eps=eps)
    for x, out in ((q, q_out), (k, k_out)):
        y, t = C.norm_rotate(x, w, float(torch.tensor(eps)), None, None, False)
        R.within(out, y, t + 2.0 ** -24 * (y.abs() + t), "normed")


def test_faults(pisa):
    """A length that does not fit skips its sequence; a page outside the pool is not written and not read."""
    p, q, k, v, pools, table, ws, scales, w = setup(pisa, 3, 300, 70, 4, 2, 64, "bf16", True, seed=9)
    lens, new = [300, 40, 200], [70, 70, 70]  # the second has fewer positions than new tokens
    table[2, 2] = table.numel() + 100
    before = [x.view(torch.uint8).clone() for x in pools]
    pisa.append_paged(p, k, v, *pools, table, i32(lens), ws, scales=scales, new_lens=i32(new), k_norm=w[1])
    assert pisa.read_device_status(ws) == pisa.DEV_BAD_SEQ_LEN
    out = [torch.full((3, 2, 70, 64), MARK, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pisa.read_paged(p, *out, *pools, table, i32(lens), ws, i32(new), scales)
    assert pisa.read_device_status(ws) == pisa.DEV_BAD_SEQ_LEN
    for which in range(2):
        for j in range(table.shape[1]):
            assert torch.equal(pools[which].view(torch.uint8)[table[1, j].long()], before[which][table[1, j].long()])
        assert bool((out[which][1] == MARK).all())
        # sequence 2: positions 130 .. 199; 130 .. 191 lie in the page that is not there
        assert bool((out[which][2, :, :62] == MARK).all()) and not bool((out[which][2, :, 62:] == MARK).any())
    table[2, 2] = -1
    pisa.append_paged(p, k, v, *pools, table, i32([300, 100, 200]), ws, scales=scales, new_lens=i32(new))
    assert pisa.read_device_status(ws) == pisa.DEV_BAD_INDEX
    pisa.read_paged(p, *out, *pools, table, i32([300, 100, 200]), ws, i32(new), scales)
    assert pisa.read_device_status(ws) == pisa.DEV_BAD_INDEX


def test_keys_in_place(pisa):
    """k_out and q_out may be k and q themselves."""
    p, q, k, v, pools, table, ws, scales, w = setup(pisa, 2, 150, 40, 8, 2, 64, "bf16", True, seed=5)
    rope = rope_table(150, 64).cuda()
    q0, k0, v0 = (x.contiguous() for x in (q, k, v))
    want_q, want_k = torch.empty_like(q0), torch.empty_like(k0)
    pisa.append_paged(p, k0, v0, *pools, table, i32([150, 40]), ws, rope, False, q0, want_q, want_k, scales=scales,
                      q_norm=w[0], k_norm=w[1])
    first = [x.view(torch.uint8).clone() for x in pools] + [scales.clone()]
    pisa.append_paged(p, k0, v0, *pools, table, i32([150, 40]), ws, rope, False, q0, q0, k0, scales=scales,
                      q_norm=w[0], k_norm=w[1])
    assert torch.equal(q0, want_q) and torch.equal(k0, want_k)
    assert all(torch.equal(a, b) for a, b in zip(first, [x.view(torch.uint8) for x in pools] + [scales]))


@pytest.mark.parametrize("n", [70, 6500])
@pytest.mark.parametrize("eps", [1e35, 3e38, 3.4e38])
@pytest.mark.parametrize("size", [1.0, 3e18, 1e19, 1e25])
def test_norms_with_a_large_eps(pisa, size, eps, n):
    """eps counts in rows whose squares leave fp32's range, too, and their sum with it may."""
    g = torch.Generator().manual_seed(5)
    p = pisa.make_params(1, n, 16, 4, 64, dtype="fp32")
    q, k = ((torch.randn(1, h, n, 64, generator=g) * size).cuda() for h in (16, 4))
    w = ((1 + torch.rand(64, generator=g)) * 1e3).cuda()
    pages = -(-n // 64)
    pool = torch.zeros(pages, 4, 64, 64, device="cuda")
    ws = torch.empty(pisa.paged_workspace_bytes(p, n), dtype=torch.uint8, device="cuda")
    q_out, k_out = torch.zeros_like(q), torch.zeros_like(k)
    pisa.append_paged(p, k, k, pool, pool.clone(), i32([list(range(pages))]), i32([n]), ws, q=q, q_out=q_out,
                      k_out=k_out, q_norm=w, k_norm=w, norm_eps=eps)
    for x, out in ((q, q_out), (k, k_out)):
        y, t = C.norm_rotate(x, w, float(torch.tensor(eps)), None, None, False)
        R.within(out, y, t + 2.0 ** -24 * (y.abs() + t) + 1e-37, "normed")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("in8,inter", [(False, False), (True, False), (True, True)])
def test_prompts_in_place(pisa, dtype, in8, inter):
    """test_keys_in_place of long calls, whose CTAs take several heads."""
    B, n, N = 2, 4000, 4100
    p, q, k, v, pools, table, ws, scales, w = setup(pisa, B, N, n, 16, 4, 128, dtype, in8, seed=6)
    rope = rope_table(N, 128).cuda()
    q0, k0, v0 = (x.contiguous() for x in (q, k, v))
    lens, new = i32([4100, 4000]), i32([4000, 3900])
    want_q, want_k = q0.clone(), k0.clone()  # (rows behind the new tokens stay as they were)
    pisa.append_paged(p, k0, v0, *pools, table, lens, ws, rope, inter, q0, want_q, want_k, new, scales=scales,
                      q_norm=w[0], k_norm=w[1])
    first = [x.view(torch.uint8).clone() for x in pools]
    pisa.append_paged(p, k0, v0, *pools, table, lens, ws, rope, inter, q0, q0, k0, new, scales=scales, q_norm=w[0],
                      k_norm=w[1])
    assert torch.equal(q0, want_q) and torch.equal(k0, want_k)
    assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(first, pools))
