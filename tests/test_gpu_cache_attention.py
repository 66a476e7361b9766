"""GPU tests of attention over 8-bit pages against its 64-bit form on the
numbers that the pages stand for, every element within the bound derived in
paged_ref.  Positions behind a sequence's length hold NaN's codes and scales
of 255 and below."""
import pytest
import torch

import cache_ref as C
import paged_ref as R
from test_gpu_paged_attention import MARK, i32, slopes_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pisa():
    from pyramid_top_block_mean_gb300 import pisa as m
    return m


def cache(B, Hkv, N, d, lens, seed, spread=3, change=None):
    """Rows whose sizes differ by up to 2^spread, so that scales do too."""
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(B, Hkv, N, d, generator=g) for _ in range(2))
    v = v * 2.0 ** torch.randint(-spread, spread + 1, (B, Hkv, N, 1), generator=g)
    k = k * 2.0 ** (-torch.rand(B, Hkv, N, 1, generator=g) * spread)
    if change is not None:
        change(k, v)
    kp, ks, table, k = C.paginate(k, lens, seed)
    vp, vs, _, v = C.paginate(v, lens, seed)
    return k.cuda(), v.cuda(), kp.cuda(), vp.cuda(), torch.stack([ks, vs]).contiguous().cuda(), table.cuda()


# ---------------------------------------------------------------- one token
def run_decode(pisa, B, Hq, Hkv, d, N, lens, seed=0, softcap=0.0, window=0, slopes=False, first=None, amp=2.0,
               scale=0.0, change=None):
    k, v, kp, vp, scales, table = cache(B, Hkv, N, d, lens, seed, change=change)
    q = (torch.randn(B, Hq, d, generator=torch.Generator().manual_seed(seed + 1)) * amp).to(torch.bfloat16).cuda()
    p = pisa.make_params(B, N, Hq, Hkv, d, scale=scale)
    layer = pisa.PagedAttention(p)
    sl = slopes_of(Hq) if slopes else None
    mask = None
    if softcap or window or slopes or first is not None:
        mask = pisa.AttentionMask(softcap, window, sl, None if first is None else i32(first)[:, None].contiguous())
    out = layer.dense_decode(q, kp, vp, table, i32(lens), mask=mask, scales=scales)
    status = layer.device_status()
    for b, n in enumerate(lens):
        if n < 1 or n > N:
            assert bool((out[b] == 0).all())
            continue
        want, tol = R.dense(q[b][:, None], k[b], v[b], n, torch.tensor([n - 1], device="cuda"),
                            scale or d ** -0.5, softcap, window, sl, None if first is None else i32([first[b]]))
        R.within(out[b], want[:, 0], tol[:, 0], f"sequence {b} of length {n}")
    return status


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (16, 4), (16, 2), (24, 3)])
def test_decode_lengths(pisa, d, Hq, Hkv):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 192, 193, 257, 700, 1000]
    assert run_decode(pisa, len(lens), Hq, Hkv, d, 1000, lens, seed=d + Hq) == 0


@pytest.mark.parametrize("kw", [dict(softcap=50.0), dict(softcap=1.5, amp=8.0), dict(window=1), dict(window=64),
                                dict(window=100), dict(slopes=True), dict(softcap=30.0, window=333, slopes=True),
                                dict(scale=0.5), dict(first=[0, 1, 64, 0, 129, 600]),
                                dict(first=[1, 1000, 65, 2 ** 31 - 1, -5, 200], window=250),
                                dict(softcap=3e4, amp=20.0), dict(amp=60.0)])
def test_decode_masks_and_scores(pisa, kw):
    assert run_decode(pisa, 6, 8, 2, 128, 777, [1, 64, 65, 300, 777, 641], seed=3, **kw) == 0


@pytest.mark.parametrize("B,N,Hq,Hkv", [(1, 40000, 8, 1), (2, 20011, 16, 8), (1, 5, 1, 1), (300, 130, 4, 2),
                                        (12, 4000, 16, 2)])
@pytest.mark.parametrize("d", [128, 64])
def test_decode_split_over_the_gpu(pisa, B, N, Hq, Hkv, d):
    lens = [max(1, N - 37 * b) for b in range(B)]
    assert run_decode(pisa, B, Hq, Hkv, d, N, lens, seed=B) == 0


def test_decode_uneven_batch(pisa):
    lens = [1] * 40 + [9000] + [64] * 40 + [1, 3000]
    assert run_decode(pisa, len(lens), 8, 2, 64, 9000, lens, seed=11) == 0


def test_decode_bad_lengths(pisa):
    assert run_decode(pisa, 5, 8, 2, 64, 300, [300, 0, 301, -3, 10], seed=12) == pisa.DEV_BAD_SEQ_LEN


@pytest.mark.parametrize("d", [64, 128])
def test_decode_rows_of_any_size(pisa, d):
    """Zero rows, and rows from 2^-100 to 2^60 of one: the powers of the values, and of keys and queries against each
    other, may be anything that fp32 holds."""
    def far(k, v):
        k[0, :, ::7], v[0, :, ::5], v[0, :, 3::5] = 0.0, 0.0, v[0, :, 3::5] * 1e-12
        k[1] *= 2.0 ** 40
        v[1] *= 2.0 ** -100
        k[2] *= 2.0 ** -60
        v[2, :, ::3] *= 2.0 ** 60
        k[3, :, 100:200] *= 2.0 ** 10  # scales over 134
        v[3, :, 50:150] *= 2.0 ** 20

    lens, B = [300, 290, 280, 270], 4
    k, v, kp, vp, scales, table = cache(B, 2, 300, d, lens, 5, change=far)
    q = torch.randn(B, 4, d, generator=torch.Generator().manual_seed(6)) * 2
    q[1] *= 2.0 ** -40
    q[2] *= 2.0 ** 60
    q[3] *= 2.0 ** -8
    q = q.to(torch.bfloat16).cuda()
    layer = pisa.PagedAttention(pisa.make_params(B, 300, 4, 2, d))
    out = layer.dense_decode(q, kp, vp, table, i32(lens), scales=scales)
    for b, n in enumerate(lens):
        want, tol = R.dense(q[b][:, None], k[b], v[b], n, torch.tensor([n - 1], device="cuda"), d ** -0.5)
        R.within(out[b], want[:, 0], tol[:, 0], f"sequence {b}")


@pytest.mark.parametrize("Hq", [2, 8])
def test_decode_queries_and_keys_at_both_ends_of_the_range(pisa, Hq):
    """Queries up to 2^127 and keys that make moderate scores of them, and the other way round."""
    d, lens = 128, [70, 70]

    def far(k, v):
        k[0] *= 2.0 ** -112
        k[1] *= 2.0 ** 110

    k, v, kp, vp, scales, table = cache(2, 1, 70, d, lens, 8, spread=0, change=far)
    q = torch.randn(2, Hq, d, generator=torch.Generator().manual_seed(9))
    q[0] *= 2.0 ** 125 / q[0].abs().amax(dim=-1, keepdim=True) * 3.5
    q[1] *= 2.0 ** -112
    q = q.to(torch.bfloat16).cuda()
    layer = pisa.PagedAttention(pisa.make_params(2, 70, Hq, 1, d, scale=2.0 ** -12))
    out = layer.dense_decode(q, kp, vp, table, i32(lens), scales=scales)
    assert layer.device_status() == 0
    for b in range(2):
        want, tol = R.dense(q[b][:, None], k[b], v[b], 70, torch.tensor([69], device="cuda"), 2.0 ** -12)
        R.within(out[b], want[:, 0], tol[:, 0], f"sequence {b}")


def test_decode_rows_that_are_not_finite(pisa):
    """A row that was not finite reads as NaN: so do the heads that see it, and no other."""
    def poke(k, v):
        v[0, 0, 70, 3] = float("inf")
        k[1, 1, 10, 9] = R.NAN
        k[2, 0, 20, 0] = v[2, 1, 21, 0] = R.NAN

    k, v, kp, vp, scales, table = cache(3, 2, 300, 64, [300] * 3, 5, change=poke)
    assert int((scales[:, table[:2].long().flatten()] == 255).sum()) >= 2
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    layer = pisa.PagedAttention(pisa.make_params(3, 300, 4, 2, 64))
    mask = pisa.AttentionMask(first_key=i32([[0], [0], [22]]))  # the third sequence's are out of sight
    out = layer.dense_decode(q, kp, vp, table, i32([300] * 3), mask=mask, scales=scales)
    assert bool(torch.isnan(out[0, :2]).all()) and bool(torch.isfinite(out[0, 2:]).all())
    assert bool(torch.isnan(out[1, 2:]).all()) and bool(torch.isfinite(out[1, :2]).all())
    want, tol = R.dense(q[2][:, None], k[2], v[2], 300, torch.tensor([299], device="cuda"), 0.125, first=i32([22]))
    R.within(out[2], want[:, 0], tol[:, 0])


@pytest.mark.parametrize("d", [64, 128])
def test_decode_small_elements_of_rows(pisa, d):
    """Elements far below their row's largest: subnormal codes, and queries whose heads and dims differ widely."""
    def far(k, v):
        v[:, :, :, 1:] *= 2.0 ** -12
        k[:, :, :, :d // 2] *= 2.0 ** -11
    lens, B = [300, 290], 2
    k, v, kp, vp, scales, table = cache(B, 2, 300, d, lens, 7, change=far)
    assert int(((kp.view(torch.uint8) & 0x78) == 0).sum()) > 1000  # subnormal codes
    q = torch.randn(B, 8, d, generator=torch.Generator().manual_seed(8)) * 4
    q[:, :, d // 2:] *= 2.0 ** -11
    q *= 2.0 ** torch.arange(-8, 8, 2)[None, :, None]
    q = q.to(torch.bfloat16).cuda()
    layer = pisa.PagedAttention(pisa.make_params(B, 300, 8, 2, d))
    out = layer.dense_decode(q, kp, vp, table, i32(lens), scales=scales)
    for b, n in enumerate(lens):
        want, tol = R.dense(q[b][:, None], k[b], v[b], n, torch.tensor([n - 1], device="cuda"), d ** -0.5)
        R.within(out[b], want[:, 0], tol[:, 0], f"sequence {b}")


def test_decode_queries_that_are_not_finite(pisa):
    k, v, kp, vp, scales, table = cache(1, 2, 300, 64, [300], 5)
    q = torch.randn(1, 8, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    q[0, 1, 60], q[0, 6, 0] = float("inf"), R.NAN
    layer = pisa.PagedAttention(pisa.make_params(1, 300, 8, 2, 64))
    out = layer.dense_decode(q, kp, vp, table, i32([300]), scales=scales)
    rest = [0, 2, 3, 4, 5, 7]
    want, tol = R.dense(q[0][:, None], k[0], v[0], 300, torch.tensor([299], device="cuda"), 0.125)
    R.within(out[0, rest], want[rest, 0], tol[rest, 0])
    assert bool(torch.isnan(out[0, [1, 6]]).all())


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 1 << 20])
def test_decode_bad_page_counts_as_unseen(pisa, bad):
    k, v, kp, vp, scales, table = cache(2, 2, 300, 64, [300, 300], 4)
    table[0, 2] = bad
    table[1, :] = bad
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    layer = pisa.PagedAttention(pisa.make_params(2, 300, 4, 2, 64))
    keep = torch.ones(1, 300, dtype=torch.bool, device="cuda")
    keep[:, 128:192] = False
    out = layer.dense_decode(q, kp, vp, table, i32([300, 300]), scales=scales)
    assert layer.device_status() == pisa.DEV_BAD_INDEX
    for h in range(4):
        o, t = R.attend(q[0, h:h + 1], k[0, h // 2], v[0, h // 2], keep, 64 ** -0.5)
        R.within(out[0, h], o[0], t[0])
    assert bool((out[1] == 0).all())


@pytest.mark.parametrize("d,Hq,Hkv,K", [(128, 16, 4, 8), (128, 8, 1, 32), (64, 4, 4, 1), (64, 8, 2, 29)])
def test_selected_decode(pisa, d, Hq, Hkv, K):
    lens = [1, 64, 65, 500, 2900, 3000]
    B, N = len(lens), 3000
    k, v, kp, vp, scales, table = cache(B, Hkv, N, d, lens, K)
    g = torch.Generator().manual_seed(K + 1)
    q = torch.randn(B, Hq, d, generator=g).to(torch.bfloat16).cuda()
    idx = torch.randint(-3, 55, (B, Hkv, K + 3), generator=g).to(torch.int32)  # unsorted, repeated, future, negative
    idx[0, 0] = -1  # nothing selected: zeros
    idx[3, :, -1] = idx[3, :, 0]
    idx = idx.cuda()
    layer = pisa.PagedAttention(pisa.make_params(B, N, Hq, Hkv, d, K=K))
    out = layer.selected_decode(q, kp, vp, table, i32(lens), idx, scales=scales)
    assert layer.device_status() == 0
    for b, n in enumerate(lens):
        want, tol = R.selected(q[b], k[b], v[b], n, idx[b], d ** -0.5)
        R.within(out[b], want, tol, f"sequence {b}")
    assert bool((out[0, :Hq // Hkv] == 0).all())


# ------------------------------------------------------------------- prompts
def run_prefill(pisa, Hq, Hkv, d, N, n, lens, new, seed=0, softcap=0.0, window=0, slopes=False, first=None,
                prefix=None, amp=2.0, scale=0.0, status=0, change=None, poke=None):
    B = len(lens)
    k, v, kp, vp, scales, table = cache(B, Hkv, N, d, lens, seed, change=change)
    if poke is not None:
        poke(scales, table)
    q = (torch.randn(B, Hq, n, d, generator=torch.Generator().manual_seed(seed + 1)) * amp).to(torch.bfloat16).cuda()
    p = pisa.make_params(B, N, Hq, Hkv, d, scale=scale)
    ws = torch.empty(pisa.paged_workspace_bytes(p, n), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, MARK)
    sl = slopes_of(Hq) if slopes else None
    mask = None
    if softcap or window or slopes or first is not None or prefix is not None:
        mask = pisa.AttentionMask(softcap, window, sl, first, None if prefix is None else i32(prefix))
    pisa.dense_prefill_paged(p, q, kp, vp, table, i32(lens), ws, out, i32(new), mask, scales=scales)
    assert pisa.read_device_status(ws) == status
    for b in range(B):
        cnt = min(max(new[b], 0), n)
        if not (0 <= new[b] <= min(n, lens[b]) and lens[b] <= N):
            assert bool((out[b, :, :cnt] == 0).all())
        elif cnt:
            pos = torch.arange(lens[b] - cnt, lens[b], device="cuda")
            want, tol = R.dense(q[b, :, :cnt], k[b], v[b], lens[b], pos, scale or d ** -0.5, softcap, window, sl,
                                None if first is None else first[b, :cnt], 0 if prefix is None else prefix[b])
            R.within(out[b, :, :cnt], want, tol, f"sequence {b}")
        assert bool((out[b, :, cnt:] == MARK).all()), "rows behind the new tokens were written"
    scratch = pisa.cache_scratch_bytes(p, n)
    if scratch:  # the same from expanded pages, bit for bit
        wide = torch.full_like(q, MARK)
        pisa.dense_prefill_paged(p, q, kp, vp, table, i32(lens), ws, wide, i32(new), mask, scales=scales,
                                 scratch=torch.full((scratch,), 255, dtype=torch.uint8, device="cuda"))
        assert pisa.read_device_status(ws) == status
        assert torch.equal(torch.nan_to_num(wide, 9.0), torch.nan_to_num(out, 9.0))
    return out


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 2, 2), (64, 16, 2), (128, 3, 3), (128, 4, 2), (128, 8, 2), (128, 8, 1)])
@pytest.mark.parametrize("n,lens,new", [
    (1, [1, 2, 130, 500], [1, 1, 1, 1]), (3, [3, 66, 500, 0], [3, 2, 1, 0]),
    (64, [64, 128, 500, 65], [64, 64, 60, 1]), (129, [129, 130, 500, 256], [129, 65, 127, 128]),
    (300, [300, 311, 500, 299], [300, 300, 257, 299])])
def test_prefill_lengths(pisa, d, Hq, Hkv, n, lens, new):
    run_prefill(pisa, Hq, Hkv, d, 500, n, lens, new, seed=n + d)


@pytest.mark.parametrize("kw", [dict(softcap=50.0), dict(softcap=1.5, amp=8.0), dict(window=1), dict(window=100),
                                dict(slopes=True), dict(prefix=[0, 50, 300, 1000]), dict(scale=0.5),
                                dict(softcap=30.0, window=200, slopes=True, prefix=[10, 0, 400, 250]),
                                dict(softcap=3e4, amp=20.0), dict(amp=60.0)])
@pytest.mark.parametrize("d,Hq,Hkv", [(128, 8, 2), (64, 2, 2)])
def test_prefill_masks_and_scores(pisa, d, Hq, Hkv, kw):
    run_prefill(pisa, Hq, Hkv, d, 600, 280, [280, 281, 600, 400], [280, 200, 280, 100], seed=9, **kw)


@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (2, 2)])
def test_prefill_documents_and_empty_rows(pisa, Hq, Hkv):
    first = torch.zeros(3, 280, dtype=torch.int32)
    pos = torch.arange(280)
    first[0] = pos // 97 * 97                 # three documents
    first[1] = 2 ** 31 - 1                    # no row sees a key
    first[1, ::3] = 5
    first[2] = torch.randint(-10, 700, (280,), generator=torch.Generator().manual_seed(3))  # no order at all
    run_prefill(pisa, Hq, Hkv, 128, 600, 280, [280, 280, 600], [280, 280, 280], seed=10, first=first.cuda())
    run_prefill(pisa, Hq, Hkv, 64, 600, 280, [280, 280, 600], [280, 280, 280], seed=10, first=first.cuda(),
                prefix=[100, 100, 600], window=150)


@pytest.mark.parametrize("n,past,B", [(1, 30000, 1), (16, 30000, 1), (61, 20000, 2), (130, 9000, 1)])
def test_prefill_few_rows_behind_a_long_cache(pisa, n, past, B):
    run_prefill(pisa, 8, 2, 128, past + n, n, [past + n - 100 * b for b in range(B)], [n] * B, seed=n)
    run_prefill(pisa, 8, 2, 64, past + n, n, [past + n - 100 * b for b in range(B)], [n] * B, seed=n, softcap=20.0,
                window=past // 2)


def test_prefill_many_sequences(pisa):
    B = 70
    lens = [1 + 7 * b for b in range(B)]
    run_prefill(pisa, 2, 1, 64, 500, 90, lens, [min(90, x) for x in lens], seed=4)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", [dict(), dict(window=300, softcap=20.0), dict(prefix=[1500, 0, 10], slopes=True)])
def test_prefill_expanded_pages(pisa, d, kw):
    """Prompts long enough to have their pages expanded: ragged, with a sequence of bad lengths, a page outside the
    pool that no row of it sees, and scales over 134."""
    def large(k, v):
        k[1, :, 700:900] *= 2.0 ** 11
        v[0, :, 1000:1100] *= 2.0 ** 20

    def poke(scales, table):
        if kw.get("window"):
            table[0, :5] = -1  # gone: the window has left them
    n = 1100
    p = pisa.make_params(3, 2000, 8, 2, d)
    assert pisa.cache_scratch_bytes(p, n) > 0
    run_prefill(pisa, 8, 2, d, 2000, n, [1777, 1200, 2001], [n, 1001, 500], seed=3, change=large, poke=poke,
                status=pisa.DEV_BAD_SEQ_LEN, **kw)


def test_prefill_expanded_pages_that_are_not_finite(pisa):
    def poke(k, v):
        v[0, 0, 900, 3] = float("inf")
        k[0, 1, 1500, 9] = R.NAN
    n, N = 1100, 1999
    k, v, kp, vp, scales, table = cache(1, 2, N, 64, [N], 6, change=poke)
    table[0, 3] = 1 << 20
    q = (torch.randn(1, 8, n, 64, generator=torch.Generator().manual_seed(7)) * 2).to(torch.bfloat16).cuda()
    layer = pisa.PagedAttention(pisa.make_params(1, N, 8, 2, 64), n=n)
    out = layer.dense_prefill(q, kp, vp, table, i32([N]), scales=scales)[0]
    assert layer._scratch is not None and layer.device_status() == pisa.DEV_BAD_INDEX
    pos = torch.arange(N - n, N, device="cuda")
    for h in range(8):
        sees = pos >= (900 if h < 4 else 1500)
        keep = torch.arange(N, device="cuda")[None] <= pos[:, None]
        keep[:, 192:256] = False  # the page that is not there
        want, tol = R.attend(q[0, h], torch.nan_to_num(k[0, h // 4]), torch.nan_to_num(v[0, h // 4]), keep, 0.125)
        assert bool(torch.isnan(out[h, sees]).all())
        R.within(out[h, ~sees], want[~sees], tol[~sees])


def test_prefill_long_prompt(pisa):
    run_prefill(pisa, 4, 1, 128, 3000, 2500, [3000, 2500], [2500, 2400], seed=7)
    run_prefill(pisa, 4, 1, 64, 3000, 2500, [3000, 2500], [2500, 2400], seed=7)


def test_prefill_bad_lengths(pisa):
    run_prefill(pisa, 8, 2, 64, 300, 70, [300, 301, 60, 100, -1, 70], [70, 70, 70, 71, 3, -2], seed=5,
                status=pisa.DEV_BAD_SEQ_LEN)


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_rows_of_any_size(pisa, d):
    def far(k, v):
        k[0, :, ::7], v[0, :, ::5], v[0, :, 3::5] = 0.0, 0.0, v[0, :, 3::5] * 1e-12
        v[1] *= 2.0 ** -100
        k[1, :, 100:200] *= 2.0 ** 12  # scales over 134
        v[1, :, 50:150] *= 2.0 ** 121
    run_prefill(pisa, 4, 2, d, 300, 200, [300, 290], [200, 180], seed=5, change=far)


def test_prefill_bad_page_counts_as_unseen(pisa):
    k, v, kp, vp, scales, table = cache(1, 2, 300, 64, [300], 4)
    for bad in (-1, 1 << 20):
        table[0, 2] = bad
        q = torch.randn(1, 4, 200, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
        layer = pisa.PagedAttention(pisa.make_params(1, 300, 4, 2, 64), n=200)
        out = layer.dense_prefill(q, kp, vp, table, i32([300]), scales=scales)
        assert layer.device_status() == pisa.DEV_BAD_INDEX
        key, pos = torch.arange(300, device="cuda"), torch.arange(100, 300, device="cuda")
        keep = (key[None] <= pos[:, None]) & (key[None] // 64 != 2)
        for h in range(4):
            o, t = R.attend(q[0, h], k[0, h // 2], v[0, h // 2], keep, 0.125)
            R.within(out[0, h], o, t)


@pytest.mark.parametrize("kw", [dict(), dict(softcap=20.0, slopes=True), dict(window=40)])
@pytest.mark.parametrize("n,N", [(280, 600), (280, 280), (30, 3000)])
@pytest.mark.parametrize("d", [64, 128])
def test_prefill_rows_that_are_not_finite(pisa, d, n, N, kw):
    """A key or value row that was not finite reads as NaN: so do the rows that see it, and no other; the last case
    is split over the keys."""
    Hq, Hkv = 4, 2
    late = N - n // 2  # seen by the later half of the new tokens alone

    def poke(k, v):
        v[0, 0, late, 3] = float("inf")
        k[0, 1, late + 3, 9] = R.NAN

    k, v, kp, vp, scales, table = cache(1, Hkv, N, d, [N], 6, change=poke)
    q = (torch.randn(1, Hq, n, d, generator=torch.Generator().manual_seed(7)) * 2).to(torch.bfloat16).cuda()
    sl = slopes_of(Hq) if kw.get("slopes") else None
    mask = pisa.AttentionMask(kw.get("softcap", 0.0), kw.get("window", 0), sl)
    layer = pisa.PagedAttention(pisa.make_params(1, N, Hq, Hkv, d), n=n)
    out = layer.dense_prefill(q, kp, vp, table, i32([N]), mask=mask, scales=scales)[0]
    assert layer.device_status() == 0
    pos = torch.arange(N - n, N, device="cuda")
    lo, _ = R.spans(pos, N, kw.get("window", 0))
    want, tol = R.dense(q[0], torch.nan_to_num(k[0]), torch.nan_to_num(v[0]), N, pos, d ** -0.5,
                        kw.get("softcap", 0.0), kw.get("window", 0), sl)
    for h in range(Hq):
        at = late if h < 2 else late + 3
        sees = (pos >= at) & (lo <= at)
        assert int(sees.sum()) > 0 and int((~sees).sum()) >= n // 2
        assert bool(torch.isnan(out[h, sees]).all())
        R.within(out[h, ~sees], want[h, ~sees], tol[h, ~sees], "rows that see finite values")
