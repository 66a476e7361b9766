"""GPU tests of attention over the paged cache (pisa_dense_decode_paged,
pisa_attend_decode_paged, pisa_dense_prefill_paged) against its 64-bit form,
every element within the bound derived in paged_ref.  Pages behind a
sequence's length, and positions of its last page behind it, hold NaN."""
import pytest
import torch

import paged_ref as R

pytestmark = pytest.mark.gpu
MARK = 77.0


@pytest.fixture(scope="module")
def pisa():
    from pyramid_top_block_mean_gb300 import pisa as m
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cache(B, Hkv, N, d, lens, seed, fill=R.NAN):
    g = torch.Generator().manual_seed(seed)
    k = torch.randn(B, Hkv, N, d, generator=g).to(torch.bfloat16)
    v = torch.randn(B, Hkv, N, d, generator=g).to(torch.bfloat16)
    kp, table = R.paginate(k, [max(0, min(n, N)) for n in lens], seed=seed, fill=fill)
    vp, _ = R.paginate(v, [max(0, min(n, N)) for n in lens], seed=seed, fill=fill)
    return k.cuda(), v.cuda(), kp.cuda(), vp.cuda(), table.cuda()


def slopes_of(Hq):
    return (2.0 ** (-8.0 * torch.arange(1, Hq + 1) / Hq)).float().cuda()


# ---------------------------------------------------------------- one token
def run_decode(pisa, B, Hq, Hkv, d, N, lens, seed=0, softcap=0.0, window=0, slopes=False, first=None, amp=2.0,
               scale=0.0, v_scale=1.0):
    k, v, kp, vp, table = cache(B, Hkv, N, d, lens, seed)
    q = (torch.randn(B, Hq, d, generator=torch.Generator().manual_seed(seed + 1)) * amp).to(torch.bfloat16).cuda()
    p = pisa.make_params(B, N, Hq, Hkv, d, scale=scale)
    layer = pisa.PagedAttention(p)
    sl = slopes_of(Hq) if slopes else None
    mask = None
    if softcap or window or slopes or first is not None:
        mask = pisa.AttentionMask(softcap, window, sl, None if first is None else i32(first)[:, None].contiguous())
    out = layer.dense_decode(q, kp, vp, table, i32(lens), mask=mask)
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
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 197, 700, 1000]
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


@pytest.mark.parametrize("bad", [-1, -2 ** 31, 1 << 20])
def test_decode_bad_page_counts_as_unseen(pisa, bad):
    k, v, kp, vp, table = cache(2, 2, 300, 64, [300, 300], 4)
    table[0, 2] = bad
    table[1, :] = bad
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    layer = pisa.PagedAttention(pisa.make_params(2, 300, 4, 2, 64))
    out = layer.dense_decode(q, kp, vp, table, i32([300, 300]))
    assert layer.device_status() == pisa.DEV_BAD_INDEX
    keep = torch.ones(1, 300, dtype=torch.bool, device="cuda")
    keep[:, 128:192] = False
    for h in range(4):
        o, t = R.attend(q[0, h:h + 1], k[0, h // 2], v[0, h // 2], keep, 64 ** -0.5)
        R.within(out[0, h], o[0], t[0])
    assert bool((out[1] == 0).all())
    idx = torch.full((2, 2, 11), -1, dtype=torch.int32, device="cuda")
    idx[:, :, :3] = i32([0, 2, 4])
    out = layer.selected_decode(q, kp, vp, table, i32([300, 300]), idx)
    assert layer.device_status() == pisa.DEV_BAD_INDEX
    keep[:, 64:256] = False
    for h in range(4):
        o, t = R.attend(q[0, h:h + 1], k[0, h // 2], v[0, h // 2], keep, 64 ** -0.5)
        R.within(out[0, h], o[0], t[0])
    assert bool((out[1] == 0).all())


def test_decode_non_finite_values_in_unseen_places(pisa):
    # keys and values before first_key, and blocks that are not selected, may hold anything
    k, v, kp, vp, table = cache(1, 2, 300, 64, [300], 5)
    for j in range(100):
        page, slot = int(table[0, j // 64]), j % 64
        kp[page, :, slot] = float("inf") if j % 2 else R.NAN
        vp[page, :, slot] = R.NAN
    q = torch.randn(1, 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    layer = pisa.PagedAttention(pisa.make_params(1, 300, 4, 2, 64))
    out = layer.dense_decode(q, kp, vp, table, i32([300]), mask=pisa.AttentionMask(first_key=i32([[100]])))
    want, tol = R.dense(q[0][:, None], k[0], v[0], 300, torch.tensor([299], device="cuda"), 0.125, first=i32([100]))
    R.within(out[0], want[:, 0], tol[:, 0])
    idx = torch.full((1, 2, 11), -1, dtype=torch.int32, device="cuda")
    idx[:, :, 3:5] = i32([4, 2])
    out = layer.selected_decode(q, kp, vp, table, i32([300]), idx)
    want, tol = R.selected(q[0], k[0], v[0], 300, idx[0], 0.125)
    R.within(out[0], want, tol)


def test_decode_non_finite_values_that_are_seen_come_through(pisa):
    k, v, kp, vp, table = cache(1, 2, 300, 64, [300], 5)
    vp[int(table[0, 1]), 0, 7, 3] = float("inf")
    kp[int(table[0, 2]), 1, 9] = R.NAN
    q = torch.randn(1, 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    layer = pisa.PagedAttention(pisa.make_params(1, 300, 4, 2, 64))
    out = layer.dense_decode(q, kp, vp, table, i32([300]))
    assert bool(torch.isinf(out[0, :2, 3]).all()) and bool(torch.isfinite(out[0, :2, 4:]).all())
    assert bool(torch.isnan(out[0, 2:]).all())


# ------------------------------------------------------------ selected blocks
@pytest.mark.parametrize("d,Hq,Hkv,K", [(128, 16, 4, 8), (128, 8, 1, 32), (64, 4, 4, 1), (64, 8, 2, 29)])
def test_selected_decode(pisa, d, Hq, Hkv, K):
    lens = [1, 64, 65, 500, 2900, 3000]
    B, N = len(lens), 3000
    k, v, kp, vp, table = cache(B, Hkv, N, d, lens, K)
    g = torch.Generator().manual_seed(K + 1)
    q = torch.randn(B, Hq, d, generator=g).to(torch.bfloat16).cuda()
    idx = torch.randint(-3, 55, (B, Hkv, K + 3), generator=g).to(torch.int32)  # unsorted, repeated, future, negative
    idx[0, 0] = -1  # nothing selected: zeros
    idx[3, :, -1] = idx[3, :, 0]
    idx = idx.cuda()
    layer = pisa.PagedAttention(pisa.make_params(B, N, Hq, Hkv, d, K=K))
    out = layer.selected_decode(q, kp, vp, table, i32(lens), idx)
    assert layer.device_status() == 0
    for b, n in enumerate(lens):
        want, tol = R.selected(q[b], k[b], v[b], n, idx[b], d ** -0.5)
        R.within(out[b], want, tol, f"sequence {b}")
    assert bool((out[0, :Hq // Hkv] == 0).all())


def test_selected_decode_bad_lengths(pisa):
    k, v, kp, vp, table = cache(3, 2, 300, 64, [300, 300, 300], 5)
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    layer = pisa.PagedAttention(pisa.make_params(3, 300, 4, 2, 64))
    idx = torch.zeros(3, 2, 11, dtype=torch.int32, device="cuda")
    out = layer.selected_decode(q, kp, vp, table, i32([0, 301, 64]), idx)
    assert layer.device_status() == pisa.DEV_BAD_SEQ_LEN
    assert bool((out[:2] == 0).all())
    want, tol = R.selected(q[2], k[2], v[2], 64, idx[2], 0.125)
    R.within(out[2], want, tol)


# ------------------------------------------------------------------- prompts
def run_prefill(pisa, Hq, Hkv, d, N, n, lens, new, seed=0, softcap=0.0, window=0, slopes=False, first=None,
                prefix=None, amp=2.0, scale=0.0, layer=None, status=0, poke=None):
    B = len(lens)
    k, v, kp, vp, table = cache(B, Hkv, N, d, lens, seed)
    if poke is not None:
        poke(kp, vp, table)
    q = (torch.randn(B, Hq, n, d, generator=torch.Generator().manual_seed(seed + 1)) * amp).to(torch.bfloat16).cuda()
    p = pisa.make_params(B, N, Hq, Hkv, d, scale=scale)
    ws = torch.empty(pisa.paged_workspace_bytes(p, n), dtype=torch.uint8, device="cuda")
    out = torch.full_like(q, MARK)
    sl = slopes_of(Hq) if slopes else None
    mask = None
    if softcap or window or slopes or first is not None or prefix is not None:
        mask = pisa.AttentionMask(softcap, window, sl, first, None if prefix is None else i32(prefix))
    pisa.dense_prefill_paged(p, q, kp, vp, table, i32(lens), ws, out, i32(new), mask)
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
    run_prefill(pisa, 8, 2, 128, past + n, n, [past + n - 100 * b for b in range(B)], [n] * B, seed=n, softcap=20.0,
                window=past // 2)


@pytest.mark.parametrize("Hq,Hkv,d", [(2, 2, 128), (8, 2, 128), (8, 1, 64)])
def test_prefill_row_tiles_with_distant_spans(pisa, Hq, Hkv, d):
    # neighbouring tokens that see far apart parts of the cache, or short ones
    n = 300
    first = torch.zeros(3, n, dtype=torch.int32)
    first[0, 20:] = 2700
    first[0, 128:] = 0
    first[1, :128] = 2500
    first[2] = (torch.arange(n) % 7) * 450
    for prefix in (None, [0, 2990, 100]):
        run_prefill(pisa, Hq, Hkv, d, 3000, n, [3000, 2900, 2999], [n, n, 290], seed=8, first=first.cuda(), prefix=prefix)


def test_prefill_many_sequences(pisa):
    B = 70
    lens = [1 + 7 * b for b in range(B)]
    run_prefill(pisa, 2, 1, 64, 500, 90, lens, [min(90, x) for x in lens], seed=4)


def test_prefill_bad_lengths(pisa):
    run_prefill(pisa, 8, 2, 64, 300, 70, [300, 301, 60, 100, -1, 70], [70, 70, 70, 71, 3, -2], seed=5,
                status=pisa.DEV_BAD_SEQ_LEN)


def test_prefill_bad_page_counts_as_unseen(pisa):
    k, v, kp, vp, table = cache(1, 2, 300, 64, [300], 4)
    for bad in (-1, 1 << 20):
        table[0, 2] = bad
        q = torch.randn(1, 4, 200, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
        layer = pisa.PagedAttention(pisa.make_params(1, 300, 4, 2, 64), n=200)
        out = layer.dense_prefill(q, kp, vp, table, i32([300]))
        assert layer.device_status() == pisa.DEV_BAD_INDEX
        key, pos = torch.arange(300, device="cuda"), torch.arange(100, 300, device="cuda")
        keep = (key[None] <= pos[:, None]) & (key[None] // 64 != 2)
        for h in range(4):
            o, t = R.attend(q[0, h], k[0, h // 2], v[0, h // 2], keep, 0.125)
            R.within(out[0, h], o, t)


def test_pages_before_the_window_may_be_gone(pisa):
    # a serving program gives pages that a window has left back: their entries are never read
    def poke(kp, vp, table):
        table[0, :(900 - 70 - 299) // 64] = -7
    run_prefill(pisa, 4, 2, 64, 900, 70, [900], [70], seed=6, window=300, poke=poke)
    k, v, kp, vp, table = cache(1, 2, 5000, 128, [5000], 7)
    table[0, :(5000 - 1000) // 64] = 2 ** 31 - 1
    q = torch.randn(1, 8, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    layer = pisa.PagedAttention(pisa.make_params(1, 5000, 8, 2, 128))
    out = layer.dense_decode(q, kp, vp, table, i32([5000]), mask=pisa.AttentionMask(window=1000))
    assert layer.device_status() == 0
    want, tol = R.dense(q[0][:, None], k[0], v[0], 5000, torch.tensor([4999], device="cuda"), 128 ** -0.5, window=1000)
    R.within(out[0], want[:, 0], tol[:, 0])


def test_sequences_that_share_pages(pisa):
    # a common prefix of two pages, own pages behind it
    k, v, kp, vp, table = cache(2, 2, 300, 64, [300, 300], 8, fill=0.0)
    table[1, :2] = table[0, :2]
    k[1, :, :128], v[1, :, :128] = k[0, :, :128], v[0, :, :128]
    layer = pisa.PagedAttention(pisa.make_params(2, 300, 4, 2, 64), n=100)
    q = torch.randn(2, 4, 100, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    out = layer.dense_prefill(q, kp, vp, table, i32([300, 250]))
    one = layer.dense_decode(q[:, :, 0].contiguous(), kp, vp, table, i32([300, 250]))
    for b, n in enumerate([300, 250]):
        want, tol = R.dense(q[b], k[b], v[b], n, torch.arange(n - 100, n, device="cuda"), 0.125)
        R.within(out[b], want, tol)
        want, tol = R.dense(q[b][:, :1], k[b], v[b], n, torch.tensor([n - 1], device="cuda"), 0.125)
        R.within(one[b], want[:, 0], tol[:, 0])


def test_prefill_non_finite_values_behind_the_window(pisa):
    # whole tiles that no row sees are never read
    def poke(kp, vp, table):
        for j in range(2):
            kp[int(table[0, j])], vp[int(table[0, j])] = R.NAN, R.NAN
    run_prefill(pisa, 4, 2, 64, 900, 70, [900], [70], seed=6, window=300, poke=poke)


@pytest.mark.parametrize("kw", [dict(), dict(softcap=20.0, slopes=True), dict(window=40)])
@pytest.mark.parametrize("n,lens", [(280, [600]), (280, [280]), (30, [3000])])
def test_prefill_non_finite_values_among_unseen_keys_of_a_tile(pisa, n, lens, kw):
    # a value reaches the rows that see its key, and no other; the last case is split over the keys
    Hq, Hkv, d, N = 4, 2, 64, lens[0]
    k, v, kp, vp, table = cache(1, Hkv, N, d, lens, 6)
    late = N - n // 2  # seen by the later half of the new tokens alone
    for j, x in ((late, float("inf")), (late + 3, R.NAN)):
        vp[int(table[0, j // 64]), :, j % 64, ::5] = x
    q = (torch.randn(1, Hq, n, d, generator=torch.Generator().manual_seed(7)) * 2).to(torch.bfloat16).cuda()
    sl = slopes_of(Hq) if kw.get("slopes") else None
    mask = pisa.AttentionMask(kw.get("softcap", 0.0), kw.get("window", 0), sl)
    layer = pisa.PagedAttention(pisa.make_params(1, N, Hq, Hkv, d), n=n)
    out = layer.dense_prefill(q, kp, vp, table, i32(lens), mask=mask)[0]
    assert layer.device_status() == 0
    pos = torch.arange(N - n, N, device="cuda")
    want, tol = R.dense(q[0], k[0], v[0], N, pos, 0.125, kw.get("softcap", 0.0), kw.get("window", 0), sl)
    lo, _ = R.spans(pos, N, kw.get("window", 0))
    clean = ~(((pos >= late) & (lo <= late)) | ((pos >= late + 3) & (lo <= late + 3)))
    assert int(clean.sum()) >= n // 2 and int((~clean).sum()) > 0
    R.within(out[:, clean], want[:, clean], tol[:, clean], "rows that see finite values")
    other = torch.arange(d, device="cuda") % 5 != 0
    R.within(out[:, ~clean][..., other], want[:, ~clean][..., other], tol[:, ~clean][..., other], "finite dims")
    assert not bool(torch.isfinite(out[:, ~clean][..., ~other]).any())


def test_prefill_long_prompt(pisa):
    run_prefill(pisa, 4, 1, 128, 3000, 2500, [3000, 2500], [2500, 2400], seed=7)
