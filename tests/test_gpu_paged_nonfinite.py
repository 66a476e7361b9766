"""GPU tests of values that are not finite in the paged prompt call: they reach
the rows that see their key, in their dims, and no others, at a cost of the
order of the call itself whatever the cache holds.  Bounds: paged_ref's."""
import pytest
import torch

import paged_ref as R

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def pisa():
    from pyramid_top_block_mean_gb300 import pisa as m
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def sprinkle(v, share, seed):
    """+inf, -inf and NaN in some dims of a share of the keys of v [B, H, N, d]; returns the poisoned copy."""
    g = torch.Generator().manual_seed(seed)
    key = torch.rand(v.shape[0], 1, v.shape[2], 1, generator=g) < share
    hit = key & (torch.rand(v.shape, generator=g) < 0.2)
    what = torch.tensor([INF, -INF, R.NAN])[torch.randint(0, 3, v.shape, generator=g)].to(v.dtype)
    return torch.where(hit, what, v)


def check(out, q, k, v, bad, length, pos, scale, dead=None, **kw):
    """One sequence's rows: finite dims within their bounds, the others what the seen values make them."""
    window, first, prefix = kw.get("window", 0), kw.get("first"), kw.get("prefix", 0)
    lo, hi = R.spans(pos, length, window, first, prefix)
    key = torch.arange(length, device=q.device)
    keep = (key[None] >= lo[:, None]) & (key[None] <= hi[:, None])
    if dead is not None:
        keep &= ~dead[None, :length]
    G = q.shape[0] // k.shape[0]
    for h in range(q.shape[0]):
        bias = None
        if kw.get("slopes") is not None:
            bias = kw["slopes"][h].double() * (key[None] - pos[:, None]).double()
        want, tol = R.attend(q[h], k[h // G, :length], v[h // G, :length], keep, scale, kw.get("softcap", 0.0), bias)
        x = bad[h // G, :length]
        up = keep.double() @ ((x == INF) | x.isnan()).double() > 0
        down = keep.double() @ ((x == -INF) | x.isnan()).double() > 0
        ok = ~(up | down)
        got = out[h].double()
        R.within(torch.where(ok, got, want), want, tol, f"head {h}")
        assert torch.equal(got.isposinf(), up & ~down) and torch.equal(got.isneginf(), down & ~up)
        assert torch.equal(got.isnan(), up & down)


def run(pisa, Hq, Hkv, d, n, lens, new, share, seed, N=None, drop=None, **kw):
    B, N = len(lens), N or max(lens)
    g = torch.Generator().manual_seed(seed)
    k, v = (torch.randn(B, Hkv, N, d, generator=g).to(torch.bfloat16) for _ in range(2))
    bad = sprinkle(v, share, seed + 1)
    kp, table = R.paginate(k, lens, seed=seed)
    vp, _ = R.paginate(bad, lens, seed=seed)
    dead = None
    if drop is not None:
        table[:, drop] = -1
        dead = (torch.arange(N) // 64 == drop).cuda()
    q = (torch.randn(B, Hq, n, d, generator=g) * 2).to(torch.bfloat16).cuda()
    k, v, bad, kp, vp, table = (x.cuda() for x in (k, v, bad, kp, vp, table))
    layer = pisa.PagedAttention(pisa.make_params(B, N, Hq, Hkv, d), n=n)
    first, prefix = kw.get("first"), kw.get("prefix")
    mask = pisa.AttentionMask(kw.get("softcap", 0.0), kw.get("window", 0), kw.get("slopes"), first,
                              None if prefix is None else i32(prefix))
    out = layer.dense_prefill(q, kp, vp, table, i32(lens), new_lens=i32(new), mask=mask).clone()
    assert layer.device_status() == (pisa.DEV_BAD_INDEX if drop is not None else 0)
    again = layer.dense_prefill(q, kp, vp, table, i32(lens), new_lens=i32(new), mask=mask)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    for b in range(B):
        pos = torch.arange(lens[b] - new[b], lens[b], device="cuda")
        kb = dict(kw)
        if first is not None:
            kb["first"] = first[b, :new[b]]
        if prefix is not None:
            kb["prefix"] = prefix[b]
        check(out[b, :, :new[b]], q[b, :, :new[b]], k[b], v[b], bad[b], lens[b], pos, d ** -0.5, dead, **kb)


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 2, 2), (128, 8, 2), (64, 8, 1), (128, 2, 2)])
@pytest.mark.parametrize("share", [0.002, 0.3, 1.0])
@pytest.mark.parametrize("n,lens,new", [(700, [700, 900, 1500], [700, 650, 1]), (30, [5000, 4000], [30, 7]),
                                        (129, [129, 128, 500], [129, 64, 0])])
def test_sprinkled_values(pisa, d, Hq, Hkv, share, n, lens, new):
    run(pisa, Hq, Hkv, d, n, lens, new, share, seed=n + d)


@pytest.mark.parametrize("kw", [dict(window=100), dict(window=1), dict(prefix=[50, 900, 0]), dict(softcap=20.0),
                                dict(softcap=20.0, window=300), dict(drop=3), dict(drop=2, window=200)])
@pytest.mark.parametrize("d,Hq,Hkv", [(64, 2, 2), (128, 8, 2)])
def test_sprinkled_values_under_masks(pisa, d, Hq, Hkv, kw):
    run(pisa, Hq, Hkv, d, 300, [300, 900, 700], [300, 290, 211], 0.02, seed=5, **kw)
    if "drop" not in kw:
        sl = (2.0 ** (-8.0 * torch.arange(1, Hq + 1) / Hq)).float().cuda()
        run(pisa, Hq, Hkv, d, 300, [300, 900, 700], [300, 290, 211], 0.02, seed=6, slopes=sl, **kw)


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 2, 2), (128, 8, 2)])
def test_sprinkled_values_among_documents(pisa, d, Hq, Hkv):
    first = torch.zeros(3, 300, dtype=torch.int32)
    first[0] = torch.arange(300) // 97 * 97
    first[1] = torch.randint(0, 900, (300,), generator=torch.Generator().manual_seed(3))  # no order at all
    first[2, ::3] = 2 ** 31 - 1  # rows that see nothing
    for share in (0.01, 0.5):
        run(pisa, Hq, Hkv, d, 300, [300, 900, 700], [300, 300, 300], share, seed=7, first=first.cuda())


@pytest.mark.parametrize("at", [0, 40, 79])
def test_many_items_on_an_sm(pisa, at):
    # 80 sequences of 2 heads x 2 items: 320 items; one sequence's are taken twice, early, in the middle or last
    B, n, d = 80, 200, 64
    g = torch.Generator().manual_seed(at)
    k, v = (torch.randn(B, 2, n, d, generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(B, 2, n, d, generator=g).to(torch.bfloat16).cuda()
    lens = i32([n] * B)
    layer = pisa.PagedAttention(pisa.make_params(B, n, 2, 2, d), n=n)
    kp, table = R.paginate(k, [n] * B, seed=1)
    vp, _ = R.paginate(v, [n] * B, seed=1)
    kp, vp, table = kp.cuda(), vp.cuda(), table.cuda()
    want = layer.dense_prefill(q, kp, vp, table, lens).clone()
    page, slot = int(table[at, 150 // 64]), 150 % 64
    vp[page, :, slot] = R.NAN
    out = layer.dense_prefill(q, kp, vp, table, lens)
    assert layer.device_status() == 0
    assert bool(out[at, :, 150:].isnan().all())
    rest = torch.ones(B, n, dtype=torch.bool, device="cuda")
    rest[at, 150:] = False
    got, want = out.transpose(1, 2)[rest], want.transpose(1, 2)[rest]
    assert torch.equal(got, want)


def test_a_sequence_of_nothing_else_beside_a_clean_one(pisa):
    # at a cost of the order of the call's: some four times, where a row at a time would be hundreds
    B, N, Hq, Hkv, d = 2, 8192, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    nb = N // 64
    kp, vp = (torch.randn(B * nb, Hkv, 64, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(B, Hq, N, d, generator=g, device="cuda").bfloat16()
    table = torch.arange(B * nb, device="cuda", dtype=torch.int32).view(B, nb)
    lens = i32([N, N])
    layer = pisa.PagedAttention(pisa.make_params(B, N, Hq, Hkv, d), n=N)

    def timed():
        layer.dense_prefill(q, kp, vp, table, lens)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        out = layer.dense_prefill(q, kp, vp, table, lens)
        b.record()
        b.synchronize()
        assert layer.device_status() == 0
        return out.clone(), a.elapsed_time(b)

    want, clean = timed()
    vp[:nb] = R.NAN
    out, poisoned = timed()
    assert bool(out[0].isnan().all()) and torch.equal(out[1], want[1])
    assert poisoned < 40 * clean, (poisoned, clean)


def test_one_value_late_in_a_long_cache(pisa):
    # 80 items, each against all of 300,000 keys; a value that half of the rows see
    N, H, d, n = 300_000, 80, 64, 100
    g = torch.Generator(device="cuda").manual_seed(2)
    nb = -(-N // 64)
    kp, vp = (torch.randn(nb, H, 64, d, generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.arange(nb, device="cuda", dtype=torch.int32).view(1, nb)
    q = torch.randn(1, H, n, d, generator=g, device="cuda").bfloat16()
    layer = pisa.PagedAttention(pisa.make_params(1, N, H, H, d), n=n)
    late = N - 50
    vp[late // 64, :, late % 64, ::3] = R.NAN
    out = layer.dense_prefill(q, kp, vp, table, i32([N]))
    assert layer.device_status() == 0
    pos = torch.arange(N - n, N, device="cuda")
    other = torch.arange(d, device="cuda") % 3 != 0
    for h in (0, 79):
        k, v = (x[:, h].reshape(-1, d)[:N] for x in (kp, vp))
        v = torch.where(v.isnan(), torch.zeros_like(v), v)
        want, tol = R.dense(q[0, h:h + 1], k[None], v[None], N, pos, d ** -0.5)
        R.within(out[0, h, :50], want[0, :50], tol[0, :50])
        R.within(out[0, h, 50:][:, other], want[0, 50:][:, other], tol[0, 50:][:, other])
    assert bool(out[0, :, 50:][..., ~other].isnan().all())


def test_rows_that_are_not_finite_for_reasons_of_their_own(pisa):
    # a query of NaN, a key of NaN: those rows alone
    B, N, Hq, Hkv, d = 1, 500, 4, 2, 64
    g = torch.Generator().manual_seed(4)
    k, v = (torch.randn(B, Hkv, N, d, generator=g).to(torch.bfloat16) for _ in range(2))
    kp, table = R.paginate(k, [N], seed=1)
    vp, _ = R.paginate(v, [N], seed=1)
    q = torch.randn(B, Hq, N, d, generator=g).to(torch.bfloat16).cuda()
    k, v, kp, vp, table = (x.cuda() for x in (k, v, kp, vp, table))
    q[0, 1, 77] = R.NAN
    kp[int(table[0, 400 // 64]), 1, 400 % 64] = R.NAN
    vp[int(table[0, 300 // 64]), 0, 300 % 64, 5] = INF
    layer = pisa.PagedAttention(pisa.make_params(B, N, Hq, Hkv, d), n=N)
    out = layer.dense_prefill(q, kp, vp, table, i32([N]))[0]
    assert layer.device_status() == 0
    pos = torch.arange(N, device="cuda")
    want, tol = R.dense(torch.nan_to_num(q[0]), k[0], v[0], N, pos, 0.125)
    nan = torch.zeros_like(out, dtype=torch.bool)
    nan[1, 77] = True
    nan[2:, 400:] = True
    inf = torch.zeros_like(nan)
    inf[:2, 300:, 5] = True
    assert torch.equal(out.isnan(), nan) and torch.equal(out.isposinf(), inf)
    ok = ~(nan | inf)
    R.within(torch.where(ok, out.double(), want), want, tol)


@pytest.mark.parametrize("d,Hq,Hkv", [(64, 8, 8), (128, 32, 8)])
def test_sprinkled_values_in_all_of_many_items(pisa, d, Hq, Hkv):
    # several items an SM, each taken twice
    run(pisa, Hq, Hkv, d, 900, [900, 1000, 1100, 900, 950, 1500], [900, 890, 700, 900, 850, 900], 0.01, seed=9)
