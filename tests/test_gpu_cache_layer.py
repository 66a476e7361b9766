"""The 8-bit cache's operators run together as a serving layer runs them: a
prompt appended in two chunks with normed heads, its dense attention, the
pyramid of the pages, then decode steps that append, select and attend; and the
selector over 8-bit pages against itself over bf16 pages of the same numbers,
bit for bit.  On other streams, captured and replayed, two layers at once."""
import pytest
import torch

import cache_ref as C
import paged_ref as R
from test_gpu_paged_layer import i32, rope_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pisa():
    from pyramid_top_block_mean_gb300 import pisa as m
    return m


class Model:
    """Projections drawn at random, and what a layer keeps."""

    def __init__(self, pisa, B, N, Hq, Hkv, d, n, K=4, seed=0):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.p = pisa.make_params(B, N, Hq, Hkv, d, K=K)
        self.w = [1 + 0.2 * torch.randn(d, generator=self.g, device="cuda") for _ in range(2)]
        self.layer = pisa.PagedAttention(self.p, n=n, rope=rope_table(N, d), q_norm=self.w[0], k_norm=self.w[1])
        nb = -(-N // 64)
        self.table = torch.randperm(B * nb, generator=self.g, device="cuda").to(torch.int32).reshape(B, nb)
        self.kp, self.vp, self.scales = pisa.quantized_pages(self.p, B * nb)
        self.scales.fill_(255)  # rows that are not written read as NaN
        self.kp.view(torch.uint8).fill_(0x7f), self.vp.view(torch.uint8).fill_(0x7f)

    def project(self, n):
        p = self.p
        x = torch.randn(p.B, n, p.H_q + 2 * p.H_kv, p.d, generator=self.g, device="cuda").to(torch.bfloat16)
        x = x.transpose(1, 2)
        return x[:, :p.H_q], x[:, p.H_q:p.H_q + p.H_kv], x[:, p.H_q + p.H_kv:]

    def cache(self):
        return self.kp, self.vp, self.table

    def append(self, n, lens, new):
        q, k, v = self.project(n)
        return self.layer.append(q, k, v, *self.cache(), i32(lens), i32(new), scales=self.scales)

    def rows(self, which, b, length):
        """The first rows of a sequence, in 64 bits, [Hkv, length, d]."""
        pages = self.table[b, :-(-length // 64)].long()
        x = C.numbers((self.kp, self.vp)[which].view(torch.uint8)[pages], self.scales[which][pages])
        return x.transpose(0, 1).flatten(1, 2)[:, :length]

    def wide_keys(self):
        """bf16 pages of the same numbers."""
        return C.numbers(self.kp, self.scales[0]).to(torch.bfloat16)


def check(m, out, q, lens, b, new=1):
    pos = torch.arange(lens[b] - new, lens[b], device="cuda")
    want, tol = R.dense(q, m.rows(0, b, lens[b]), m.rows(1, b, lens[b]), lens[b], pos, m.p.d ** -0.5)
    R.within(out, want, tol)


def test_prompt_then_decode(pisa):
    B, N, Hq, Hkv, d = 2, 1000, 8, 2, 128
    m = Model(pisa, B, N, Hq, Hkv, d, n=400)
    lens = [0, 0]
    for new in ([400, 313], [350, 400]):
        lens = [a + b for a, b in zip(lens, new)]
        q = m.append(400, lens, new)
        out = m.layer.dense_prefill(q, *m.cache(), i32(lens), new_lens=i32(new), scales=m.scales)
        assert m.layer.device_status() == 0
        for b in range(B):
            check(m, out[b, :, :new[b]], q[b, :, :new[b]], lens, b, new[b])
    sel = pisa.Selector(m.p, mode="decode")
    sel.build_paged(m.kp, m.table, i32(lens), scales=m.scales)
    assert sel.device_status() == 0
    wide = pisa.Selector(m.p, mode="decode")
    wide.build_paged(m.wide_keys(), m.table, i32(lens))
    assert torch.equal(sel.pyramid, wide.pyramid)
    for step in range(70):
        lens = [x + 1 for x in lens]
        q = m.append(1, lens, [1, 1])[:, :, 0].contiguous()
        idx, score = sel.decode_paged(q, m.kp, m.table, i32(lens), scales=m.scales)
        want_idx, want_score = wide.decode_paged(q, m.wide_keys(), m.table, i32(lens))
        assert torch.equal(idx, want_idx) and torch.equal(score, want_score)
        assert torch.equal(sel.pyramid, wide.pyramid)
        out = m.layer.selected_decode(q, *m.cache(), i32(lens), idx, scales=m.scales)
        if step % 23 == 0:
            for b in range(B):
                want, tol = R.selected(q[b], m.rows(0, b, lens[b]), m.rows(1, b, lens[b]), lens[b], idx[b], d ** -0.5)
                R.within(out[b], want, tol)
        out = m.layer.dense_decode(q, *m.cache(), i32(lens), scales=m.scales)
        if step % 23 == 0:
            for b in range(B):
                check(m, out[b][:, None], q[b][:, None], lens, b)
    assert m.layer.device_status() == 0 and sel.device_status() == 0


@pytest.mark.parametrize("d,Hq,Hkv,K,scorer", [(128, 16, 4, 8, 0), (64, 8, 1, 5, 0), (128, 4, 4, 32, 1),
                                               (64, 4, 2, 3, 2), (128, 2, 1, 4, 0)])
def test_selector_equals_itself_over_wide_pages(pisa, d, Hq, Hkv, K, scorer):
    lens = [5000, 4999, 64, 1, 130, 4097]
    B, N = len(lens), 5000
    g = torch.Generator().manual_seed(d + K)
    k = torch.randn(B, Hkv, N, d, generator=g) * 2.0 ** torch.randint(-3, 12, (B, Hkv, N, 1), generator=g)
    k[4, 0, 77] = float("nan")
    kp, ks, table, _ = C.paginate(k, lens, seed=1)
    kp, scales, table = kp.cuda(), torch.stack([ks, ks]).contiguous().cuda(), table.cuda()
    wide_pages = C.numbers(kp, scales[0]).to(torch.bfloat16)
    p = pisa.make_params(B, N, Hq, Hkv, d, K=K, scorer=scorer)
    before = i32([n - 1 for n in lens])
    got, want = pisa.Selector(p, mode="decode"), pisa.Selector(p, mode="decode")
    for s in (got, want):
        s.pyramid.zero_()
    got.build_paged(kp, table, before, scales=scales)
    want.build_paged(wide_pages, table, before)
    assert got.device_status() == 0
    assert torch.equal(torch.nan_to_num(got.pyramid, 3.0), torch.nan_to_num(want.pyramid, 3.0))
    q = torch.randn(B, Hq, d, generator=g).to(torch.bfloat16).cuda()
    a, x = got.decode_paged(q, kp, table, i32(lens), scales=scales)
    b, y = want.decode_paged(q, wide_pages, table, i32(lens))
    assert got.device_status() == 0
    assert torch.equal(a, b) and torch.equal(torch.nan_to_num(x, 3.0), torch.nan_to_num(y, 3.0))
    assert torch.equal(torch.nan_to_num(got.pyramid, 3.0), torch.nan_to_num(want.pyramid, 3.0))


def test_selector_faults(pisa):
    p = pisa.make_params(2, 1000, 4, 2, 64)
    k = torch.randn(2, 2, 1000, 64, generator=torch.Generator().manual_seed(0))
    kp, ks, table, _ = C.paginate(k, [1000, 1000], seed=1)
    kp, scales, table = kp.cuda(), torch.stack([ks, ks]).contiguous().cuda(), table.cuda()
    table[1, 3] = 1 << 20
    sel = pisa.Selector(p, mode="decode")
    sel.build_paged(kp, table, i32([1000, 1000]), scales=scales)
    assert sel.device_status() == pisa.DEV_BAD_INDEX
    q = torch.randn(2, 4, 64, device="cuda").to(torch.bfloat16)
    idx, _ = sel.decode_paged(q, kp, table, i32([1000, 1000]), scales=scales)
    assert sel.device_status() == pisa.DEV_BAD_INDEX
    assert bool((idx[1] == -1).all()) and bool((idx[0, :, 0] == 0).all())
    idx, _ = sel.decode_paged(q, kp, table, i32([0, 1001]), scales=scales)
    assert sel.device_status() == pisa.DEV_BAD_SEQ_LEN and bool((idx == -1).all())


def test_captured_step_replays_with_new_contents(pisa):
    m = Model(pisa, 3, 900, 8, 2, 128, n=500)
    m.append(500, [500, 400, 64], [500, 400, 64])
    lens = i32([501, 401, 65])
    q, k, v = (x.clone() for x in m.project(1))
    idx = torch.full((3, 2, 7), -1, dtype=torch.int32, device="cuda")
    idx[:, :, :2] = i32([0, 1])
    n_q = m.project(400)[0].contiguous()
    p_lens, p_new = i32([500, 400, 64]), i32([400, 100, 64])
    back = [torch.zeros(3, 2, 64, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def step():
        r = m.layer.append(q, k, v, *m.cache(), lens, scales=m.scales)[:, :, 0].clone()
        a = m.layer.dense_decode(r, *m.cache(), lens, scales=m.scales)
        b = m.layer.selected_decode(r, *m.cache(), lens, idx, scales=m.scales)
        c = m.layer.dense_prefill(n_q, *m.cache(), p_lens, new_lens=p_new, scales=m.scales)
        m.layer.read(*back, *m.cache(), lens, new_lens=i64, scales=m.scales)
        return r, a, b, c, *back

    i64 = i32([64, 10, 1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):  # (the first prompt's scratch is made within)
        outs = step()
    for new_lens in ([502, 402, 66], [577, 64, 129], [501, 401, 65]):
        for x, y in zip((q, k, v), m.project(1)):
            x.copy_(y)
        lens.copy_(i32(new_lens))
        # positions between the prompt and the step hold something finite
        m.scales.copy_(torch.where(m.scales == 255, 127, m.scales))
        for x in (m.kp.view(torch.uint8), m.vp.view(torch.uint8)):
            x.copy_(torch.where(x == 0x7f, 0x38, x))
        graph.replay()
        got = [x.clone() for x in outs]
        want = [x.clone() for x in step()]
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert m.layer.device_status() == 0


def test_two_layers_on_two_streams(pisa):
    ms = [Model(pisa, 2, 3000, 8, 2, 128, n=2500, seed=s) for s in range(2)]
    qs, prompts = [], []
    for m in ms:
        prompts.append(m.append(2500, [2500, 2000], [2500, 2000]).clone())
        qs.append(m.project(1)[0][:, :, 0].contiguous())
    lens, new = i32([2500, 2000]), i32([2500, 2000])
    alone = [(m.layer.dense_decode(q, *m.cache(), lens, scales=m.scales).clone(),
              m.layer.dense_prefill(x, *m.cache(), lens, new_lens=new, scales=m.scales).clone())
             for m, q, x in zip(ms, qs, prompts)]
    streams = [torch.cuda.Stream() for _ in ms]
    torch.cuda.synchronize()
    for _ in range(10):
        for m, q, x, s in zip(ms, qs, prompts, streams):
            m.layer.dense_decode(q, *m.cache(), lens, stream=s, scales=m.scales)
            m.layer.dense_prefill(x, *m.cache(), lens, new_lens=new, stream=s, scales=m.scales)
    torch.cuda.synchronize()
    for m, q, x, (a, b) in zip(ms, qs, prompts, alone):
        assert torch.equal(m.layer._buffer("dense", q), a) and torch.equal(m.layer._buffer("prefill", x), b)


def test_without_room_for_a_scratch(pisa):
    m = Model(pisa, 1, 3000, 8, 2, 128, n=2500)
    q = m.append(2500, [2500], [2500]).clone()
    want = m.layer.dense_prefill(q, *m.cache(), i32([2500]), scales=m.scales).clone()
    assert m.layer._scratch is not None
    m.layer._scratch, m.layer._scratch_bytes = None, 1 << 45
    for _ in range(2):
        assert torch.equal(m.layer.dense_prefill(q, *m.cache(), i32([2500]), scales=m.scales), want)
    assert m.layer._scratch is None


def test_repeated_calls_agree_bit_for_bit(pisa):
    m = Model(pisa, 2, 5000, 8, 2, 128, n=4000)
    m.append(4000, [4000, 3777], [4000, 3777])
    q = m.project(1)[0][:, :, 0].contiguous()
    n_q = m.project(37)[0].contiguous()
    runs = []
    for _ in range(5):
        runs.append((m.layer.dense_decode(q, *m.cache(), i32([4000, 3777]), scales=m.scales).clone(),
                     m.layer.dense_prefill(n_q, *m.cache(), i32([4000, 3777]), scales=m.scales).clone()))
    for r in runs[1:]:
        assert torch.equal(r[0], runs[0][0]) and torch.equal(r[1], runs[0][1])


def test_offsets_past_32_bits(pisa):
    """A pool of more than 2^31 codes, its last pages in use."""
    p = pisa.make_params(1, 200, 2, 1, 128)
    num = (1 << 31) // (64 * 128) + 100
    kp = torch.empty(num, 1, 64, 128, dtype=torch.float8_e4m3fn, device="cuda")
    vp = torch.empty_like(kp)
    scales = torch.empty(2, num, 1, 64, dtype=torch.uint8, device="cuda")
    table = i32([[num - 1, num - 3, 0, num - 2]])
    g = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn(1, 1, 200, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(1, 2, 200, 128, generator=g, device="cuda").to(torch.bfloat16)
    layer = pisa.PagedAttention(p, n=200)
    layer.append(None, k, v, kp, vp, table, i32([200]), scales=scales)
    got = [torch.empty_like(k) for _ in range(2)]
    layer.read(*got, kp, vp, table, i32([200]), scales=scales)
    for x, y in zip((k, v), got):
        codes, s = C.quantize(x.cpu())
        assert torch.equal(y.cpu().double(), C.numbers(codes, s))
    out = layer.dense_prefill(q, kp, vp, table, i32([200]), scales=scales)
    one = layer.dense_decode(q[:, :, 199].contiguous(), kp, vp, table, i32([200]), scales=scales)
    want, tol = R.dense(q[0], got[0][0], got[1][0], 200, torch.arange(200, device="cuda"), 128 ** -0.5)
    R.within(out[0], want, tol)
    R.within(one[0], want[:, 199], tol[:, 199])


def test_a_scratch_belongs_to_the_stream_of_its_call(pisa):
    """Memory that the current stream may still write is not taken for a call on another."""
    m = Model(pisa, 1, 2048, 16, 4, 128, n=512)
    q = m.append(512, [512], [512])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy = torch.ones(m.layer._scratch_bytes, dtype=torch.uint8, device="cuda")
    at = busy.data_ptr()
    del busy
    out = m.layer.dense_prefill(q, *m.cache(), i32([512]), scales=m.scales, stream=side)
    torch.cuda.synchronize()
    assert m.layer._scratch.data_ptr() != at
    check(m, out[0], q[0], [512], 0, 512)


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 16, 4), (64, 8, 1)])
def test_selector_equals_itself_for_keys_of_any_size(pisa, d, Hq, Hkv):
    """Scales over 134 in some leaves, among others and alone, and rows near the smallest power."""
    lens = [1000, 999, 700, 1000]
    g = torch.Generator().manual_seed(d)
    k = torch.randn(4, Hkv, 1000, d, generator=g)
    k[0, :, 100:300] *= 2.0 ** 20
    k[1] *= 2.0 ** torch.randint(0, 40, (Hkv, 1000, 1), generator=g)
    k[2] *= 2.0 ** -112
    k[3, :, ::7] = 0.0
    k[3, :, 640:704] *= 2.0 ** -130
    kp, ks, table, _ = C.paginate(k, lens, seed=2)
    kp, scales, table = kp.cuda(), torch.stack([ks, ks]).contiguous().cuda(), table.cuda()
    wide_pages = C.numbers(kp, scales[0]).to(torch.bfloat16)
    p = pisa.make_params(4, 1000, Hq, Hkv, d, K=4)
    before = i32([n - 1 for n in lens])
    got, want = pisa.Selector(p, mode="decode"), pisa.Selector(p, mode="decode")
    for s in (got, want):
        s.pyramid.zero_()
    got.build_paged(kp, table, before, scales=scales)
    want.build_paged(wide_pages, table, before)
    assert torch.equal(got.pyramid, want.pyramid)
    q = torch.randn(4, Hq, d, generator=g)
    q[2] *= 2.0 ** 100
    q = q.to(torch.bfloat16).cuda()
    a, x = got.decode_paged(q, kp, table, i32(lens), scales=scales)
    b, y = want.decode_paged(q, wide_pages, table, i32(lens))
    assert got.device_status() == 0
    assert torch.equal(a, b) and torch.equal(x, y) and torch.equal(got.pyramid, want.pyramid)
