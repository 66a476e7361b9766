"""The paged operators run together as a serving layer runs them: a prompt
appended in two chunks, its dense attention, the pyramid of the pages, then
decode steps that append, select and attend; on other streams, captured into a
CUDA graph and replayed with new contents, and with two layers at once."""
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


def rope_table(N, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(N, dtype=torch.float64)[:, None] * f[None]
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous().cuda()


class Model:
    """Projections drawn at random, and what a layer keeps."""

    def __init__(self, pisa, B, N, Hq, Hkv, d, n, K=4, seed=0):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.p = pisa.make_params(B, N, Hq, Hkv, d, K=K)
        self.rope = rope_table(N, d)
        self.layer = pisa.PagedAttention(self.p, n=n, rope=self.rope)
        nb = -(-N // 64)
        self.table = torch.randperm(B * nb, generator=self.g, device="cuda").to(torch.int32).reshape(B, nb)
        self.kp = torch.full((B * nb, Hkv, 64, d), R.NAN, dtype=torch.bfloat16, device="cuda")
        self.vp = self.kp.clone()
        # the same cache, contiguous
        self.k = torch.zeros(B, Hkv, N, d, dtype=torch.bfloat16, device="cuda")
        self.v = torch.zeros_like(self.k)

    def project(self, n):
        p = self.p
        x = torch.randn(p.B, n, p.H_q + 2 * p.H_kv, p.d, generator=self.g, device="cuda").to(torch.bfloat16)
        x = x.transpose(1, 2)
        return x[:, :p.H_q], x[:, p.H_q:p.H_q + p.H_kv], x[:, p.H_q + p.H_kv:]

    def append(self, n, lens, new):
        q, k, v = self.project(n)
        k_out = torch.empty(k.shape, dtype=k.dtype, device="cuda")
        q = self.layer.append(q, k, v, self.kp, self.vp, self.table, i32(lens), i32(new), k_out=k_out)
        for b, (length, cnt) in enumerate(zip(lens, new)):
            self.k[b, :, length - cnt:length] = k_out[b, :, :cnt]
            self.v[b, :, length - cnt:length] = v[b, :, :cnt]
        return q


def test_prompt_then_decode(pisa):
    B, N, Hq, Hkv, d = 2, 1000, 8, 2, 128
    m = Model(pisa, B, N, Hq, Hkv, d, n=400)
    lens = [0, 0]
    for new in ([400, 313], [350, 400]):
        lens = [a + b for a, b in zip(lens, new)]
        q = m.append(400, lens, new)
        out = m.layer.dense_prefill(q, m.kp, m.vp, m.table, i32(lens), new_lens=i32(new))
        assert m.layer.device_status() == 0
        for b in range(B):
            pos = torch.arange(lens[b] - new[b], lens[b], device="cuda")
            want, tol = R.dense(q[b, :, :new[b]], m.k[b], m.v[b], lens[b], pos, d ** -0.5)
            R.within(out[b, :, :new[b]], want, tol)
    sel = pisa.Selector(m.p, mode="decode")
    sel.build_paged(m.kp, m.table, i32(lens))
    assert sel.device_status() == 0
    contig = pisa.Selector(m.p, mode="decode")
    contig.build(m.k, i32(lens))
    for step in range(70):
        lens = [x + 1 for x in lens]
        q = m.append(1, lens, [1, 1])[:, :, 0].contiguous()
        idx, _ = sel.decode_paged(q, m.kp, m.table, i32(lens))
        want_idx, _ = contig.decode(q, m.k, i32(lens))
        assert torch.equal(idx, want_idx)
        out = m.layer.selected_decode(q, m.kp, m.vp, m.table, i32(lens), idx)
        if step % 23 == 0:
            for b in range(B):
                want, tol = R.selected(q[b], m.k[b], m.v[b], lens[b], idx[b], d ** -0.5)
                R.within(out[b], want, tol)
        out = m.layer.dense_decode(q, m.kp, m.vp, m.table, i32(lens))
        if step % 23 == 0:
            for b in range(B):
                want, tol = R.dense(q[b][:, None], m.k[b], m.v[b], lens[b], i32([lens[b] - 1]).long(), d ** -0.5)
                R.within(out[b], want[:, 0], tol[:, 0])
    assert m.layer.device_status() == 0 and sel.device_status() == 0


def test_one_new_token_of_a_prompt_call_equals_decode(pisa):
    m = Model(pisa, 2, 500, 8, 2, 64, n=300)
    lens = [300, 211]
    m.append(300, lens, lens)
    lens = [301, 212]
    q = m.append(1, lens, [1, 1])
    a = m.layer.dense_prefill(q, m.kp, m.vp, m.table, i32(lens))[:, :, 0].double()
    b = m.layer.dense_decode(q[:, :, 0].contiguous(), m.kp, m.vp, m.table, i32(lens)).double()
    for s in range(2):
        _, tol = R.dense(q[s], m.k[s], m.v[s], lens[s], i32([lens[s] - 1]).long(), 0.125)
        R.within(a[s], b[s], 2 * tol[:, 0])


def test_captured_step_replays_with_new_contents(pisa):
    m = Model(pisa, 3, 600, 8, 2, 128, n=500)
    m.append(500, [500, 400, 64], [500, 400, 64])
    lens = i32([501, 401, 65])
    q, k, v = (x.clone() for x in m.project(1))
    idx = torch.full((3, 2, 7), -1, dtype=torch.int32, device="cuda")
    idx[:, :, :2] = i32([0, 1])
    n_q, n_k, n_v = (x.contiguous() for x in m.project(200))
    p_lens, p_new = i32([500, 400, 64]), i32([200, 100, 64])

    def step():
        r = m.layer.append(q, k, v, m.kp, m.vp, m.table, lens)[:, :, 0].clone()
        a = m.layer.dense_decode(r, m.kp, m.vp, m.table, lens)
        b = m.layer.selected_decode(r, m.kp, m.vp, m.table, lens, idx)
        c = m.layer.dense_prefill(n_q, m.kp, m.vp, m.table, p_lens, new_lens=p_new)
        return a, b, c

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for new_lens in ([502, 402, 66], [577, 10, 129], [501, 401, 65]):
        for x, y in zip((q, k, v), m.project(1)):
            x.copy_(y)
        lens.copy_(i32(new_lens))
        # positions between the prompt and the step hold something finite
        m.kp.copy_(torch.nan_to_num(m.kp)), m.vp.copy_(torch.nan_to_num(m.vp))
        graph.replay()
        got = [x.clone() for x in outs]
        want = [x.clone() for x in step()]
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert m.layer.device_status() == 0


def test_repeated_calls_agree_bit_for_bit(pisa):
    m = Model(pisa, 2, 5000, 8, 2, 128, n=4000)
    m.append(4000, [4000, 3777], [4000, 3777])
    q = m.project(1)[0][:, :, 0].contiguous()
    n_q = m.project(37)[0].contiguous()
    runs = []
    for _ in range(5):
        runs.append((m.layer.dense_decode(q, m.kp, m.vp, m.table, i32([4000, 3777])).clone(),
                     m.layer.dense_prefill(n_q, m.kp, m.vp, m.table, i32([4000, 3777])).clone()))
    for r in runs[1:]:
        assert torch.equal(r[0], runs[0][0]) and torch.equal(r[1], runs[0][1])


def test_two_layers_on_two_streams(pisa):
    ms = [Model(pisa, 2, 3000, 8, 2, 128, n=2500, seed=s) for s in range(2)]
    for m in ms:
        m.append(2500, [2500, 2000], [2500, 2000])
    qs = [m.project(1)[0][:, :, 0].contiguous() for m in ms]
    lens = i32([2500, 2000])
    alone = [m.layer.dense_decode(q, m.kp, m.vp, m.table, lens).clone() for m, q in zip(ms, qs)]
    streams = [torch.cuda.Stream() for _ in ms]
    torch.cuda.synchronize()
    for _ in range(20):
        for m, q, s in zip(ms, qs, streams):
            m.layer.dense_decode(q, m.kp, m.vp, m.table, lens, stream=s)
    torch.cuda.synchronize()
    for m, q, want in zip(ms, qs, alone):
        assert torch.equal(m.layer._buffer("dense", q), want)


@pytest.mark.parametrize("n", [1, 61, 200, 700, 2048])
def test_a_layer_takes_fewer_tokens_than_asked_for(pisa, n):
    """A call of fewer tokens splits its keys where the largest call does not."""
    B, N, Hq, Hkv, d = 1, 4096, 8, 1, 128
    m = Model(pisa, B, N, Hq, Hkv, d, n=2560)
    m.kp.normal_(generator=m.g)
    m.vp.normal_(generator=m.g)
    q = torch.randn(B, Hq, n, d, generator=m.g, device="cuda").bfloat16()
    lens = i32([3700])
    out = m.layer.dense_prefill(q, m.kp, m.vp, m.table, lens)
    assert m.layer.device_status() == 0
    ws = torch.empty(pisa.paged_workspace_bytes(m.p, n), dtype=torch.uint8, device="cuda")
    want = torch.full_like(q, R.NAN)
    pisa.dense_prefill_paged(m.p, q, m.kp, m.vp, m.table, lens, ws, want)
    assert torch.equal(out, want)


def test_calls_without_a_new_token_between_others(pisa):
    """Rows all absent, then present, back to back on one workspace."""
    B, N, Hq, Hkv, d, n = 2, 8192, 8, 2, 128, 32
    m = Model(pisa, B, N, Hq, Hkv, d, n=n)
    m.kp.normal_(generator=m.g)
    m.vp.normal_(generator=m.g)
    q = torch.randn(B, Hq, n, d, generator=m.g, device="cuda").bfloat16()
    lens, some, none = i32([8000, 5001]), i32([n, 5]), i32([0, 0])
    want = m.layer.dense_prefill(q, m.kp, m.vp, m.table, lens, new_lens=some).clone()
    for _ in range(20):
        out = torch.zeros_like(want)
        rest = torch.full_like(want, R.NAN)
        pisa.dense_prefill_paged(m.p, q, m.kp, m.vp, m.table, lens, m.layer.ws, rest, new_lens=none)
        pisa.dense_prefill_paged(m.p, q, m.kp, m.vp, m.table, lens, m.layer.ws, out, new_lens=some)
        pisa.dense_prefill_paged(m.p, q, m.kp, m.vp, m.table, lens, m.layer.ws, rest, new_lens=none)
        assert m.layer.device_status() == 0
        assert torch.equal(out, want) and bool(rest.isnan().all())
