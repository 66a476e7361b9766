"""GPU tests of a PagedAttention on streams other than the one it was made on,
and of one made during a capture."""
import pytest
import torch

from test_gpu_paged_layer import Model, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pisa():
    from pyramid_top_block_mean_gb300 import pisa as m
    return m


def test_outputs_are_ready_for_any_stream(pisa):
    """The first call may run on another stream than the one that the layer was made on."""
    m = Model(pisa, 2, 500, 8, 2, 64, n=300)
    m.append(300, [300, 211], [300, 211])
    lens = i32([300, 211])
    q, n_q = m.project(1)[0][:, :, 0].contiguous(), m.project(40)[0].contiguous()
    want = m.layer.dense_decode(q, m.kp, m.vp, m.table, lens).clone()
    n_want = m.layer.dense_prefill(n_q, m.kp, m.vp, m.table, lens).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)  # the making stream is busy for some 25 ms
    layer = pisa.PagedAttention(m.p, n=40)
    out = layer.dense_decode(q, m.kp, m.vp, m.table, lens, stream=side)
    n_out = layer.dense_prefill(n_q, m.kp, m.vp, m.table, lens, stream=side)
    torch.cuda.synchronize()
    assert layer.device_status() == 0
    assert torch.equal(out, want) and torch.equal(n_out, n_want)


def test_a_layer_made_during_a_capture(pisa):
    m = Model(pisa, 2, 500, 8, 2, 64, n=300)
    m.append(300, [300, 211], [300, 211])
    lens = i32([300, 211])
    q = m.project(1)[0][:, :, 0].contiguous()
    want = m.layer.dense_decode(q, m.kp, m.vp, m.table, lens).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pisa.PagedAttention(m.p, n=40).dense_decode(q, m.kp, m.vp, m.table, lens)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
