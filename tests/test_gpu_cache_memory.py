"""GPU tests of what a PagedAttention owns: its buffers stay whole until calls
on other streams have run."""
import pytest
import torch

from test_gpu_cache_layer import Model, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pisa():
    from pyramid_top_block_mean_gb300 import pisa as m
    return m


def taken(nbytes, addresses):
    """Whether the allocator would hand out one of the addresses on the current stream."""
    held = []
    for _ in range(8):
        held.append(torch.empty(nbytes, dtype=torch.uint8, device="cuda"))
        if held[-1].data_ptr() in addresses:
            return True
    return False


@pytest.mark.parametrize("what", ["scratch", "workspace", "outputs"])
def test_buffers_outlive_pending_calls_on_another_stream(pisa, what):
    m = Model(pisa, 1, 2048, 16, 4, 128, n=1024)
    q = m.append(1024, [1024], [1024]).clone()
    lens = i32([1024])
    if what == "scratch":  # made on the current stream
        m.layer.dense_prefill(q, *m.cache(), lens, scales=m.scales)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)  # some 200 ms
    m.layer.dense_prefill(q, *m.cache(), lens, scales=m.scales, stream=side)
    block = {"scratch": m.layer._scratch, "workspace": m.layer.ws, "outputs": m.layer._out["dense"]}[what]
    block = block.untyped_storage()
    address, nbytes = block.data_ptr(), block.nbytes()
    del block, m.layer
    assert not taken(nbytes, {address}) or side.query()
    torch.cuda.synchronize()
