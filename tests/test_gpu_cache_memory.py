"""GPU tests of what a PagedAttention owns: its buffers stay whole until calls
on other streams have run, and the scratch of long prompts over 8-bit pages is
made when a prompt needs it, and when there is room."""
import pytest
import torch

from test_gpu_cache_layer import Model, check, i32

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


def test_a_prompt_of_few_tokens_makes_no_scratch(pisa):
    m = Model(pisa, 1, 3000, 8, 2, 128, n=2500)
    q = m.append(10, [10], [10]).clone()
    out = m.layer.dense_prefill(q, *m.cache(), i32([10]), scales=m.scales)
    check(m, out[0], q[0], [10], 0, 10)
    assert m.layer._scratch is None
    q = m.append(2400, [2410], [2400]).clone()
    out = m.layer.dense_prefill(q, *m.cache(), i32([2410]), scales=m.scales)
    check(m, out[0], q[0], [2410], 0, 2400)
    assert m.layer._scratch is not None


def test_a_scratch_is_asked_for_again(pisa):
    """A prompt that found no room does not take it from all that follow."""
    m = Model(pisa, 1, 3000, 8, 2, 128, n=2500)
    q = m.append(2500, [2500], [2500]).clone()
    want = m.layer.dense_prefill(q, *m.cache(), i32([2500]), scales=m.scales).clone()
    size = m.layer._scratch_bytes
    m.layer._scratch, m.layer._scratch_bytes = None, 1 << 45
    assert torch.equal(m.layer.dense_prefill(q, *m.cache(), i32([2500]), scales=m.scales), want)
    assert m.layer._scratch is None
    m.layer._scratch_bytes = m.layer._scratch_bytes and size  # there is room again
    for _ in range(5):
        assert torch.equal(m.layer.dense_prefill(q, *m.cache(), i32([2500]), scales=m.scales), want)
    assert m.layer._scratch is not None


def test_layers_share_a_scratch(pisa):
    """Two layers of one scratch: calls in turn, results of their own, and nothing else allocated."""
    ms = [Model(pisa, 1, 3000, 8, 2, 128, n=2500, seed=s) for s in range(2)]
    qs = [m.append(2500, [2500], [2500]).clone() for m in ms]
    lens = i32([2500])
    want = [m.layer.dense_prefill(q, *m.cache(), lens, scales=m.scales).clone() for m, q in zip(ms, qs)]
    shared = torch.zeros(pisa.cache_scratch_bytes(ms[0].p, 2500), dtype=torch.uint8, device="cuda")
    layers = [pisa.PagedAttention(m.p, n=2500, scratch=shared) for m in ms]
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for _ in range(2):
        for m, layer, q, y in zip(ms, layers, qs, want):
            assert torch.equal(layer.dense_prefill(q, *m.cache(), lens, scales=m.scales), y)
    assert torch.cuda.memory_allocated() == before
    assert shared.any()  # the pages went through it
