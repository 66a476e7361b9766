"""The entry points of the 8-bit cache and of normed appending refuse bad
arguments on the host, before any launch (fake addresses: none of these calls
reaches a GPU)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def pisa():
    from pyramid_top_block_mean_gb300 import build
    build.build()
    from pyramid_top_block_mean_gb300 import pisa as m
    return m


A, MIS, ODD, BIG = 0x10000, 0x10008, 0x10002, 1 << 40
FIELDS = ("k_pages", "v_pages", "k_scales", "v_scales")


def cache(pisa, **kw):
    c = pisa.Cache(ctypes.sizeof(pisa.Cache), pisa.CACHE_E4M3, A, A, A, A, 10, A, None, 0)
    for name, value in kw.items():
        setattr(c, name, value)
    return ctypes.byref(c)


def norm(pisa, **kw):
    c = pisa.HeadNorm(ctypes.sizeof(pisa.HeadNorm), 1e-6, A, A)
    for name, value in kw.items():
        setattr(c, name, value)
    return ctypes.byref(c)


def calls(pisa, p):
    """name -> call(cache, **changes) of every entry point that takes a cache."""
    L, P = pisa.lib(), ctypes.byref(p)

    def append(c, lens=A, ws=A, size=BIG, n=4, norm=None, k=A):
        return L.pisa_cache_append(P, n, A, None, k, None, A, None, lens, A, norm, A, 64, 0, c, ws, size, A, A, None)

    def read(c, lens=A, ws=A, size=BIG, n=4, out=A, new=A):
        return L.pisa_cache_read(P, n, c, lens, new, ws, size, out, A, None)

    def dense(c, lens=A, ws=A, size=BIG, q=A, out=A, mask=None):
        return L.pisa_cache_dense_decode(P, mask, q, c, lens, ws, size, out, None)

    def selected(c, lens=A, ws=A, size=BIG, q=A, out=A, idx=A):
        return L.pisa_cache_attend_decode(P, q, c, lens, idx, ws, size, out, None)

    def prefill(c, lens=A, ws=A, size=BIG, q=A, out=A, mask=None, n=4, new=A):
        return L.pisa_cache_dense_prefill(P, mask, n, q, c, lens, new, ws, size, out, None)

    return dict(append=append, read=read, dense=dense, selected=selected, prefill=prefill)


def test_caches_are_checked(pisa):
    p = pisa.make_params(2, 4096, 16, 4, 128, K=8)
    for name, call in calls(pisa, p).items():
        assert call(None) == -1, name
        assert call(cache(pisa, struct_size=8)) == -1, name
        assert call(cache(pisa, format=2)) == -2 and call(cache(pisa, format=-1)) == -2, name
        assert call(cache(pisa, num_pages=0)) == -1 and call(cache(pisa, num_pages=1 << 31)) == -2, name
        assert call(cache(pisa, page_table=None)) == -1 and call(cache(pisa, page_table=ODD)) == -3, name
        for f in FIELDS:
            assert call(cache(pisa, **{f: None})) == -1, (name, f)
            assert call(cache(pisa, **{f: MIS})) == -3, (name, f)
        assert call(cache(pisa, scratch=MIS)) == -3, name
        c = cache(pisa)
        assert call(c, lens=None) == -1 and call(c, lens=ODD) == -3, name
        assert call(c, ws=None) == -1 and call(c, ws=MIS) == -3 and call(c, size=16) == -4, name


def test_scales_are_not_asked_of_pages_in_the_models_type(pisa):
    p = pisa.make_params(2, 4096, 16, 4, 128, K=8)
    own = dict(format=pisa.CACHE_PARAMS, k_scales=None, v_scales=None)
    for name, call in calls(pisa, p).items():
        assert call(cache(pisa, **own), size=16) == -4, name  # nothing else is missing


def test_norms_are_checked(pisa):
    p = pisa.make_params(2, 4096, 16, 4, 128, K=8)
    append = calls(pisa, p)["append"]
    for kw, code in ((dict(struct_size=4), -1), (dict(eps=0.0), -1), (dict(eps=-1.0), -1), (dict(eps=1e-31), -1),
                     (dict(eps=float("inf")), -1), (dict(eps=float("nan")), -1), (dict(q_weight=MIS), -3),
                     (dict(k_weight=MIS), -3)):
        assert append(cache(pisa), norm=norm(pisa, **kw)) == code, kw
    assert append(cache(pisa), norm=norm(pisa), size=16) == -4


def test_read_refusals(pisa):
    p = pisa.make_params(2, 4096, 16, 4, 128, K=8)
    read = calls(pisa, p)["read"]
    c = cache(pisa)
    assert read(c, n=-1) == -1 and read(c, n=4097) == -1 and read(c, out=MIS) == -3 and read(c, new=ODD) == -3
    assert read(c, size=255) == -4 and read(None, n=0) == 0
    assert calls(pisa, pisa.make_params(2, 4096, 16, 4, 96))["read"](c) == -2


def test_binding_checks_8_bit_pages(pisa):
    p = pisa.make_params(2, 128, 4, 2, 64)
    k = torch.zeros(2, 2, 3, 64, dtype=torch.bfloat16)
    kp, vp, scales = pisa.quantized_pages(p, 4, device="cpu")
    assert kp.shape == vp.shape == (4, 2, 64, 64) and kp.dtype is torch.float8_e4m3fn and scales.shape == (2, 4, 2, 64)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    layer = pisa.PagedAttention(p, n=3, device="cpu")
    for call in (lambda **kw: layer.append(None, k, k, **kw), lambda **kw: layer.read(k, k, **kw)):
        for bad in (dict(k_pages=kp.view(torch.uint8)), dict(v_pages=vp.float()), dict(scales=scales[:1]),
                    dict(scales=scales.float()), dict(scales=scales[:, :3]), dict(scales=None), dict(k_pages=kp[:, :1])):
            a = dict(k_pages=kp, v_pages=vp, page_table=table, seq_lens=lens, scales=scales) | bad
            with pytest.raises(ValueError, match="expected contiguous"):
                call(**a)
        with pytest.raises(ValueError, match="expected CUDA tensors"):
            call(k_pages=kp, v_pages=vp, page_table=table, seq_lens=lens, scales=scales)
    with pytest.raises(ValueError):
        layer.read(None, None, kp, vp, table, lens, scales=scales)
    for bad in (torch.ones(32), torch.ones(64).double()):
        with pytest.raises(ValueError, match="norm"):
            pisa.PagedAttention(p, n=3, device="cpu", q_norm=bad)
        with pytest.raises(ValueError, match="norm"):
            pisa.PagedAttention(p, n=3, device="cpu", k_norm=bad)


def test_attention_refusals(pisa):
    p = pisa.make_params(2, 4096, 16, 4, 128, K=8)
    c = cache(pisa)
    on = calls(pisa, p)
    for name in set(on) - {"append", "read"}:
        assert on[name](c, q=None) == -1 and on[name](c, q=MIS) == -3, name
        for dtype, d, code in (("fp32", 128, -2), ("bf16", 96, -2)):
            assert calls(pisa, pisa.make_params(2, 4096, 16, 4, d, K=8, dtype=dtype))[name](c) == code, name
    for name in ("dense", "selected", "prefill"):
        assert on[name](c, out=None) == -1 and on[name](c, out=MIS) == -3, name
    assert on["selected"](c, idx=None) == -1 and on["selected"](c, idx=ODD) == -3
    bad = pisa.Mask(ctypes.sizeof(pisa.Mask), -1.0, 0, None, None, None)
    assert on["dense"](c, mask=ctypes.byref(bad)) == -1 and on["prefill"](c, mask=ctypes.byref(bad)) == -1
    assert on["prefill"](c, n=-1) == -1 and on["prefill"](c, n=4097) == -1 and on["prefill"](c, new=ODD) == -3
    assert on["prefill"](None, n=0) == 0


def test_scratch_sizes(pisa):
    p = pisa.make_params(2, 4096, 16, 4, 128, K=8)
    sizes = [pisa.cache_scratch_bytes(p, n) for n in (0, 1, 61, 2048, 4096)]
    assert sizes[:3] == [0, 0, 0] and sizes[3] == sizes[4] >= 4 * 2 * 4096 * 4 * 128
    assert pisa.cache_scratch_bytes(p, -1) == 0 and pisa.cache_scratch_bytes(p, 4097) == 0
    assert pisa.cache_scratch_bytes(pisa.make_params(64, 131072, 32, 8, 128), 8192) == 0  # 34 GB
    assert pisa.lib().pisa_cache_scratch_bytes(ctypes.byref(p), pisa.CACHE_PARAMS, 4096) == 0


def test_selector_refusals(pisa):
    L = pisa.lib()
    p, f32 = (pisa.make_params(2, 4096, 16, 4, 128, K=8, dtype=t) for t in ("bf16", "fp32"))

    def build(c, p=p, ws=A, size=BIG, pyramid=A):
        return L.pisa_cache_build_pyramid(ctypes.byref(p), c, A, pyramid, ws, size, None)

    def select(c, p=p, ws=A, size=BIG, pyramid=A, q=A, lens=A, idx=A):
        return L.pisa_cache_select_decode(ctypes.byref(p), q, c, lens, pyramid, ws, size, idx, None, None, None)

    for call in (build, select):
        assert call(None) == -1 and call(cache(pisa, struct_size=8)) == -1
        assert call(cache(pisa, format=2)) == -2 and call(cache(pisa), p=f32) == -2
        for f in ("k_pages", "k_scales"):
            assert call(cache(pisa, **{f: None})) == -1 and call(cache(pisa, **{f: MIS})) == -3
        assert call(cache(pisa, num_pages=0)) == -1
        assert call(cache(pisa, page_table=None)) == -1 and call(cache(pisa, page_table=ODD)) == -3
        c = cache(pisa, v_pages=None, v_scales=None)
        assert call(c, pyramid=None) == -1 and call(c, pyramid=MIS) == -3 and call(c, size=16) == -4
        assert call(c, ws=None) == -1 and call(c, ws=MIS) == -3
    c = cache(pisa)
    assert select(c, q=None) == -1 and select(c, lens=None) == -1 and select(c, idx=None) == -1
    kp, _, scales = pisa.quantized_pages(p, 4, device="cpu")
    table = torch.zeros(2, 64, dtype=torch.int32)
    for bad in (dict(k_pages=kp.float()), dict(scales=scales[:1]), dict(scales=scales.float())):
        with pytest.raises(ValueError, match="expected contiguous"):
            pisa.build_pyramid_paged(p, **(dict(k_pages=kp, page_table=table, pyramid=None, ws=None, scales=scales) | bad))
