"""The paged serving entry points refuse bad arguments on the host, before
any launch (fake addresses: none of these calls reaches a GPU), and their
64-bit references agree with independent forms."""
import ctypes

import pytest
import torch

import paged_ref as R


@pytest.fixture(scope="module")
def pisa():
    from pyramid_top_block_mean_gb300 import build
    build.build()
    from pyramid_top_block_mean_gb300 import pisa as m
    return m


A = ctypes.c_void_p(0x10000)
MIS = ctypes.c_void_p(0x10008)
ODD = ctypes.c_void_p(0x10002)
BIG = 1 << 40


def strides(*x):
    return (ctypes.c_int64 * 3)(*x)


def append(L, p, n=4, q=A, qs=None, k=A, ks=None, v=A, vs=None, lens=A, new=A, rope=A, rot=64, inter=0, kp=A, vp=A,
           pages=10, table=A, ws=A, size=BIG, q_out=A, k_out=A):
    return L.pisa_append_paged(ctypes.byref(p), n, q, qs, k, ks, v, vs, lens, new, rope, rot, inter, kp, vp, pages,
                               table, ws, size, q_out, k_out, None)


@pytest.mark.parametrize("change,code", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(lens=None), -1), (dict(kp=None), -1), (dict(vp=None), -1),
    (dict(table=None), -1), (dict(ws=None), -1), (dict(pages=0), -1), (dict(n=-1), -1), (dict(n=4097), -1),
    (dict(q=None), -1), (dict(q_out=None), -1), (dict(rope=None), -1), (dict(rot=0), -1), (dict(rot=-16), -1),
    (dict(rot=144), -1), (dict(rot=24), -2), (dict(k=MIS), -3), (dict(vp=MIS), -3), (dict(rope=MIS), -3),
    (dict(q_out=MIS), -3), (dict(k_out=MIS), -3), (dict(lens=ODD), -3), (dict(new=ODD), -3), (dict(table=ODD), -3),
    (dict(size=16), -4), (dict(ks=strides(512, 128, 4)), -3), (dict(vs=strides(512, -128, 128)), -1),
    (dict(pages=1 << 31), -2),
])
def test_append_refusals(pisa, change, code):
    p = pisa.make_params(2, 4096, 16, 4, 128, K=8)
    assert append(pisa.lib(), p, **change) == code


def mask(pisa, **kw):
    m = pisa.Mask(ctypes.sizeof(pisa.Mask), 0.0, 0, None, None, None)
    for key, val in kw.items():
        setattr(m, key, val)
    return ctypes.byref(m)


@pytest.mark.parametrize("bad", [dict(struct_size=8), dict(softcap=-1.0), dict(softcap=float("nan")),
                                 dict(softcap=float("inf")), dict(window=-1)])
def test_masks_are_checked(pisa, bad):
    L = pisa.lib()
    p = pisa.make_params(2, 4096, 16, 4, 128, K=8)
    m = mask(pisa, **bad)
    assert L.pisa_dense_decode_paged(ctypes.byref(p), m, A, A, A, 10, A, A, A, BIG, A, None) == -1
    assert L.pisa_dense_prefill_paged(ctypes.byref(p), m, 4, A, A, A, 10, A, A, A, A, BIG, A, None) == -1


def test_attention_refusals(pisa):
    L = pisa.lib()
    p = pisa.make_params(2, 4096, 16, 4, 128, K=8)
    f32 = pisa.make_params(2, 4096, 16, 4, 128, K=8, dtype="fp32")
    d96 = pisa.make_params(2, 4096, 16, 4, 96, K=8)

    def dense(p=p, q=A, k=A, v=A, pages=10, table=A, lens=A, ws=A, size=BIG, out=A):
        return L.pisa_dense_decode_paged(ctypes.byref(p), None, q, k, v, pages, table, lens, ws, size, out, None)

    def sel(p=p, q=A, k=A, v=A, pages=10, table=A, lens=A, idx=A, ws=A, size=BIG, out=A):
        return L.pisa_attend_decode_paged(ctypes.byref(p), q, k, v, pages, table, lens, idx, ws, size, out, None)

    def pre(p=p, n=4, q=A, k=A, v=A, pages=10, table=A, lens=A, new=A, ws=A, size=BIG, out=A):
        return L.pisa_dense_prefill_paged(ctypes.byref(p), None, n, q, k, v, pages, table, lens, new, ws, size, out,
                                          None)

    for call in (dense, sel, pre):
        assert call(p=f32) == -2 and call(p=d96) == -2
        for name in ("q", "k", "v", "table", "lens", "ws", "out"):
            assert call(**{name: None}) == -1, name
        for name in ("q", "k", "v", "ws", "out"):
            assert call(**{name: MIS}) == -3, name
        for name in ("table", "lens"):
            assert call(**{name: ODD}) == -3, name
        assert call(pages=0) == -1 and call(size=16) == -4
    assert sel(idx=None) == -1 and sel(idx=ODD) == -3
    assert pre(n=-1) == -1 and pre(n=4097) == -1 and pre(new=ODD) == -3


def test_empty_calls_are_no_ops(pisa):
    L = pisa.lib()
    p0 = pisa.make_params(0, 4096, 16, 4, 128, K=8)
    p = pisa.make_params(2, 4096, 16, 4, 128, K=8)
    assert append(L, p0, k=None, ws=None) == 0 and append(L, p, n=0, k=None, ws=None) == 0
    assert L.pisa_dense_decode_paged(ctypes.byref(p0), None, *[None] * 3, 0, *[None] * 3, 0, None, None) == 0
    assert L.pisa_dense_prefill_paged(ctypes.byref(p), None, 0, *[None] * 3, 0, *[None] * 4, 0, None, None) == 0


def test_workspace_sizes(pisa):
    p = pisa.make_params(2, 4096, 16, 4, 128, K=8)
    sizes = [pisa.paged_workspace_bytes(p, n) for n in (0, 1, 64, 4096)]
    assert all(s >= 256 for s in sizes)
    assert pisa.paged_workspace_bytes(p, -1) == 0 and pisa.paged_workspace_bytes(p, 4097) == 0
    assert pisa.paged_workspace_bytes(pisa.make_params(2, 4096, 16, 4, 96, K=8), 1) == 0


@pytest.mark.parametrize("B,N,Hkv,d", [(1, 16384, 1, 128), (2, 4096, 4, 128), (1, 1024, 4, 64), (3, 65536, 5, 64),
                                       (1, 65536, 76, 128), (1, 65536, 77, 128), (2, 200, 1, 64)])
@pytest.mark.parametrize("G", [1, 4, 8])
def test_a_workspace_for_n_tokens_serves_fewer(pisa, B, N, Hkv, d, G):
    p = pisa.make_params(B, N, G * Hkv, Hkv, d, K=8)
    at = [n for n in (0, 1, 2, 17, 61, 128, 129, 200, 256, 511, 1000, 1024, 2047, 4096, 8192, 16384, 65536) if n <= N]
    sizes = [pisa.paged_workspace_bytes(p, n) for n in at]
    assert sizes[0] >= 256 and sizes == sorted(sizes), list(zip(at, sizes))


def test_binding_checks_tensors(pisa):
    p = pisa.make_params(2, 128, 4, 2, 64)
    k = torch.zeros(2, 2, 3, 64, dtype=torch.bfloat16)
    pool = torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)

    def call(**kw):
        a = dict(k=k, v=k, k_pages=pool, v_pages=pool, page_table=table, seq_lens=lens, ws=ws) | kw
        return pisa.append_paged(p, **a)

    for bad in (dict(v=k.float()), dict(v=k[:, :1]), dict(k_pages=pool[:, :1]), dict(page_table=table.long()),
                dict(page_table=table[:, :1]), dict(seq_lens=lens[:1]), dict(k=k.transpose(2, 3).contiguous()
                                                                             .transpose(2, 3)),
                dict(new_lens=lens.long()), dict(rope=torch.zeros(100, 64)), {}):  # {}: tensors not on a GPU
        with pytest.raises(ValueError):
            call(**bad)


def test_layer_checks_its_tensors(pisa):
    p = pisa.make_params(2, 128, 4, 2, 64)
    for bad in (dict(n=129), dict(n=-1), dict(rope=torch.zeros(100, 64)), dict(rope=torch.zeros(128, 64).double())):
        with pytest.raises((ValueError, RuntimeError)):
            pisa.PagedAttention(p, **(dict(n=3, device="cpu") | bad))
    layer = pisa.PagedAttention(p, n=3, rope=torch.zeros(128, 64), device="cpu")
    q, k = (torch.zeros(2, h, 3, 64, dtype=torch.bfloat16) for h in (4, 2))
    pool = torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    for call in (lambda: layer.append(q, k, k, pool, pool, table, lens),  # not on a GPU
                 lambda: layer.append(None, k, k, pool, pool, table, lens),
                 lambda: layer.dense_prefill(q.repeat(1, 1, 2, 1), pool, pool, table, lens),  # six new tokens
                 lambda: layer.dense_decode(q, pool, pool, table, lens)):
        with pytest.raises(ValueError):
            call()


def test_reference_attention_against_a_library_routine():
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(n, 16, generator=g, dtype=torch.float64) for n in (5, 9, 9))
    keep = torch.rand(5, 9, generator=g) > 0.4
    keep[:, 0] = True
    keep[2] = False
    o, tol = R.attend(q, k, v, keep, 0.25)
    want = torch.nn.functional.scaled_dot_product_attention(q[None], k[None], v[None], attn_mask=keep[None],
                                                            scale=0.25)[0]
    rows = [0, 1, 3, 4]
    assert torch.allclose(o[rows], want[rows], atol=1e-12) and bool((o[2] == 0).all()) and bool((tol > 0).all())
    # a key that no row sees may hold anything
    keep[:, 3] = False
    v2 = v.clone(); v2[3] = float("nan")
    assert torch.equal(R.attend(q, k, v2, keep, 0.25)[0], R.attend(q, k, v, keep, 0.25)[0])


def test_reference_rotation_against_complex_products():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 7, 32, generator=g, dtype=torch.float64)
    ang = torch.rand(50, 8, generator=g, dtype=torch.float64) * 6
    rope = torch.cat([ang.cos(), ang.sin()], 1)
    pos = torch.tensor([0, 3, 4, 9, 20, 48, 49])
    turn = torch.polar(torch.ones(7, 8, dtype=torch.float64), ang[pos])
    y, _ = R.rotate(x, rope, pos, True)
    want = torch.view_as_real(torch.view_as_complex(x[..., :16].reshape(3, 7, 8, 2)) * turn).reshape(3, 7, 16)
    assert torch.allclose(y[..., :16], want) and torch.equal(y[..., 16:], x[..., 16:])
    y, _ = R.rotate(x, rope, pos, False)
    z = torch.complex(x[..., :8], x[..., 8:16]) * turn
    assert torch.allclose(y[..., :16], torch.cat([z.real, z.imag], -1))


def test_reference_spans():
    pos = torch.tensor([3, 4, 5, 6])
    lo, hi = R.spans(pos, 7, window=2, first=torch.tensor([0, 9, 0, 6]), prefix=6)
    assert lo.tolist() == [2, 9, 4, 6] and hi.tolist() == [5, 5, 5, 6]
    assert R.spans(pos, 7, prefix=20)[1].tolist() == [6, 6, 6, 6]
