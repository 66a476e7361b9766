"""Thin ctypes binding of the selector's C ABI (include/pisa.h).

Argument marshalling only: every step of the selection runs in the CUDA
kernels of libpisa.so.  PyTorch provides device memory and streams.  Importing
this module loads the library and raises ImportError when it is missing; there
is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpisa.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
        "(the selector has no CPU fallback)")

_lib = ctypes.CDLL(LIB_PATH)

PISA_OK = 0
STATUS_NAMES = {0: "PISA_OK", -1: "PISA_ERR_INVALID_ARG", -2: "PISA_ERR_UNSUPPORTED",
                -3: "PISA_ERR_MISALIGNED", -4: "PISA_ERR_WORKSPACE", -5: "PISA_ERR_CUDA",
                -6: "PISA_ERR_DEVICE"}
BF16, FP32 = 0, 1
SCORER_LSE, SCORER_MEAN, SCORER_MEAN_VAR = 0, 1, 2
SUMMARIES_ALL, SUMMARIES_PREFIX = 0, 1
MODE_PREFILL, MODE_DECODE, MODE_FLAT, MODE_ATTEND = 0, 1, 2, 3
DEV_OK, DEV_BAD_SEQ_LEN, DEV_TIMEOUT, DEV_BAD_INDEX = 0, 1, 2, 3

EXPORTED = ["pisa_abi_version", "pisa_status_string", "pisa_pyramid_levels", "pisa_pyramid_nodes",
            "pisa_pyramid_bytes", "pisa_workspace_bytes", "pisa_build_pyramid", "pisa_select_prefill",
            "pisa_prefill_route", "pisa_prefill_leaves", "pisa_select_decode", "pisa_select_flat",
            "pisa_read_device_status", "pisa_select_prefill_static", "pisa_kernel_launches",
            "pisa_attend_prefill", "pisa_build_pyramid_paged", "pisa_select_decode_paged", "pisa_attend_decode",
            "pisa_read_static_status", "pisa_test_inject_leaf_timeout", "pisa_append_paged",
            "pisa_dense_decode_paged", "pisa_attend_decode_paged", "pisa_dense_prefill_paged",
            "pisa_paged_workspace_bytes"]


class Params(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("dtype", ctypes.c_int32),
                ("B", ctypes.c_int64), ("N", ctypes.c_int64),
                ("H_q", ctypes.c_int32), ("H_kv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("C", ctypes.c_int32), ("g", ctypes.c_int32), ("K", ctypes.c_int32),
                ("qtile", ctypes.c_int32), ("scale", ctypes.c_float), ("scorer", ctypes.c_int32),
                ("summaries", ctypes.c_int32)]


class Mask(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("softcap", ctypes.c_float), ("window", ctypes.c_int64),
                ("slopes", ctypes.c_void_p), ("first_key", ctypes.c_void_p), ("prefix_lens", ctypes.c_void_p)]


_P = ctypes.POINTER(Params)
_M = ctypes.POINTER(Mask)
_strides_t = ctypes.c_int64 * 9
_vp = ctypes.c_void_p
_lib.pisa_abi_version.restype = ctypes.c_int
_lib.pisa_kernel_launches.restype = ctypes.c_uint64
_lib.pisa_status_string.argtypes = [ctypes.c_int]
_lib.pisa_status_string.restype = ctypes.c_char_p
_lib.pisa_pyramid_levels.argtypes = [_P]
_lib.pisa_pyramid_levels.restype = ctypes.c_int32
_lib.pisa_pyramid_nodes.argtypes = [_P]
_lib.pisa_pyramid_nodes.restype = ctypes.c_int64
_lib.pisa_pyramid_bytes.argtypes = [_P]
_lib.pisa_pyramid_bytes.restype = ctypes.c_size_t
_lib.pisa_workspace_bytes.argtypes = [_P, ctypes.c_int32]
_lib.pisa_workspace_bytes.restype = ctypes.c_size_t
_lib.pisa_build_pyramid.argtypes = [_P, _vp, _vp, _vp, _vp]
_lib.pisa_build_pyramid.restype = ctypes.c_int
_lib.pisa_select_prefill.argtypes = [_P, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp, _vp, _vp, _vp]
_lib.pisa_select_prefill.restype = ctypes.c_int
_lib.pisa_prefill_route.argtypes = [_P, _vp, _vp, _vp, ctypes.c_size_t, _vp, _vp]
_lib.pisa_prefill_route.restype = ctypes.c_int
_lib.pisa_prefill_leaves.argtypes = [_P, _vp, _vp, _vp, ctypes.c_size_t, _vp, _vp, _vp]
_lib.pisa_prefill_leaves.restype = ctypes.c_int
_lib.pisa_select_decode.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp, _vp, _vp, _vp]
_lib.pisa_select_decode.restype = ctypes.c_int
_lib.pisa_select_flat.argtypes = [_P, _vp, _vp, _vp, ctypes.c_size_t, _vp, _vp, _vp]
_lib.pisa_select_flat.restype = ctypes.c_int
_lib.pisa_build_pyramid_paged.argtypes = [_P, _vp, ctypes.c_int64, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
_lib.pisa_build_pyramid_paged.restype = ctypes.c_int
_lib.pisa_select_decode_paged.argtypes = [_P, _vp, _vp, ctypes.c_int64, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp,
                                          _vp, _vp, _vp]
_lib.pisa_select_decode_paged.restype = ctypes.c_int
_lib.pisa_attend_decode.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp, _vp]
_lib.pisa_attend_decode.restype = ctypes.c_int
_lib.pisa_attend_prefill.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp, _vp]
_lib.pisa_attend_prefill.restype = ctypes.c_int
_lib.pisa_append_paged.argtypes = [_P, ctypes.c_int64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int32,
                                   ctypes.c_int32, _vp, _vp, ctypes.c_int64, _vp, _vp, ctypes.c_size_t, _vp, _vp, _vp]
_lib.pisa_append_paged.restype = ctypes.c_int
_lib.pisa_dense_decode_paged.argtypes = [_P, _M, _vp, _vp, _vp, ctypes.c_int64, _vp, _vp, _vp, ctypes.c_size_t, _vp,
                                         _vp]
_lib.pisa_dense_decode_paged.restype = ctypes.c_int
_lib.pisa_attend_decode_paged.argtypes = [_P, _vp, _vp, _vp, ctypes.c_int64, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp,
                                          _vp]
_lib.pisa_attend_decode_paged.restype = ctypes.c_int
_lib.pisa_dense_prefill_paged.argtypes = [_P, _M, ctypes.c_int64, _vp, _vp, _vp, ctypes.c_int64, _vp, _vp, _vp, _vp,
                                          ctypes.c_size_t, _vp, _vp]
_lib.pisa_dense_prefill_paged.restype = ctypes.c_int
_lib.pisa_paged_workspace_bytes.argtypes = [_P, ctypes.c_int64]
_lib.pisa_paged_workspace_bytes.restype = ctypes.c_size_t
_lib.pisa_read_device_status.argtypes = [_vp, ctypes.POINTER(ctypes.c_int32), _vp]
_lib.pisa_read_device_status.restype = ctypes.c_int
_lib.pisa_select_prefill_static.argtypes = [_P, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.pisa_select_prefill_static.restype = ctypes.c_int
_lib.pisa_read_static_status.argtypes = [ctypes.POINTER(ctypes.c_int32), _vp]
_lib.pisa_read_static_status.restype = ctypes.c_int
_lib.pisa_test_inject_leaf_timeout.argtypes = [ctypes.c_uint64, ctypes.c_int32]
_lib.pisa_test_inject_leaf_timeout.restype = None


class PisaError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)}")


def lib() -> ctypes.CDLL:
    return _lib


def status_string(code: int) -> str:
    return _lib.pisa_status_string(code).decode()


def abi_version() -> int:
    return _lib.pisa_abi_version()


def kernel_launches() -> int:
    """Kernel launches the library has issued in this process so far."""
    return _lib.pisa_kernel_launches()


def make_params(B: int, N: int, H_q: int, H_kv: int, d: int, C: int = 64, g: int = 2, K: int = 8,
                qtile: int = 4, dtype: str = "bf16", scale: float = 0.0, scorer: int = 0,
                summaries: int = 0) -> Params:
    """scorer: SCORER_LSE (PISA), SCORER_MEAN (PISA-1) or SCORER_MEAN_VAR (PISA-2);
    summaries: SUMMARIES_ALL or SUMMARIES_PREFIX (prefix-consistent prefill)."""
    return Params(ctypes.sizeof(Params), BF16 if dtype == "bf16" else FP32, B, N, H_q, H_kv, d, C, g, K,
                  qtile, scale, scorer, summaries)


def params_from_shape(s, N: Optional[int] = None, scorer: int = 0, summaries: int = 0) -> Params:
    return make_params(s.B, s.N if N is None else N, s.Hq, s.Hkv, s.d, s.C, s.g, s.K, s.qtile, s.dtype,
                       scorer=scorer, summaries=summaries)


def pyramid_levels(p: Params) -> int:
    return _lib.pisa_pyramid_levels(ctypes.byref(p))


def pyramid_nodes(p: Params) -> int:
    return _lib.pisa_pyramid_nodes(ctypes.byref(p))


def pyramid_bytes(p: Params) -> int:
    return _lib.pisa_pyramid_bytes(ctypes.byref(p))


def workspace_bytes(p: Params, mode: int) -> int:
    return _lib.pisa_workspace_bytes(ctypes.byref(p), mode)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(rc: int, what: str):
    if rc != PISA_OK:
        raise PisaError(rc, what)


def build_pyramid(p: Params, k: torch.Tensor, pyramid: torch.Tensor, seq_lens: Optional[torch.Tensor] = None,
                  stream=None, check: bool = True) -> int:
    rc = _lib.pisa_build_pyramid(ctypes.byref(p), _ptr(k), _ptr(seq_lens), _ptr(pyramid), _stream(stream))
    if check:
        _check(rc, "pisa_build_pyramid")
    return rc


def select_prefill(p: Params, q, k, pyramid, ws, out_idx, out_score=None, trace=None, stream=None,
                   check: bool = True) -> int:
    rc = _lib.pisa_select_prefill(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(pyramid), _ptr(ws),
                                  0 if ws is None else ws.numel() * ws.element_size(),
                                  _ptr(out_idx), _ptr(out_score), _ptr(trace), _stream(stream))
    if check:
        _check(rc, "pisa_select_prefill")
    return rc


def prefill_route(p: Params, q, pyramid, ws, trace=None, stream=None, check: bool = True) -> int:
    rc = _lib.pisa_prefill_route(ctypes.byref(p), _ptr(q), _ptr(pyramid), _ptr(ws),
                                 ws.numel() * ws.element_size(), _ptr(trace), _stream(stream))
    if check:
        _check(rc, "pisa_prefill_route")
    return rc


def prefill_leaves(p: Params, q, k, ws, out_idx, out_score=None, stream=None, check: bool = True) -> int:
    rc = _lib.pisa_prefill_leaves(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(ws), ws.numel() * ws.element_size(),
                                  _ptr(out_idx), _ptr(out_score), _stream(stream))
    if check:
        _check(rc, "pisa_prefill_leaves")
    return rc


def select_decode(p: Params, q, k_cache, seq_lens, pyramid, ws, out_idx, out_score=None, trace=None,
                  stream=None, check: bool = True) -> int:
    rc = _lib.pisa_select_decode(ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(seq_lens), _ptr(pyramid),
                                 _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                 _ptr(out_idx), _ptr(out_score), _ptr(trace), _stream(stream))
    if check:
        _check(rc, "pisa_select_decode")
    return rc


def select_flat(p: Params, q, pyramid, ws, out_idx, out_score=None, stream=None, check: bool = True) -> int:
    rc = _lib.pisa_select_flat(ctypes.byref(p), _ptr(q), _ptr(pyramid), _ptr(ws),
                               0 if ws is None else ws.numel() * ws.element_size(),
                               _ptr(out_idx), _ptr(out_score), _stream(stream))
    if check:
        _check(rc, "pisa_select_flat")
    return rc


def build_pyramid_paged(p: Params, k_pages, page_table, pyramid, ws, seq_lens=None, stream=None,
                        check: bool = True) -> int:
    """k_pages [num_pages, H_kv, C, d]; page_table int32 [B, ceil(N / C)]."""
    rc = _lib.pisa_build_pyramid_paged(ctypes.byref(p), _ptr(k_pages), k_pages.shape[0], _ptr(page_table),
                                       _ptr(seq_lens), _ptr(pyramid), _ptr(ws), ws.numel() * ws.element_size(),
                                       _stream(stream))
    if check:
        _check(rc, "pisa_build_pyramid_paged")
    return rc


def select_decode_paged(p: Params, q, k_pages, page_table, seq_lens, pyramid, ws, out_idx, out_score=None,
                        trace=None, stream=None, check: bool = True) -> int:
    rc = _lib.pisa_select_decode_paged(ctypes.byref(p), _ptr(q), _ptr(k_pages), k_pages.shape[0], _ptr(page_table),
                                       _ptr(seq_lens), _ptr(pyramid), _ptr(ws), ws.numel() * ws.element_size(),
                                       _ptr(out_idx), _ptr(out_score), _ptr(trace), _stream(stream))
    if check:
        _check(rc, "pisa_select_decode_paged")
    return rc


def attend_prefill(p: Params, q, k, v, idx, ws, out, stream=None, check: bool = True) -> int:
    rc = _lib.pisa_attend_prefill(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(idx), _ptr(ws),
                                  0 if ws is None else ws.numel() * ws.element_size(), _ptr(out),
                                  _stream(stream))
    if check:
        _check(rc, "pisa_attend_prefill")
    return rc


def attend_decode(p: Params, q, k_cache, v_cache, seq_lens, idx, ws, out, stream=None, check: bool = True) -> int:
    rc = _lib.pisa_attend_decode(ctypes.byref(p), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seq_lens), _ptr(idx),
                                 _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), _ptr(out),
                                 _stream(stream))
    if check:
        _check(rc, "pisa_attend_decode")
    return rc


def paged_workspace_bytes(p: Params, n: int = 1) -> int:
    return _lib.pisa_paged_workspace_bytes(ctypes.byref(p), n)


# What the paged calls ask of their tensors (the C side sees only addresses):
# dtype, shape, one device, and adjacent elements.  These run before every
# decode step, so they only touch attributes that cost a fraction of a
# microsecond.
def _refuse(t, name: str, shape, dtype, index: int, layout: str):
    raise ValueError(f"{name}: expected {layout} {dtype} {tuple(shape)} on cuda:{index}, got {t.dtype} "
                     f"{tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _want(t, name: str, shape, dtype, index: int) -> int:
    """Address of a contiguous tensor."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _refuse(t, name, shape, dtype, index, "contiguous")
    return t.data_ptr()


def _want_rows(t, name: str, shape, dtype, index: int):
    """Address and strides of a [B, H, n, d] view with adjacent elements in a row."""
    st = t.stride()
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or st[3] != 1:
        _refuse(t, name, shape, dtype, index, "row-contiguous")
    return t.data_ptr(), st


def _want_cache(p: Params, k_pages, v_pages, page_table, seq_lens, dtype, index: int):
    """(k_pages, v_pages, number of pages, page_table, seq_lens) as the calls take them."""
    num = k_pages.shape[0]
    shape = (num, p.H_kv, p.C, p.d)
    B = p.B
    return (_want(k_pages, "k_pages", shape, dtype, index), _want(v_pages, "v_pages", shape, dtype, index), num,
            _want(page_table, "page_table", (B, -(-p.N // 64)), torch.int32, index),
            _want(seq_lens, "seq_lens", (B,), torch.int32, index))


def _want_space(ws, index: int):
    """Address and bytes of a workspace."""
    if ws.get_device() != index or not ws.is_contiguous():
        _refuse(ws, "ws", ws.shape, ws.dtype, index, "contiguous")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _dtype(p: Params) -> torch.dtype:
    return torch.bfloat16 if p.dtype == BF16 else torch.float32


def _launch(index: int, stream, what: str, check: bool, fn, *args) -> int:
    """Calls fn(*args, stream) with the tensors' device current, on the given
    stream or the device's current one."""
    if index < 0:
        raise ValueError(f"{what}: expected CUDA tensors")
    if stream is None:
        st = torch._C._cuda_getCurrentRawStream(index)
    elif stream.device.index != index:
        raise ValueError(f"{what}: the stream is on {stream.device}, the tensors on cuda:{index}")
    else:
        st = stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, st)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, st)
    if check and rc != PISA_OK:
        raise PisaError(rc, what)
    return rc


class AttentionMask:
    """What a dense paged attention call does to its scores and which keys it
    sees (pisa_mask): a tanh cap, a window, per-head distance slopes [H_q]
    fp32, first visible keys [B, n] int32, prefix lengths [B] int32."""

    def __init__(self, softcap: float = 0.0, window: int = 0, slopes: Optional[torch.Tensor] = None,
                 first_key: Optional[torch.Tensor] = None, prefix_lens: Optional[torch.Tensor] = None):
        self.slopes, self.first_key, self.prefix_lens = slopes, first_key, prefix_lens
        self.c = Mask(ctypes.sizeof(Mask), softcap, window, None, None, None)  # addresses: at each call


def _mask_arg(mask: Optional[AttentionMask], p: Params, n: int, index: int):
    if mask is None:
        return None
    c = mask.c
    c.slopes = None if mask.slopes is None else _want(mask.slopes, "slopes", (p.H_q,), torch.float32, index)
    c.first_key = None if mask.first_key is None else _want(mask.first_key, "first_key", (p.B, n), torch.int32, index)
    c.prefix_lens = (None if mask.prefix_lens is None else
                     _want(mask.prefix_lens, "prefix_lens", (p.B,), torch.int32, index))
    return ctypes.byref(c)


# The calls proper, with a workspace, outputs and angles (addresses) that their
# callers have looked at already: the functions below at each call,
# PagedAttention when it makes them.
def _append(p, k, v, k_pages, v_pages, page_table, seq_lens, space, rope, rot, interleaved, q, q_out, k_out, new_lens,
            stream, check) -> int:
    index, dt = k.get_device(), _dtype(p)
    n = k.shape[2]
    kv_shape = (p.B, p.H_kv, n, p.d)
    kp, ks = _want_rows(k, "k", kv_shape, dt, index)
    vp, vs = _want_rows(v, "v", kv_shape, dt, index)
    qp, qs = (None, ks) if q is None else _want_rows(q, "q", (p.B, p.H_q, n, p.d), dt, index)
    strides = _strides_t(*qs[:3], *ks[:3], *vs[:3])
    at = ctypes.addressof(strides)
    kpp, vpp, num, table, lens = _want_cache(p, k_pages, v_pages, page_table, seq_lens, dt, index)
    return _launch(index, stream, "pisa_append_paged", check, _lib.pisa_append_paged, ctypes.byref(p), n, qp, at, kp,
                   at + 24, vp, at + 48, lens,
                   None if new_lens is None else _want(new_lens, "new_lens", (p.B,), torch.int32, index), rope, rot,
                   interleaved, kpp, vpp, num, table, *space, q_out,
                   None if k_out is None else _want(k_out, "k_out", kv_shape, dt, index))


def _dense_decode(p, q, k_pages, v_pages, page_table, seq_lens, space, out, mask, stream, check) -> int:
    index, dt = q.get_device(), _dtype(p)
    cache = _want_cache(p, k_pages, v_pages, page_table, seq_lens, dt, index)
    return _launch(index, stream, "pisa_dense_decode_paged", check, _lib.pisa_dense_decode_paged, ctypes.byref(p),
                   _mask_arg(mask, p, 1, index), _want(q, "q", (p.B, p.H_q, p.d), dt, index), *cache, *space, out)


def _selected_decode(p, q, k_pages, v_pages, page_table, seq_lens, idx, space, out, stream, check) -> int:
    index, dt = q.get_device(), _dtype(p)
    cache = _want_cache(p, k_pages, v_pages, page_table, seq_lens, dt, index)
    return _launch(index, stream, "pisa_attend_decode_paged", check, _lib.pisa_attend_decode_paged, ctypes.byref(p),
                   _want(q, "q", (p.B, p.H_q, p.d), dt, index), *cache,
                   _want(idx, "idx", (p.B, p.H_kv, p.K + 3), torch.int32, index), *space, out)


def _dense_prefill(p, q, k_pages, v_pages, page_table, seq_lens, new_lens, space, out, mask, stream, check) -> int:
    index, dt, n = q.get_device(), _dtype(p), q.shape[2]
    cache = _want_cache(p, k_pages, v_pages, page_table, seq_lens, dt, index)
    return _launch(index, stream, "pisa_dense_prefill_paged", check, _lib.pisa_dense_prefill_paged, ctypes.byref(p),
                   _mask_arg(mask, p, n, index), n, _want(q, "q", (p.B, p.H_q, n, p.d), dt, index), *cache,
                   None if new_lens is None else _want(new_lens, "new_lens", (p.B,), torch.int32, index), *space, out)


def append_paged(p: Params, k, v, k_pages, v_pages, page_table, seq_lens, ws, rope=None, interleaved: bool = False,
                 q=None, q_out=None, k_out=None, new_lens=None, stream=None, check: bool = True) -> int:
    """k, v [B, H_kv, n, d] and q [B, H_q, n, d], strided views allowed; rope
    fp32 [N, rot_dim] (cosines, then sines); seq_lens counts the new tokens."""
    index, rot = k.get_device(), 0 if rope is None else rope.shape[-1]
    if q_out is not None:
        q_out = _want(q_out, "q_out", (p.B, p.H_q, k.shape[2], p.d), _dtype(p), index)
    if rope is not None:
        rope = _want(rope, "rope", (p.N, rot), torch.float32, index)
    return _append(p, k, v, k_pages, v_pages, page_table, seq_lens, _want_space(ws, index), rope, rot, interleaved, q,
                   q_out, k_out, new_lens, stream, check)


def dense_decode_paged(p: Params, q, k_pages, v_pages, page_table, seq_lens, ws, out,
                       mask: Optional[AttentionMask] = None, stream=None, check: bool = True) -> int:
    """q and out [B, H_q, d]: attention of one new token per sequence over its whole cache."""
    index = q.get_device()
    return _dense_decode(p, q, k_pages, v_pages, page_table, seq_lens, _want_space(ws, index),
                         _want(out, "out", (p.B, p.H_q, p.d), _dtype(p), index), mask, stream, check)


def attend_decode_paged(p: Params, q, k_pages, v_pages, page_table, seq_lens, idx, ws, out, stream=None,
                        check: bool = True) -> int:
    """attend_decode over a paged cache; idx int32 [B, H_kv, K+3]."""
    index = q.get_device()
    return _selected_decode(p, q, k_pages, v_pages, page_table, seq_lens, idx, _want_space(ws, index),
                            _want(out, "out", (p.B, p.H_q, p.d), _dtype(p), index), stream, check)


def dense_prefill_paged(p: Params, q, k_pages, v_pages, page_table, seq_lens, ws, out, new_lens=None,
                        mask: Optional[AttentionMask] = None, stream=None, check: bool = True) -> int:
    """q and out [B, H_q, n, d]: attention of n new tokens per sequence over the pages that hold them already."""
    index = q.get_device()
    return _dense_prefill(p, q, k_pages, v_pages, page_table, seq_lens, new_lens, _want_space(ws, index),
                          _want(out, "out", (p.B, p.H_q, q.shape[2], p.d), _dtype(p), index), mask, stream, check)


def read_device_status(ws: torch.Tensor, stream=None) -> int:
    code = ctypes.c_int32(0)
    rc = _lib.pisa_read_device_status(_ptr(ws), ctypes.byref(code), _stream(stream))
    if rc not in (PISA_OK, -6):
        _check(rc, "pisa_read_device_status")
    return code.value


class Selector:
    """Owns the device buffers (torch tensors) for one problem shape and runs
    the selector through the C ABI.  `mode` is "prefill", "decode" or "flat"."""

    def __init__(self, p: Params, device="cuda", mode: str = "prefill", with_scores: bool = True):
        self.p = p
        self.device = torch.device(device)
        W = p.K + 3
        P = pyramid_nodes(p)
        self.pyramid = torch.empty(p.B, p.H_kv, P, p.d, dtype=torch.float32, device=self.device)
        m = {"prefill": MODE_PREFILL, "decode": MODE_DECODE, "flat": MODE_FLAT}[mode]
        nbytes = workspace_bytes(p, m)
        self.ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
        if mode == "decode":
            shape = (p.B, p.H_kv, W)
        else:
            shape = (p.B, p.H_kv, p.N, W)
        self.out_idx = torch.empty(shape, dtype=torch.int32, device=self.device)
        self.out_score = torch.empty(shape, dtype=torch.float32, device=self.device) if with_scores else None

    def build(self, k, seq_lens=None, stream=None):
        build_pyramid(self.p, k, self.pyramid, seq_lens, stream)

    def prefill(self, q, k, trace=None, stream=None, build: bool = True):
        if build:
            build_pyramid(self.p, k, self.pyramid, None, stream)
        select_prefill(self.p, q, k, self.pyramid, self.ws, self.out_idx, self.out_score, trace, stream)
        return self.out_idx, self.out_score

    def decode(self, q, k_cache, seq_lens, trace=None, stream=None):
        select_decode(self.p, q, k_cache, seq_lens, self.pyramid, self.ws, self.out_idx, self.out_score, trace,
                      stream)
        return self.out_idx, self.out_score

    def build_paged(self, k_pages, page_table, seq_lens=None, stream=None):
        build_pyramid_paged(self.p, k_pages, page_table, self.pyramid, self.ws, seq_lens, stream)

    def decode_paged(self, q, k_pages, page_table, seq_lens, trace=None, stream=None):
        select_decode_paged(self.p, q, k_pages, page_table, seq_lens, self.pyramid, self.ws, self.out_idx,
                            self.out_score, trace, stream)
        return self.out_idx, self.out_score

    def flat(self, q, k=None, stream=None, build: bool = True):
        if build:
            build_pyramid(self.p, k, self.pyramid, None, stream)
        select_flat(self.p, q, self.pyramid, self.ws, self.out_idx, self.out_score, stream)
        return self.out_idx, self.out_score

    def device_status(self, stream=None) -> int:
        return read_device_status(self.ws, stream)


class Attention:
    """Owns the workspace and output of block-sparse attention over a
    selection for one problem shape: prefill (pisa_attend_prefill, every
    query position) or decode (pisa_attend_decode, one query per sequence)."""

    def __init__(self, p: Params, device="cuda", mode: str = "prefill"):
        self.p = p
        self.mode = mode
        self.device = torch.device(device)
        m = MODE_ATTEND if mode == "prefill" else MODE_DECODE
        self.ws = torch.empty(max(workspace_bytes(p, m), 256), dtype=torch.uint8, device=self.device)
        shape = (p.B, p.H_q, p.N, p.d) if mode == "prefill" else (p.B, p.H_q, p.d)
        self.out = torch.empty(shape, dtype=torch.bfloat16, device=self.device)

    def __call__(self, q, k, v, idx, stream=None):
        attend_prefill(self.p, q, k, v, idx, self.ws, self.out, stream)
        return self.out

    def decode(self, q, k_cache, v_cache, seq_lens, idx, stream=None):
        attend_decode(self.p, q, k_cache, v_cache, seq_lens, idx, self.ws, self.out, stream)
        return self.out

    def device_status(self, stream=None) -> int:
        return read_device_status(self.ws, stream)


class PagedAttention:
    """A serving layer's calls over a paged cache for one problem shape, with
    up to n new tokens per sequence in a call: appending rotated keys and
    values, dense attention of one token or of a prompt, and attention over
    the selector's blocks.  Owns the workspace and one output buffer per kind
    of call, zeroed when it is made and written again by the next call of its
    kind (a call of fewer tokens uses its front).  Rows behind a sequence's new
    tokens are not written: they hold zeros or what an earlier call left there.
    Calls may run on any stream, one after the other.
    rope: fp32 [N, rot_dim] as append_paged takes it, or None."""

    def __init__(self, p: Params, n: int = 1, rope: Optional[torch.Tensor] = None, interleaved: bool = False,
                 device="cuda"):
        p = Params.from_buffer_copy(p)  # the buffers below are made for these numbers
        self.p, self.n, self.rope, self.interleaved = p, n, rope, interleaved
        self.device = torch.device(device)
        nbytes = paged_workspace_bytes(p, n)
        if nbytes == 0:
            raise ValueError("unsupported problem shape, or n outside [0, N]")
        nbytes = max(nbytes, paged_workspace_bytes(p, min(p.N, 1)))  # (n = 0: decode calls)
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        self.device = self.ws.device
        self._index = self.ws.get_device()
        self._space = _want_space(self.ws, self._index)
        self._rot = 0 if rope is None else rope.shape[-1]
        self._rope = None if rope is None else _want(rope, "rope", (p.N, self._rot), torch.float32, self._index)
        one, many = (p.B, p.H_q, p.d), (p.B, p.H_q, n, p.d)
        rows = p.B * p.H_q * p.d
        flat = torch.zeros(rows * (2 + 2 * n), dtype=_dtype(p), device=self.device)
        self._out = {"dense": flat[:rows].view(one), "selected": flat[rows:2 * rows].view(one),
                     "q": flat[2 * rows:(2 + n) * rows].view(many), "prefill": flat[(2 + n) * rows:].view(many)}
        if self._index >= 0:  # the zeros are there before the first call, whatever stream that runs on
            with torch.cuda.device(self._index):
                if not torch.cuda.is_current_stream_capturing():
                    torch.cuda.current_stream().synchronize()

    def _fits(self, x, ok: bool):
        if x.get_device() != self._index:
            raise ValueError(f"expected tensors on {self.device}, got {x.device}")
        if not ok:
            raise ValueError(f"{tuple(x.shape)}: more than the {self.n} new tokens per sequence asked for")

    def _buffer(self, kind: str, like):
        out = self._out[kind]
        same = out.shape == like.shape
        self._fits(like, same or (like.dim() == out.dim() and like.numel() <= out.numel()))
        if same:
            return out
        return out.view(-1)[:like.numel()].view(like.shape)

    def append(self, q, k, v, k_pages, v_pages, page_table, seq_lens, new_lens=None, k_out=None, stream=None):
        """Rotates and appends k and v; returns the rotated queries [B, H_q, n, d] (None when q is None)."""
        if q is None:
            self._fits(k, k.dim() == 4 and k.shape[2] <= self.n)
        q_out = None if q is None else self._buffer("q", q)
        _append(self.p, k, v, k_pages, v_pages, page_table, seq_lens, self._space, self._rope, self._rot,
                self.interleaved, q, None if q is None else q_out.data_ptr(), k_out, new_lens, stream, True)
        return None if q is None else q_out

    def dense_decode(self, q, k_pages, v_pages, page_table, seq_lens, mask=None, stream=None):
        out = self._buffer("dense", q)
        _dense_decode(self.p, q, k_pages, v_pages, page_table, seq_lens, self._space, out.data_ptr(), mask, stream,
                      True)
        return out

    def selected_decode(self, q, k_pages, v_pages, page_table, seq_lens, idx, stream=None):
        out = self._buffer("selected", q)
        _selected_decode(self.p, q, k_pages, v_pages, page_table, seq_lens, idx, self._space, out.data_ptr(), stream,
                         True)
        return out

    def dense_prefill(self, q, k_pages, v_pages, page_table, seq_lens, new_lens=None, mask=None, stream=None):
        out = self._buffer("prefill", q)
        _dense_prefill(self.p, q, k_pages, v_pages, page_table, seq_lens, new_lens, self._space, out.data_ptr(), mask,
                       stream, True)
        return out

    def device_status(self, stream=None) -> int:
        return read_device_status(self.ws, stream)
