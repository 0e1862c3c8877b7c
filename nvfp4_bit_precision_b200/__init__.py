"""Python binding of libnvfp4 -- the B200 (sm_100a) NVFP4 quantizer and
block-scaled GEMM.

The C functions keep their names (``nvfp4_quantize``, ``nvfp4_dequantize``,
``mxfp8_quantize``, ``mxfp4_quantize``, ``nvfp4_gemm``, ``nvfp4_grouped_gemm``, ``nvfp4_rmsnorm``,
``nvfp4_route``, ``nvfp4_combine``, ``nvfp4_gemv``, ``nvfp4_grouped_gemv``, ``nvfp4_expert_mlp``,
``nvfp4_kv_append``, ``nvfp4_kv_attention`` and the backward calls); this
module only marshals arguments: torch tensors become device pointers and the current torch
stream becomes the ``cudaStream_t``.  Every arithmetic step runs in the CUDA
kernels of ``libnvfp4.so``.  There is no fallback: importing this package
raises if the library is missing, and every call raises ``NVFP4Error`` on a
non-zero status.

The convenience wrappers (``quantize``, ``dequantize``, ``mxfp8``, ``mxfp4``, ``gemm``,
``grouped_gemm``, ``rmsnorm``, ``route``, ``combine``, ``gemv``, ``grouped_gemv``, ``expert_mlp``, ``kv_append``,
``kv_attention``) allocate their outputs with torch and call the C functions.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass
from typing import Optional

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4.so")

from . import build as _build

if _build.stale():
    try:
        _build.build()
    except Exception as exc:  # no nvcc / compile error: there is no CPU fallback
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing and could not be built: {exc}") from exc

_lib = ctypes.CDLL(LIB_PATH)


class _Torch:
    """torch, imported at its first use, when it takes this object's place: the C functions need addresses only."""

    def __getattr__(self, name):
        global torch
        import torch
        return getattr(torch, name)


torch = _Torch()

# ----------------------------------------------------------------- constants
NVFP4_OK = 0
NVFP4_RNE, NVFP4_SR = 0, 1
NVFP4_1D16, NVFP4_2D16x16 = 0, 1
NVFP4_ROWWISE, NVFP4_COLWISE = 1, 2
NVFP4_SF_ROWMAJOR, NVFP4_SF_MMA = 0, 1
NVFP4_OUT_F32, NVFP4_OUT_BF16 = 0, 1
NVFP4_SOFTMAX, NVFP4_SIGMOID = 0, 1

EXPORTED = [
    "nvfp4_quantize", "nvfp4_dequantize", "mxfp8_quantize", "nvfp4_gemm", "nvfp4_grouped_gemm",
    "nvfp4_quantize_workspace_size", "nvfp4_gemm_workspace_size", "nvfp4_sf_mma_bytes",
    "nvfp4_sf_mma_grouped_bytes", "nvfp4_workspace_status", "nvfp4_status_string",
    "nvfp4_version", "nvfp4_quantize_noalloc", "nvfp4_quantize_noalloc_status",
    "nvfp4_gather_rows", "mxfp4_quantize", "mxfp8_gemm", "mxfp8_sf_mma_bytes", "mxfp4_gemm",
    "mxfp8_combine", "nvfp4_gemm_cycles", "nvfp4_rmsnorm", "nvfp4_rmsnorm_backward",
    "nvfp4_rmsnorm_backward_workspace_size", "nvfp4_route", "nvfp4_route_backward",
    "nvfp4_route_workspace_size", "nvfp4_combine", "nvfp4_combine_backward",
    "nvfp4_combine_backward_workspace_size", "nvfp4_gemv", "nvfp4_grouped_gemv", "nvfp4_kv_append",
    "nvfp4_kv_attention", "nvfp4_kv_attention_workspace_size", "nvfp4_expert_mlp",
    "nvfp4_expert_mlp_workspace_size",
]


class QuantParams(ctypes.Structure):
    """Mirror of ``nvfp4_quant_params`` (include/nvfp4.h)."""
    _fields_ = [
        ("rounding", ctypes.c_int), ("scaling", ctypes.c_int), ("outputs", ctypes.c_int),
        ("rht_colwise", ctypes.c_int), ("sf_layout", ctypes.c_int),
        ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint32),
        ("amax_in", ctypes.c_void_p),
        ("row_index", ctypes.c_void_p), ("src_rows", ctypes.c_int64),
        ("group_offsets", ctypes.c_void_p), ("num_groups", ctypes.c_int),
        ("mx_outputs", ctypes.c_int), ("mx_rounding", ctypes.c_int),
        ("mx_q_row", ctypes.c_void_p), ("mx_sf_row", ctypes.c_void_p),
        ("mx_q_col", ctypes.c_void_p), ("mx_sf_col", ctypes.c_void_p),
        ("mx_sf_layout", ctypes.c_int),
    ]


class RouteParams(ctypes.Structure):
    """Mirror of ``nvfp4_route_params`` (include/nvfp4.h)."""
    _fields_ = [
        ("top_k", ctypes.c_int), ("score", ctypes.c_int), ("groups", ctypes.c_int),
        ("topk_groups", ctypes.c_int), ("group_top", ctypes.c_int), ("renormalize", ctypes.c_int),
        ("scale", ctypes.c_float),
    ]


class KVCacheView(ctypes.Structure):
    """Mirror of ``nvfp4_kv_cache`` (include/nvfp4.h)."""
    _fields_ = [
        ("q", ctypes.c_void_p), ("sf", ctypes.c_void_p), ("amax", ctypes.c_void_p),
        ("pages", ctypes.c_int64), ("kv_heads", ctypes.c_int), ("page_size", ctypes.c_int),
        ("dim", ctypes.c_int),
    ]


_P, _I64, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
_lib.nvfp4_quantize.argtypes = [_P, _I64, _I64, _I64, ctypes.POINTER(QuantParams), _P, _P, _P,
                                _P, _P, _P, _P, _SZ, _P]
_lib.nvfp4_quantize_noalloc.argtypes = [_P, _I64, _I64, _I64, ctypes.POINTER(QuantParams), _P,
                                        _P, _P, _P, _P, _P, _P]
_lib.mxfp8_quantize.argtypes = [_P, _I64, _I64, _I64, ctypes.c_int, ctypes.c_int,
                                ctypes.c_uint64, ctypes.c_uint32, _P, _P, _P, _P, _P]
_lib.mxfp4_quantize.argtypes = [_P, _I64, _I64, _I64, ctypes.c_int, ctypes.c_int, _P, _P, _P,
                                _P, _P]
_lib.mxfp4_gemm.argtypes = [_P, _P, _P, _P, _I64, _I64, _I64, ctypes.c_int, _P, _I64, _P, _P, _SZ,
                            _P]
_lib.nvfp4_dequantize.argtypes = [_P, _P, _P, _I64, _I64, ctypes.c_int, ctypes.c_int, _P, _P]
_lib.nvfp4_gemm.argtypes = [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, ctypes.c_int, _P, _I64, _P,
                            _P, _SZ, _P]
_lib.mxfp8_gemm.argtypes = [_P, _P, _P, _P, _I64, _I64, _I64, ctypes.c_int, _P, _I64, _P, _P, _SZ,
                            _P]
_lib.mxfp8_combine.argtypes = [_P, _P, _I64, _I64, _P, _P, _I64, ctypes.c_int, _P, _P, _SZ, _P]
_lib.mxfp8_sf_mma_bytes.argtypes = [_I64, _I64]
_lib.mxfp8_sf_mma_bytes.restype = _SZ
_lib.nvfp4_grouped_gemm.argtypes = [ctypes.c_int, _P, _I64, _P, _P, _P, _P, _P, _P, _I64, _I64,
                                    ctypes.c_int, _P, _P, _P, _SZ, _P]
_lib.nvfp4_gather_rows.argtypes = [_P, _P, _I64, _I64, _P, _I64, _P, ctypes.c_int, _P, _P, _P,
                                   _SZ, _P]
_lib.nvfp4_quantize_workspace_size.argtypes = [_I64, _I64, ctypes.POINTER(QuantParams)]
_lib.nvfp4_quantize_workspace_size.restype = _SZ
_lib.nvfp4_gemm_workspace_size.argtypes = [_I64, _I64, _I64]
_lib.nvfp4_gemm_workspace_size.restype = _SZ
_lib.nvfp4_sf_mma_bytes.argtypes = [_I64, _I64]
_lib.nvfp4_sf_mma_bytes.restype = _SZ
_lib.nvfp4_sf_mma_grouped_bytes.argtypes = [_I64, ctypes.c_int, _I64]
_lib.nvfp4_sf_mma_grouped_bytes.restype = _SZ
_lib.nvfp4_workspace_status.argtypes = [_P, _P]
_lib.nvfp4_gemm_cycles.argtypes = [_P, _P, ctypes.POINTER(ctypes.c_uint64)]
_lib.nvfp4_quantize_noalloc_status.argtypes = [_P]
_lib.nvfp4_status_string.argtypes = [ctypes.c_int]
_lib.nvfp4_status_string.restype = ctypes.c_char_p
_lib.nvfp4_version.restype = ctypes.c_int
_INT, _F32 = ctypes.c_int, ctypes.c_float
_lib.nvfp4_rmsnorm.argtypes = [_P, _I64, _P, _I64, _P, _INT, _F32, _I64, _I64, _P, _I64, _P, _I64, _P, _P,
                               _P, _P, _INT, _P]
_lib.nvfp4_rmsnorm_backward.argtypes = [_P, _I64, _P, _I64, _P, _I64, _P, _INT, _P, _I64, _I64, _P, _I64,
                                        _P, _P, _SZ, _P]
_lib.nvfp4_rmsnorm_backward_workspace_size.argtypes = [_I64, _I64]
_lib.nvfp4_rmsnorm_backward_workspace_size.restype = _SZ
_lib.nvfp4_route.argtypes = [_P, _INT, _I64, _P, _I64, _INT, ctypes.POINTER(RouteParams), _P, _P, _P, _P,
                             _P, _P, _SZ, _P]
_lib.nvfp4_route_backward.argtypes = [_P, _P, _INT, _I64, _P, _I64, _INT, ctypes.POINTER(RouteParams), _P,
                                      _I64, _P]
_lib.nvfp4_route_workspace_size.argtypes = [_I64, _INT]
_lib.nvfp4_route_workspace_size.restype = _SZ
_lib.nvfp4_combine.argtypes = [_P, _INT, _I64, _I64, _P, _P, _I64, _INT, _P, _P, _P, _SZ, _P]
_lib.nvfp4_combine_backward.argtypes = [_P, _P, _INT, _I64, _I64, _P, _P, _I64, _INT, _P, _P, _P, _P, _SZ,
                                        _P]
_lib.nvfp4_combine_backward_workspace_size.argtypes = [_I64]
_lib.nvfp4_combine_backward_workspace_size.restype = _SZ
_lib.nvfp4_gemv.argtypes = [_P, _I64, _I64, _P, _P, _P, _I64, _I64, _INT, _P, _I64, _P]
_lib.nvfp4_grouped_gemv.argtypes = [_INT, _P, _I64, _P, _I64, _I64, _P, _P, _P, _P, _I64, _I64, _INT, _P,
                                    _I64, _P, _SZ, _P]
_lib.nvfp4_kv_append.argtypes = [ctypes.POINTER(KVCacheView), _P, _I64, _I64, _P, _I64, _I64, _I64, _P, _I64,
                                 _I64, _I64, _P, _P, _P, _P, _I64, _INT, _INT, _P, _I64, _I64, _INT, _P, _I64,
                                 _I64, _P, _SZ, _P]
_lib.nvfp4_kv_attention.argtypes = [_P, _I64, _I64, _I64, _I64, _INT, _INT, ctypes.POINTER(KVCacheView), _P, _I64,
                                    _I64, _P, _F32, _I64, _P, _P, _P, _SZ, _P]
_lib.nvfp4_kv_attention_workspace_size.argtypes = [_I64, _INT, _INT, _INT, _INT, _I64]
_lib.nvfp4_kv_attention_workspace_size.restype = _SZ
_lib.nvfp4_expert_mlp.argtypes = [_INT, _P, _I64, _P, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64,
                                  _P, _P, _INT, _P, _P, _P, _SZ, _P]
_lib.nvfp4_expert_mlp_workspace_size.argtypes = [_I64, _I64, _I64]
_lib.nvfp4_expert_mlp_workspace_size.restype = _SZ
for _n in ("nvfp4_quantize", "nvfp4_quantize_noalloc", "mxfp8_quantize", "mxfp4_quantize",
           "nvfp4_dequantize", "nvfp4_gemm", "mxfp8_gemm", "mxfp4_gemm", "mxfp8_combine",
           "nvfp4_grouped_gemm", "nvfp4_gather_rows", "nvfp4_workspace_status",
           "nvfp4_quantize_noalloc_status", "nvfp4_gemm_cycles", "nvfp4_rmsnorm",
           "nvfp4_rmsnorm_backward", "nvfp4_route", "nvfp4_route_backward", "nvfp4_combine",
           "nvfp4_combine_backward", "nvfp4_gemv", "nvfp4_grouped_gemv", "nvfp4_kv_append",
           "nvfp4_kv_attention", "nvfp4_expert_mlp"):
    getattr(_lib, _n).restype = ctypes.c_int


class NVFP4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


def status_string(s: int) -> str:
    return _lib.nvfp4_status_string(int(s)).decode()


def _check(status: int, where: str) -> None:
    if status != NVFP4_OK:
        raise NVFP4Error(status, where)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        torch.cuda.init()  # (returns at once where it has been)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ----------------------------------------------------------------- raw C calls
def nvfp4_quantize(x, rows, cols, ld, params: QuantParams, q_row, sf_row, g_row, q_col, sf_col,
                   g_col, workspace, ws_bytes, stream=None) -> None:
    _check(_lib.nvfp4_quantize(_ptr(x), rows, cols, ld, ctypes.byref(params), _ptr(q_row),
                               _ptr(sf_row), _ptr(g_row), _ptr(q_col), _ptr(sf_col), _ptr(g_col),
                               _ptr(workspace), ws_bytes, _stream(stream)), "nvfp4_quantize")


def nvfp4_quantize_noalloc(x, rows, cols, ld, params: QuantParams, q_row, sf_row, g_row, q_col,
                           sf_col, g_col, stream=None) -> None:
    """nvfp4_quantize without a workspace, for callers that cannot allocate device
    memory; its scratch lives in an array inside the library (see include/nvfp4.h)."""
    _check(_lib.nvfp4_quantize_noalloc(_ptr(x), rows, cols, ld, ctypes.byref(params), _ptr(q_row),
                                       _ptr(sf_row), _ptr(g_row), _ptr(q_col), _ptr(sf_col),
                                       _ptr(g_col), _stream(stream)), "nvfp4_quantize_noalloc")


def mxfp8_quantize(x, rows, cols, ld, directions, rounding, seed, offset, q_row, e8_row, q_col,
                   e8_col, stream=None) -> None:
    _check(_lib.mxfp8_quantize(_ptr(x), rows, cols, ld, directions, rounding, seed, offset,
                               _ptr(q_row), _ptr(e8_row), _ptr(q_col), _ptr(e8_col),
                               _stream(stream)), "mxfp8_quantize")


def mxfp4_quantize(x, rows, cols, ld, directions, q_row, e8_row, q_col, e8_col,
                   stream=None, sf_layout=NVFP4_SF_ROWMAJOR) -> None:
    _check(_lib.mxfp4_quantize(_ptr(x), rows, cols, ld, directions, sf_layout, _ptr(q_row),
                               _ptr(e8_row), _ptr(q_col), _ptr(e8_col), _stream(stream)),
           "mxfp4_quantize")


def mxfp4_gemm(qa, sfa, qb, sfb, M, N, K, out_dtype, D, ldd, amax_out, workspace, ws_bytes,
               stream=None) -> None:
    _check(_lib.mxfp4_gemm(_ptr(qa), _ptr(sfa), _ptr(qb), _ptr(sfb), M, N, K, out_dtype, _ptr(D),
                           ldd, _ptr(amax_out), _ptr(workspace), ws_bytes, _stream(stream)),
           "mxfp4_gemm")


def nvfp4_dequantize(q, sf, g, rows, cols, sf_layout, out_dtype, out, stream=None) -> None:
    _check(_lib.nvfp4_dequantize(_ptr(q), _ptr(sf), _ptr(g), rows, cols, sf_layout, out_dtype,
                                 _ptr(out), _stream(stream)), "nvfp4_dequantize")


def nvfp4_gemm(qa, sfa, ga, qb, sfb, gb, M, N, K, out_dtype, D, ldd, amax_out, workspace,
               ws_bytes, stream=None) -> None:
    _check(_lib.nvfp4_gemm(_ptr(qa), _ptr(sfa), _ptr(ga), _ptr(qb), _ptr(sfb), _ptr(gb), M, N, K,
                           out_dtype, _ptr(D), ldd, _ptr(amax_out), _ptr(workspace), ws_bytes,
                           _stream(stream)),
           "nvfp4_gemm")


def mxfp8_gemm(qa, sfa, qb, sfb, M, N, K, out_dtype, D, ldd, amax_out, workspace, ws_bytes,
               stream=None) -> None:
    _check(_lib.mxfp8_gemm(_ptr(qa), _ptr(sfa), _ptr(qb), _ptr(sfb), M, N, K, out_dtype, _ptr(D),
                           ldd, _ptr(amax_out), _ptr(workspace), ws_bytes, _stream(stream)),
           "mxfp8_gemm")


def mxfp8_combine(q, e8, rows, cols, slot_row, weight, tokens, k, out, workspace=None,
                  ws_bytes=0, stream=None) -> None:
    _check(_lib.mxfp8_combine(_ptr(q), _ptr(e8), rows, cols, _ptr(slot_row), _ptr(weight), tokens,
                              k, _ptr(out), _ptr(workspace), ws_bytes, _stream(stream)),
           "mxfp8_combine")


def nvfp4_grouped_gemm(G, group_offsets, total_rows, qa, sfa, ga, qb, sfb, gb, N, K, out_dtype, D,
                       amax_out, workspace, ws_bytes, stream=None) -> None:
    _check(_lib.nvfp4_grouped_gemm(G, _ptr(group_offsets), total_rows, _ptr(qa), _ptr(sfa),
                                   _ptr(ga), _ptr(qb), _ptr(sfb), _ptr(gb), N, K, out_dtype,
                                   _ptr(D), _ptr(amax_out), _ptr(workspace), ws_bytes,
                                   _stream(stream)),
           "nvfp4_grouped_gemm")


def nvfp4_gather_rows(q_src, sf_src, src_rows, k, row_index, rows, group_offsets, num_groups,
                      q_dst, sf_dst, workspace, ws_bytes, stream=None) -> None:
    _check(_lib.nvfp4_gather_rows(_ptr(q_src), _ptr(sf_src), src_rows, k, _ptr(row_index), rows,
                                  _ptr(group_offsets), num_groups, _ptr(q_dst), _ptr(sf_dst),
                                  _ptr(workspace), ws_bytes, _stream(stream)),
           "nvfp4_gather_rows")


def nvfp4_rmsnorm(x, ldx, residual, ldr, weight, weight_dtype, eps, rows, cols, h, ldh, y, ldy, rstd,
                  amax_out, mx_q, mx_sf, mx_sf_layout, stream=None) -> None:
    _check(_lib.nvfp4_rmsnorm(_ptr(x), ldx, _ptr(residual), ldr, _ptr(weight), weight_dtype, eps, rows, cols,
                              _ptr(h), ldh, _ptr(y), ldy, _ptr(rstd), _ptr(amax_out), _ptr(mx_q),
                              _ptr(mx_sf), mx_sf_layout, _stream(stream)), "nvfp4_rmsnorm")


def nvfp4_rmsnorm_backward(dy, lddy, h, ldh, dh, lddh, weight, weight_dtype, rstd, rows, cols, dx, lddx,
                           dweight, workspace, ws_bytes, stream=None) -> None:
    _check(_lib.nvfp4_rmsnorm_backward(_ptr(dy), lddy, _ptr(h), ldh, _ptr(dh), lddh, _ptr(weight),
                                       weight_dtype, _ptr(rstd), rows, cols, _ptr(dx), lddx, _ptr(dweight),
                                       _ptr(workspace), ws_bytes, _stream(stream)),
           "nvfp4_rmsnorm_backward")


def nvfp4_route(logits, logits_dtype, ld, bias, tokens, experts, params: RouteParams, expert, weight,
                group_offsets, row_index, slot_row, workspace, ws_bytes, stream=None) -> None:
    _check(_lib.nvfp4_route(_ptr(logits), logits_dtype, ld, _ptr(bias), tokens, experts,
                            ctypes.byref(params), _ptr(expert), _ptr(weight), _ptr(group_offsets),
                            _ptr(row_index), _ptr(slot_row), _ptr(workspace), ws_bytes, _stream(stream)),
           "nvfp4_route")


def nvfp4_route_backward(dweight, logits, logits_dtype, ld, expert, tokens, experts, params: RouteParams,
                         dlogits, ldd, stream=None) -> None:
    _check(_lib.nvfp4_route_backward(_ptr(dweight), _ptr(logits), logits_dtype, ld, _ptr(expert), tokens,
                                     experts, ctypes.byref(params), _ptr(dlogits), ldd, _stream(stream)),
           "nvfp4_route_backward")


def nvfp4_combine(rows, rows_dtype, n_rows, cols, slot_row, weight, tokens, k, base, out, workspace=None,
                  ws_bytes=0, stream=None) -> None:
    _check(_lib.nvfp4_combine(_ptr(rows), rows_dtype, n_rows, cols, _ptr(slot_row), _ptr(weight), tokens, k,
                              _ptr(base), _ptr(out), _ptr(workspace), ws_bytes, _stream(stream)),
           "nvfp4_combine")


def nvfp4_combine_backward(dout, rows, rows_dtype, n_rows, cols, slot_row, weight, tokens, k, used_rows,
                           drows, dweight, workspace=None, ws_bytes=0, stream=None) -> None:
    _check(_lib.nvfp4_combine_backward(_ptr(dout), _ptr(rows), rows_dtype, n_rows, cols, _ptr(slot_row),
                                       _ptr(weight), tokens, k, _ptr(used_rows), _ptr(drows), _ptr(dweight),
                                       _ptr(workspace), ws_bytes, _stream(stream)),
           "nvfp4_combine_backward")


def nvfp4_expert_mlp(G, group_offsets, total_rows, x, ldx, tokens, row_index, gate_q, gate_sf, gate_g, up_q, up_sf,
                     up_g, down_q, down_sf, down_g, hidden, ffn, slot_row, weight, k, base, out, workspace, ws_bytes,
                     stream=None) -> None:
    _check(_lib.nvfp4_expert_mlp(G, _ptr(group_offsets), total_rows, _ptr(x), ldx, tokens, _ptr(row_index),
                                 _ptr(gate_q), _ptr(gate_sf), _ptr(gate_g), _ptr(up_q), _ptr(up_sf), _ptr(up_g),
                                 _ptr(down_q), _ptr(down_sf), _ptr(down_g), hidden, ffn, _ptr(slot_row), _ptr(weight),
                                 k, _ptr(base), _ptr(out), _ptr(workspace), ws_bytes, _stream(stream)),
           "nvfp4_expert_mlp")


def nvfp4_expert_mlp_workspace_size(total_rows: int, hidden: int, ffn: int) -> int:
    return _lib.nvfp4_expert_mlp_workspace_size(total_rows, hidden, ffn)


def nvfp4_kv_append(cache: KVCacheView, k, ldk, hsk, v, ldv, hsv, tokens, table, ldt, sequences, table_pages,
                    position, sequence, cos, sin, angles, rot, neighbours, q, ldq, hsq, heads, q_out, ldo, hso,
                    workspace=None, ws_bytes=0, stream=None) -> None:
    _check(_lib.nvfp4_kv_append(ctypes.byref(cache), _ptr(k), ldk, hsk, _ptr(v), ldv, hsv, tokens, _ptr(table), ldt,
                                sequences, table_pages, _ptr(position), _ptr(sequence), _ptr(cos), _ptr(sin), angles,
                                rot, neighbours, _ptr(q), ldq, hsq, heads, _ptr(q_out), ldo, hso, _ptr(workspace),
                                ws_bytes, _stream(stream)), "nvfp4_kv_append")


def nvfp4_kv_attention(q, ldb, ldi, ldh, sequences, queries, heads, cache: KVCacheView, table, ldt, table_pages,
                       lengths, scale, window, out, lse, workspace, ws_bytes, stream=None) -> None:
    _check(_lib.nvfp4_kv_attention(_ptr(q), ldb, ldi, ldh, sequences, queries, heads, ctypes.byref(cache),
                                   _ptr(table), ldt, table_pages, _ptr(lengths), scale, window, _ptr(out), _ptr(lse),
                                   _ptr(workspace), ws_bytes, _stream(stream)), "nvfp4_kv_attention")


def nvfp4_kv_attention_workspace_size(sequences: int, queries: int, heads: int, kv_heads: int, dim: int,
                                      capacity: int) -> int:
    return _lib.nvfp4_kv_attention_workspace_size(sequences, queries, heads, kv_heads, dim, capacity)


def nvfp4_gemv(x, ldx, rows, q, sf, g, N, K, out_dtype, D, ldd, stream=None) -> None:
    _check(_lib.nvfp4_gemv(_ptr(x), ldx, rows, _ptr(q), _ptr(sf), _ptr(g), N, K, out_dtype, _ptr(D), ldd,
                           _stream(stream)), "nvfp4_gemv")


def nvfp4_grouped_gemv(G, group_offsets, total_rows, x, ldx, src_rows, row_index, q, sf, g, N, K, out_dtype,
                       D, ldd, workspace=None, ws_bytes=0, stream=None) -> None:
    _check(_lib.nvfp4_grouped_gemv(G, _ptr(group_offsets), total_rows, _ptr(x), ldx, src_rows,
                                   _ptr(row_index), _ptr(q), _ptr(sf), _ptr(g), N, K, out_dtype, _ptr(D),
                                   ldd, _ptr(workspace), ws_bytes, _stream(stream)),
           "nvfp4_grouped_gemv")


@functools.lru_cache(maxsize=1024)
def nvfp4_rmsnorm_backward_workspace_size(rows: int, cols: int) -> int:
    return int(_lib.nvfp4_rmsnorm_backward_workspace_size(rows, cols))


@functools.lru_cache(maxsize=1024)
def nvfp4_route_workspace_size(tokens: int, experts: int) -> int:
    return int(_lib.nvfp4_route_workspace_size(tokens, experts))


def nvfp4_combine_backward_workspace_size(n_rows: int) -> int:
    return int(_lib.nvfp4_combine_backward_workspace_size(n_rows))


def nvfp4_workspace_status(workspace, stream=None) -> int:
    return int(_lib.nvfp4_workspace_status(_ptr(workspace), _stream(stream)))


def nvfp4_gemm_cycles(workspace, stream=None) -> int:
    """SM cycles (entry to exit) of the longest CTA of the last GEMM call on
    `workspace`; synchronises the stream."""
    v = ctypes.c_uint64(0)
    _check(_lib.nvfp4_gemm_cycles(_ptr(workspace), _stream(stream), ctypes.byref(v)),
           "nvfp4_gemm_cycles")
    return int(v.value)


def nvfp4_quantize_noalloc_status(stream=None) -> int:
    return int(_lib.nvfp4_quantize_noalloc_status(_stream(stream)))


def nvfp4_sf_mma_bytes(rows: int, k: int) -> int:
    return int(_lib.nvfp4_sf_mma_bytes(rows, k))


def mxfp8_sf_mma_bytes(rows: int, k: int) -> int:
    return int(_lib.mxfp8_sf_mma_bytes(rows, k))


def nvfp4_sf_mma_grouped_bytes(total_rows: int, num_groups: int, k: int) -> int:
    return int(_lib.nvfp4_sf_mma_grouped_bytes(total_rows, num_groups, k))


def nvfp4_quantize_workspace_size(rows: int = 0, cols: int = 0) -> int:
    return int(_lib.nvfp4_quantize_workspace_size(rows, cols, None))


def nvfp4_gemm_workspace_size(M: int = 0, N: int = 0, K: int = 0) -> int:
    return int(_lib.nvfp4_gemm_workspace_size(M, N, K))


def nvfp4_version() -> int:
    return int(_lib.nvfp4_version())


# ----------------------------------------------------------------- convenience wrappers
@dataclass
class NVFP4Tensor:
    """Codes [rows, k/2] u8, scale bytes (row-major [rows, k/16] or tiled bytes), g [1] f32."""
    q: object
    sf: object
    g: object
    rows: int
    k: int
    sf_layout: int


def _workspace(device, nbytes: int = 256):
    import torch
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def quantize(x, *, rowwise: bool = True, colwise: bool = False, rounding: int = NVFP4_RNE,
             scaling: int = NVFP4_1D16, rht: bool = False, sf_layout: int = NVFP4_SF_ROWMAJOR,
             seed: int = 0, offset: int = 0, amax=None, mx_outputs: int = 0,
             mx_rounding: int = NVFP4_RNE, mx_sf_layout: int = NVFP4_SF_ROWMAJOR,
             row_index=None, src_rows: int = 0, group_offsets=None, num_groups: int = 0,
             rows: Optional[int] = None, workspace=None, stream=None):
    """Quantise a bf16 [rows, cols] CUDA tensor.  Returns dict with 'row', 'col'
    (NVFP4Tensor or None), 'mx_row', 'mx_col' ((codes, e8m0) or None)."""
    import torch
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.is_cuda
    cols = x.shape[1]
    ld = x.stride(0)
    assert x.stride(1) == 1
    n_rows = rows if rows is not None else x.shape[0]
    dev = x.device
    u8 = dict(dtype=torch.uint8, device=dev)

    def sf_alloc(r, k, grouped=False):
        if sf_layout == NVFP4_SF_MMA:
            n = (nvfp4_sf_mma_grouped_bytes(r, num_groups, k) if grouped
                 else nvfp4_sf_mma_bytes(r, k))
            return torch.zeros(n, **u8)
        return torch.empty((r, k // 16), **u8)

    out = {"row": None, "col": None, "mx_row": None, "mx_col": None}
    q_row = sf_row = g_row = q_col = sf_col = g_col = None
    if rowwise:
        q_row = torch.empty((n_rows, cols // 2), **u8)
        sf_row = sf_alloc(n_rows, cols, grouped=group_offsets is not None)
        g_row = torch.empty(1, dtype=torch.float32, device=dev)
        out["row"] = NVFP4Tensor(q_row, sf_row, g_row, n_rows, cols, sf_layout)
    if colwise:
        q_col = torch.empty((cols, n_rows // 2), **u8)
        sf_col = sf_alloc(cols, n_rows)
        g_col = torch.empty(1, dtype=torch.float32, device=dev)
        out["col"] = NVFP4Tensor(q_col, sf_col, g_col, cols, n_rows, sf_layout)
    p = QuantParams()
    p.rounding, p.scaling = rounding, scaling
    p.outputs = (NVFP4_ROWWISE if rowwise else 0) | (NVFP4_COLWISE if colwise else 0)
    p.rht_colwise = 1 if rht else 0
    p.sf_layout = sf_layout
    p.seed, p.offset = seed, offset
    p.amax_in = _ptr(amax)
    p.row_index = _ptr(row_index)
    p.src_rows = src_rows if row_index is not None else 0
    p.group_offsets = _ptr(group_offsets)
    p.num_groups = num_groups
    p.mx_outputs, p.mx_rounding, p.mx_sf_layout = mx_outputs, mx_rounding, mx_sf_layout

    def mx_sf_alloc(r, k):
        if mx_sf_layout == NVFP4_SF_MMA:
            return torch.zeros(mxfp8_sf_mma_bytes(r, k), **u8)
        return torch.empty((r, k // 32), **u8)

    if mx_outputs & NVFP4_ROWWISE:
        mq, me = torch.empty((n_rows, cols), **u8), mx_sf_alloc(n_rows, cols)
        p.mx_q_row, p.mx_sf_row = mq.data_ptr(), me.data_ptr()
        out["mx_row"] = (mq, me)
    if mx_outputs & NVFP4_COLWISE:
        mq, me = torch.empty((cols, n_rows), **u8), mx_sf_alloc(cols, n_rows)
        p.mx_q_col, p.mx_sf_col = mq.data_ptr(), me.data_ptr()
        out["mx_col"] = (mq, me)
    ws = workspace if workspace is not None else _workspace(dev)
    nvfp4_quantize(x, n_rows, cols, ld, p, q_row, sf_row, g_row, q_col, sf_col, g_col,
                   *_scratch("quantize", ws), stream)
    out["workspace"] = ws
    return out


def mxfp8(x, directions: int = NVFP4_COLWISE, rounding: int = NVFP4_RNE, seed: int = 0,
          offset: int = 0, stream=None):
    import torch
    rows, cols = x.shape
    u8 = dict(dtype=torch.uint8, device=x.device)
    qr = er = qc = ec = None
    if directions & NVFP4_ROWWISE:
        qr, er = torch.empty((rows, cols), **u8), torch.empty((rows, cols // 32), **u8)
    if directions & NVFP4_COLWISE:
        qc, ec = torch.empty((cols, rows), **u8), torch.empty((cols, rows // 32), **u8)
    mxfp8_quantize(x, rows, cols, x.stride(0), directions, rounding, seed, offset, qr, er, qc, ec,
                   stream)
    return (qr, er), (qc, ec)


def mxfp4(x, directions: int = NVFP4_ROWWISE | NVFP4_COLWISE, stream=None,
          sf_layout: int = NVFP4_SF_ROWMAJOR):
    """MXFP4 codes and E8M0 scales of a bf16 [rows, cols] tensor:
    ((q_row [rows, cols/2], e8 [rows, cols/32]) or (None, None),
     (q_col [cols, rows/2], e8 [cols, rows/32]) or (None, None)); with
    sf_layout = NVFP4_SF_MMA the scales are flat tiled buffers (mxfp4_gemm's layout)."""
    import torch
    rows, cols = x.shape
    u8 = dict(dtype=torch.uint8, device=x.device)

    def e8(r, k):
        if sf_layout == NVFP4_SF_MMA:
            return torch.zeros(mxfp8_sf_mma_bytes(r, k), **u8)
        return torch.empty((r, k // 32), **u8)

    qr = er = qc = ec = None
    if directions & NVFP4_ROWWISE:
        qr, er = torch.empty((rows, cols // 2), **u8), e8(rows, cols)
    if directions & NVFP4_COLWISE:
        qc, ec = torch.empty((cols, rows // 2), **u8), e8(cols, rows)
    mxfp4_quantize(x, rows, cols, x.stride(0), directions, qr, er, qc, ec, stream, sf_layout)
    return (qr, er), (qc, ec)


def mx4_gemm(qa, sfa, qb, sfb, out_dtype: int = NVFP4_OUT_BF16, out=None, amax_out=None,
             workspace=None, stream=None):
    """D = A_hat B_hat^T of MXFP4 operands: qa [M, K/2], qb [N, K/2] codes with E8M0 scales
    in the tiled layout (mxfp4(..., sf_layout=NVFP4_SF_MMA))."""
    import torch
    M, K = qa.shape[0], qa.shape[1] * 2
    N = qb.shape[0]
    dt = torch.bfloat16 if out_dtype == NVFP4_OUT_BF16 else torch.float32
    D = out if out is not None else torch.empty((M, N), dtype=dt, device=qa.device)
    ws = workspace if workspace is not None else _workspace(qa.device)
    mxfp4_gemm(qa, sfa, qb, sfb, M, N, K, out_dtype, D, D.stride(0), amax_out, *_scratch("mx4_gemm", ws),
               stream)
    return D


def dequantize(t: NVFP4Tensor, out_dtype: int = NVFP4_OUT_F32, stream=None):
    dt = torch.float32 if out_dtype == NVFP4_OUT_F32 else torch.bfloat16
    q = t.q
    out = _matrix(q.device, dt, t.rows, t.k)
    _check(_lib.nvfp4_dequantize(q.data_ptr(), _ptr(t.sf), _ptr(t.g), t.rows, t.k, t.sf_layout, out_dtype,
                                 out.data_ptr(), _stream(stream)), "nvfp4_dequantize")
    return out


def gemm(a: NVFP4Tensor, b: NVFP4Tensor, out_dtype: int = NVFP4_OUT_BF16, out=None,
         amax_out=None, workspace=None, stream=None):
    """D = A B^T for NVFP4 operands A [M, K] and B [N, K] (tiled scale layout).
    ``amax_out`` (optional device f32 [1]) receives max |D| as stored."""
    import torch
    assert a.k == b.k and a.sf_layout == NVFP4_SF_MMA and b.sf_layout == NVFP4_SF_MMA
    M, N, K = a.rows, b.rows, a.k
    dt = torch.float32 if out_dtype == NVFP4_OUT_F32 else torch.bfloat16
    if out is None:
        out = torch.empty((M, N), dtype=dt, device=a.q.device)
    ws = workspace if workspace is not None else _workspace(a.q.device)
    nvfp4_gemm(a.q, a.sf, a.g, b.q, b.sf, b.g, M, N, K, out_dtype, out, out.stride(0), amax_out,
               *_scratch("gemm", ws), stream)
    return out


def mx_gemm(qa, sfa, qb, sfb, out_dtype: int = NVFP4_OUT_BF16, out=None, amax_out=None,
            workspace=None, stream=None):
    """D = A_hat B_hat^T of MXFP8 operands: qa [M, K], qb [N, K] E4M3 codes with E8M0
    scales in the tiled layout (quantize(..., mx_sf_layout=NVFP4_SF_MMA))."""
    import torch
    M, K = qa.shape
    N = qb.shape[0]
    dt = torch.bfloat16 if out_dtype == NVFP4_OUT_BF16 else torch.float32
    D = out if out is not None else torch.empty((M, N), dtype=dt, device=qa.device)
    ws = workspace if workspace is not None else _workspace(qa.device)
    mxfp8_gemm(qa, sfa, qb, sfb, M, N, K, out_dtype, D, D.stride(0), amax_out, *_scratch("mx_gemm", ws),
               stream)
    return D


def grouped_gemm(group_offsets, a: NVFP4Tensor, qb, sfb, gb, N: int, out_dtype: int = NVFP4_OUT_BF16,
                 out=None, amax_out=None, workspace=None, stream=None):
    """MoE grouped D = A_e B_e^T; qb [G, N, K/2], sfb tiled per expert, gb [G]."""
    import torch
    G = group_offsets.numel() - 1
    dt = torch.float32 if out_dtype == NVFP4_OUT_F32 else torch.bfloat16
    if out is None:
        out = torch.empty((a.rows, N), dtype=dt, device=a.q.device)
    ws = workspace if workspace is not None else _workspace(a.q.device)
    nvfp4_grouped_gemm(G, group_offsets, a.rows, a.q, a.sf, a.g, qb, sfb, gb, N, a.k, out_dtype,
                       out, amax_out, *_scratch("grouped_gemm", ws), stream)
    return out


def gather_rows(t: NVFP4Tensor, row_index, group_offsets=None, workspace=None, stream=None):
    """MoE dispatch of an already quantised operand: row i of the result is row
    ``row_index[i]`` of ``t`` (codes and tiled scales), laid out per expert
    group when ``group_offsets`` (device int32 [G+1]) is given."""
    import torch
    assert t.sf_layout == NVFP4_SF_MMA
    rows = row_index.numel()
    G = 0 if group_offsets is None else group_offsets.numel() - 1
    u8 = dict(dtype=torch.uint8, device=t.q.device)
    q = torch.empty((rows, t.k // 2), **u8)
    n = nvfp4_sf_mma_grouped_bytes(rows, G, t.k) if G else nvfp4_sf_mma_bytes(rows, t.k)
    sf = torch.zeros(n, **u8)
    ws = workspace if workspace is not None else _workspace(t.q.device)
    nvfp4_gather_rows(t.q, t.sf, t.rows, t.k, row_index, rows, group_offsets, G, q, sf,
                      *_scratch("gather_rows", ws), stream)
    return NVFP4Tensor(q, sf, t.g, rows, t.k, NVFP4_SF_MMA)


# ------------------------------------------------- the MoE block around the experts' products
@dataclass
class Routing:
    """What ``route`` gives: the experts and weights of each token's slots, and the order of the
    routed rows that ``gather_rows``, ``grouped_gemm``, ``grouped_gemv`` and ``combine`` read."""
    expert: object         # int32 [tokens, top_k], -1 = no expert
    weight: object         # f32 [tokens, top_k]
    group_offsets: object  # int32 [experts + 1]
    row_index: object      # int32 [tokens * top_k]: the token of each routed row
    slot_row: object       # int32 [tokens, top_k]: the row of each slot, -1 = none
    params: RouteParams


# The calls below serve single tokens too, where the kernel takes a few microseconds: their checks read
# each property once, and they hand addresses to the library without further wrapping.
def _need(ok, message: str) -> None:
    if not ok:
        raise ValueError(message)


def _one_device(name: str, *tensors):
    """The device of the tensors: one CUDA device, the current one (the calls launch there)."""
    first = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != first:
            raise ValueError(f"{name}: tensors on {tensors[0].device} and {t.device}")
    if first < 0:
        raise ValueError(f"{name}: CUDA tensors expected, got {tensors[0].device}")
    current = torch._C._cuda_getDevice()
    if first != current:
        raise ValueError(f"{name}: tensors on cuda:{first}, but the current device is cuda:{current}")
    return tensors[0].device


def _raw_stream(dev) -> int:
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _matrix(dev, dtype, rows: int, cols: int):
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=dev)


def _dtype_code(name: str, t) -> int:
    dt = t.dtype
    if dt is torch.bfloat16:
        return NVFP4_OUT_BF16
    if dt is torch.float32:
        return NVFP4_OUT_F32
    raise ValueError(f"{name} must be bfloat16 or float32, got {dt}")


def _rows_of(name: str, t, rows=None, cols=None):
    """A bf16 matrix with contiguous rows; returns its row stride in elements."""
    shape = t.shape
    if t.dtype is not torch.bfloat16 or len(shape) != 2:
        raise ValueError(f"{name} must be a bfloat16 matrix, got {t.dtype} {tuple(shape)}")
    n, c = shape
    if (rows is not None and n != rows) or (cols is not None and c != cols):
        raise ValueError(f"{name}: [{rows}, {cols}] expected, got {tuple(shape)}")
    if t.is_contiguous():  # (the stride of a single row is never used, and torch leaves it arbitrary)
        return c
    if c > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: rows must be contiguous")
    return t.stride(0) if n > 1 else c


def _flat(name: str, t, dtype, *shape) -> None:
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous {dtype} {shape} expected, got {t.dtype} {tuple(t.shape)}")


def _bytes(name: str, t, least: int) -> None:
    if t.element_size() != 1 or not t.is_contiguous() or t.numel() < least:
        raise ValueError(f"{name}: at least {least} contiguous bytes expected, got {t.dtype} {tuple(t.shape)}")


def _scratch(name: str, workspace):
    """Address and bytes of a caller's workspace (an expanded one has fewer than its elements say)."""
    if not workspace.is_contiguous():
        raise ValueError(f"{name}: contiguous workspace expected, got strides {workspace.stride()}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _on(stream):
    if isinstance(stream, int):  # (ExternalStream(0) would be a new stream, not the default one)
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def rmsnorm(x, weight, residual=None, eps: float = 1e-6, *, y: bool = True, mx: bool = False,
            mx_sf_layout: int = NVFP4_SF_ROWMAJOR, amax: bool = False, rstd: bool = False, stream=None):
    """Root-mean-square norm of x + residual (bf16 [rows, cols]) times weight (bf16 or f32 [cols]).

    Returns a dict: 'h' the sum in bf16 (x itself without a residual), 'y' the norm in bf16, 'mx' its MXFP8
    (codes, e8m0) for ``mx_gemm``, 'amax' max |y| ([1], for ``quantize``'s amax), 'rstd' [rows] for
    ``rmsnorm_backward``; None for what was not asked for.  With ``stream`` the outputs belong to it."""
    if stream is not None:
        with _on(stream):
            return rmsnorm(x, weight, residual, eps, y=y, mx=mx, mx_sf_layout=mx_sf_layout, amax=amax,
                           rstd=rstd)
    dev = _one_device("rmsnorm", x, weight, residual)
    ldx = _rows_of("rmsnorm: x", x)
    rows, cols = x.shape
    wdt = _dtype_code("rmsnorm: weight", weight)
    _flat("rmsnorm: weight", weight, weight.dtype, cols)
    if not y:
        _need(mx, "rmsnorm: neither y nor mx asked for")
        _need(not amax, "rmsnorm: amax is that of y")
    out = {"h": x, "y": None, "mx": None, "amax": None, "rstd": None}
    res = h = yp = mq = ms = ap = rp = None
    ldr = 0
    if residual is not None:
        ldr = _rows_of("rmsnorm: residual", residual, rows, cols)
        res = residual.data_ptr()
        out["h"] = _matrix(dev, torch.bfloat16, rows, cols)
        h = out["h"].data_ptr()
    if y:
        out["y"] = _matrix(dev, torch.bfloat16, rows, cols)
        yp = out["y"].data_ptr()
    if mx:
        q = _matrix(dev, torch.uint8, rows, cols)
        s = (torch.empty(mxfp8_sf_mma_bytes(rows, cols), dtype=torch.uint8, device=dev)
             if mx_sf_layout == NVFP4_SF_MMA else _matrix(dev, torch.uint8, rows, cols // 32))
        out["mx"] = (q, s)
        mq, ms = q.data_ptr(), s.data_ptr()
    if amax:
        out["amax"] = torch.empty(1, dtype=torch.float32, device=dev)
        ap = out["amax"].data_ptr()
    if rstd:
        out["rstd"] = torch.empty(rows, dtype=torch.float32, device=dev)
        rp = out["rstd"].data_ptr()
    _check(_lib.nvfp4_rmsnorm(x.data_ptr(), ldx, res, ldr, weight.data_ptr(), wdt, eps, rows, cols, h, cols,
                              yp, cols, rp, ap, mq, ms, mx_sf_layout, _raw_stream(dev)), "nvfp4_rmsnorm")
    return out


def rmsnorm_backward(dy, h, weight, rstd, dh=None, *, dweight: bool = True, workspace=None, stream=None):
    """(dx, dweight) of ``rmsnorm`` from the gradients of its y and (dh, optional) of its h.  dx is the
    gradient of x and of residual; dweight (in weight's dtype) is None where not asked for."""
    if stream is not None:
        with _on(stream):
            return rmsnorm_backward(dy, h, weight, rstd, dh, dweight=dweight, workspace=workspace)
    dev = _one_device("rmsnorm_backward", dy, h, weight, rstd, dh, workspace)
    ldy = _rows_of("rmsnorm_backward: dy", dy)
    rows, cols = dy.shape
    ldh = _rows_of("rmsnorm_backward: h", h, rows, cols)
    lddh = _rows_of("rmsnorm_backward: dh", dh, rows, cols) if dh is not None else 0
    wdt = _dtype_code("rmsnorm_backward: weight", weight)
    _flat("rmsnorm_backward: weight", weight, weight.dtype, cols)
    _flat("rmsnorm_backward: rstd", rstd, torch.float32, rows)
    dx = _matrix(dev, torch.bfloat16, rows, cols)
    dw = wp = dwp = None
    nb = 0
    if dweight:
        dw = torch.empty_like(weight)
        if workspace is None:
            nb = nvfp4_rmsnorm_backward_workspace_size(rows, cols)
            workspace = torch.empty(nb, dtype=torch.uint8, device=dev)
            wp = workspace.data_ptr()
        else:
            wp, nb = _scratch("rmsnorm_backward", workspace)
        dwp = dw.data_ptr()
    _check(_lib.nvfp4_rmsnorm_backward(dy.data_ptr(), ldy, h.data_ptr(), ldh,
                                       dh.data_ptr() if dh is not None else None, lddh, weight.data_ptr(), wdt,
                                       rstd.data_ptr(), rows, cols, dx.data_ptr(), cols, dwp, wp, nb,
                                       _raw_stream(dev)), "nvfp4_rmsnorm_backward")
    return dx, dw


def _logits_of(name: str, logits):
    dt = _dtype_code(f"{name}: logits", logits)
    shape = logits.shape
    _need(len(shape) == 2, f"{name}: logits [tokens, experts] expected")
    if logits.is_contiguous():
        return dt, shape[1]
    _need(shape[1] <= 1 or logits.stride(1) == 1, f"{name}: rows of logits must be contiguous")
    return dt, logits.stride(0) if shape[0] > 1 else shape[1]


def route(logits, top_k: int, *, score: int = NVFP4_SOFTMAX, bias=None, groups: int = 1,
          topk_groups: Optional[int] = None, group_top: int = 2, renormalize: bool = True,
          scale: float = 1.0, workspace=None, stream=None) -> Routing:
    """Experts and weights of each token (logits [tokens, experts], bf16 or f32), and the order of the routed
    rows.  bias (f32 [experts]) steers the choice only; ``topk_groups`` of ``groups`` expert groups, ranked by
    the sum of their ``group_top`` best scores, may be chosen from.  Logits at or below bf16's lowest finite
    value mask their experts; slots without an expert have expert -1, weight 0 and row -1."""
    if stream is not None:
        with _on(stream):
            return route(logits, top_k, score=score, bias=bias, groups=groups, topk_groups=topk_groups,
                         group_top=group_top, renormalize=renormalize, scale=scale, workspace=workspace)
    dev = _one_device("route", logits, bias, workspace)
    dt, ld = _logits_of("route", logits)
    tokens, experts = logits.shape
    if bias is not None:
        _flat("route: bias", bias, torch.float32, experts)
    _need(top_k >= 1, "route: top_k must be at least 1")
    p = RouteParams(top_k, score, groups, groups if topk_groups is None else topk_groups, group_top,
                    1 if renormalize else 0, scale)
    i32 = torch.int32
    r = Routing(_matrix(dev, i32, tokens, top_k), _matrix(dev, torch.float32, tokens, top_k),
                torch.empty(experts + 1, dtype=i32, device=dev),
                torch.empty(tokens * top_k, dtype=i32, device=dev), _matrix(dev, i32, tokens, top_k), p)
    wp = None
    if workspace is not None:
        wp, n = _scratch("route", workspace)
    else:
        n = nvfp4_route_workspace_size(tokens, experts)
        if n > 256:
            workspace = torch.empty(n, dtype=torch.uint8, device=dev)
            wp = workspace.data_ptr()
    _check(_lib.nvfp4_route(logits.data_ptr(), dt, ld, bias.data_ptr() if bias is not None else None, tokens,
                            experts, ctypes.byref(p), r.expert.data_ptr(), r.weight.data_ptr(),
                            r.group_offsets.data_ptr(), r.row_index.data_ptr(), r.slot_row.data_ptr(), wp, n,
                            _raw_stream(dev)), "nvfp4_route")
    return r


def route_backward(dweight, logits, routing: Routing, *, stream=None):
    """The logits' gradient (their dtype) from that of ``routing.weight`` (f32 [tokens, top_k])."""
    if stream is not None:
        with _on(stream):
            return route_backward(dweight, logits, routing)
    dev = _one_device("route_backward", dweight, logits, routing.expert)
    dt, ld = _logits_of("route_backward", logits)
    tokens, experts = logits.shape
    k = routing.params.top_k
    _flat("route_backward: dweight", dweight, torch.float32, tokens, k)
    _flat("route_backward: expert", routing.expert, torch.int32, tokens, k)
    d = _matrix(dev, logits.dtype, tokens, experts)
    _check(_lib.nvfp4_route_backward(dweight.data_ptr(), logits.data_ptr(), dt, ld, routing.expert.data_ptr(),
                                     tokens, experts, ctypes.byref(routing.params), d.data_ptr(), experts,
                                     _raw_stream(dev)), "nvfp4_route_backward")
    return d


def _combine_args(name: str, rows, slot_row, weight):
    dt = _dtype_code(f"{name}: rows", rows)
    shape, slots = rows.shape, slot_row.shape
    _need(len(shape) == 2 and rows.is_contiguous(), f"{name}: contiguous rows [n, cols] expected")
    _need(len(slots) == 2, f"{name}: slot_row [tokens, k] expected")
    _flat(f"{name}: slot_row", slot_row, torch.int32, *slots)
    _flat(f"{name}: weight", weight, torch.float32, *slots)
    return dt, shape[0], shape[1], slots[0], slots[1]


def combine(rows, slot_row, weight, base=None, *, workspace=None, stream=None):
    """out[t] = base[t] + sum_j weight[t, j] * rows[slot_row[t, j]], bf16 [tokens, cols]; rows bf16 or f32,
    slots with a negative row left out.  ``workspace`` (256 bytes, optional) receives the status word."""
    if stream is not None:
        with _on(stream):
            return combine(rows, slot_row, weight, base, workspace=workspace)
    dev = _one_device("combine", rows, slot_row, weight, base, workspace)
    dt, n, cols, tokens, k = _combine_args("combine", rows, slot_row, weight)
    bp = wp = None
    if base is not None:
        _flat("combine: base", base, torch.bfloat16, tokens, cols)
        bp = base.data_ptr()
    nb = 0
    if workspace is not None:
        wp, nb = _scratch("combine", workspace)
    out = _matrix(dev, torch.bfloat16, tokens, cols)
    _check(_lib.nvfp4_combine(rows.data_ptr(), dt, n, cols, slot_row.data_ptr(), weight.data_ptr(), tokens, k,
                              bp, out.data_ptr(), wp, nb, _raw_stream(dev)), "nvfp4_combine")
    return out


def combine_backward(dout, rows, slot_row, weight, group_offsets=None, *, workspace=None, stream=None):
    """(drows, dweight) of ``combine`` (the base's gradient is dout).  Rows that no slot names get a zero gradient;
    with the routing's ``group_offsets``, whose last rows few are, without a pass over all of them.  Each row
    belongs to one slot at most, as a routing's do; a ``workspace`` of
    ``nvfp4_combine_backward_workspace_size(n)`` bytes has that checked and receives the status word."""
    if stream is not None:
        with _on(stream):
            return combine_backward(dout, rows, slot_row, weight, group_offsets, workspace=workspace)
    dev = _one_device("combine_backward", dout, rows, slot_row, weight, group_offsets, workspace)
    dt, n, cols, tokens, k = _combine_args("combine_backward", rows, slot_row, weight)
    _flat("combine_backward: dout", dout, torch.bfloat16, tokens, cols)
    used = None
    if group_offsets is not None:
        _need(group_offsets.dim() == 1 and group_offsets.numel() >= 2,
              "combine_backward: group_offsets [groups + 1] expected")
        _flat("combine_backward: group_offsets", group_offsets, torch.int32, group_offsets.numel())
        used = group_offsets.data_ptr() + 4 * (group_offsets.numel() - 1)
    drows = torch.empty_like(rows) if used is not None else torch.zeros_like(rows)
    dweight = _matrix(dev, torch.float32, tokens, k)
    wp, nb = None, 0
    if workspace is not None:
        wp, nb = _scratch("combine_backward", workspace)
    _check(_lib.nvfp4_combine_backward(dout.data_ptr(), rows.data_ptr(), dt, n, cols, slot_row.data_ptr(),
                                       weight.data_ptr(), tokens, k, used, drows.data_ptr(), dweight.data_ptr(),
                                       wp, nb, _raw_stream(dev)), "nvfp4_combine_backward")
    return drows, dweight


def _gemv_out(name: str, out_dtype: int, rows: int, N: int, out, dev):
    dt = torch.float32 if out_dtype == NVFP4_OUT_F32 else torch.bfloat16
    if out is None:
        return _matrix(dev, dt, rows, N), N
    _need(out.dtype is dt and out.shape == (rows, N) and (N <= 1 or out.stride(1) == 1),
          f"{name}: out {dt} [{rows}, {N}] with contiguous rows expected")
    _need(rows <= 1 or out.stride(0) >= N, f"{name}: rows of out overlap")
    return out, out.stride(0) if rows > 1 else N


def gemv(x, w: NVFP4Tensor, out_dtype: int = NVFP4_OUT_BF16, out=None, *, stream=None):
    """D = x W^T of a few bf16 rows x [rows, K] and an NVFP4 matrix [N, K] (tiled scales): ``gemm`` for
    single tokens, x not quantised."""
    if stream is not None:
        with _on(stream):
            return gemv(x, w, out_dtype, out)
    q, sf, g, N, K = w.q, w.sf, w.g, w.rows, w.k
    dev = _one_device("gemv", x, q, sf, g, out)
    ldx = _rows_of("gemv: x", x, None, K)
    rows = x.shape[0]
    _need(w.sf_layout == NVFP4_SF_MMA, "gemv: w must have tiled scales (NVFP4_SF_MMA)")
    _flat("gemv: w.q", q, torch.uint8, N, K // 2)
    _need(g.dtype is torch.float32 and g.numel() == 1, "gemv: w.g must be one float32 number")
    _bytes("gemv: w.sf", sf, nvfp4_sf_mma_bytes(N, K))
    out, ldd = _gemv_out("gemv", out_dtype, rows, N, out, dev)
    _check(_lib.nvfp4_gemv(x.data_ptr(), ldx, rows, q.data_ptr(), sf.data_ptr(), g.data_ptr(), N, K, out_dtype,
                           out.data_ptr(), ldd, _raw_stream(dev)), "nvfp4_gemv")
    return out


def grouped_gemv(group_offsets, x, qb, sfb, gb, N: int, row_index=None, out_dtype: int = NVFP4_OUT_BF16,
                 out=None, *, workspace=None, stream=None):
    """``gemv`` with one matrix per group: row i of D (in group e by group_offsets) is row row_index[i] of x
    (row i without row_index) times matrix e; qb [G, N, K/2], sfb tiled per matrix, gb [G]."""
    if stream is not None:
        with _on(stream):
            return grouped_gemv(group_offsets, x, qb, sfb, gb, N, row_index, out_dtype, out,
                                workspace=workspace)
    dev = _one_device("grouped_gemv", x, group_offsets, qb, sfb, gb, row_index, out, workspace)
    ldx = _rows_of("grouped_gemv: x", x)
    src, K = x.shape
    G = group_offsets.numel() - 1
    _flat("grouped_gemv: group_offsets", group_offsets, torch.int32, G + 1)
    _flat("grouped_gemv: qb", qb, torch.uint8, G, N, K // 2)
    _flat("grouped_gemv: gb", gb, torch.float32, G)
    _bytes("grouped_gemv: sfb", sfb, G * nvfp4_sf_mma_bytes(N, K))
    rows, ip, wp, nb = src, None, None, 0
    if row_index is not None:
        rows = row_index.numel()
        _flat("grouped_gemv: row_index", row_index, torch.int32, rows)
        ip = row_index.data_ptr()
    if workspace is not None:
        wp, nb = _scratch("grouped_gemv", workspace)
    out, ldd = _gemv_out("grouped_gemv", out_dtype, rows, N, out, dev)
    _check(_lib.nvfp4_grouped_gemv(G, group_offsets.data_ptr(), rows, x.data_ptr(), ldx, src, ip,
                                   qb.data_ptr(), sfb.data_ptr(), gb.data_ptr(), N, K, out_dtype,
                                   out.data_ptr(), ldd, wp, nb, _raw_stream(dev)), "nvfp4_grouped_gemv")
    return out


def expert_mlp(x, routing: Routing, up, down, gate=None, base=None, *, workspace=None, stream=None):
    """The experts of a MoE layer for a few tokens x [tokens, hidden] bf16: each routed row through its expert's gate
    and up matrices, silu(gate) * up (without a gate max(up, 0)^2), its down matrix, and the weighted sum per token
    on top of base.  up, down and gate: ``moe.ExpertWeights`` (or the like: q, sf, g, n).  ``workspace``:
    nvfp4_expert_mlp_workspace_size bytes, which then hold the status word too.  For inference: no gradients; meant for
    up to about eight rows an expert (with more, ``grouped_gemm`` of quantised rows is faster)."""
    if stream is not None:
        with _on(stream):
            return expert_mlp(x, routing, up, down, gate, base, workspace=workspace)
    offsets, row_index, slot_row, weight = routing.group_offsets, routing.row_index, routing.slot_row, routing.weight
    uq, us, ug, dq, ds, dg = up.q, up.sf, up.g, down.q, down.sf, down.g
    gq, gs, gg = (None, None, None) if gate is None else (gate.q, gate.sf, gate.g)
    dev = _one_device("expert_mlp", x, offsets, row_index, slot_row, weight, uq, us, ug, dq, ds, dg, gq, gs, gg, base,
                      workspace)
    ldx = _rows_of("expert_mlp: x", x)
    tokens, hidden = x.shape
    G, ffn, rows = offsets.numel() - 1, up.n, row_index.numel()
    i32, f32 = torch.int32, torch.float32
    _flat("expert_mlp: group_offsets", offsets, i32, G + 1)
    _flat("expert_mlp: row_index", row_index, i32, rows)
    if slot_row.dim() != 2:
        raise ValueError("expert_mlp: slot_row [tokens, top_k] expected")
    k = slot_row.shape[1]
    _flat("expert_mlp: slot_row", slot_row, i32, tokens, k)
    _flat("expert_mlp: weight", weight, f32, tokens, k)
    if down.n != hidden:
        raise ValueError(f"expert_mlp: down has {down.n} rows, x {hidden} columns")
    _experts_matrix("expert_mlp: up", uq, us, ug, G, ffn, hidden)
    _experts_matrix("expert_mlp: down", dq, ds, dg, G, hidden, ffn)
    bp = gp = gsp = ggp = None
    if gate is not None:
        if gate.n != ffn:
            raise ValueError(f"expert_mlp: gate has {gate.n} rows, up {ffn}")
        _experts_matrix("expert_mlp: gate", gq, gs, gg, G, ffn, hidden)
        gp, gsp, ggp = gq.data_ptr(), gs.data_ptr(), gg.data_ptr()
    if base is not None:
        _flat("expert_mlp: base", base, torch.bfloat16, tokens, hidden)
        bp = base.data_ptr()
    if workspace is None:
        nb = nvfp4_expert_mlp_workspace_size(rows, hidden, ffn)
        workspace = torch.empty(nb, dtype=torch.uint8, device=dev)
        wp = workspace.data_ptr()
    else:
        wp, nb = _scratch("expert_mlp", workspace)
    out = _matrix(dev, torch.bfloat16, tokens, hidden)
    _check(_lib.nvfp4_expert_mlp(G, offsets.data_ptr(), rows, x.data_ptr(), ldx, tokens, row_index.data_ptr(), gp, gsp,
                                 ggp, uq.data_ptr(), us.data_ptr(), ug.data_ptr(), dq.data_ptr(), ds.data_ptr(),
                                 dg.data_ptr(), hidden, ffn, slot_row.data_ptr(), weight.data_ptr(), k, bp,
                                 out.data_ptr(), wp, nb, _raw_stream(dev)), "nvfp4_expert_mlp")
    return out


def _experts_matrix(name: str, q, sf, g, G: int, n: int, k: int) -> None:
    """One NVFP4 matrix [n, k] per expert, tiled scales."""
    if q.shape != (G, n, k // 2) or q.dtype is not torch.uint8 or not q.is_contiguous():
        raise ValueError(f"{name}.q: contiguous uint8 {(G, n, k // 2)} expected, got {q.dtype} {tuple(q.shape)}")
    if g.shape != (G,) or g.dtype is not torch.float32 or not g.is_contiguous():
        raise ValueError(f"{name}.g: contiguous float32 {(G,)} expected, got {g.dtype} {tuple(g.shape)}")
    least = G * ((n + 127) // 128 * 128) * (k // 16)
    if sf.numel() < least or sf.element_size() != 1 or not sf.is_contiguous():
        raise ValueError(f"{name}.sf: at least {least} contiguous bytes expected, got {sf.dtype} {tuple(sf.shape)}")


# ------------------------------------------------- the cache of a decoding step, and attention over it
@dataclass
class KVCache:
    """A paged cache of keys and values in NVFP4, blocks along the head dimension: codes uint8 [2, pages, kv_heads,
    page_size, dim/2] and E4M3 bytes uint8 [2, pages, kv_heads, page_size, dim/16], the keys first; amax f32 [2], the
    largest magnitudes that keys and values are expected to have (larger ones saturate), and g = amax / 2688.  The two
    belong together (append and attention read amax, ``dequantize`` g) and stay as they are while the cache holds anything:
    what is in it was quantised with them."""
    q: object
    sf: object
    amax: object
    g: object

    def _half(self, which: int) -> NVFP4Tensor:
        q, sf, g = self.q, self.sf, self.g
        _, pages, heads, size, half = q.shape
        rows, blocks = pages * heads * size, half // 8
        return NVFP4Tensor(q.as_strided((rows, half), (half, 1), q.storage_offset() + which * rows * half),
                           sf.as_strided((rows, blocks), (blocks, 1), sf.storage_offset() + which * rows * blocks),
                           g.as_strided((1,), (1,), g.storage_offset() + which), rows, 2 * half, NVFP4_SF_ROWMAJOR)

    def keys(self) -> NVFP4Tensor:
        """The keys as one matrix [pages * kv_heads * page_size, dim], a view (for ``dequantize``)."""
        return self._half(0)

    def values(self) -> NVFP4Tensor:
        """The values, likewise."""
        return self._half(1)


def kv_cache(pages: int, kv_heads: int, page_size: int, dim: int, amax_k: float = 2688.0, amax_v: float = 2688.0,
             device=None) -> KVCache:
    """A cache of zeros."""
    dev = torch.device("cuda") if device is None else device
    amax = torch.tensor([amax_k, amax_v], dtype=torch.float32)
    # (2688 as a tensor: a division by a number may come out as a product with its reciprocal)
    g = torch.where(amax > 0, amax / torch.full_like(amax, 2688.0), 1.0)
    return KVCache(torch.zeros((2, pages, kv_heads, page_size, dim // 2), dtype=torch.uint8, device=dev),
                   torch.zeros((2, pages, kv_heads, page_size, dim // 16), dtype=torch.uint8, device=dev),
                   amax.to(dev), g.to(dev))


def _cache_view(name: str, cache: KVCache) -> KVCacheView:
    q, sf, amax = cache.q, cache.sf, cache.amax
    u8 = torch.uint8
    shape = q.shape
    if len(shape) != 5 or shape[0] != 2 or q.dtype is not u8 or not q.is_contiguous():
        raise ValueError(f"{name}: cache.q contiguous uint8 [2, pages, kv_heads, page_size, dim/2] expected, got {q.dtype} "
                         f"{tuple(shape)}")
    _, pages, heads, size, half = shape
    if sf.shape != (2, pages, heads, size, half // 8) or sf.dtype is not u8 or not sf.is_contiguous():
        raise ValueError(f"{name}: cache.sf contiguous uint8 {(2, pages, heads, size, half // 8)} expected, got {sf.dtype} "
                         f"{tuple(sf.shape)}")
    if amax.shape != (2,) or amax.dtype is not torch.float32 or not amax.is_contiguous():
        raise ValueError(f"{name}: cache.amax float32 [2] expected, got {amax.dtype} {tuple(amax.shape)}")
    return KVCacheView(q.data_ptr(), sf.data_ptr(), amax.data_ptr(), pages, heads, size, 2 * half)


def _table_of(name: str, table):
    shape = table.shape
    if len(shape) != 2 or table.dtype is not torch.int32:
        raise ValueError(f"{name}: int32 table [sequences, pages] expected, got {table.dtype} {tuple(shape)}")
    n, pages = shape
    if table.is_contiguous():
        return n, pages, pages
    _need(pages <= 1 or table.stride(1) == 1, f"{name}: rows of the table must be contiguous")
    return n, pages, table.stride(0) if n > 1 else pages


def _heads_of(name: str, t, tokens, heads, dim):
    """A bf16 tensor [tokens, heads, dim] with contiguous heads; returns its strides in elements."""
    if t.shape != (tokens, heads, dim) or t.dtype is not torch.bfloat16:
        raise ValueError(f"{name}: bfloat16 {(tokens, heads, dim)} expected, got {t.dtype} {tuple(t.shape)}")
    ld, hs, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}: heads must be contiguous")
    # (the stride of a single row or head is never used, and torch leaves it arbitrary)
    return ld if tokens > 1 else heads * dim, hs if heads > 1 else dim


def kv_append(cache: KVCache, k, v, table, position, sequence=None, *, cos=None, sin=None, interleaved: bool = False,
              q=None, q_out=None, workspace=None, stream=None):
    """Keys and values of new tokens (bf16 [tokens, kv_heads, dim]) into the cache: token t at place ``position[t]`` of
    sequence ``sequence[t]`` (sequence t without it), whose pages are ``table[sequence]`` (all int32).  With cos and
    sin (f32 [angles, rot/2], rows by position) the first rot elements of the keys' heads are turned by their
    position, pairs (i, i + rot/2) or with ``interleaved`` (2i, 2i + 1), and q's (bf16 [tokens, heads, dim]) into
    ``q_out`` (a new tensor; q itself may be given), which is returned.  Tokens with a negative position or sequence are
    left out (their rows of q_out too); tokens without a place in the cache are left out and reported in the optional
    ``workspace`` (256 bytes).  For inference: no gradients."""
    if stream is not None:
        with _on(stream):
            return kv_append(cache, k, v, table, position, sequence, cos=cos, sin=sin, interleaved=interleaved, q=q,
                             q_out=q_out, workspace=workspace)
    dev = _one_device("kv_append", k, v, cache.q, cache.sf, cache.amax, table, position, sequence, cos, sin, q, q_out,
                      workspace)
    view = _cache_view("kv_append", cache)
    kv, dim = view.kv_heads, view.dim
    tokens = k.shape[0]
    ldk, hsk = _heads_of("kv_append: k", k, tokens, kv, dim)
    ldv, hsv = _heads_of("kv_append: v", v, tokens, kv, dim)
    sequences, pages, ldt = _table_of("kv_append", table)
    i32 = torch.int32
    if position.dtype is not i32 or position.shape != (tokens,) or not position.is_contiguous():
        raise ValueError(f"kv_append: position int32 {(tokens,)} expected, got {position.dtype} {tuple(position.shape)}")
    sp = cp = np = qp = op = wp = None
    if sequence is not None:
        if sequence.dtype is not i32 or sequence.shape != (tokens,) or not sequence.is_contiguous():
            raise ValueError(f"kv_append: sequence int32 {(tokens,)} expected, got {sequence.dtype} {tuple(sequence.shape)}")
        sp = sequence.data_ptr()
    angles = rot = heads = ldq = hsq = ldo = hso = nb = 0
    if cos is not None or sin is not None:
        if cos is None or sin is None or len(cos.shape) != 2:
            raise ValueError("kv_append: cos and sin [angles, rot/2] go together")
        shape = cos.shape
        f32 = torch.float32
        if (sin.shape != shape or cos.dtype is not f32 or sin.dtype is not f32 or not cos.is_contiguous()
                or not sin.is_contiguous()):
            raise ValueError(f"kv_append: cos and sin contiguous float32 of one shape expected, got {cos.dtype} "
                             f"{tuple(shape)} and {sin.dtype} {tuple(sin.shape)}")
        angles, rot = shape[0], 2 * shape[1]
        cp, np = cos.data_ptr(), sin.data_ptr()
    if q is not None:
        if cp is None:
            raise ValueError("kv_append: q is turned by cos and sin, which are missing")
        heads = q.shape[1] if q.dim() == 3 else 0
        ldq, hsq = _heads_of("kv_append: q", q, tokens, heads, dim)
        if q_out is None:
            ldo, hso = heads * dim, dim
            q_out = torch.empty_strided((tokens, heads, dim), (ldo, dim, 1), dtype=torch.bfloat16, device=dev)
        else:
            ldo, hso = _heads_of("kv_append: q_out", q_out, tokens, heads, dim)
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("kv_append: q_out without q")
    if workspace is not None:
        wp, nb = _scratch("kv_append", workspace)
    _check(_lib.nvfp4_kv_append(ctypes.byref(view), k.data_ptr(), ldk, hsk, v.data_ptr(), ldv, hsv, tokens,
                                table.data_ptr(), ldt, sequences, pages, position.data_ptr(), sp, cp, np, angles, rot,
                                1 if interleaved else 0, qp, ldq, hsq, heads, op, ldo, hso, wp, nb,
                                torch._C._cuda_getCurrentRawStream(dev.index)), "nvfp4_kv_append")
    return q_out


def kv_attention(q, cache: KVCache, table, lengths, *, scale: Optional[float] = None, window: int = 0, lse: bool = False,
                 workspace=None, stream=None):
    """Attention of the last tokens of each sequence, q bf16 [sequences, queries, heads, dim], over the cache: query i
    sees the cached tokens up to its own place lengths[s] - queries + i (lengths int32 [sequences], the queries' tokens
    included), of them the ``window`` last ones (0: all; pages before the first query's may be gone).  Query heads share
    the kv heads in order; scale is 1 / sqrt(dim) without one.  Returns bf16 [sequences, queries, heads, dim]; with
    ``lse`` also the logarithm of each row's sum of exponentials, f32 [sequences, queries, heads].  Rows that see nothing
    are 0, their lse -inf.  ``workspace``: nvfp4_kv_attention_workspace_size bytes, which then hold the status word too.
    For inference: no gradients; meant for few rows (the cache is decoded again for every eight of queries * heads /
    kv_heads)."""
    if stream is not None:
        with _on(stream):
            return kv_attention(q, cache, table, lengths, scale=scale, window=window, lse=lse, workspace=workspace)
    dev = _one_device("kv_attention", q, cache.q, cache.sf, cache.amax, table, lengths, workspace)
    view = _cache_view("kv_attention", cache)
    shape = q.shape
    if len(shape) != 4 or shape[3] != view.dim or q.dtype is not torch.bfloat16:
        raise ValueError(f"kv_attention: q bfloat16 [sequences, queries, heads, {view.dim}] expected, got {q.dtype} "
                         f"{tuple(shape)}")
    n, new, heads, dim = shape
    ldb, ldi, ldh, one = q.stride()
    if one != 1:
        raise ValueError("kv_attention: heads of q must be contiguous")
    sequences, pages, ldt = _table_of("kv_attention", table)
    if sequences != n:
        raise ValueError(f"kv_attention: a table of {sequences} sequences for {n}")
    _flat("kv_attention: lengths", lengths, torch.int32, n)
    if workspace is None:
        nb = _attention_bytes(n, new, heads, view.kv_heads, dim, pages * view.page_size)
        workspace = torch.empty(nb, dtype=torch.uint8, device=dev)
        wp = workspace.data_ptr()
    else:
        wp, nb = _scratch("kv_attention", workspace)
    out = torch.empty_strided(shape, (new * heads * dim, heads * dim, dim, 1), dtype=torch.bfloat16, device=dev)
    sums = torch.empty((n, new, heads), dtype=torch.float32, device=dev) if lse else None
    # (strides over a single sequence, token or head are never used, and torch leaves them arbitrary)
    _check(_lib.nvfp4_kv_attention(q.data_ptr(), ldb if n > 1 else 0, ldi if new > 1 else 0, ldh if heads > 1 else dim, n,
                                   new, heads, ctypes.byref(view), table.data_ptr(), ldt, pages, lengths.data_ptr(),
                                   dim ** -0.5 if scale is None else scale, window, out.data_ptr(),
                                   sums.data_ptr() if lse else None, wp, nb, _raw_stream(dev)), "nvfp4_kv_attention")
    return (out, sums) if lse else out


@functools.lru_cache(maxsize=256)
def _attention_bytes(*sizes) -> int:
    return _lib.nvfp4_kv_attention_workspace_size(*sizes)
