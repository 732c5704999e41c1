"""Thin Python binding of libqfp4.so (see include/qfp4.h).

Argument marshalling only: every function takes torch tensors (or raw
integers for pointers), passes their device addresses and sizes to the C ABI
and raises ``Qfp4Error`` on a non-zero status.  All computation happens in
the CUDA kernels of the library.  There is no fallback: if the library is
missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

MXFP4 = 0
NVFP4 = 1
NVFP4_B32 = 2
E4M3 = 0
E5M2 = 1
SCALE_FP32 = 0
SCALE_POW2 = 1
CACHE_BF16 = 0
CACHE_E4M3 = 1
CACHE_NVFP4 = 2
OUT_BF16 = 0
OUT_FP32 = 1
SF_ROWMAJOR = 0
SF_MMA = 1

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqfp4.so")
_lock = threading.Lock()
_lib = None

# (restype, argtypes) per exported symbol, mirroring include/qfp4.h
_i32, _i64, _sz, _vp, _cp = ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_char_p
_f32 = ctypes.c_float
SIGNATURES = {
    "qfp4_version": (_i32, []),
    "qfp4_status_string": (_cp, [_i32]),
    "qfp4_device_check": (_i32, []),
    "qfp4_poll_device_status": (_i32, [_vp]),
    "qfp4_block_size": (_i32, [_i32]),
    "qfp4_sf_mma_bytes": (_sz, [_i64, _i64]),
    "qfp4_sf_mma_grouped_bytes": (_sz, [_i64, _i64, _i64]),
    "qfp4_global_scale": (_i32, [_vp, _i64, _i64, _vp, _vp]),
    "qfp4_global_scale_grouped": (_i32, [_vp, _i64, _i64, _i64, _vp, _vp, _vp]),
    "qfp4_quantize": (_i32, [_i32, _vp, _i64, _i64, _vp, _vp, _vp, _i32, _vp]),
    "qfp4_global_scale_rows": (_i32, [_vp, _i64, _i64, _vp, _vp]),
    "qfp4_quantize_rows": (_i32, [_i32, _vp, _i64, _i64, _vp, _vp, _vp, _i32, _vp]),
    "qfp4_gemm_nt_scaled": (_i32, [_i32, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                   _sz, _vp]),
    "qfp4_quantize_grouped_rows": (_i32, [_i32, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "qfp4_gemm_nt_grouped_scaled": (_i32, [_i32, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp,
                                           _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "qfp4_absmax_gs": (_i32, [_i64, _vp, _vp, _i64, _vp, _vp]),
    "qfp4_sparse24_meta_bytes": (_sz, [_i64, _i64, _i32]),
    "qfp4_sparse24_compress": (_i32, [_vp, _i64, _i64, _vp, _vp, _i32, _vp]),
    "qfp4_gemm_nt_sparse24": (_i32, [_i32, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                     _vp]),
    "qfp4_gemm_swiglu_quantize": (_i32, [_i32, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                         _vp]),
    "qfp4_gemm_swiglu_quantize_grouped": (_i32, [_i32, _i64, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp,
                                                 _vp, _vp, _vp, _vp, _vp]),
    "qfp4_quantize_grouped": (_i32, [_i32, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "qfp4_residual_rmsnorm_quantize": (_i32, [_i32, _vp, _vp, _vp, _i64, _i64, ctypes.c_float, _vp, _vp, _vp,
                                              _vp, _i32, _vp]),
    "qfp4_sf_interleave": (_i32, [_vp, _i64, _i64, _vp, _i32, _vp]),
    "qfp4_gemm_workspace_bytes": (_sz, [_i32, _i64, _i64, _i64]),
    "qfp4_gemm_nt": (_i32, [_i32, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "qfp4_gemm_nt_noalloc": (_i32, [_i32, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "qfp4_gemm_nt_grouped": (_i32, [_i32, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp,
                                    _vp, _vp, _vp, _vp, _sz, _vp]),
    "qfp4_fp8_quantize": (_i32, [_i32, _i32, _vp, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "qfp4_fp8_quantize_weight": (_i32, [_i32, _i32, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "qfp4_gemm_nt_fp8": (_i32, [_i32, _i32, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp]),
    "qfp4_gemm_nt_fp8_grouped": (_i32, [_i32, _i32, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _i32, _vp,
                                        _vp]),
    "qfp4_fp8_grouped_cols": (_sz, [_i64, _i64]),
    "qfp4_fp8_quantize_grouped": (_i32, [_i32, _i32, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
    "qfp4_gemm_nt_fp8_kgrouped": (_i32, [_i32, _i32, _i64, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _i32, _vp,
                                         _vp]),
    "qfp4_moe_route_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "qfp4_moe_route": (_i32, [_i32, _vp, _i64, _i64, _i64, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                              _vp, _sz, _vp]),
    "qfp4_moe_route_backward": (_i32, [_i32, _vp, _i64, _i64, _i64, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "qfp4_gemv_nt": (_i32, [_i32, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _vp, _i64, _vp]),
    "qfp4_qk_norm_rope": (_i32, [_vp, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _f32, _vp, _i64, _i64, _i32, _vp, _vp,
                                 _i64, _vp, _i64, _vp]),
    "qfp4_qk_norm_rope_cache": (_i32, [_vp, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _f32, _vp, _i64, _i64, _i32, _vp,
                                       _vp, _i64, _i32, _vp, _i64, _i64, _vp, _vp, _vp, _vp]),
    "qfp4_qk_norm_rope_backward_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "qfp4_qk_norm_rope_backward": (_i32, [_vp, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _f32, _vp, _i64, _i64, _i32,
                                          _vp, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _sz, _vp]),
    "qfp4_kv_cache_page_bytes": (_sz, [_i32, _i64, _i64, _i64]),
    "qfp4_kv_cache_write": (_i32, [_i32, _vp, _i64, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _i64,
                                   _vp]),
    "qfp4_kv_cache_read": (_i32, [_i32, _vp, _i64, _i64, _i64, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _i64,
                                  _vp]),
    "qfp4_attention_decode_workspace_bytes": (_sz, [_i64, _i64, _i64, _i64]),
    "qfp4_attention_decode": (_i32, [_i32, _vp, _i64, _i64, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i64,
                                     _f32, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
}


# Calls with many arguments, which take them as one array of 64-bit words:
# (function, packer), filled by load().
_WORDS = ("qfp4_fp8_quantize", "qfp4_fp8_quantize_grouped", "qfp4_fp8_quantize_weight", "qfp4_gemm_nt_fp8",
          "qfp4_gemm_nt_fp8_grouped", "qfp4_gemm_nt_fp8_kgrouped", "qfp4_moe_route", "qfp4_moe_route_backward")
_LAYER_WORDS = ("qfp4_gemv_nt", "qfp4_qk_norm_rope", "qfp4_qk_norm_rope_cache", "qfp4_qk_norm_rope_backward",
                "qfp4_kv_cache_write", "qfp4_kv_cache_read", "qfp4_attention_decode")
_words = {}


class Qfp4Error(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")


def load() -> ctypes.CDLL:
    """Open libqfp4.so (built by build.py / __graft_entry__.build())."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"libqfp4.so not built ({LIB_PATH}); run __graft_entry__.build()")
            lib = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            for name in _WORDS + _LAYER_WORDS:
                fn = getattr(lib, name + "_words")
                fn.restype = _i32
                fn.argtypes = [ctypes.c_char_p]
                form = "".join("f4x" if a is _f32 else "q" for a in SIGNATURES[name][1])
                _words[name] = fn, struct.Struct("=" + form).pack
            _lib = lib
        return _lib


FAULTINJ_PATH = os.path.join(_HERE, "libqfp4_faultinj.so")
_faultinj = None


def load_fault_injection() -> ctypes.CDLL:
    """Open the test build (libqfp4_faultinj.so, built by
    build.build(variant="faultinj")): the same entry points with a 5 ms wait
    limit, plus qfp4_test_inject_skip_release(int), its counterpart for the
    8-bit products qfp4_test_inject_fp8_skip_release(int), that of the attention and
    the head norms' gradient qfp4_test_inject_skip_copy(int), and the encoder probes
    qfp4_test_scale_codes / qfp4_test_element_codes.  For tests only; the
    product path always uses load()."""
    global _faultinj
    with _lock:
        if _faultinj is None:
            if not os.path.exists(FAULTINJ_PATH):
                raise RuntimeError(f"fault-injection build missing ({FAULTINJ_PATH})")
            lib = ctypes.CDLL(FAULTINJ_PATH)
            for name, (res, args) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            for name in ("qfp4_test_inject_skip_release", "qfp4_test_inject_fp8_skip_release",
                         "qfp4_test_inject_skip_copy"):
                getattr(lib, name).restype = _i32
                getattr(lib, name).argtypes = [_i32]
            for name in ("qfp4_test_scale_codes", "qfp4_test_element_codes"):
                fn = getattr(lib, name)
                fn.restype = _i32
                fn.argtypes = [_i32, ctypes.c_uint32, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p]
            _faultinj = lib
        return _faultinj


def status_string(status: int) -> str:
    return load().qfp4_status_string(int(status)).decode()


def _torch_stream(device) -> int:
    return torch.cuda.current_stream().cuda_stream      # on a torch without CUDA: its own error


# The current stream's handle, without building a torch Stream around it
# (0.1 us instead of 3).  A torch built without CUDA has neither lookup, and
# what needs no GPU (sizes, refusals, status texts) works there too.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _torch_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", lambda: 0)


def _p(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        return _current_stream(_current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, rc: int) -> None:
    if rc != 0:
        raise Qfp4Error(fn, rc)


def _call(fn: str, *args) -> None:
    if _lib is None:
        load()
    function, pack = _words[fn]
    rc = function(pack(*args))
    if rc != 0:
        raise Qfp4Error(fn, rc)


def version() -> int:
    return load().qfp4_version()


def device_check() -> int:
    return load().qfp4_device_check()


def poll_device_status(stream=None) -> int:
    return load().qfp4_poll_device_status(_stream(stream))


def block_size(fmt: int) -> int:
    return load().qfp4_block_size(fmt)


def sf_mma_bytes(rows: int, cols: int) -> int:
    return int(load().qfp4_sf_mma_bytes(rows, cols))


def sf_mma_grouped_bytes(total_rows: int, groups: int, cols: int) -> int:
    return int(load().qfp4_sf_mma_grouped_bytes(total_rows, groups, cols))


def gemm_workspace_bytes(fmt: int, M: int, N: int, K: int) -> int:
    return int(load().qfp4_gemm_workspace_bytes(fmt, M, N, K))


def global_scale(X, gs_out, stream=None) -> None:
    rows, cols = X.shape
    _check("qfp4_global_scale",
           load().qfp4_global_scale(_p(X), rows, cols, _p(gs_out), _stream(stream)))


def global_scale_grouped(X, row_offsets, gs_out, stream=None) -> None:
    rows, cols = X.shape
    groups = row_offsets.numel() - 1
    _check("qfp4_global_scale_grouped",
           load().qfp4_global_scale_grouped(_p(X), rows, cols, groups, _p(row_offsets), _p(gs_out),
                                            _stream(stream)))


def absmax_gs(row_offsets, X, gs_out, stream=None) -> None:
    """Per-group global scales with the row count read on the device from
    row_offsets[groups]; X is [>= that many rows, K]."""
    K = X.shape[1]
    groups = row_offsets.numel() - 1
    _check("qfp4_absmax_gs",
           load().qfp4_absmax_gs(groups, _p(row_offsets), _p(X), K, _p(gs_out), _stream(stream)))


def quantize(fmt, X, gs, Q, SF, sf_layout=SF_ROWMAJOR, stream=None) -> None:
    M, K = X.shape
    _check("qfp4_quantize",
           load().qfp4_quantize(fmt, _p(X), M, K, _p(gs), _p(Q), _p(SF), sf_layout, _stream(stream)))


def global_scale_rows(X, gs_out, stream=None) -> None:
    """Per-row NVFP4 global scales: gs_out[r] = amax(row r) / (6*448)."""
    rows, cols = X.shape
    _check("qfp4_global_scale_rows",
           load().qfp4_global_scale_rows(_p(X), rows, cols, _p(gs_out), _stream(stream)))


def quantize_rows(fmt, X, gs_rows, Q, SF, sf_layout=SF_ROWMAJOR, stream=None) -> None:
    """Quantise with one global scale per row (two-level NVFP4)."""
    M, K = X.shape
    _check("qfp4_quantize_rows",
           load().qfp4_quantize_rows(fmt, _p(X), M, K, _p(gs_rows), _p(Q), _p(SF), sf_layout, _stream(stream)))


def quantize_grouped(fmt, X, row_offsets, gs, Q, SF_mma, stream=None) -> None:
    rows, K = X.shape
    groups = row_offsets.numel() - 1
    _check("qfp4_quantize_grouped",
           load().qfp4_quantize_grouped(fmt, _p(X), rows, K, groups, _p(row_offsets), _p(gs), _p(Q),
                                        _p(SF_mma), _stream(stream)))


def quantize_grouped_rows(fmt, X, row_offsets, gs_rows, Q, SF_mma, stream=None) -> None:
    """Grouped quantiser with one global scale per row (per-group MMA scale layout)."""
    rows, K = X.shape
    groups = row_offsets.numel() - 1
    _check("qfp4_quantize_grouped_rows",
           load().qfp4_quantize_grouped_rows(fmt, _p(X), rows, K, groups, _p(row_offsets), _p(gs_rows), _p(Q),
                                             _p(SF_mma), _stream(stream)))


def residual_rmsnorm_quantize(fmt, X, R, gamma, eps, Y, gs_rows, Q, SF, sf_layout=SF_MMA, stream=None) -> None:
    """y = bf16(X + R) into Y (R and Y may be None), z = RMSNorm(y) * gamma,
    per-row global scales of z into gs_rows (NVFP4) and z quantised into Q, SF."""
    M, K = X.shape
    _check("qfp4_residual_rmsnorm_quantize",
           load().qfp4_residual_rmsnorm_quantize(fmt, _p(X), _p(R), _p(gamma), M, K, float(eps), _p(Y), _p(gs_rows),
                                                 _p(Q), _p(SF), sf_layout, _stream(stream)))


def sf_interleave(SF_in, rows, cols, SF_out, layout=SF_MMA, stream=None) -> None:
    _check("qfp4_sf_interleave",
           load().qfp4_sf_interleave(_p(SF_in), rows, cols, _p(SF_out), layout, _stream(stream)))


def gemm_nt_scaled(fmt, M, N, K, A, A_sf, B, B_sf, gs_a, gs_b, row_scale, col_scale, D, workspace=None,
                   ws_bytes=0, stream=None) -> None:
    """The GEMM with the two-level epilogue: row m of D times row_scale[m],
    column n times col_scale[n] (either may be None)."""
    _check("qfp4_gemm_nt_scaled",
           load().qfp4_gemm_nt_scaled(fmt, M, N, K, _p(A), _p(A_sf), _p(B), _p(B_sf), _p(gs_a), _p(gs_b),
                                      _p(row_scale), _p(col_scale), _p(D), _p(workspace), ws_bytes,
                                      _stream(stream)))


def gemm_nt(fmt, M, N, K, A, A_sf, B, B_sf, gs_a, gs_b, D, workspace=None, ws_bytes=0,
            stream=None) -> None:
    _check("qfp4_gemm_nt",
           load().qfp4_gemm_nt(fmt, M, N, K, _p(A), _p(A_sf), _p(B), _p(B_sf), _p(gs_a), _p(gs_b),
                               _p(D), _p(workspace), ws_bytes, _stream(stream)))


def gemm_nt_grouped(fmt, row_offsets, total_rows, max_group_rows, N, K, A, A_sf, B, B_sf,
                    gs_a, gs_b, D, workspace=None, ws_bytes=0, stream=None) -> None:
    groups = row_offsets.numel() - 1
    _check("qfp4_gemm_nt_grouped",
           load().qfp4_gemm_nt_grouped(fmt, groups, _p(row_offsets), total_rows, max_group_rows, N, K,
                                       _p(A), _p(A_sf), _p(B), _p(B_sf), _p(gs_a), _p(gs_b), _p(D),
                                       _p(workspace), ws_bytes, _stream(stream)))


def gemm_nt_grouped_scaled(fmt, row_offsets, total_rows, max_group_rows, N, K, A, A_sf, B, B_sf,
                           gs_a, gs_b, row_scale, col_scale, D, workspace=None, ws_bytes=0,
                           stream=None) -> None:
    """Grouped GEMM with the two-level epilogue: row m times row_scale[m],
    column n of group e times col_scale[e*N + n] (either may be None)."""
    groups = row_offsets.numel() - 1
    _check("qfp4_gemm_nt_grouped_scaled",
           load().qfp4_gemm_nt_grouped_scaled(fmt, groups, _p(row_offsets), total_rows, max_group_rows, N, K,
                                              _p(A), _p(A_sf), _p(B), _p(B_sf), _p(gs_a), _p(gs_b),
                                              _p(row_scale), _p(col_scale), _p(D), _p(workspace), ws_bytes,
                                              _stream(stream)))


def sparse24_meta_bytes(rows: int, K: int, layout: int = SF_MMA) -> int:
    return int(load().qfp4_sparse24_meta_bytes(rows, K, layout))


def sparse24_compress(W, W_comp, W_meta, layout=SF_MMA, stream=None) -> None:
    """2:4 pair-sparse packed W [rows, K/2] -> kept bytes [rows, K/4] and metadata."""
    rows, K = W.shape[0], W.shape[1] * 2
    _check("qfp4_sparse24_compress",
           load().qfp4_sparse24_compress(_p(W), rows, K, _p(W_comp), _p(W_meta), layout, _stream(stream)))


def gemm_nt_sparse24(fmt, M, N, K, X, X_sf, W_comp, W_meta, W_sf, gs_x, gs_w, D, row_scale=None, col_scale=None,
                     stream=None) -> None:
    _check("qfp4_gemm_nt_sparse24",
           load().qfp4_gemm_nt_sparse24(fmt, M, N, K, _p(X), _p(X_sf), _p(W_comp), _p(W_meta), _p(W_sf), _p(gs_x),
                                        _p(gs_w), _p(row_scale), _p(col_scale), _p(D), _stream(stream)))


def gemm_swiglu_quantize(fmt, M, I, K, A, A_sf, W, W_sf, gs_a, gs_w, gs_out, Q_out, SF_out,
                         stream=None) -> None:
    """Up-projection with SwiGLU, requantised: W holds the gate and up rows
    interleaved in groups of the block size; writes H = silu(gate) * up
    quantised into Q_out [M, I/2] and SF_out (MMA layout for [M, I/g])."""
    _check("qfp4_gemm_swiglu_quantize",
           load().qfp4_gemm_swiglu_quantize(fmt, M, I, K, _p(A), _p(A_sf), _p(W), _p(W_sf), _p(gs_a), _p(gs_w),
                                            _p(gs_out), _p(Q_out), _p(SF_out), _stream(stream)))


def gemm_swiglu_quantize_grouped(fmt, row_offsets, total_rows, I, K, A, A_sf, W, W_sf, gs_a, gs_w, gs_out,
                                 Q_out, SF_out, stream=None) -> None:
    """Per-expert version; SF_out in the per-group MMA layout."""
    groups = row_offsets.numel() - 1
    _check("qfp4_gemm_swiglu_quantize_grouped",
           load().qfp4_gemm_swiglu_quantize_grouped(fmt, groups, _p(row_offsets), total_rows, I, K, _p(A),
                                                    _p(A_sf), _p(W), _p(W_sf), _p(gs_a), _p(gs_w), _p(gs_out),
                                                    _p(Q_out), _p(SF_out), _stream(stream)))


def _at(t, dtype, least=0):
    """Address of a whole row-major matrix on the GPU (a strided view or a host
    tensor would be read as something else), of the given type and with at least
    so many elements (the C ABI sees an address and cannot tell: a kernel would
    write past a shorter one's end).  A router call has fifteen of these: the
    usual path asks each question once."""
    if t is None:
        return 0
    try:
        if t.dtype is dtype and t.is_cuda and t.numel() >= least and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        if isinstance(t, int):
            return t
        raise
    if not (t.is_cuda and t.is_contiguous()):
        raise ValueError("qfp4: tensors must be contiguous and on the GPU")
    if t.dtype is not dtype:
        raise ValueError(f"qfp4: expected {dtype}, got {t.dtype}")
    raise ValueError(f"qfp4: expected at least {least} elements, got {t.numel()} ({tuple(t.shape)})")


_F32, _BF16, _I32, _U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8
_CODES = {E4M3: (torch.float8_e4m3fn, torch.uint8), E5M2: (torch.float8_e5m2, torch.uint8)}


def _codes(t, kind, least=0):
    """Address of a matrix of 8-bit codes: of that type, or plain bytes."""
    if t is None:
        return 0
    try:
        if t.dtype in _CODES[kind] and t.is_cuda and t.numel() >= least and t.is_contiguous():
            return t.data_ptr()
    except (AttributeError, KeyError):      # an address; a type that the library refuses
        if isinstance(t, int):
            return t
    if kind in _CODES and t.dtype not in _CODES[kind]:
        raise ValueError(f"qfp4: expected codes of {_CODES[kind][0]}, got {t.dtype}")
    return _at(t, t.dtype, least)


def fp8_quantize(type, X, Q=None, SF=None, Q_t=None, SF_t=None, scale=SCALE_FP32, row_index=None, stream=None) -> None:
    """BF16 X -> 8-bit codes with a scale per 128 elements: along the rows
    (Q [M, K], SF [ceil(K/128), M]) and / or along the columns, transposed
    (Q_t [K, ceil16(M)], SF_t [ceil(M/128), K]).  row_index (int32 [M]) gathers
    rows of X."""
    rows, K = X.shape
    M = rows if row_index is None else row_index.numel()
    _call("qfp4_fp8_quantize", type, scale, _at(X, _BF16), rows, _at(row_index, _I32), M, K,
          _codes(Q, type, M * K), _at(SF, _F32, (K + 127) // 128 * M),
          _codes(Q_t, type, K * ((M + 15) // 16 * 16)), _at(SF_t, _F32, (M + 127) // 128 * K), _stream(stream))


def fp8_grouped_cols(total_rows: int, groups: int) -> int:
    """Columns of Q_t when every group's rows begin a block of 128 of their own."""
    return int(load().qfp4_fp8_grouped_cols(total_rows, groups))


def fp8_quantize_grouped(type, X, row_offsets, Q_t, SF_t, Q=None, SF=None, scale=SCALE_FP32, row_index=None,
                         stream=None) -> None:
    """fp8_quantize for one product per expert: Q_t [K, cols], SF_t [cols/128, K]
    with cols = fp8_grouped_cols(rows, groups)."""
    rows, K = X.shape
    M = rows if row_index is None else row_index.numel()
    groups = row_offsets.numel() - 1
    cols = fp8_grouped_cols(M, groups)
    _call("qfp4_fp8_quantize_grouped", type, scale, _at(X, _BF16), rows, _at(row_index, _I32), groups,
          _at(row_offsets, _I32), M, K, _codes(Q, type, M * K), _at(SF, _F32, (K + 127) // 128 * M),
          _codes(Q_t, type, K * cols), _at(SF_t, _F32, cols // 128 * K), _stream(stream))


def fp8_quantize_weight(type, W, Q, SF, Q_t=None, SF_t=None, scale=SCALE_FP32, stream=None) -> None:
    """Weights W [N, K] or [groups, N, K] -> codes with a scale per 128 x 128
    block, and optionally their transpose (Q_t [.., K, ceil16(N)])."""
    groups, (N, K) = (1 if W.dim() == 2 else W.shape[0]), W.shape[-2:]
    blocks = groups * ((N + 127) // 128) * ((K + 127) // 128)
    _call("qfp4_fp8_quantize_weight", type, scale, groups, _at(W, _BF16, groups * N * K), N, K,
          _codes(Q, type, groups * N * K), _at(SF, _F32, blocks),
          _codes(Q_t, type, groups * K * ((N + 15) // 16 * 16)), _at(SF_t, _F32, blocks), _stream(stream))


def gemm_nt_fp8(a_type, b_type, M, N, K, A, A_sf, B, B_sf, D, b_rows=128, out=OUT_BF16, accumulate=False,
                stream=None) -> None:
    """D = A B^T with a scale per 128 elements of K: A_sf [ceil(K/128), M], B_sf
    per 128 x 128 block (b_rows=128) or [ceil(K/128), N] (b_rows=1)."""
    blocks = (K + 127) // 128
    _call("qfp4_gemm_nt_fp8", a_type, b_type, M, N, K, _codes(A, a_type, M * K), _at(A_sf, _F32, blocks * M),
          _codes(B, b_type, N * K), _at(B_sf, _F32, blocks * (N if b_rows == 1 else (N + 127) // 128)), b_rows, out,
          1 if accumulate else 0, _at(D, _F32 if out == OUT_FP32 else _BF16, M * N), _stream(stream))


def gemm_nt_fp8_grouped(a_type, b_type, row_offsets, total_rows, max_group_rows, N, K, A, A_sf, B, B_sf, D,
                        out=OUT_BF16, stream=None) -> None:
    """One product per expert: rows [row_offsets[e], row_offsets[e+1]) with B[e]."""
    groups = row_offsets.numel() - 1
    blocks = (K + 127) // 128
    _call("qfp4_gemm_nt_fp8_grouped", a_type, b_type, groups, _at(row_offsets, _I32), total_rows, max_group_rows, N, K,
          _codes(A, a_type, total_rows * K), _at(A_sf, _F32, blocks * total_rows),
          _codes(B, b_type, groups * N * K), _at(B_sf, _F32, groups * ((N + 127) // 128) * blocks), out,
          _at(D, _F32 if out == OUT_FP32 else _BF16, total_rows * N), _stream(stream))


def gemm_nt_fp8_kgrouped(a_type, b_type, row_offsets, total_rows, M, N, A, A_sf, B, B_sf, D, accumulate=False,
                         stream=None) -> None:
    """Every expert's weight gradient: D[e] (+)= A_e B_e^T over the columns that
    fp8_quantize_grouped gave group e; D fp32 [groups, M, N]."""
    groups = row_offsets.numel() - 1
    cols = fp8_grouped_cols(total_rows, groups)
    _call("qfp4_gemm_nt_fp8_kgrouped", a_type, b_type, groups, _at(row_offsets, _I32), total_rows, M, N,
          _codes(A, a_type, M * cols), _at(A_sf, _F32, cols // 128 * M),
          _codes(B, b_type, N * cols), _at(B_sf, _F32, cols // 128 * N),
          1 if accumulate else 0, _at(D, _F32, groups * M * N), _stream(stream))


def moe_route_workspace_bytes(T: int, E: int, topk: int) -> int:
    return int(load().qfp4_moe_route_workspace_bytes(T, E, topk))


def _logits(t):
    """(type, address)"""
    return (OUT_FP32, _at(t, _F32)) if t.dtype == _F32 else (OUT_BF16, _at(t, _BF16))


def moe_route(logits, topk, ids, gates, counts, row_offsets, dest, src, n_valid, mean_prob, loss, workspace,
              valid=None, renorm=True, stream=None) -> None:
    """Top-k experts of each token, gates, per-expert counts and row order, and
    the balance loss; valid is uint8 [T] or None."""
    T, E = logits.shape
    pairs = T * topk
    _call("qfp4_moe_route", *_logits(logits), T, E, topk, _at(valid, _U8, T), 1 if renorm else 0,
          _at(ids, _I32, pairs), _at(gates, _F32, pairs), _at(counts, _I32, E), _at(row_offsets, _I32, E + 1),
          _at(dest, _I32, pairs), _at(src, _I32, pairs), _at(n_valid, _I32, 1), _at(mean_prob, _F32, E),
          _at(loss, _F32, 1), _at(workspace, workspace.dtype), workspace.nbytes, _stream(stream))


def moe_route_backward(logits, ids, counts, n_valid, dgates, dloss, dlogits, valid=None, renorm=True,
                       stream=None) -> None:
    """dlogits of (gates . dgates + dloss * loss), choices and counts held fixed;
    dgates and dloss may be None."""
    T, E = logits.shape
    topk = ids.shape[1]
    pairs = T * topk
    _call("qfp4_moe_route_backward", *_logits(logits), T, E, topk, _at(valid, _U8, T), 1 if renorm else 0,
          _at(ids, _I32, pairs), _at(counts, _I32, E), _at(n_valid, _I32, 1), _at(dgates, _F32, pairs),
          _at(dloss, _F32, 1), _at(dlogits, logits.dtype, T * E), _stream(stream))


def _rows(t, width, want=None):
    """(address, elements from row to row) of BF16 rows of `width` elements that lie
    together: a contiguous matrix, or some columns of one (the heads of one kind in a
    projection's output).  want: (rows, width) or (rows, heads, elements of each); the
    heads may also be given as one row.  None: the shape that the tensor has, where the
    call's sizes were taken from it.  The usual path asks each question once."""
    if t is None:
        return 0, width
    if t.dtype is _BF16 and t.is_cuda and (want is None or t.shape == want) and t.is_contiguous():
        return t.data_ptr(), width
    if t.dtype is not _BF16 or not t.is_cuda:
        raise ValueError(f"qfp4: expected {_BF16} on the GPU, got {t.dtype} on {t.device}")
    shape, stride = t.shape, t.stride()
    rows = shape[0] if want is None else want[0]
    if len(shape) == 3:
        if shape[2] != 1 and stride[2] != 1 or shape[1] != 1 and stride[1] != shape[2]:
            raise ValueError("qfp4: the heads of a row must lie together")
        if want is not None and len(want) == 3 and shape[2] != want[2]:
            raise ValueError(f"qfp4: expected heads of {want[2]} elements, got {tuple(shape)}")
        got = shape[1] * shape[2]
    elif len(shape) == 2:
        if shape[1] != 1 and stride[1] != 1:
            raise ValueError("qfp4: the elements of a row must lie together")
        got = shape[1]
    else:
        raise ValueError(f"qfp4: expected rows, got {tuple(shape)}")
    if shape[0] != rows or got != width:
        raise ValueError(f"qfp4: expected {rows} rows of {width} elements, got {tuple(shape)}")
    return t.data_ptr(), stride[0] if rows > 1 and width > 0 else width


def gemv_nt(fmt, X, W, W_sf, gs_w, D, stream=None) -> None:
    """D = X W^T: up to 16 BF16 rows X [M, K] times 4-bit weights W [N, K/2] with
    scales in the MMA layout (B of gemm_nt); gs_w may be None."""
    M, K = X.shape
    N, row = W.shape
    if row * 2 != K:
        raise ValueError(f"qfp4: W has {row * 2} columns, X {K}")
    x, ldx = _rows(X, K)
    d, ldd = _rows(D, N, (M, N))
    g = 16 if fmt == NVFP4 else 32
    _call("qfp4_gemv_nt", fmt, M, N, K, x, ldx, _at(W, _U8, N * row),
          _at(W_sf, _U8, (N + 127) // 128 * 128 * ((K // g + 3) // 4 * 4)), _at(gs_w, _F32, 1), d, ldd, _stream(stream))


def _space(t):
    """(address, bytes) of a workspace, of whatever type."""
    if not (t.is_cuda and t.is_contiguous()):
        raise ValueError("qfp4: tensors must be contiguous and on the GPU")
    return t.data_ptr(), t.nbytes


def _head_args(QKV, T, width, q_heads, kv_heads, head_dim, value_heads, q_weight, k_weight, cos_sin, positions, eps,
               interleaved):
    """What the calls on query and key heads share, in the C ABI's order."""
    if width < (q_heads + kv_heads + value_heads) * head_dim:
        raise ValueError(f"qfp4: {q_heads} + {kv_heads} heads of {head_dim} do not fit in rows of {width}")
    x, ld = _rows(QKV, width)
    rows, rotary = (0, 0) if cos_sin is None else cos_sin.shape
    return (x, ld, T, q_heads, kv_heads, head_dim, _at(q_weight, _BF16, head_dim), _at(k_weight, _BF16, head_dim), eps,
            _at(cos_sin, _F32), rows, rotary, 1 if interleaved else 0, _at(positions, _I32, T))


def qk_norm_rope(QKV, q_heads, kv_heads, Q_out, K_out, q_weight=None, k_weight=None, cos_sin=None, positions=None,
                 eps=1e-6, interleaved=False, stream=None) -> None:
    """RMS norms of the query and key heads (weights None: none) and the rotation
    by cos_sin [positions, rotary_dim] (None: none), from the QKV projection's
    output [T, (q_heads + kv_heads + ...) * head_dim].  Q_out [T, q_heads,
    head_dim] and K_out [T, kv_heads, head_dim] may be views of QKV itself."""
    (T, width), D = QKV.shape, Q_out.shape[2]
    args = _head_args(QKV, T, width, q_heads, kv_heads, D, 0, q_weight, k_weight, cos_sin, positions, eps, interleaved)
    q, ldq = _rows(Q_out, q_heads * D, (T, q_heads, D))
    k, ldk = _rows(K_out, kv_heads * D, (T, kv_heads, D))
    _call("qfp4_qk_norm_rope", *args, q, ldq, k, ldk, _stream(stream))


def qk_norm_rope_backward_workspace_bytes(T: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(load().qfp4_qk_norm_rope_backward_workspace_bytes(T, q_heads, kv_heads, head_dim))


def qk_norm_rope_backward(QKV, q_heads, kv_heads, dQ, dK, dQKV, dq_weight, dk_weight, workspace, q_weight=None,
                          k_weight=None, cos_sin=None, positions=None, eps=1e-6, interleaved=False,
                          stream=None) -> None:
    """Gradient of qk_norm_rope: the query and key heads of dQKV (its value heads
    stay) and, fp32 [head_dim], those of the weights; without weights they and
    the workspace may be None."""
    (T, width), D = QKV.shape, dQ.shape[2]
    args = _head_args(QKV, T, width, q_heads, kv_heads, D, 0, q_weight, k_weight, cos_sin, positions, eps, interleaved)
    q, ldq = _rows(dQ, q_heads * D, (T, q_heads, D))
    k, ldk = _rows(dK, kv_heads * D, (T, kv_heads, D))
    dx, ldx = _rows(dQKV, width, (T, width))
    ws, nbytes = (0, 0) if workspace is None else _space(workspace)
    _call("qfp4_qk_norm_rope_backward", *args, q, ldq, k, ldk, dx, ldx, _at(dq_weight, _F32, D),
          _at(dk_weight, _F32, D), ws, nbytes, _stream(stream))


def kv_cache_page_bytes(type: int, kv_heads: int, head_dim: int, page_size: int) -> int:
    """Bytes of a page; a cache is a uint8 tensor of that many per page."""
    return int(load().qfp4_kv_cache_page_bytes(type, kv_heads, head_dim, page_size))


_CACHE_TOKEN = {CACHE_BF16: (32, 0), CACHE_E4M3: (16, 64), CACHE_NVFP4: (9, 0)}     # bits per element and more


def _cache(type, cache, kv_heads, D, page_size):
    """(address, pages) of a cache whose pages have that layout's size."""
    pages, token = cache.shape[0], _CACHE_TOKEN.get(type)
    page = (token[0] * D + token[1]) // 8 * kv_heads * page_size if token else 0
    if cache.numel() != pages * page and token:
        raise ValueError(f"qfp4: a page of this cache has {page} bytes, got {tuple(cache.shape)}")
    return _at(cache, _U8), pages


def kv_cache_write(type, K, V, slots, cache, page_size, gs_k=None, gs_v=None, stream=None) -> None:
    """Quantises K and V [T, kv_heads, head_dim] (BF16; heads of a projection's
    output, or whole) into the slots (int32 [T], negative: skipped) of the cache
    [pages, ...] (uint8, kv_cache_page_bytes per page)."""
    T, H, D = K.shape
    k, ldk = _rows(K, H * D)
    v, ldv = _rows(V, H * D, (T, H, D))
    c, pages = _cache(type, cache, H, D, page_size)
    _call("qfp4_kv_cache_write", type, k, ldk, v, ldv, T, H, D, _at(slots, _I32, T), _at(gs_k, _F32, 1),
          _at(gs_v, _F32, 1), c, pages, page_size, _stream(stream))


def kv_cache_read(type, cache, page_size, slots, K_out, V_out, gs_k=None, gs_v=None, stream=None) -> None:
    """The tokens at these slots in BF16, K_out and V_out [T, kv_heads, head_dim]
    (either may be None); a negative slot gives zeros."""
    T, H, D = (V_out if K_out is None else K_out).shape
    k, ldk = _rows(K_out, H * D, (T, H, D))
    v, ldv = _rows(V_out, H * D, (T, H, D))
    c, pages = _cache(type, cache, H, D, page_size)
    _call("qfp4_kv_cache_read", type, c, pages, page_size, H, D, _at(slots, _I32, T), T, _at(gs_k, _F32, 1),
          _at(gs_v, _F32, 1), k, ldk, v, ldv, _stream(stream))


def qk_norm_rope_cache(QKV, q_heads, kv_heads, Q_out, type, cache, page_size, slots, q_weight=None, k_weight=None,
                       cos_sin=None, positions=None, gs_k=None, gs_v=None, eps=1e-6, interleaved=False,
                       stream=None) -> None:
    """qk_norm_rope with the keys and the value heads behind them quantised
    straight into the cache."""
    (T, width), D = QKV.shape, Q_out.shape[2]
    args = _head_args(QKV, T, width, q_heads, kv_heads, D, kv_heads, q_weight, k_weight, cos_sin, positions, eps, interleaved)
    q, ldq = _rows(Q_out, q_heads * D, (T, q_heads, D))
    c, pages = _cache(type, cache, kv_heads, D, page_size)
    _call("qfp4_qk_norm_rope_cache", *args, q, ldq, type, c, pages, page_size, _at(slots, _I32, T),
          _at(gs_k, _F32, 1), _at(gs_v, _F32, 1), _stream(stream))


def attention_decode_workspace_bytes(B: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(load().qfp4_attention_decode_workspace_bytes(B, q_heads, kv_heads, head_dim))


def attention_decode(type, Q, cache, page_size, page_table, lengths, scale, O, workspace, gs_k=None, gs_v=None,
                     kv_heads=None, lse=None, window=0, stream=None) -> None:
    """Attention of one new token per sequence, Q and O [B, q_heads, head_dim],
    over the paged cache [pages, kv_heads, ...] (kv_heads: where the cache has
    another shape); page_table int32 [B, max_pages], lengths int32 [B].  The
    workspace is zeroed once, before its first use."""
    B, H, D = Q.shape
    heads = cache.shape[1] if kv_heads is None else kv_heads
    q, ldq = _rows(Q, H * D)
    c, pages = _cache(type, cache, heads, D, page_size)
    rows, max_pages = page_table.shape
    if rows != B:
        raise ValueError(f"qfp4: page_table has {rows} rows for {B} sequences")
    _call("qfp4_attention_decode", type, q, ldq, B, H, heads, D, c, pages, page_size, _at(page_table, _I32),
          max_pages, _at(lengths, _I32, B), window, scale, _at(gs_k, _F32, 1), _at(gs_v, _F32, 1),
          _at(O, _BF16, B * H * D), _at(lse, _F32, B * H), *_space(workspace), _stream(stream))
