"""Python binding of libgq, the GB300 quantized skinny MUL_MAT library.

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``_lib/libgq.so`` (built by ``_build.py``); PyTorch supplies device
memory and streams.  There is no CPU fallback: when the library is missing or
the device is not a GB300, the calls raise.

The functions below carry the names of the C entry points in ``include/gq.h``
and take the same arguments, with torch CUDA tensors (or raw device addresses
as ints) in place of pointers and an optional stream (default: torch's current
stream).  They raise ``GQError`` when the C call returns a non-zero status.
The lower-case helpers at the end allocate the outputs with torch and call them.
"""
from __future__ import annotations

import ctypes
import os
import threading

_PKG = os.path.dirname(os.path.abspath(__file__))
# GQ_LIBRARY may name another build of the same ABI (the GQ_DEBUG build, _lib/libgq_debug.so)
LIB_PATH = os.environ.get("GQ_LIBRARY") or os.path.join(_PKG, "_lib", "libgq.so")

GQ_OK = 0
GQ_ERR_INVALID_ARG = 1
GQ_ERR_MISALIGNED = 2
GQ_ERR_UNSUPPORTED_DEVICE = 3
GQ_ERR_CUDA = 4
GQ_ERR_TIMEOUT = 5
GQ_ERR_NO_MEMORY = 6
GQ_ERR_DEVICE_CHECK = 7

GQ_PATH_AUTO = 0
GQ_PATH_GEMV = 1
GQ_PATH_TC = 2

_lock = threading.Lock()
_lib = None


class GQError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        self.status = status
        super().__init__(f"{where}: status {status}: {message}")


_P = ctypes.c_void_p
_I = ctypes.c_int64
_S = ctypes.c_int

GQ_KV_I8 = 0
GQ_KV_E4M3 = 1


class KVPagesStruct(ctypes.Structure):
    """gq_kv_pages."""
    _fields_ = ([(n, _I) for n in ("kind", "B", "Hkv", "D", "P", "NB", "pages")]
                + [(n, _P) for n in ("k", "v", "ks", "vs", "table", "base", "held", "seen")])


class AttnScoresStruct(ctypes.Structure):
    """gq_attn_scores."""
    _fields_ = [("scale", ctypes.c_float), ("cap", ctypes.c_float), ("window", _I),
                ("slopes", _P), ("first", _P), ("prefix", _P)]


GQ_MX_E2M1 = 0
GQ_MX_E4M3 = 1
GQ_TYPE_F32 = 0
GQ_TYPE_BF16 = 1
GQ_SCORE_SOFTMAX = 0
GQ_SCORE_SIGMOID = 1


class MXRowsStruct(ctypes.Structure):
    """gq_mx_rows."""
    _fields_ = [("rows", _I), ("codes", _P), ("scales", _P)]


class ExpertRowsStruct(ctypes.Structure):
    """gq_expert_rows."""
    _fields_ = [("E", _I), ("R", _I), ("offsets", _P), ("rows", _P)]


class RouterStruct(ctypes.Structure):
    """gq_router."""
    _fields_ = ([(n, _I) for n in ("E", "top_k", "score", "groups", "top_groups", "group_best", "renormalize")]
                + [("factor", ctypes.c_float), ("bias", _P)])


# name -> (argtypes, restype); the signatures of include/gq.h
SIGNATURES = {
    "gq_debug_wait_timeout": ([ctypes.c_uint32, _P], _S),
    "gq_debug_dp4a_probe": ([_I, _P, _I, _P], _S),
    "gq_kv_quantize_i8": ([_P, _P, _P, _I, _I, _P], _S),
    "gq_kv_append_i8": ([_P, _P, _P, _P, _I, _I, _I, _I, _P], _S),
    "gq_attn_decode_i8": ([_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, ctypes.c_float, _P], _S),
    "gq_kv_pages_append": ([ctypes.POINTER(KVPagesStruct), _P, _I, _P, _I, _P, _I, _I, _P], _S),
    "gq_kv_pages_read": ([ctypes.POINTER(KVPagesStruct), _P, _P, _I, _I, _P, _P, _P], _S),
    "gq_attn_pages": ([ctypes.POINTER(KVPagesStruct), ctypes.POINTER(AttnScoresStruct), _P, _I, _P, _I, _I, _I, _P, _I,
                       _P, _P, ctypes.c_float, _P], _S),
    "gq_kv_pages_evict": ([ctypes.POINTER(KVPagesStruct), _P, _I, _I, _I, _P, _P, _P, _P, _P], _S),
    "gq_mx_scale_cols": ([_I], ctypes.c_size_t),
    "gq_quantize_mx": ([_P, _I, _S, _S, _P, _P, _I, _I, _P], _S),
    "gq_dequantize_mx": ([_P, _P, _S, _P, _S, _I, _I, _P], _S),
    "gq_rms_norm_mx": ([_P, _I, _P, _I, _S, _P, ctypes.c_double, _P, _I, _P, _S, _P, _P, _I, _I, _P], _S),
    "gq_mxfp4_repacked_bytes": ([_I, _I, _I], ctypes.c_size_t),
    "gq_repack_mxfp4": ([_P, _P, _P, _I, _I, _I, _P], _S),
    "gq_mul_mat_mxfp4_mx": ([_P, ctypes.POINTER(MXRowsStruct), ctypes.POINTER(ExpertRowsStruct), _P, _I, _S, _I, _I, _P], _S),
    "gq_mul_mat_mxfp4": ([_P, _P, _I, _S, _P, _I, _S, _I, _I, _I, _P], _S),
    "gq_swiglu_mxfp4_mx": ([_P, ctypes.POINTER(MXRowsStruct), ctypes.POINTER(ExpertRowsStruct), _P, _P, _I, _I, _P], _S),
    "gq_route": ([ctypes.POINTER(RouterStruct), _P, _I, _S, _P, _P, _P, _P, _P, _P, _I, _P], _S),
    "gq_experts_combine": ([_P, _I, _P, _P, _I, _P, _I, _S, _P, _I, _S, _I, _I, _P], _S),
    "gq_abi_version": ([], ctypes.c_int),
    "gq_status_string": ([_S], ctypes.c_char_p),
    "gq_last_error_message": ([], ctypes.c_char_p),
    "gq_last_error": ([], _S),
    "gq_q4_0_bytes": ([_I, _I], ctypes.c_size_t),
    "gq_q8_0_bytes": ([_I, _I], ctypes.c_size_t),
    "gq_q4_0_repacked_bytes": ([_I, _I], ctypes.c_size_t),
    "gq_quantize_q4_0": ([_P, _P, _I, _I, _P], _S),
    "gq_quantize_rows_q8_0": ([_P, _P, _I, _I, _P], _S),
    "gq_repack_q4_0": ([_P, _P, _I, _I, _P], _S),
    "gq_mul_mat_q4_0_f32": ([_P, _P, _P, _I, _I, _I, _P], _S),
    "gq_mul_mat_f16_f32": ([_P, _P, _P, _I, _I, _I, _P], _S),
    "gq_mul_mat_q4_0_f32_path": ([_P, _P, _P, _I, _I, _I, _S, _P], _S),
    "gq_mul_mat_f16_f32_path": ([_P, _P, _P, _I, _I, _I, _S, _P], _S),
    "gq_reserve_workspace": ([_I, _I, _I, _P], _S),
    "gq_set_m_threshold": ([_I], _S),
    "gq_set_static_weights": ([ctypes.c_int], _S),
    "gq_get_static_weights": ([], ctypes.c_int),
    "gq_get_m_threshold": ([], _I),
    "gq_debug_block_dots_q4_0": ([_P, _P, _P, _I, _I, _I, _P], _S),
    "gq_mul_mat_q4_0_f32_noalloc": ([_P, _P, _P, _I, _I, _I, _P], _S),
    "gq_mul_mat_q4_0_f32_host": ([_P, _P, _P, _I, _I, _I, _P], _S),
    "gq_set_dispatch_profile": ([ctypes.c_int, _I, _I, _P, _P, _P, _I], _S),
    "gq_clear_dispatch_profiles": ([], _S),
    "gq_choose_path": ([ctypes.c_int, _I, _I, _I], ctypes.c_int),
    "gq_q4_1_bytes": ([_I, _I], ctypes.c_size_t),
    "gq_q4_1_repacked_bytes": ([_I, _I], ctypes.c_size_t),
    "gq_quantize_q4_1": ([_P, _P, _I, _I, _P], _S),
    "gq_repack_q4_1": ([_P, _P, _I, _I, _P], _S),
    "gq_mul_mat_q4_1_f32": ([_P, _P, _P, _I, _I, _I, _P], _S),
    "gq_q5_0_bytes": ([_I, _I], ctypes.c_size_t),
    "gq_q5_0_repacked_bytes": ([_I, _I], ctypes.c_size_t),
    "gq_quantize_q5_0": ([_P, _P, _I, _I, _P], _S),
    "gq_repack_q5_0": ([_P, _P, _I, _I, _P], _S),
    "gq_mul_mat_q5_0_f32": ([_P, _P, _P, _I, _I, _I, _P], _S),
    "gq_q8_0_repacked_bytes": ([_I, _I], ctypes.c_size_t),
    "gq_repack_q8_0": ([_P, _P, _I, _I, _P], _S),
    "gq_mul_mat_q8_0_f32": ([_P, _P, _P, _I, _I, _I, _P], _S),
    "gq_f16_repacked_bytes": ([_I, _I], ctypes.c_size_t),
    "gq_repack_f16": ([_P, _P, _I, _I, _P], _S),
    "gq_mul_mat_f16r_f32": ([_P, _P, _P, _I, _I, _I, _P], _S),
}


def lib() -> ctypes.CDLL:
    """The loaded libgq.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(
                        f"{LIB_PATH} is missing: build it with "
                        "`python -m quantized_skinny_matmul_gb300._build` (nvcc, sm_103a)")
                handle = ctypes.CDLL(LIB_PATH)
                for name, (args, res) in SIGNATURES.items():
                    fn = getattr(handle, name)
                    fn.argtypes = args
                    fn.restype = res
                _lib = handle
    return _lib


def _ptr(t) -> int:
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _torch_stream():
    """A function that gives the handle of torch's current stream (3 us for the Stream object, 0.1 us raw)."""
    import torch
    raw, device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
    if raw is None or device is None:
        return lambda: torch.cuda.current_stream().cuda_stream
    return lambda: raw(device())


def _current_stream() -> int:
    global _current
    if _current is None:
        _current = _torch_stream()
    return _current()


_current = None


def _stream(stream) -> int:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, where: str) -> None:
    if status != GQ_OK:
        msg = lib().gq_last_error_message().decode(errors="replace")
        raise GQError(status, where, msg or lib().gq_status_string(status).decode())


# ---------------------------------------------------------------------------
# the entry points of include/gq.h
# ---------------------------------------------------------------------------
def gq_abi_version() -> int:
    return lib().gq_abi_version()


def gq_last_error() -> int:
    """Status of the device-side sticky word (synchronizes the device)."""
    return lib().gq_last_error()


def gq_q4_0_bytes(N: int, K: int) -> int:
    return lib().gq_q4_0_bytes(N, K)


def gq_q8_0_bytes(M: int, K: int) -> int:
    return lib().gq_q8_0_bytes(M, K)


def gq_q4_0_repacked_bytes(N: int, K: int) -> int:
    return lib().gq_q4_0_repacked_bytes(N, K)


def gq_quantize_q4_0(w, q4_blocks, N: int, K: int, stream=None) -> None:
    _check(lib().gq_quantize_q4_0(_ptr(w), _ptr(q4_blocks), N, K, _stream(stream)), "gq_quantize_q4_0")


def gq_quantize_rows_q8_0(x, q8_blocks, M: int, K: int, stream=None) -> None:
    _check(lib().gq_quantize_rows_q8_0(_ptr(x), _ptr(q8_blocks), M, K, _stream(stream)),
           "gq_quantize_rows_q8_0")


def gq_repack_q4_0(q4_blocks, q4_repacked, N: int, K: int, stream=None) -> None:
    _check(lib().gq_repack_q4_0(_ptr(q4_blocks), _ptr(q4_repacked), N, K, _stream(stream)),
           "gq_repack_q4_0")


def gq_mul_mat_q4_0_f32(q4_repacked, src1, dst, M: int, N: int, K: int, stream=None) -> None:
    _check(lib().gq_mul_mat_q4_0_f32(_ptr(q4_repacked), _ptr(src1), _ptr(dst), M, N, K, _stream(stream)),
           "gq_mul_mat_q4_0_f32")


def gq_mul_mat_f16_f32(src0_f16, src1, dst, M: int, N: int, K: int, stream=None) -> None:
    _check(lib().gq_mul_mat_f16_f32(_ptr(src0_f16), _ptr(src1), _ptr(dst), M, N, K, _stream(stream)),
           "gq_mul_mat_f16_f32")


def gq_mul_mat_q4_0_f32_path(q4_repacked, src1, dst, M: int, N: int, K: int, path: int,
                             stream=None) -> None:
    _check(lib().gq_mul_mat_q4_0_f32_path(_ptr(q4_repacked), _ptr(src1), _ptr(dst), M, N, K, path,
                                          _stream(stream)), "gq_mul_mat_q4_0_f32_path")


def gq_mul_mat_f16_f32_path(src0_f16, src1, dst, M: int, N: int, K: int, path: int,
                            stream=None) -> None:
    _check(lib().gq_mul_mat_f16_f32_path(_ptr(src0_f16), _ptr(src1), _ptr(dst), M, N, K, path,
                                         _stream(stream)), "gq_mul_mat_f16_f32_path")


def gq_reserve_workspace(M: int, N: int, K: int, stream=None) -> None:
    _check(lib().gq_reserve_workspace(M, N, K, _stream(stream)), "gq_reserve_workspace")


def gq_set_m_threshold(t: int) -> None:
    _check(lib().gq_set_m_threshold(t), "gq_set_m_threshold")


def gq_get_m_threshold() -> int:
    return lib().gq_get_m_threshold()


def gq_set_static_weights(enable: bool) -> None:
    _check(lib().gq_set_static_weights(1 if enable else 0), "gq_set_static_weights")


def gq_get_static_weights() -> bool:
    return bool(lib().gq_get_static_weights())


def gq_mul_mat_q4_0_f32_noalloc(q4_repacked, src1, dst, M: int, N: int, K: int, stream=None) -> None:
    """The Q4_0 product with no device allocation (static scratch in the library)."""
    _check(lib().gq_mul_mat_q4_0_f32_noalloc(_ptr(q4_repacked), _ptr(src1), _ptr(dst), M, N, K,
                                             _stream(stream)), "gq_mul_mat_q4_0_f32_noalloc")


def _host_ptr(a) -> int:
    if isinstance(a, int):
        return a
    if getattr(a, "is_cuda", False):
        raise ValueError("expected a host (CPU) tensor")
    if not a.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return a.data_ptr()


def gq_mul_mat_q4_0_f32_host(q4_repacked, src1_host, dst_host, M: int, N: int, K: int, stream=None) -> None:
    """The Q4_0 product from host src1 into host dst (copies enqueued on the stream)."""
    _check(lib().gq_mul_mat_q4_0_f32_host(_ptr(q4_repacked), _host_ptr(src1_host), _host_ptr(dst_host), M, N, K,
                                          _stream(stream)), "gq_mul_mat_q4_0_f32_host")


GQ_KIND_Q4_0 = 0
GQ_KIND_F16 = 1


def gq_set_dispatch_profile(kind: int, N: int, K: int, Ms, t_gemv, t_tc) -> None:
    """Install the benched times of both kernel families at the given M for one shape."""
    n = len(Ms)
    if len(t_gemv) != n or len(t_tc) != n:
        raise ValueError("one time per M and family")
    m_arr = (ctypes.c_int64 * n)(*[int(m) for m in Ms])
    g_arr = (ctypes.c_double * n)(*[float(t) for t in t_gemv])
    t_arr = (ctypes.c_double * n)(*[float(t) for t in t_tc])
    _check(lib().gq_set_dispatch_profile(kind, N, K, ctypes.addressof(m_arr), ctypes.addressof(g_arr),
                                         ctypes.addressof(t_arr), n), "gq_set_dispatch_profile")


def gq_clear_dispatch_profiles() -> None:
    _check(lib().gq_clear_dispatch_profiles(), "gq_clear_dispatch_profiles")


def gq_choose_path(kind: int, N: int, K: int, M: int) -> int:
    return lib().gq_choose_path(kind, N, K, M)


def gq_q4_1_bytes(N: int, K: int) -> int:
    return lib().gq_q4_1_bytes(N, K)


def gq_q4_1_repacked_bytes(N: int, K: int) -> int:
    return lib().gq_q4_1_repacked_bytes(N, K)


def gq_quantize_q4_1(w, q41_blocks, N: int, K: int, stream=None) -> None:
    _check(lib().gq_quantize_q4_1(_ptr(w), _ptr(q41_blocks), N, K, _stream(stream)), "gq_quantize_q4_1")


def gq_repack_q4_1(q41_blocks, q41_repacked, N: int, K: int, stream=None) -> None:
    _check(lib().gq_repack_q4_1(_ptr(q41_blocks), _ptr(q41_repacked), N, K, _stream(stream)), "gq_repack_q4_1")


def gq_mul_mat_q4_1_f32(q41_repacked, src1, dst, M: int, N: int, K: int, stream=None) -> None:
    _check(lib().gq_mul_mat_q4_1_f32(_ptr(q41_repacked), _ptr(src1), _ptr(dst), M, N, K, _stream(stream)),
           "gq_mul_mat_q4_1_f32")


def gq_q5_0_bytes(N: int, K: int) -> int:
    return lib().gq_q5_0_bytes(N, K)


def gq_q5_0_repacked_bytes(N: int, K: int) -> int:
    return lib().gq_q5_0_repacked_bytes(N, K)


def gq_quantize_q5_0(w, q5_blocks, N: int, K: int, stream=None) -> None:
    _check(lib().gq_quantize_q5_0(_ptr(w), _ptr(q5_blocks), N, K, _stream(stream)), "gq_quantize_q5_0")


def gq_repack_q5_0(q5_blocks, q5_repacked, N: int, K: int, stream=None) -> None:
    _check(lib().gq_repack_q5_0(_ptr(q5_blocks), _ptr(q5_repacked), N, K, _stream(stream)), "gq_repack_q5_0")


def gq_mul_mat_q5_0_f32(q5_repacked, src1, dst, M: int, N: int, K: int, stream=None) -> None:
    _check(lib().gq_mul_mat_q5_0_f32(_ptr(q5_repacked), _ptr(src1), _ptr(dst), M, N, K, _stream(stream)),
           "gq_mul_mat_q5_0_f32")


def gq_q8_0_repacked_bytes(N: int, K: int) -> int:
    return lib().gq_q8_0_repacked_bytes(N, K)


def gq_repack_q8_0(q8_blocks, q8_repacked, N: int, K: int, stream=None) -> None:
    _check(lib().gq_repack_q8_0(_ptr(q8_blocks), _ptr(q8_repacked), N, K, _stream(stream)), "gq_repack_q8_0")


def gq_mul_mat_q8_0_f32(q8_repacked, src1, dst, M: int, N: int, K: int, stream=None) -> None:
    _check(lib().gq_mul_mat_q8_0_f32(_ptr(q8_repacked), _ptr(src1), _ptr(dst), M, N, K, _stream(stream)),
           "gq_mul_mat_q8_0_f32")


def gq_f16_repacked_bytes(N: int, K: int) -> int:
    return lib().gq_f16_repacked_bytes(N, K)


def gq_repack_f16(src0_f16, f16_repacked, N: int, K: int, stream=None) -> None:
    _check(lib().gq_repack_f16(_ptr(src0_f16), _ptr(f16_repacked), N, K, _stream(stream)), "gq_repack_f16")


def gq_mul_mat_f16r_f32(f16_repacked, src1, dst, M: int, N: int, K: int, stream=None) -> None:
    _check(lib().gq_mul_mat_f16r_f32(_ptr(f16_repacked), _ptr(src1), _ptr(dst), M, N, K, _stream(stream)),
           "gq_mul_mat_f16r_f32")


def gq_debug_block_dots_q4_0(q4_repacked, q8_blocks, sumi, M: int, N: int, K: int, stream=None) -> None:
    _check(lib().gq_debug_block_dots_q4_0(_ptr(q4_repacked), _ptr(q8_blocks), _ptr(sumi), M, N, K,
                                          _stream(stream)), "gq_debug_block_dots_q4_0")


def gq_debug_wait_timeout(limit: int, stream=None) -> None:
    _check(lib().gq_debug_wait_timeout(limit, _stream(stream)), "gq_debug_wait_timeout")


def gq_debug_dp4a_probe(iters: int, sink, blocks: int, stream=None) -> None:
    _check(lib().gq_debug_dp4a_probe(iters, _ptr(sink), blocks, _stream(stream)), "gq_debug_dp4a_probe")


def gq_kv_quantize_i8(x, q, scale, rows: int, D: int, stream=None) -> None:
    _check(lib().gq_kv_quantize_i8(_ptr(x), _ptr(q), _ptr(scale), rows, D, _stream(stream)), "gq_kv_quantize_i8")


def gq_kv_append_i8(x, q, scale, pos, B: int, Hkv: int, Tcap: int, D: int, stream=None) -> None:
    _check(lib().gq_kv_append_i8(_ptr(x), _ptr(q), _ptr(scale), _ptr(pos), B, Hkv, Tcap, D, _stream(stream)),
           "gq_kv_append_i8")


def gq_attn_decode_i8(q, k, k_scale, v, v_scale, lens, out, B: int, Hq: int, Hkv: int, Tcap: int, D: int,
                      softmax_scale: float, stream=None) -> None:
    _check(lib().gq_attn_decode_i8(_ptr(q), _ptr(k), _ptr(k_scale), _ptr(v), _ptr(v_scale), _ptr(lens), _ptr(out),
                                   B, Hq, Hkv, Tcap, D, float(softmax_scale), _stream(stream)),
           "gq_attn_decode_i8")


def gq_kv_pages_append(cache, k, ldk: int, v, ldv: int, cu, T: int, max_n: int, stream=None) -> None:
    """``cache``: a KVPages; k, v: packed rows (first row's tensor or address) of row strides ldk, ldv."""
    _check(lib().gq_kv_pages_append(_struct(cache), _rows_ptr(k), ldk, _rows_ptr(v), ldv, _ptr(cu), T, max_n,
                                    _stream(stream)), "gq_kv_pages_append")


def gq_kv_pages_read(cache, start, cu, T: int, max_n: int, k, v, stream=None) -> None:
    _check(lib().gq_kv_pages_read(_struct(cache), _ptr(start), _ptr(cu), T, max_n, _ptr(k), _ptr(v), _stream(stream)),
           "gq_kv_pages_read")


def gq_attn_pages(cache, scores, q, ldq: int, cu, T: int, max_n: int, Hq: int, out, ldo: int, weights_in, weights_out,
                  decay: float, stream=None) -> None:
    _check(lib().gq_attn_pages(_struct(cache), _struct(scores), _rows_ptr(q), ldq, _ptr(cu), T, max_n, Hq,
                               _rows_ptr(out), ldo, _ptr(weights_in), _ptr(weights_out), decay, _stream(stream)),
           "gq_attn_pages")


def gq_kv_pages_evict(cache, weights, budget: int, keep_first: int, keep_last: int, table_out, base_out, weights_out,
                      held_out, stream=None) -> None:
    _check(lib().gq_kv_pages_evict(_struct(cache), _ptr(weights), budget, keep_first, keep_last, _ptr(table_out),
                                   _ptr(base_out), _ptr(weights_out), _ptr(held_out), _stream(stream)),
           "gq_kv_pages_evict")


def gq_mx_scale_cols(K: int) -> int:
    return lib().gq_mx_scale_cols(K)


def gq_quantize_mx(x, ldx: int, type: int, kind: int, codes, scales, M: int, K: int, stream=None) -> None:
    _check(lib().gq_quantize_mx(_rows_ptr(x), ldx, type, kind, _ptr(codes), _ptr(scales), M, K, _stream(stream)), "gq_quantize_mx")


def gq_dequantize_mx(codes, scales, kind: int, y, type: int, M: int, K: int, stream=None) -> None:
    _check(lib().gq_dequantize_mx(_ptr(codes), _ptr(scales), kind, _ptr(y), type, M, K, _stream(stream)), "gq_dequantize_mx")


def gq_rms_norm_mx(x, ldx: int, residual, ldr: int, type: int, weight, eps: float, h, ldh: int, y, ytype: int, codes, scales,
                   M: int, K: int, stream=None) -> None:
    _check(lib().gq_rms_norm_mx(_rows_ptr(x), ldx, _rows_ptr(residual), ldr, type, _ptr(weight), eps, _rows_ptr(h), ldh, _ptr(y),
                                ytype, _ptr(codes), _ptr(scales), M, K, _stream(stream)), "gq_rms_norm_mx")


def gq_mxfp4_repacked_bytes(count: int, N: int, K: int) -> int:
    return lib().gq_mxfp4_repacked_bytes(count, N, K)


def gq_repack_mxfp4(codes, scales, repacked, count: int, N: int, K: int, stream=None) -> None:
    _check(lib().gq_repack_mxfp4(_ptr(codes), _ptr(scales), _ptr(repacked), count, N, K, _stream(stream)), "gq_repack_mxfp4")


def gq_mul_mat_mxfp4_mx(repacked, x, plan, dst, ldd: int, type: int, N: int, K: int, stream=None) -> None:
    """``x``: an MXRowsStruct; ``plan``: an ExpertRowsStruct or None; dst: rows of stride ldd."""
    _check(lib().gq_mul_mat_mxfp4_mx(_ptr(repacked), _ref(x), _ref(plan), _rows_ptr(dst), ldd, type, N, K, _stream(stream)),
           "gq_mul_mat_mxfp4_mx")


def gq_mul_mat_mxfp4(repacked, x, ldx: int, xtype: int, dst, ldd: int, type: int, M: int, N: int, K: int, stream=None) -> None:
    _check(lib().gq_mul_mat_mxfp4(_ptr(repacked), _rows_ptr(x), ldx, xtype, _rows_ptr(dst), ldd, type, M, N, K, _stream(stream)),
           "gq_mul_mat_mxfp4")


def gq_swiglu_mxfp4_mx(repacked, x, plan, codes, scales, F: int, K: int, stream=None) -> None:
    _check(lib().gq_swiglu_mxfp4_mx(_ptr(repacked), _ref(x), _ref(plan), _ptr(codes), _ptr(scales), F, K, _stream(stream)),
           "gq_swiglu_mxfp4_mx")


def gq_route(router, logits, ldl: int, type: int, used, ids, weights, offsets, rows, pos, T: int, stream=None) -> None:
    """``router``: a RouterStruct."""
    _check(lib().gq_route(_ref(router), _rows_ptr(logits), ldl, type, _ptr(used), _ptr(ids), _ptr(weights), _ptr(offsets),
                          _ptr(rows), _ptr(pos), T, _stream(stream)), "gq_route")


def gq_experts_combine(y, R: int, pos, weights, top_k: int, residual, ldr: int, rtype: int, out, ldo: int, type: int, T: int,
                       N: int, stream=None) -> None:
    _check(lib().gq_experts_combine(_ptr(y), R, _ptr(pos), _ptr(weights), top_k, _rows_ptr(residual), ldr, rtype, _rows_ptr(out),
                                    ldo, type, T, N, _stream(stream)), "gq_experts_combine")


def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


def _struct(x):
    return x if x is None else x.by_ref


def _rows_ptr(t) -> int:
    """Address of packed rows: each row contiguous, any stride between rows."""
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    return t.data_ptr()


def _f32():
    global _float32
    if _float32 is None:
        import torch
        _float32 = torch.float32
    return _float32


_float32 = None


def _lengths(cu, n: int, name: str = "cu") -> int:
    """The address of int32 [n] on the device."""
    if cu.shape != (n,) or not cu.is_cuda or not cu.is_contiguous() or str(cu.dtype) != "torch.int32":
        raise ValueError(f"{name}: expected a contiguous CUDA int32 tensor of {n} values, got {cu.dtype} {tuple(cu.shape)}")
    return cu.data_ptr()


def _page_weights(cache, w) -> int:
    """The address of f32 [B, Hkv, NB] on the device."""
    if (w.shape != (cache.B, cache.Hkv, cache.NB) or w.dtype is not _f32() or not w.is_cuda or not w.is_contiguous()):
        raise ValueError(f"weights: expected a contiguous CUDA float32 tensor of shape "
                         f"{(cache.B, cache.Hkv, cache.NB)}, got {w.dtype} {tuple(w.shape)}")
    return w.data_ptr()


def _packed(x, D: int, name: str):
    """(rows, heads, row stride) of packed f32 rows: [T, heads * D] or [T, heads, D], each row contiguous."""
    shape, stride = x.shape, x.stride()
    if not x.is_cuda:
        raise ValueError(f"{name}: expected a CUDA tensor")
    if x.dtype is not _f32():
        raise ValueError(f"{name}: expected float32, got {x.dtype}")
    if len(shape) == 2:
        heads, rest = divmod(shape[1], D)
        if rest:
            raise ValueError(f"{name}: rows of {shape[1]} values are not a multiple of D = {D}")
        whole = stride[1] == 1 or shape[1] == 1
    elif len(shape) == 3 and shape[2] == D:
        heads = shape[1]
        whole = stride[2] == 1 and (stride[1] == D or heads == 1)
    else:
        raise ValueError(f"{name}: expected shape [T, heads * {D}] or [T, heads, {D}], got {tuple(shape)}")
    if not whole:
        raise ValueError(f"{name}: each row must be contiguous")
    return shape[0], heads, stride[0] if shape[0] > 1 else heads * D


# the tensors of gq_kv_pages (None: any type of one byte)
_PAGES_DTYPES = dict(k=None, v=None, ks="float32", vs="float32", table="int32", base="int32", held="int32", seen="int32")


class KVPages:
    """One layer's 8-bit KV cache in pages (gq_kv_pages): the tensors, kept alive, and their struct.

    k, v: one-byte codes [pages, P, D]; ks, vs: f32 [pages]; table, base: int32 [B, Hkv, NB];
    held, seen: int32 [B], the tokens held and the next position before the step.  Each may be
    assigned another tensor of the same shape and type (what was captured into a graph keeps the
    old one's address).
    """

    def __init__(self, kind, k, v, ks, vs, table, base, held, seen):
        pages, P, D = k.shape
        B, Hkv, NB = table.shape
        tensors = dict(k=k, v=v, ks=ks, vs=vs, table=table, base=base, held=held, seen=seen)
        shapes = dict(k=(pages, P, D), v=(pages, P, D), ks=(pages,), vs=(pages,), table=(B, Hkv, NB), base=(B, Hkv, NB),
                      held=(B,), seen=(B,))
        for name, t in tensors.items():
            _shape(t, shapes[name], _PAGES_DTYPES[name], name)
        struct = KVPagesStruct(kind, B, Hkv, D, P, NB, pages, *(_ptr(t) for t in tensors.values()))
        vars(self).update(tensors, kind=kind, B=B, Hkv=Hkv, D=D, P=P, NB=NB, pages=pages, struct=struct,
                          by_ref=ctypes.pointer(struct))

    def __setattr__(self, name, value):
        """Another tensor in the place of one: checked like the first, and its address goes into the struct."""
        if name in _PAGES_DTYPES:
            _shape(value, tuple(getattr(self, name).shape), _PAGES_DTYPES[name], name)
            setattr(self.struct, name, _ptr(value))
        elif name in vars(self):
            raise AttributeError(f"{name}: a cache's kind and sizes are fixed, make another KVPages")
        vars(self)[name] = value

    @classmethod
    def empty(cls, B: int, Hkv: int, D: int, tokens: int, page: int = 32, kind: int = GQ_KV_I8, device="cuda"):
        """A cache with room for `tokens` tokens per sequence, each head owning its pages."""
        import torch
        NB = -(-tokens // page)
        n = B * Hkv * NB
        codes = [torch.zeros((n, page, D), dtype=torch.int8 if kind == GQ_KV_I8 else torch.uint8, device=device)
                 for _ in range(2)]
        scales = [torch.zeros(n, dtype=torch.float32, device=device) for _ in range(2)]
        table = torch.arange(n, dtype=torch.int32, device=device).reshape(B, Hkv, NB)
        ints = [torch.zeros(B, dtype=torch.int32, device=device) for _ in range(2)]
        return cls(kind, *codes, *scales, table, torch.zeros_like(table), *ints)


# the tensors of gq_attn_scores
_SCORES_DTYPES = dict(slopes="float32", first="int32", prefix="int32")


class AttnScores:
    """What attn_pages does to scores (gq_attn_scores); tensors are kept alive here.  Every field may be assigned."""

    def __init__(self, scale: float, cap: float = 0.0, window: int = 0, slopes=None, first=None, prefix=None):
        struct = AttnScoresStruct()
        vars(self).update(struct=struct, by_ref=ctypes.pointer(struct))
        self.scale, self.cap, self.window = scale, cap, window
        self.slopes, self.first, self.prefix = slopes, first, prefix

    def __setattr__(self, name, value):
        if name in ("struct", "by_ref"):
            raise AttributeError(f"{name} cannot be assigned")
        dtype = _SCORES_DTYPES.get(name)
        if dtype and value is not None:
            _shape(value, tuple(value.shape), dtype, name)
        if dtype or name in ("scale", "cap", "window"):
            setattr(self.struct, name, _ptr(value) if dtype else value)
        vars(self)[name] = value


def _shape(t, shape, dtype, name: str) -> None:
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is None and t.element_size() != 1 or dtype is not None and str(t.dtype) != "torch." + dtype:
        raise ValueError(f"{name}: wrong dtype {t.dtype}")


# ---------------------------------------------------------------------------
# allocating helpers (torch tensors in, torch tensors out)
# ---------------------------------------------------------------------------
def quantize_q4_0(w):
    """f32 CUDA tensor [N, K] -> canonical Q4_0 bytes, uint8 [N, K/32, 18]."""
    import torch
    N, K = w.shape
    out = torch.empty((N, K // 32, 18), dtype=torch.uint8, device=w.device)
    gq_quantize_q4_0(w, out, N, K)
    return out


def quantize_rows_q8_0(x):
    import torch
    M, K = x.shape
    out = torch.empty((M, K // 32, 34), dtype=torch.uint8, device=x.device)
    gq_quantize_rows_q8_0(x, out, M, K)
    return out


def repack_q4_0(q4, N: int, K: int):
    import torch
    out = torch.empty(gq_q4_0_repacked_bytes(N, K), dtype=torch.uint8, device=q4.device)
    gq_repack_q4_0(q4, out, N, K)
    return out


def concat_rows_q4_0(repacked, Ns, K: int):
    """Several repacked weight matrices with the same K as one matrix of sum(Ns) rows.

    The repacked layout stores whole 16-row groups one after the other, so when
    every N is a multiple of 16 the concatenated buffers are the repacked layout
    of the stacked matrix: one product then computes [x W1^T | x W2^T | ...]
    (for example Q, K and V, or gate and up, which share their input) with one
    weight stream and one quantized copy of the activations.
    """
    import torch
    if len(repacked) != len(Ns):
        raise ValueError("one N per matrix")
    for r, n in zip(repacked, Ns):
        if n % 16:
            raise ValueError(f"N={n} is not a multiple of 16: row groups would be padded")
        if r.numel() != gq_q4_0_repacked_bytes(n, K):
            raise ValueError(f"a buffer of {r.numel()} bytes is not the repacked layout of N={n}, K={K}")
    return torch.cat([r.reshape(-1) for r in repacked])


def mul_mat_q4_0_f32(q4_repacked, src1, N: int, path: int = GQ_PATH_AUTO, out=None):
    import torch
    M, K = src1.shape
    dst = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=src1.device)
    gq_mul_mat_q4_0_f32_path(q4_repacked, src1, dst, M, N, K, path)
    return dst


def mul_mat_f16_f32(src0_f16, src1, path: int = GQ_PATH_AUTO, out=None):
    import torch
    N, K = src0_f16.shape
    M = src1.shape[0]
    dst = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=src1.device)
    gq_mul_mat_f16_f32_path(src0_f16, src1, dst, M, N, K, path)
    return dst


def repack_f16(src0_f16):
    """F16 CUDA tensor [N, K] -> the 16 x 32 tile layout of gq_repack_f16 (uint8)."""
    import torch
    N, K = src0_f16.shape
    out = torch.empty(gq_f16_repacked_bytes(N, K), dtype=torch.uint8, device=src0_f16.device)
    gq_repack_f16(src0_f16, out, N, K)
    return out


def mul_mat_f16r_f32(f16_repacked, src1, N: int, out=None):
    import torch
    M, K = src1.shape
    dst = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=src1.device)
    gq_mul_mat_f16r_f32(f16_repacked, src1, dst, M, N, K)
    return dst


def repack_q8_0(q8, N: int, K: int):
    """Q8_0 weight blocks (uint8 [N, K/32, 34], e.g. from quantize_rows_q8_0) -> the tile layout."""
    import torch
    out = torch.empty(gq_q8_0_repacked_bytes(N, K), dtype=torch.uint8, device=q8.device)
    gq_repack_q8_0(q8, out, N, K)
    return out


def mul_mat_q8_0_f32(q8_repacked, src1, N: int, out=None):
    import torch
    M, K = src1.shape
    dst = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=src1.device)
    gq_mul_mat_q8_0_f32(q8_repacked, src1, dst, M, N, K)
    return dst


def quantize_q5_0(w):
    """f32 CUDA tensor [N, K] -> Q5_0 bytes, uint8 [N, K/32, 22]."""
    import torch
    N, K = w.shape
    out = torch.empty((N, K // 32, 22), dtype=torch.uint8, device=w.device)
    gq_quantize_q5_0(w, out, N, K)
    return out


def repack_q5_0(q5, N: int, K: int):
    import torch
    out = torch.empty(gq_q5_0_repacked_bytes(N, K), dtype=torch.uint8, device=q5.device)
    gq_repack_q5_0(q5, out, N, K)
    return out


def mul_mat_q5_0_f32(q5_repacked, src1, N: int, out=None):
    import torch
    M, K = src1.shape
    dst = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=src1.device)
    gq_mul_mat_q5_0_f32(q5_repacked, src1, dst, M, N, K)
    return dst


def quantize_q4_1(w):
    """f32 CUDA tensor [N, K] -> Q4_1 bytes, uint8 [N, K/32, 20]."""
    import torch
    N, K = w.shape
    out = torch.empty((N, K // 32, 20), dtype=torch.uint8, device=w.device)
    gq_quantize_q4_1(w, out, N, K)
    return out


def repack_q4_1(q41, N: int, K: int):
    import torch
    out = torch.empty(gq_q4_1_repacked_bytes(N, K), dtype=torch.uint8, device=q41.device)
    gq_repack_q4_1(q41, out, N, K)
    return out


def mul_mat_q4_1_f32(q41_repacked, src1, N: int, out=None):
    import torch
    M, K = src1.shape
    dst = out if out is not None else torch.empty((M, N), dtype=torch.float32, device=src1.device)
    gq_mul_mat_q4_1_f32(q41_repacked, src1, dst, M, N, K)
    return dst


def tune_dispatch(weights, N: int, K: int, kind: int = GQ_KIND_Q4_0,
                  Ms=(1, 2, 4, 8, 16, 32, 64, 128, 256, 512), reps: int = 20, install: bool = True):
    """Bench both kernel families on the current device for one shape and install the profile.

    ``weights`` are the product's weights on the device (Q4_0 repacked, or row-major F16).
    Each M is timed with CUDA events over ``reps`` back-to-back products after a warm-up.
    Returns {"M": [...], "gemv_us": [...], "tc_us": [...]}.
    """
    import torch
    fn = gq_mul_mat_q4_0_f32_path if kind == GQ_KIND_Q4_0 else gq_mul_mat_f16_f32_path
    out = {"M": [], "gemv_us": [], "tc_us": []}
    gen = torch.Generator(device=weights.device).manual_seed(1234)
    for M in Ms:
        x = torch.randn((M, K), generator=gen, device=weights.device, dtype=torch.float32)
        dst = torch.empty((M, N), device=weights.device, dtype=torch.float32)
        times = []
        for path in (GQ_PATH_GEMV, GQ_PATH_TC):
            for _ in range(3):
                fn(weights, x, dst, M, N, K, path)
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            for _ in range(reps):
                fn(weights, x, dst, M, N, K, path)
            end.record()
            end.synchronize()
            times.append(start.elapsed_time(end) * 1e3 / reps)
        out["M"].append(int(M))
        out["gemv_us"].append(times[0])
        out["tc_us"].append(times[1])
    if install:
        gq_set_dispatch_profile(kind, N, K, out["M"], out["gemv_us"], out["tc_us"])
    return out


def kv_quantize_i8(x):
    """f32 CUDA tensor [..., D] -> (int8 codes [..., D], f32 scales [...]), one scale per row of D."""
    import torch
    x = x.contiguous()
    D = x.shape[-1]
    q = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    s = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    gq_kv_quantize_i8(x, q, s, x.numel() // D, D)
    return q, s


def attn_decode_i8(q, k, k_scale, v, v_scale, lens, softmax_scale=None, out=None):
    """Decode attention over an INT8 cache: q f32 [B, Hq, D]; k, v int8 [B, Hkv, Tcap, D];
    scales f32 [B, Hkv, Tcap]; lens int32 [B].  Returns f32 [B, Hq, D]."""
    import torch
    B, Hq, D = q.shape
    Hkv, Tcap = k.shape[1], k.shape[2]
    if softmax_scale is None:
        softmax_scale = D ** -0.5
    if out is None:
        out = torch.empty((B, Hq, D), dtype=torch.float32, device=q.device)
    gq_attn_decode_i8(q, k, k_scale, v, v_scale, lens, out, B, Hq, Hkv, Tcap, D, softmax_scale)
    return out


def kv_pages_append(cache: KVPages, k, v, cu, max_n: int) -> None:
    """Write a step's packed keys and values (f32 [T, Hkv * D] or [T, Hkv, D], rows may be strided)."""
    T, heads, ldk = _packed(k, cache.D, "k")
    Tv, heads_v, ldv = _packed(v, cache.D, "v")
    if T != Tv or heads != cache.Hkv or heads_v != heads:
        raise ValueError(f"expected {cache.Hkv} heads in the rows of k and v, and as many rows in both: got {heads} "
                         f"and {heads_v} heads, {T} and {Tv} rows")
    _check(lib().gq_kv_pages_append(cache.by_ref, k.data_ptr(), ldk, v.data_ptr(), ldv, _lengths(cu, cache.B + 1), T, max_n,
                                    _current_stream()), "gq_kv_pages_append")


def kv_pages_read(cache: KVPages, start, cu, T: int, max_n: int):
    """Slots start[b] .. of each sequence as f32: (k, v), each [T, Hkv, D], packed by cu."""
    import torch
    shape = (T, cache.Hkv, cache.D)
    k, v = (torch.empty(shape, dtype=torch.float32, device=cache.ks.device) for _ in range(2))
    _check(lib().gq_kv_pages_read(cache.by_ref, _lengths(start, cache.B, "start"), _lengths(cu, cache.B + 1), T, max_n,
                                  k.data_ptr(), v.data_ptr(), _current_stream()), "gq_kv_pages_read")
    return k, v


def attn_pages(cache: KVPages, q, cu, max_n: int, scores: AttnScores, weights=None, decay: float = 1.0, out=None):
    """Attention of a step's packed queries (f32 [T, Hq * D] or [T, Hq, D]) over the cache: f32 [T, Hq, D].

    With ``weights`` (f32 [B, Hkv, NB], what each page gathered so far) the result is
    (out, new weights), the new ones being decay * weights + this step's shares.
    """
    T, Hq, ldq = _packed(q, cache.D, "q")
    if scores.slopes is not None and scores.slopes.shape[0] != Hq:
        raise ValueError(f"slopes: expected {Hq} values, got {scores.slopes.shape[0]}")
    for t, name in ((scores.first, "first"), (scores.prefix, "prefix")):
        if t is not None and t.shape[0] != T:
            raise ValueError(f"{name}: expected {T} values, got {t.shape[0]}")
    if out is None:
        import torch
        out, ldo = torch.empty((T, Hq, cache.D), dtype=torch.float32, device=cache.ks.device), Hq * cache.D
    else:
        To, Ho, ldo = _packed(out, cache.D, "out")
        if To != T or Ho != Hq:
            raise ValueError(f"out: expected {T} rows of {Hq} heads, got {To} and {Ho}")
    new = w_in = w_out = None
    if weights is not None:
        import torch
        w_in, new = _page_weights(cache, weights), torch.empty_like(weights)
        w_out = new.data_ptr()
    _check(lib().gq_attn_pages(cache.by_ref, scores.by_ref, q.data_ptr(), ldq, _lengths(cu, cache.B + 1), T, max_n, Hq,
                               out.data_ptr(), ldo, w_in, w_out, decay, _current_stream()), "gq_attn_pages")
    return out if weights is None else (out, new)


def kv_pages_evict(cache: KVPages, weights, budget: int, keep_first: int = 1, keep_last: int = 1):
    """Drop the pages that gathered least until `budget` are left: (table, base, weights, held), new tensors."""
    w = _page_weights(cache, weights)
    from torch import empty_like
    table, base, new, held = empty_like(cache.table), empty_like(cache.base), empty_like(weights), empty_like(cache.held)
    _check(lib().gq_kv_pages_evict(cache.by_ref, w, budget, keep_first, keep_last, table.data_ptr(), base.data_ptr(),
                                   new.data_ptr(), held.data_ptr(), _current_stream()), "gq_kv_pages_evict")
    return table, base, new, held


# ---------------------------------------------------------------------------
# microscaled formats, routing, experts
# ---------------------------------------------------------------------------
# (a call on few rows takes the GPU some microseconds, so what a call costs on the host counts here: a torch.empty is
# 1.5 us, a launch 2 to 3 us)
def _torch():
    """torch, and its types as gq_type, once."""
    global _th, _types, _float32, _bfloat16, _uint8, _int32
    import torch
    _th, _types = torch, {torch.float32: GQ_TYPE_F32, torch.bfloat16: GQ_TYPE_BF16}
    _float32, _bfloat16, _uint8, _int32 = torch.float32, torch.bfloat16, torch.uint8, torch.int32
    return torch


_th = _types = _bfloat16 = _uint8 = _int32 = None


def _mx_type(dtype, name: str) -> int:
    """gq_type of a torch dtype."""
    if _types is None:
        _torch()
    t = _types.get(dtype)
    if t is None:
        raise ValueError(f"{name}: expected float32 or bfloat16, got {dtype}")
    return t


def _cuda(t, dtype: str, shape, name: str) -> int:
    """The address of a contiguous CUDA tensor of this type and shape."""
    if not t.is_cuda or not t.is_contiguous() or str(t.dtype) != "torch." + dtype or t.shape != shape:
        raise ValueError(f"{name}: expected a contiguous CUDA {dtype} tensor of shape {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _matrix(x, name: str):
    """(rows, columns, row stride, gq_type) of a CUDA matrix whose rows are contiguous."""
    shape = x.shape
    if not x.is_cuda or len(shape) != 2:
        raise ValueError(f"{name}: expected a CUDA matrix, got {tuple(shape)}")
    (M, K), (ld, one) = shape, x.stride()
    if one != 1 and K > 1:
        raise ValueError(f"{name}: each row must be contiguous")
    return M, K, ld if M > 1 else K, _mx_type(x.dtype, name)


class _Fixed:
    """What calls are given pointers and sizes of: its fields stay as they were made."""

    def __setattr__(self, name, value):
        raise AttributeError(f"{type(self).__name__}.{name} cannot be changed; make a new {type(self).__name__}")


class MXRows(_Fixed):
    """Rows in microscaled blocks: codes uint8 [rows, K] (e4m3) or [rows, K / 2] (e2m1), scales uint8 [rows, S]."""

    def __init__(self, codes, scales, kind: int = GQ_MX_E4M3):
        rows, width = codes.shape
        K = width * (2 if kind == GQ_MX_E2M1 else 1)
        c, s = _cuda(codes, "uint8", codes.shape, "codes"), _cuda(scales, "uint8", (rows, gq_mx_scale_cols(K)), "scales")
        self.__dict__.update(kind=kind, rows=rows, K=K, codes_ptr=c, scales_ptr=s, _codes=codes, _scales=scales, _buffer=None, _struct=None)

    @classmethod
    def empty(cls, rows: int, K: int, kind: int = GQ_MX_E4M3, device="cuda"):
        """Room for rows of K values: one tensor that holds the codes, then the scales."""
        if K <= 0 or K % 32 or rows <= 0:
            raise ValueError(f"expected rows of a multiple of 32 values, got {(rows, K)}")
        self = cls.__new__(cls)
        width = K // 2 if kind == GQ_MX_E2M1 else K
        buffer = (_th or _torch()).empty(rows * (width + (K + 511) // 512 * 16), dtype=_uint8, device=device)
        at = buffer.data_ptr()
        self.__dict__.update(kind=kind, rows=rows, K=K, codes_ptr=at, scales_ptr=at + rows * width, _codes=None, _scales=None,
                             _buffer=buffer, _struct=None)
        return self

    @property
    def codes(self):
        if self._codes is None:
            n = self.scales_ptr - self.codes_ptr
            self.__dict__["_codes"] = self._buffer[:n].view(self.rows, n // self.rows)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            self.__dict__["_scales"] = self._buffer[self.scales_ptr - self.codes_ptr:].view(self.rows, -1)
        return self._scales

    @property
    def device(self):
        return (self._codes if self._buffer is None else self._buffer).device

    @property
    def by_ref(self):
        """The gq_mx_rows, for a call."""
        if self._struct is None:
            self.__dict__["_struct"] = ctypes.pointer(MXRowsStruct(self.rows, self.codes_ptr, self.scales_ptr))
        return self._struct


class MXWeights(_Fixed):
    """`count` repacked 4-bit matrices [N, K] (gq_repack_mxfp4)."""

    def __init__(self, data, count: int, N: int, K: int):
        address = _cuda(data, "uint8", (gq_mxfp4_repacked_bytes(count, N, K),), "data")
        self.__dict__.update(address=address, data=data, device=data.device, count=count, N=N, K=K)


class ExpertPlan(_Fixed):
    """Rows sorted by expert (gq_expert_rows): offsets int32 [E + 1], the token of each row, the row of each choice [T, top_k]."""

    def __init__(self, offsets, rows, pos):
        _cuda(offsets, "int32", offsets.shape[:1], "offsets")
        _cuda(rows, "int32", rows.shape[:1], "rows")
        _cuda(pos, "int32", pos.shape, "pos")
        self._set(offsets, rows, pos, offsets.shape[0] - 1, rows.shape[0])

    def _set(self, offsets, rows, pos, E: int, R: int):
        self.__dict__.update(offsets=offsets, rows=rows, pos=pos, E=E, R=R, _gathered=None, _in_order=None)

    def by_ref(self, gather: bool):
        """The gq_expert_rows, for a call: with the rows to gather, or without."""
        if self._gathered is None:
            o, r = self.offsets.data_ptr(), self.rows.data_ptr()
            self.__dict__.update(_gathered=ctypes.pointer(ExpertRowsStruct(self.E, self.R, o, r)),
                                 _in_order=ctypes.pointer(ExpertRowsStruct(self.E, self.R, o, None)))
        return self._gathered if gather else self._in_order


class Router(_Fixed):
    """How tokens choose their experts (gq_router)."""

    def __init__(self, E: int, top_k: int, score: str = "softmax", bias=None, groups: int = 1, top_groups: int = 1,
                 group_best: int = 1, renormalize: bool = True, factor: float = 1.0):
        scores = {"softmax": GQ_SCORE_SOFTMAX, "sigmoid": GQ_SCORE_SIGMOID}
        if score not in scores:
            raise ValueError(f"score: expected softmax or sigmoid, got {score}")
        struct = RouterStruct(E, top_k, scores[score], groups, top_groups, group_best, renormalize, factor,
                              None if bias is None else _cuda(bias, "float32", (E,), "bias"))
        self.__dict__.update(E=E, top_k=top_k, bias=bias, struct=struct, by_ref=ctypes.pointer(struct))


def quantize_mx(x, kind: int = GQ_MX_E4M3) -> MXRows:
    """Rows f32 or bf16 [M, K] in microscaled blocks."""
    M, K, ld, t = _matrix(x, "x")
    out = MXRows.empty(M, K, kind, x.device)
    status = lib().gq_quantize_mx(x.data_ptr(), ld, t, kind, out.codes_ptr, out.scales_ptr, M, K, _current_stream())
    if status:
        _check(status, "gq_quantize_mx")
    return out


def dequantize_mx(rows: MXRows, dtype=None):
    """The values of microscaled rows, f32 (or bf16) [rows, K]."""
    th = _th or _torch()
    dtype = dtype or _float32
    t = _mx_type(dtype, "dtype")
    y = th.empty((rows.rows, rows.K), dtype=dtype, device=rows.device)
    status = lib().gq_dequantize_mx(rows.codes_ptr, rows.scales_ptr, rows.kind, y.data_ptr(), t, rows.rows, rows.K, _current_stream())
    if status:
        _check(status, "gq_dequantize_mx")
    return y


def repack_mxfp4(codes, scales, N: int, K: int) -> MXWeights:
    """e2m1 codes [count * N, K / 2] and scales [count * N, S] as matrices [N, K] for the products."""
    import torch
    rows = codes.shape[0]
    if N <= 0 or rows % N:
        raise ValueError(f"codes: {rows} rows are not a multiple of N = {N}")
    c = _cuda(codes, "uint8", (rows, K // 2), "codes")
    s = _cuda(scales, "uint8", (rows, gq_mx_scale_cols(K)), "scales")
    data = torch.empty(gq_mxfp4_repacked_bytes(rows // N, N, K), dtype=torch.uint8, device=codes.device)
    _check(lib().gq_repack_mxfp4(c, s, data.data_ptr(), rows // N, N, K, _current_stream()), "gq_repack_mxfp4")
    return MXWeights(data, rows // N, N, K)


def _operands(w: MXWeights, x: MXRows, plan, gather: bool, parts: int):
    """(output rows, the plan's struct) of a product, its arguments checked."""
    if x.kind != GQ_MX_E4M3 or x.K != w.K:
        raise ValueError(f"x: expected e4m3 rows of K = {w.K}, got kind {x.kind}, K = {x.K}")
    if w.count != (1 if plan is None else plan.E) * parts:
        raise ValueError(f"weights: expected {(1 if plan is None else plan.E) * parts} matrices, got {w.count}")
    if plan is None:
        if gather:
            raise ValueError("gather: there is no plan")
        return x.rows, None
    return plan.R, plan.by_ref(gather)


def _output(out, rows: int, N: int, dtype, device):
    """(tensor, row stride, gq_type) of an output [rows, N]: `out` if given (of `dtype`, if that is too), else a new one."""
    if out is None:
        dtype = dtype or _f32()
        t = _mx_type(dtype, "dtype")
        return _th.empty((rows, N), dtype=dtype, device=device), N, t
    Ro, No, ld, t = _matrix(out, "out")
    if Ro != rows or No != N:
        raise ValueError(f"out: expected shape {(rows, N)}, got {(Ro, No)}")
    if dtype is not None and dtype != out.dtype:
        raise ValueError(f"out: expected {dtype}, got {out.dtype}")
    return out, ld, t


def mul_mat_mxfp4(w: MXWeights, x, plan: ExpertPlan = None, gather: bool = False, dtype=None, out=None):
    """Rows times 4-bit weights, f32 (or bf16) [rows, N].  x: MXRows, or f32 / bf16 rows (quantized inside).

    With a plan, row r is the product of x's row plan.rows[r] (gather) or r with the weights of its expert;
    rows from plan.offsets[E] on are left as they are.
    """
    if isinstance(x, MXRows):
        R, ref = _operands(w, x, plan, gather, 1)
        out, ldd, otype = _output(out, R, w.N, dtype, w.device)
        status = lib().gq_mul_mat_mxfp4_mx(w.address, x.by_ref, ref, out.data_ptr(), ldd, otype, w.N, w.K, _current_stream())
    else:
        R, K, ldx, xtype = _matrix(x, "x")
        if plan is not None or gather or K != w.K or w.count != 1:
            raise ValueError(f"x: expected rows of K = {w.K} and one matrix without a plan, got K = {K} and {w.count}")
        out, ldd, otype = _output(out, R, w.N, dtype, w.device)
        status = lib().gq_mul_mat_mxfp4(w.address, x.data_ptr(), ldx, xtype, out.data_ptr(), ldd, otype, R, w.N, K, _current_stream())
    if status:
        _check(status, "gq_mul_mat_mxfp4")
    return out


def swiglu_mxfp4(w: MXWeights, x: MXRows, plan: ExpertPlan = None, gather: bool = False) -> MXRows:
    """silu(x Wg^T) * (x Wu^T) in e4m3 blocks; w holds Wg and Wu, each [F, K], one after the other (for each expert)."""
    R, ref = _operands(w, x, plan, gather, 2)
    out = MXRows.empty(R, w.N, GQ_MX_E4M3, w.device)
    status = lib().gq_swiglu_mxfp4_mx(w.address, x.by_ref, ref, out.codes_ptr, out.scales_ptr, w.N, w.K, _current_stream())
    if status:
        _check(status, "gq_swiglu_mxfp4_mx")
    return out


def rms_norm_mx(x, weight, eps: float, residual=None, y_dtype=None):
    """(h, blocks): h = x + residual (x itself without one) and the e4m3 blocks of its norm; with y_dtype (h, blocks, y)."""
    M, K, ldx, t = _matrix(x, "x")
    w = None if weight is None else _cuda(weight, "float32", (K,), "weight")
    device = x.device
    h, y, res, ldr, h_ptr, y_ptr, yt = x, None, None, K, None, None, GQ_TYPE_F32
    if residual is not None:
        Mr, Kr, ldr, tr = _matrix(residual, "residual")
        if Mr != M or Kr != K or tr != t:
            raise ValueError(f"residual: expected {x.dtype} {(M, K)}, got {residual.dtype} {(Mr, Kr)}")
        h, res = _th.empty((M, K), dtype=x.dtype, device=device), residual.data_ptr()
        h_ptr = h.data_ptr()
    if y_dtype is not None:
        yt = _mx_type(y_dtype, "y_dtype")
        y = _th.empty((M, K), dtype=y_dtype, device=device)
        y_ptr = y.data_ptr()
    out = MXRows.empty(M, K, GQ_MX_E4M3, device)
    status = lib().gq_rms_norm_mx(x.data_ptr(), ldx, res, ldr, t, w, eps, h_ptr, K, y_ptr, yt, out.codes_ptr, out.scales_ptr, M, K,
                                  _current_stream())
    if status:
        _check(status, "gq_rms_norm_mx")
    return (h, out) if y is None else (h, out, y)


def route(logits, router: Router, used=None):
    """(ids, weights, plan) of f32 or bf16 logits [T, E]; `used`: int32 [1], tokens from it on are padding."""
    T, E, ldl, t = _matrix(logits, "logits")
    if E != router.E:
        raise ValueError(f"logits: expected {router.E} experts, got {E}")
    k, dev, empty = router.top_k, logits.device, _th.empty
    u = None if used is None else _cuda(used, "int32", (1,), "used")
    ids, pos = empty((T, k), dtype=_int32, device=dev), empty((T, k), dtype=_int32, device=dev)
    rows, offsets = empty(T * k, dtype=_int32, device=dev), empty(E + 1, dtype=_int32, device=dev)
    weights = empty((T, k), dtype=_float32, device=dev)
    status = lib().gq_route(router.by_ref, logits.data_ptr(), ldl, t, u, ids.data_ptr(), weights.data_ptr(), offsets.data_ptr(),
                            rows.data_ptr(), pos.data_ptr(), T, _current_stream())
    if status:
        _check(status, "gq_route")
    plan = ExpertPlan.__new__(ExpertPlan)
    plan._set(offsets, rows, pos, E, T * k)
    return ids, weights, plan


def experts_combine(y, plan: ExpertPlan, weights, residual=None, dtype=None, out=None):
    """residual + the weighted sum of each token's rows of y (f32 [R, N]): f32 (or `dtype`) [T, N]."""
    T, k = plan.pos.shape
    R, N = y.shape
    a, w = _cuda(y, "float32", (plan.R, N), "y"), _cuda(weights, "float32", (T, k), "weights")
    res, ldr, rtype = None, N, GQ_TYPE_F32
    if residual is not None:
        Tr, Nr, ldr, rtype = _matrix(residual, "residual")
        if Tr != T or Nr != N:
            raise ValueError(f"residual: expected shape {(T, N)}, got {(Tr, Nr)}")
        res = residual.data_ptr()
    out, ldo, otype = _output(out, T, N, dtype, y.device)
    status = lib().gq_experts_combine(a, R, plan.pos.data_ptr(), w, k, res, ldr, rtype, out.data_ptr(), ldo, otype, T, N, _current_stream())
    if status:
        _check(status, "gq_experts_combine")
    return out
