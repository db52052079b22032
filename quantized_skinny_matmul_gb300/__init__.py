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
