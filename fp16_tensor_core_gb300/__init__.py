"""Python binding of libdg (include/dg.h): argument marshalling only.

Every function below has the name of the C entry point it calls and does no
arithmetic of its own: it turns torch tensors (device memory) into pointers
and sizes, calls the library, and raises DgError on a non-zero status.
PyTorch is used only for device memory and streams.  There is no fallback:
if ``_build/libdg.so`` has not been built, every call raises.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import sysconfig
import threading

import torch

__all__ = [
    "DG_OK", "DG_ERR_INVALID_VALUE", "DG_ERR_MISALIGNED", "DG_ERR_UNSUPPORTED",
    "DG_ERR_CUDA", "DG_ERR_TIMEOUT", "DG_BF16", "DG_E4M3", "DG_FP16", "DgError",
    "lib", "library_path", "dg_amax", "dg_amax_pow2", "dg_quantize_e4m3",
    "dg_quantize_e4m3_amax", "dg_fp8_gemm",
    "dg_fp8_gemm_amax", "dg_fp8_gemm_grouped", "dg_fp8_gemm_splitk_static",
    "dg_hgemm", "dg_hgemm_scaled", "dg_fp16_range_scale", "dg_convert_f16",
    "dg_gemm_plan", "dg_init", "dg_sync_status", "dg_set_wait_timeout_us",
    "dg_debug_skip_first_load", "dg_status_string", "dg_version", "dg_release_stream",
    "dg_reload_env", "dg_convert_f16_amax", "dg_convert_f16_amax_pair", "dg_quantize_e4m3_pair",
    "DG_ROPE_HALF", "DG_ROPE_INTERLEAVED", "DG_ROPE_UNSCALED", "DG_ROPE_LINEAR", "DG_ROPE_NTK",
    "DG_ROPE_BY_PARTS", "DgRotary", "DgKvCache", "dg_rope_table", "dg_rope", "dg_kv_append",
    "dg_kv_read", "dg_attn_decode", "dg_attn_decode_scratch",
    "DG_ACT_NONE", "DG_ACT_RELU", "DG_ACT_GELU", "DG_ACT_GELU_TANH", "DG_ACT_SILU", "dg_rmsnorm",
    "dg_rmsnorm_e4m3", "dg_rmsnorm_e4m3_amax", "dg_rmsnorm_grad", "dg_rmsnorm_grad_scratch",
    "dg_activate", "dg_activate_grad", "dg_activate_grad_scratch", "dg_fp8_gemm_fused", "dg_hgemm_fused",
    "EXPORTED_SYMBOLS",
]

DG_OK, DG_ERR_INVALID_VALUE, DG_ERR_MISALIGNED, DG_ERR_UNSUPPORTED, DG_ERR_CUDA, DG_ERR_TIMEOUT = range(6)
DG_BF16, DG_E4M3, DG_FP16 = 0, 1, 2
DG_ROPE_HALF, DG_ROPE_INTERLEAVED = 0, 1
DG_ROPE_UNSCALED, DG_ROPE_LINEAR, DG_ROPE_NTK, DG_ROPE_BY_PARTS = range(4)
DG_ACT_NONE, DG_ACT_RELU, DG_ACT_GELU, DG_ACT_GELU_TANH, DG_ACT_SILU = range(5)

#: Every function include/dg.h declares.
EXPORTED_SYMBOLS = (
    "dg_amax", "dg_amax_pow2", "dg_quantize_e4m3", "dg_quantize_e4m3_amax", "dg_fp8_gemm",
    "dg_fp8_gemm_amax",
    "dg_fp8_gemm_grouped", "dg_fp8_gemm_splitk_static", "dg_hgemm", "dg_hgemm_scaled",
    "dg_fp16_range_scale", "dg_convert_f16", "dg_gemm_plan",
    "dg_init", "dg_sync_status", "dg_set_wait_timeout_us", "dg_debug_skip_first_load",
    "dg_status_string", "dg_version", "dg_release_stream", "dg_reload_env", "dg_convert_f16_amax",
    "dg_convert_f16_amax_pair", "dg_quantize_e4m3_pair",
    "dg_rope_table", "dg_rope", "dg_kv_append", "dg_kv_read", "dg_attn_decode",
    "dg_attn_decode_scratch", "dg_rmsnorm", "dg_rmsnorm_e4m3", "dg_rmsnorm_e4m3_amax",
    "dg_rmsnorm_grad", "dg_rmsnorm_grad_scratch", "dg_activate", "dg_activate_grad",
    "dg_activate_grad_scratch", "dg_fp8_gemm_fused", "dg_hgemm_fused",
)

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_build", "libdg.so")
_NATIVE_PATH = os.path.join(_HERE, "_build", "dg_python" + sysconfig.get_config_var("EXT_SUFFIX"))
_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return _LIB_PATH


class DgError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {dg_status_string(status)} ({status})")


class _Plan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in
                ("path", "block_m", "block_n", "block_k", "stages", "grid", "tiles", "smem_bytes")]


class _Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class _RopeScaling(ctypes.Structure):
    _fields_ = [("base", ctypes.c_double), ("scaling", ctypes.c_int), ("factor", ctypes.c_double),
                ("original_positions", ctypes.c_double), ("slow_rotations", ctypes.c_double),
                ("fast_rotations", ctypes.c_double), ("magnitude", ctypes.c_double)]


class _Rotary(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("positions", ctypes.c_int64),
                ("rotary_dim", ctypes.c_int), ("layout", ctypes.c_int)]


class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("stride", ctypes.c_int64)]


class _Epilogue(ctypes.Structure):
    _fields_ = [("scale_a", ctypes.c_void_p), ("scale_b", ctypes.c_void_p), ("scale_a_rows", ctypes.c_int),
                ("scale_b_rows", ctypes.c_int), ("bias", ctypes.c_void_p), ("act", ctypes.c_int),
                ("residual", ctypes.c_void_p), ("residual_type", ctypes.c_int),
                ("scale_d", ctypes.c_void_p), ("amax_d", ctypes.c_void_p)]


class _KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64), ("kv_heads", ctypes.c_int),
                ("page_size", ctypes.c_int), ("head_dim", ctypes.c_int)]


def lib():
    """The loaded libdg (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise RuntimeError(
                    f"libdg.so not found at {_LIB_PATH}; build it with "
                    "`python -c 'import __graft_entry__ as g; g.build()'`")
            L = ctypes.CDLL(_LIB_PATH)
            vp, i64, st = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
            L.dg_amax.argtypes = [vp, i64, vp, vp, vp]
            L.dg_amax_pow2.argtypes = [vp, i64, vp, vp, vp]
            L.dg_quantize_e4m3.argtypes = [vp, i64, vp, vp, vp]
            L.dg_quantize_e4m3_amax.argtypes = [vp, i64, vp, vp, vp, vp, vp]
            L.dg_fp8_gemm.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, vp, ctypes.c_int, vp]
            L.dg_fp8_gemm_amax.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, vp, ctypes.c_int,
                                           vp, vp]
            L.dg_fp8_gemm_grouped.argtypes = [vp, vp, vp, i64, i64, i64, ctypes.c_int, vp, vp, vp,
                                              vp, ctypes.c_int, vp]
            L.dg_fp8_gemm_splitk_static.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, vp,
                                                     ctypes.c_int, vp, vp]
            L.dg_hgemm.argtypes = [vp, vp, vp, i64, i64, i64, ctypes.c_int, vp]
            L.dg_hgemm_scaled.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, ctypes.c_int, vp]
            L.dg_fp16_range_scale.argtypes = [vp, vp, vp, vp]
            L.dg_convert_f16.argtypes = [vp, i64, vp, vp, vp]
            L.dg_convert_f16_amax.argtypes = [vp, i64, vp, vp, vp, vp]
            L.dg_convert_f16_amax_pair.argtypes = [vp, i64, vp, i64, vp, vp, vp, vp, vp, vp]
            L.dg_quantize_e4m3_pair.argtypes = [vp, i64, vp, i64, vp, vp, vp, vp, vp, vp, vp]
            L.dg_gemm_plan.argtypes = [i64, i64, i64, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                       ctypes.POINTER(_Plan)]
            heads, i32 = ctypes.POINTER(_Heads), ctypes.c_int
            rotary, cache = ctypes.POINTER(_Rotary), ctypes.POINTER(_KvCache)
            L.dg_rope_table.argtypes = [vp, i64, i32, ctypes.POINTER(_RopeScaling), vp]
            L.dg_rope.argtypes = [heads, heads, i64, i32, i32, vp, rotary, i32, i32, vp]
            L.dg_kv_append.argtypes = [heads, heads, i32, heads, heads, i64, vp, rotary, vp, cache,
                                       i32, vp]
            L.dg_kv_read.argtypes = [cache, vp, i64, heads, heads, i32, vp]
            L.dg_attn_decode.argtypes = [heads, heads, vp, i32, i32, i32, cache, vp, i64, i64, vp, vp,
                                         i64, ctypes.c_double, i32, vp, i64, vp]
            L.dg_attn_decode_scratch.argtypes = [i32, i32, i32, i32, i64, i32, ctypes.POINTER(i64)]
            rows, f64 = ctypes.POINTER(_Rows), ctypes.c_double
            norm = [rows, rows, rows, vp, i64, i64, f64, i32]
            L.dg_rmsnorm.argtypes = [*norm, rows, vp]
            L.dg_rmsnorm_e4m3.argtypes = [*norm, vp, vp, vp]
            L.dg_rmsnorm_e4m3_amax.argtypes = [*norm, vp, vp, vp, vp, vp]
            L.dg_rmsnorm_grad.argtypes = [rows, vp, rows, rows, i64, i64, f64, i32, rows, vp, vp, i64, vp]
            L.dg_rmsnorm_grad_scratch.argtypes = [i64, i64, i32, ctypes.POINTER(i64)]
            fused = [vp, vp, vp, i64, i64, i64, ctypes.POINTER(_Epilogue), i32, vp]
            L.dg_fp8_gemm_fused.argtypes = fused
            L.dg_hgemm_fused.argtypes = fused
            L.dg_activate.argtypes = [rows, i32, i32, i64, i64, i32, rows, vp, vp, vp, vp, vp]
            L.dg_activate_grad.argtypes = [rows, rows, vp, vp, i32, i32, i64, i64, i32, rows, vp, vp, i64, vp]
            L.dg_activate_grad_scratch.argtypes = [i64, i64, i32, i32, ctypes.POINTER(i64)]
            L.dg_init.argtypes = []
            L.dg_sync_status.argtypes = [vp]
            L.dg_set_wait_timeout_us.argtypes = [ctypes.c_uint64]
            L.dg_set_wait_timeout_us.restype = None
            L.dg_debug_skip_first_load.argtypes = [ctypes.c_int]
            L.dg_debug_skip_first_load.restype = None
            L.dg_status_string.argtypes = [ctypes.c_int]
            L.dg_status_string.restype = ctypes.c_char_p
            L.dg_version.argtypes = []
            L.dg_release_stream.argtypes = [vp]
            L.dg_reload_env.argtypes = []
            L.dg_reload_env.restype = None
            for name in ("dg_amax", "dg_amax_pow2", "dg_quantize_e4m3", "dg_fp8_gemm", "dg_fp8_gemm_amax", "dg_hgemm",
                         "dg_fp8_gemm_grouped", "dg_fp8_gemm_splitk_static", "dg_gemm_plan", "dg_init",
                         "dg_sync_status", "dg_version", "dg_hgemm_scaled", "dg_fp16_range_scale",
                         "dg_convert_f16", "dg_quantize_e4m3_amax", "dg_release_stream",
                         "dg_convert_f16_amax", "dg_convert_f16_amax_pair",
                         "dg_quantize_e4m3_pair", "dg_rope_table", "dg_rope", "dg_kv_append",
                         "dg_kv_read", "dg_attn_decode", "dg_attn_decode_scratch", "dg_rmsnorm",
                         "dg_rmsnorm_e4m3", "dg_rmsnorm_e4m3_amax", "dg_rmsnorm_grad",
                         "dg_rmsnorm_grad_scratch", "dg_activate", "dg_activate_grad",
                         "dg_activate_grad_scratch", "dg_fp8_gemm_fused", "dg_hgemm_fused"):
                getattr(L, name).restype = st
            _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensor must be in CUDA device memory")
    if not t.is_contiguous():
        raise ValueError("tensor must be contiguous")
    return t.data_ptr()


# The current stream's handle without building a torch.cuda.Stream (which
# takes longer than a launch).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None and _current_device is not None and torch.cuda.is_initialized():
            return _raw_stream(_current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, where: str):
    if rc != DG_OK:
        raise DgError(rc, where)


def dg_status_string(status: int) -> str:
    return lib().dg_status_string(int(status)).decode()


def dg_version() -> int:
    return lib().dg_version()


def dg_init() -> None:
    _check(lib().dg_init(), "dg_init")


def dg_amax(x, amax_out, scale_out=None, stream=None) -> None:
    """amax_out[0] = max |x|; scale_out[0] = amax / 448 (1 if amax == 0)."""
    _check(lib().dg_amax(_ptr(x), x.numel(), _ptr(amax_out), _ptr(scale_out), _stream(stream)),
           "dg_amax")


def dg_amax_pow2(x, amax_out, scale_out, stream=None) -> None:
    """amax_out[0] = max |x|; scale_out[0] = smallest power of two p with 448 p >= amax."""
    _check(lib().dg_amax_pow2(_ptr(x), x.numel(), _ptr(amax_out), _ptr(scale_out), _stream(stream)),
           "dg_amax_pow2")


def dg_quantize_e4m3(x, scale, q, stream=None) -> None:
    """q = E4M3(x / scale[0]) elementwise (uint8 codes)."""
    if q.numel() != x.numel():
        raise ValueError("q must have as many elements as x")
    _check(lib().dg_quantize_e4m3(_ptr(x), x.numel(), _ptr(scale), _ptr(q), _stream(stream)),
           "dg_quantize_e4m3")


def dg_quantize_e4m3_pair(a, b, amax_a, amax_b, scale_a, scale_b, qa, qb, stream=None) -> None:
    """amax, scale and E4M3 codes of both GEMM operands in one call (as
    dg_amax + dg_quantize_e4m3 on each)."""
    _check(lib().dg_quantize_e4m3_pair(_ptr(a), a.numel(), _ptr(b), b.numel(), _ptr(amax_a),
                                       _ptr(amax_b), _ptr(scale_a), _ptr(scale_b), _ptr(qa),
                                       _ptr(qb), _stream(stream)), "dg_quantize_e4m3_pair")


def dg_quantize_e4m3_amax(x, scale, q, amax_out, next_scale_out=None, stream=None) -> None:
    """q = E4M3(x / scale[0]) and amax_out[0] = max |x| in one pass; optionally
    next_scale_out[0] = amax / 448 (delayed scaling)."""
    _check(lib().dg_quantize_e4m3_amax(_ptr(x), x.numel(), _ptr(scale), _ptr(q), _ptr(amax_out),
                                       _ptr(next_scale_out), _stream(stream)),
           "dg_quantize_e4m3_amax")


def dg_fp8_gemm(A, B, D, scale_a, scale_b, scale_d=None, out=DG_BF16, stream=None,
                M=None, N=None, K=None) -> None:
    """D (M x N) = out(scale_a * scale_b * A (M x K, E4M3) @ B (N x K, E4M3)^T)."""
    if M is None:
        M, K = A.shape
        N = B.shape[0]
    _check(lib().dg_fp8_gemm(_ptr(A), _ptr(B), _ptr(D), M, N, K, _ptr(scale_a), _ptr(scale_b),
                             _ptr(scale_d), int(out), _stream(stream)), "dg_fp8_gemm")


def dg_fp8_gemm_amax(A, B, D, scale_a, scale_b, scale_d=None, out=DG_BF16, amax_d=None,
                     stream=None, M=None, N=None, K=None) -> None:
    """dg_fp8_gemm, and amax_d[0] = max |scale_a * scale_b * acc| (delayed output scaling)."""
    if M is None:
        M, K = A.shape
        N = B.shape[0]
    _check(lib().dg_fp8_gemm_amax(_ptr(A), _ptr(B), _ptr(D), M, N, K, _ptr(scale_a), _ptr(scale_b),
                                  _ptr(scale_d), int(out), _ptr(amax_d), _stream(stream)),
           "dg_fp8_gemm_amax")


def dg_fp8_gemm_splitk_static(A, B, D, scale_a, scale_b, scale_d=None, out=DG_BF16,
                              status_out=None, stream=None, M=None, N=None, K=None) -> None:
    """dg_fp8_gemm for M <= 16 on the split-K kernel with the library's static
    workspace (no allocation); kernel error bits are ORed into status_out."""
    if M is None:
        M, K = A.shape
        N = B.shape[0]
    _check(lib().dg_fp8_gemm_splitk_static(_ptr(A), _ptr(B), _ptr(D), M, N, K, _ptr(scale_a),
                                           _ptr(scale_b), _ptr(scale_d), int(out),
                                           _ptr(status_out), _stream(stream)),
           "dg_fp8_gemm_splitk_static")


def dg_fp8_gemm_grouped(A, B, D, group_offsets, scale_a, scale_b, scale_d=None, out=DG_BF16,
                        stream=None, M=None, N=None, K=None, groups=None) -> None:
    """Grouped GEMM: group g computes rows [off[g], off[g+1]) of D from B rows [g*N, g*N + N)."""
    if groups is None:
        groups = group_offsets.numel() - 1
    if M is None:
        M, K = A.shape
        N = D.shape[1]
    _check(lib().dg_fp8_gemm_grouped(_ptr(A), _ptr(B), _ptr(D), M, N, K, int(groups),
                                     _ptr(group_offsets), _ptr(scale_a), _ptr(scale_b),
                                     _ptr(scale_d), int(out), _stream(stream)),
           "dg_fp8_gemm_grouped")


def dg_hgemm(A, B, D, out=DG_FP16, stream=None, M=None, N=None, K=None) -> None:
    """D (M x N) = out(A (M x K, FP16) @ B (N x K, FP16)^T), FP32 accumulation."""
    if M is None:
        M, K = A.shape
        N = B.shape[0]
    _check(lib().dg_hgemm(_ptr(A), _ptr(B), _ptr(D), M, N, K, int(out), _stream(stream)),
           "dg_hgemm")


def dg_hgemm_scaled(A, B, D, scale_a, scale_b, out=DG_BF16, stream=None, M=None, N=None,
                    K=None) -> None:
    """D = out(scale_a * scale_b * A @ B^T), FP16 operands, FP32 accumulation."""
    if M is None:
        M, K = A.shape
        N = B.shape[0]
    _check(lib().dg_hgemm_scaled(_ptr(A), _ptr(B), _ptr(D), M, N, K, _ptr(scale_a),
                                 _ptr(scale_b), int(out), _stream(stream)), "dg_hgemm_scaled")


def dg_fp16_range_scale(amax_a, amax_b, factors, stream=None) -> None:
    """factors[0..3] = scale, sqrt(scale), 1/scale, 1 with
    scale = min(1, 65504 / (amax_a * amax_b)) (FP16 dynamic-range scaling)."""
    _check(lib().dg_fp16_range_scale(_ptr(amax_a), _ptr(amax_b), _ptr(factors),
                                     _stream(stream)), "dg_fp16_range_scale")


def dg_convert_f16(x, out, factor=None, stream=None) -> None:
    """out = fp16_rn(x * factor[0]) elementwise (binary16 bit patterns)."""
    _check(lib().dg_convert_f16(_ptr(x), x.numel(), _ptr(factor), _ptr(out), _stream(stream)),
           "dg_convert_f16")


def dg_convert_f16_amax(x, out, factor, amax_out, stream=None) -> None:
    """out = fp16_rn(x * factor[0]) and amax_out[0] = max |x| in one pass
    (the next call's factors come from dg_fp16_range_scale on such maxima)."""
    _check(lib().dg_convert_f16_amax(_ptr(x), x.numel(), _ptr(factor), _ptr(out), _ptr(amax_out),
                                     _stream(stream)), "dg_convert_f16_amax")


def dg_convert_f16_amax_pair(a, b, out_a, out_b, factor, amax_a, amax_b, stream=None) -> None:
    """dg_convert_f16_amax for both HGEMM operands in one pass (one factor)."""
    _check(lib().dg_convert_f16_amax_pair(_ptr(a), a.numel(), _ptr(b), b.numel(), _ptr(factor),
                                          _ptr(out_a), _ptr(out_b), _ptr(amax_a), _ptr(amax_b),
                                          _stream(stream)), "dg_convert_f16_amax_pair")


# The arguments of the serving calls and of those around a layer's products
# are read natively: see csrc/dg_python.c.
_native = None


def _load_native():
    global _native
    L = lib()
    with _lock:
        if _native is None:
            spec = importlib.util.spec_from_file_location("dg_python", _NATIVE_PATH)
            if spec is None or not os.path.exists(_NATIVE_PATH):
                raise RuntimeError(f"{_NATIVE_PATH} not found; build it with the library "
                                   "(needs gcc and Python's headers)")
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            if _raw_stream is not None and _current_device is not None:
                stream, device = _raw_stream, _current_device
            else:
                stream, device = lambda _: torch.cuda.current_stream().cuda_stream, torch.cuda.current_device
            module.bind(*(ctypes.cast(f, ctypes.c_void_p).value
                          for f in (L.dg_rope, L.dg_kv_append, L.dg_kv_read, L.dg_attn_decode)),
                        torch.bfloat16, torch.float16, torch.int32, torch.float32, stream, device, _check)
            module.bind_layer(*(ctypes.cast(f, ctypes.c_void_p).value
                                for f in (L.dg_rmsnorm, L.dg_rmsnorm_e4m3, L.dg_rmsnorm_e4m3_amax,
                                          L.dg_rmsnorm_grad, L.dg_activate, L.dg_activate_grad,
                                          L.dg_fp8_gemm_fused, L.dg_hgemm_fused)),
                              torch.uint8)
            _native = module
    return _native


class DgRotary:
    """A rotary table (FP32 [positions, rotary_dim / 2, 2], see dg_rope_table)
    with its layout; keeps the tensor alive."""

    def __init__(self, table, layout=DG_ROPE_HALF):
        if table.dtype != torch.float32 or table.dim() != 3 or table.shape[2] != 2:
            raise ValueError("table must be FP32 [positions, rotary_dim / 2, 2]")
        self.table = table
        self.c = _Rotary(_ptr(table), table.shape[0], 2 * table.shape[1], int(layout))
        self.rotary_address = ctypes.addressof(self.c)


class DgKvCache:
    """A paged E4M3 key/value cache: codes k, v uint8 [pages, kv_heads,
    page_size, head_dim] and scales FP32 [pages, kv_heads, page_size]; keeps
    the tensors alive."""

    def __init__(self, k, v, k_scale, v_scale):
        if k.dtype != torch.uint8 or v.dtype != torch.uint8 or k.dim() != 4 or v.shape != k.shape:
            raise ValueError("k and v must be uint8 [pages, kv_heads, page_size, head_dim]")
        for s in (k_scale, v_scale):
            if s.dtype != torch.float32 or s.shape != k.shape[:3]:
                raise ValueError("scales must be FP32 [pages, kv_heads, page_size]")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        pages, self.kv_heads, page_size, self.head_dim = k.shape
        self.c = _KvCache(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), pages, self.kv_heads,
                          page_size, self.head_dim)
        self.cache_address = ctypes.addressof(self.c)


def dg_rope_table(table, base=10000.0, scaling=DG_ROPE_UNSCALED, factor=1.0,
                  original_positions=0.0, slow_rotations=1.0, fast_rotations=32.0, magnitude=1.0,
                  stream=None) -> None:
    """Fill table (FP32 [positions, rotary_dim / 2, 2]) with cosines and sines."""
    if table.dtype != torch.float32 or table.dim() != 3 or table.shape[2] != 2:
        raise ValueError("table must be FP32 [positions, rotary_dim / 2, 2]")
    sc = _RopeScaling(base, int(scaling), factor, original_positions, slow_rotations,
                      fast_rotations, magnitude)
    _check(lib().dg_rope_table(_ptr(table), table.shape[0], 2 * table.shape[1], ctypes.byref(sc),
                               _stream(stream)), "dg_rope_table")


def dg_rope(x, out, positions, rotary, inverse=False, stream=None) -> None:
    """out = x with each head's first rotary_dim elements turned (inverse: back)."""
    (_native or _load_native()).rope(x, out, positions, rotary, inverse, stream)


def dg_kv_append(k, v, slots, cache, positions=None, rotary=None, q=None, q_out=None,
                 stream=None) -> None:
    """Turn (with rotary) and quantise k, v [tokens, kv_heads, head_dim] into the
    cache's slots; q is turned into q_out (given together) in the same launch."""
    (_native or _load_native()).kv_append(k, v, slots, cache, positions, rotary, q, q_out, stream)


def dg_kv_read(cache, slots, k=None, v=None, stream=None) -> None:
    """k[t], v[t] = the cached key and value of slots[t] (code times scale)."""
    if k is not None or v is not None:
        (_native or _load_native()).kv_read(cache, slots, k, v, stream)


def dg_attn_decode_scratch(batch, q_len, q_heads, cache, prefix_len=0, sm_count=0) -> int:
    """Bytes of scratch dg_attn_decode needs for these sizes."""
    n = ctypes.c_int64()
    _check(lib().dg_attn_decode_scratch(batch, q_len, q_heads, cache.head_dim, prefix_len, sm_count,
                                        ctypes.byref(n)), "dg_attn_decode_scratch")
    return n.value


def dg_attn_decode(q, out, cache, page_table, kv_lens, scratch, scale=None, lse=None,
                   prefix_pages=None, prefix_len=None, stream=None) -> None:
    """Attention of q [batch * q_len, q_heads, head_dim] over the cache: own
    tokens by page_table [batch, max_pages] and kv_lens [batch], after a prefix
    that the whole batch shares (prefix_pages and prefix_len, given together)."""
    (_native or _load_native()).attn_decode(q, out, cache, page_table, kv_lens, scratch, scale, lse,
                                            prefix_pages, prefix_len, stream)


def dg_rmsnorm(x, y, weight=None, residual=None, sum=None, eps=1e-6, stream=None) -> None:
    """y = norm(x + residual) * weight on rows [rows, cols]; sum receives x + residual."""
    (_native or _load_native()).rmsnorm(x, y, weight, residual, sum, eps, stream)


def dg_rmsnorm_e4m3(x, q, row_scale, weight=None, residual=None, sum=None, eps=1e-6, stream=None) -> None:
    """dg_rmsnorm with E4M3 codes (uint8) and an FP32 scale per row in place of y."""
    (_native or _load_native()).rmsnorm_e4m3(x, q, row_scale, weight, residual, sum, eps, stream)


def dg_rmsnorm_e4m3_amax(x, scale, q, amax_out, next_scale_out=None, weight=None, residual=None, sum=None,
                         eps=1e-6, stream=None) -> None:
    """dg_rmsnorm with codes E4M3(y / scale[0]); amax_out[0] = max |y| and
    optionally next_scale_out[0] = amax / 448 for the next call (delayed scaling)."""
    (_native or _load_native()).rmsnorm_e4m3_amax(x, scale, q, amax_out, next_scale_out, weight, residual, sum,
                                                  eps, stream)


def dg_rmsnorm_grad_scratch(rows, cols, sm_count=0) -> int:
    """Bytes of scratch dg_rmsnorm_grad needs for dweight."""
    n = ctypes.c_int64()
    _check(lib().dg_rmsnorm_grad_scratch(rows, cols, sm_count, ctypes.byref(n)), "dg_rmsnorm_grad_scratch")
    return n.value


def dg_rmsnorm_grad(s, dy, dx, weight=None, dsum=None, dweight=None, scratch=None, eps=1e-6, stream=None) -> None:
    """dx (of x and residual alike, plus dsum) and FP32 dweight of dg_rmsnorm, from s = x + residual."""
    (_native or _load_native()).rmsnorm_grad(s, dy, dx, weight, dsum, dweight, scratch, eps, stream)


def dg_activate(x, act, y=None, q=None, q_scale=None, x_q=None, x_scale=None, gated=False, stream=None) -> None:
    """act(x), or act(gate) * up of x = [gate, up], as y and/or as E4M3 codes q with a
    scale per row; x_q and x_scale [rows, 1 or 2] receive an 8-bit checkpoint of x."""
    (_native or _load_native()).activate(x, act, y, q, q_scale, x_q, x_scale, gated, stream)


def dg_activate_grad_scratch(rows, cols, gated=False, sm_count=0) -> int:
    """Bytes of scratch dg_activate_grad needs for dbias (cols: of dy)."""
    n = ctypes.c_int64()
    _check(lib().dg_activate_grad_scratch(rows, cols, 1 if gated else 0, sm_count, ctypes.byref(n)),
           "dg_activate_grad_scratch")
    return n.value


def dg_activate_grad(dy, act, dx, x=None, x_q=None, x_scale=None, gated=False, dbias=None, scratch=None,
                     stream=None) -> None:
    """dx of dg_activate from its input x or the checkpoint x_q, x_scale; dbias (FP32) = column sums of dx."""
    (_native or _load_native()).activate_grad(dy, act, dx, x, x_q, x_scale, gated, dbias, scratch, stream)


def dg_fp8_gemm_fused(A, B, D, scale_a, scale_b, bias=None, act=DG_ACT_NONE, residual=None, scale_d=None,
                      amax_d=None, out=DG_BF16, stream=None) -> None:
    """D = out(act(scale_a * scale_b * A @ B^T + bias) + residual) on E4M3 operands
    A [M, K], B [N, K]: scales of one element or of one a row, bias FP32 [N],
    residual BF16 or FP16 [M, N] (may be D)."""
    (_native or _load_native()).fp8_gemm_fused(A, B, D, scale_a, scale_b, bias, act, residual, scale_d, amax_d,
                                               out, stream)


def dg_hgemm_fused(A, B, D, bias=None, act=DG_ACT_NONE, residual=None, scale_a=None, scale_b=None, amax_d=None,
                   out=DG_FP16, stream=None) -> None:
    """dg_fp8_gemm_fused on FP16 operands; scales are optional (both or neither)."""
    (_native or _load_native()).hgemm_fused(A, B, D, scale_a, scale_b, bias, act, residual, None, amax_d, out,
                                            stream)


def dg_gemm_plan(M, N, K, in_dtype=DG_E4M3, out_dtype=DG_BF16, sm_count=0) -> dict:
    """The path and tile the library picks for this shape (host only)."""
    p = _Plan()
    _check(lib().dg_gemm_plan(M, N, K, int(in_dtype), int(out_dtype), int(sm_count),
                              ctypes.byref(p)), "dg_gemm_plan")
    return {f: getattr(p, f) for f, _ in _Plan._fields_}


def dg_sync_status(stream=None) -> int:
    """Synchronise the stream; return (without raising) the status code."""
    return lib().dg_sync_status(_stream(stream))


def dg_set_wait_timeout_us(us: int) -> None:
    lib().dg_set_wait_timeout_us(int(us))


def dg_debug_skip_first_load(enable: bool = True) -> None:
    lib().dg_debug_skip_first_load(1 if enable else 0)


def dg_release_stream(stream=None) -> None:
    """Free the split-K workspace the stream holds (synchronises the stream)."""
    _check(lib().dg_release_stream(_stream(stream)), "dg_release_stream")


def dg_reload_env() -> None:
    """Re-read the DG_* tuning variables (otherwise read once, at first use)."""
    lib().dg_reload_env()
