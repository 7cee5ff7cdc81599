"""Python binding for libtg_gemm.so, the GB300 fp16 tiled tensor-core GEMM.

C[i,j] = epi(sum_k A[i,k] B[k,j] + bias[j]), epi = identity or exact-erf GELU:
the GEMM of "TileLang: writing LLM GPU kernels by thinking in tiles"
(sections 2-3) with the GELU(MatMul + Bias) epilogue of "Designing
high-performance GPU kernels with TileLang ..." (section 3).

This module only marshals arguments into the C ABI declared in
include/tg_gemm.h: every step of the computation runs in the library's CUDA
kernels. Functions named tg_* mirror the C entry points one to one (raw
pointers as ints, sizes, a stream handle); ``gemm`` and ``gemm_staged`` accept
torch tensors and pass their pointers and torch's current stream. There is no
CPU path: if the library has not been built, importing this package raises.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtg_gemm.so")

EPI_NONE, EPI_GELU = 0, 1
NOALLOC_SCRATCH_BYTES = 8 * 1024 * 1024  # TG_NOALLOC_SCRATCH_BYTES
KERNEL_AUTO, KERNEL_TILED_TMA, KERNEL_TILED_LSU, KERNEL_SPLITK, KERNEL_TILED_PAIR = 0, 1, 2, 3, 4
W4_INT4, W4_FP4_E2M1 = 0, 1
W4_KERNEL_AUTO, W4_KERNEL_TMEM, W4_KERNEL_REG = 0, 1, 2
FP16, BF16 = 0, 1
KV_E4M3, KV_INT8 = 0, 1
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED_DEVICE, ERR_CUDA, ERR_TIMEOUT, ERR_NO_MEMORY, ERR_BOUNDS = range(7)

# every symbol include/tg_gemm.h declares
EXPORTS = ("tg_gemm", "tg_gemm_ex", "tg_gemm_plan", "tg_gemm_staged", "tg_gemm_splitk_noalloc", "tg_gemm_w4", "tg_gemm_w4_ex",
           "tg_gemm_w4_kernel", "tg_attention_fwd",
           "tg_softmax_rows", "tg_bias_gelu",
           "tg_rope", "tg_kv_append", "tg_kv_read", "tg_attention_kv_workspace", "tg_attention_kv",
           "tg_device_status", "tg_debug_status",
           "tg_set_watchdog_ns",
           "tg_debug_skip_first_arrive", "tg_debug_bounds_limit", "tg_debug_build", "tg_status_string",
           "tg_last_error", "tg_version",
           "tg_ring_bytes", "tg_shutdown")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
                      "(or python tiled_tensor_core_tcgen05_gb300/build.py); there is no fallback path")

_vp, _i64, _int, _u64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint64
_dbl = ctypes.c_double


def bind(path: str) -> ctypes.CDLL:
    """Load a build of the library (this package's, or its debug build
    libtg_gemm_debug.so) with every entry point's C signature set."""
    lib = ctypes.CDLL(path)
    lib.tg_gemm.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp]
    lib.tg_gemm_ex.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _int, _int, _vp]
    lib.tg_gemm_plan.argtypes = [_vp, _vp, _i64, _i64, _i64, ctypes.POINTER(_int), ctypes.POINTER(_int),
                                 ctypes.POINTER(_int)]
    lib.tg_gemm_staged.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _vp]
    lib.tg_gemm_splitk_noalloc.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _int, _vp]
    lib.tg_gemm_w4.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _int, _vp]
    lib.tg_gemm_w4_ex.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _int, _int, _vp]
    lib.tg_gemm_w4_kernel.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _int, _int, _int, _int, _vp]
    lib.tg_attention_fwd.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _int, _vp]
    lib.tg_softmax_rows.argtypes = [_vp, _vp, _i64, _i64, _vp]
    lib.tg_bias_gelu.argtypes = [_vp, _vp, _i64, _i64, _int, _vp]
    cache = [_vp] * 4 + [_i64] * 4 + [_int]   # codes, scales, pages, kv_heads, page, dim, format
    strided = [_vp, _i64, _i64]               # pointer, token stride, head stride
    batch = [_vp, _i64, _vp, _vp, _i64, _i64]  # table, its width, lens, cu, batch, total
    lib.tg_rope.argtypes = strided + strided + [_vp, _i64, _i64, _i64, _vp, _i64, _dbl, _int, _int, _int, _vp]
    lib.tg_kv_append.argtypes = (cache + strided + strided + batch + [_i64, _vp, _i64, _dbl, _int] + strided + strided
                                 + [_i64, _int, _vp])
    lib.tg_kv_read.argtypes = cache + batch + [_vp, _vp, _int, _vp]
    lib.tg_attention_kv_workspace.argtypes = [_i64, _i64, _i64, _int] + [_i64] * 6 + [_int, ctypes.POINTER(_i64)]
    lib.tg_attention_kv.argtypes = (strided + [_vp, _vp] + cache + batch + [_i64, _i64, _i64, _int, _i64, _dbl, _int,
                                                                            _vp, _i64, _vp])
    lib.tg_device_status.argtypes = [_vp, ctypes.POINTER(_int)]
    lib.tg_debug_status.argtypes = [_vp]
    lib.tg_set_watchdog_ns.argtypes = [_u64]
    lib.tg_debug_skip_first_arrive.argtypes = [_int]
    lib.tg_debug_bounds_limit.argtypes = [_i64]
    lib.tg_debug_build.argtypes = []
    lib.tg_status_string.argtypes = [_int]
    lib.tg_status_string.restype = ctypes.c_char_p
    lib.tg_last_error.argtypes = []
    lib.tg_last_error.restype = ctypes.c_char_p
    lib.tg_version.argtypes = []
    lib.tg_ring_bytes.argtypes = [_int]
    lib.tg_ring_bytes.restype = _i64
    lib.tg_shutdown.argtypes = []
    lib.tg_shutdown.restype = None
    for name in ("tg_gemm", "tg_gemm_ex", "tg_gemm_plan", "tg_gemm_staged", "tg_gemm_splitk_noalloc", "tg_gemm_w4", "tg_gemm_w4_ex",
                 "tg_gemm_w4_kernel", "tg_attention_fwd", "tg_softmax_rows", "tg_bias_gelu", "tg_rope", "tg_kv_append", "tg_kv_read", "tg_attention_kv_workspace",
                 "tg_attention_kv", "tg_device_status", "tg_debug_status",
                 "tg_set_watchdog_ns", "tg_debug_skip_first_arrive", "tg_debug_bounds_limit", "tg_debug_build",
                 "tg_version"):
        getattr(lib, name).restype = _int
    return lib


_lib = bind(LIB_PATH)


class TgError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{tg_status_string(status)}: {message}")
        self.status = status


def _check(status: int) -> None:
    if status != OK:
        raise TgError(status, tg_last_error())


def library() -> ctypes.CDLL:
    return _lib


# ---------------------------------------------------------------- raw C ABI

def tg_gemm(A: int, B: int, bias: int | None, C: int, M: int, N: int, K: int, epilogue: int,
            stream: int | None) -> None:
    _check(_lib.tg_gemm(A, B, bias, C, M, N, K, epilogue, stream))


def tg_gemm_ex(A: int, B: int, bias: int | None, C: int, M: int, N: int, K: int, epilogue: int,
               kernel: int, split_k: int, stream: int | None) -> None:
    _check(_lib.tg_gemm_ex(A, B, bias, C, M, N, K, epilogue, kernel, split_k, stream))


def tg_gemm_plan(A: int | None, B: int | None, M: int, N: int, K: int) -> tuple[int, int, int]:
    """(kernel, K slices, aligned copy 0/1) that tg_gemm would take for these operands."""
    k, s, c = _int(), _int(), _int()
    _check(_lib.tg_gemm_plan(A, B, M, N, K, ctypes.byref(k), ctypes.byref(s), ctypes.byref(c)))
    return k.value, s.value, c.value


def tg_gemm_staged(hA, hB, hbias, hC, dA, dB, dbias, dC, M, N, K, epilogue, stream) -> None:
    _check(_lib.tg_gemm_staged(hA, hB, hbias, hC, dA, dB, dbias, dC, M, N, K, epilogue, stream))


def tg_gemm_splitk_noalloc(A: int, B: int, bias: int | None, C: int, M: int, N: int, K: int, epilogue: int,
                           split_k: int, stream: int | None) -> None:
    """The skinny split-K GEMM with its scratch in the library's fixed device
    array, for callers that must not have the library allocate device memory
    (see include/tg_gemm.h for the size limit and the sharing rules)."""
    _check(_lib.tg_gemm_splitk_noalloc(A, B, bias, C, M, N, K, epilogue, split_k, stream))


def tg_gemm_w4(A: int, Bq: int, scales: int, bias: int | None, C: int, M: int, N: int, K: int, epilogue: int,
               split_k: int, stream: int | None) -> None:
    _check(_lib.tg_gemm_w4(A, Bq, scales, bias, C, M, N, K, epilogue, split_k, stream))


def tg_gemm_w4_ex(A: int, Bq: int, scales: int, bias: int | None, C: int, M: int, N: int, K: int, epilogue: int,
                  weight_format: int, split_k: int, stream: int | None) -> None:
    _check(_lib.tg_gemm_w4_ex(A, Bq, scales, bias, C, M, N, K, epilogue, weight_format, split_k, stream))


def tg_gemm_w4_kernel(A: int, Bq: int, scales: int, bias: int | None, C: int, M: int, N: int, K: int,
                      epilogue: int, weight_format: int, kernel: int, split_k: int, stream: int | None) -> None:
    _check(_lib.tg_gemm_w4_kernel(A, Bq, scales, bias, C, M, N, K, epilogue, weight_format, kernel, split_k,
                                  stream))


def tg_attention_fwd(Q: int, K: int, V: int, O: int, B: int, S: int, H: int, D: int, causal: bool,
                     stream: int | None) -> None:
    _check(_lib.tg_attention_fwd(Q, K, V, O, B, S, H, D, 1 if causal else 0, stream))


def attention(Q, K, V, causal: bool = False, out=None, stream=None):
    """O = softmax(Q K^T / sqrt(D)) V for CUDA float16 tensors of shape
    (batch, sequence, heads, 128), contiguous; optional causal mask."""
    import torch
    if Q.dim() != 4 or Q.shape != K.shape or Q.shape != V.shape:
        raise ValueError(f"Q, K, V must share one (B, S, H, D) shape: {tuple(Q.shape)} {tuple(K.shape)} {tuple(V.shape)}")
    B, S, H, D = Q.shape
    if out is None:
        out = torch.empty_like(Q)
    elif out.shape != Q.shape:
        raise ValueError("out has the wrong shape")
    if Q.numel() == 0:
        return out
    tg_attention_fwd(_dev_fp16(Q, "Q"), _dev_fp16(K, "K"), _dev_fp16(V, "V"), _dev_fp16(out, "out"), B, S, H, D,
                     causal, _stream_handle(stream))
    return out


def tg_softmax_rows(X: int, Y: int, M: int, N: int, stream: int | None) -> None:
    _check(_lib.tg_softmax_rows(X, Y, M, N, stream))


def softmax(X, out=None, stream=None):
    """Row softmax of a CUDA float16 matrix (contiguous); ``out`` may be X."""
    import torch
    if X.dim() != 2:
        raise ValueError("X must be a matrix")
    if out is None:
        out = torch.empty_like(X)
    elif out.shape != X.shape:
        raise ValueError("out has the wrong shape")
    if X.numel():
        tg_softmax_rows(_dev_fp16(X, "X"), _dev_fp16(out, "out"), X.shape[0], X.shape[1], _stream_handle(stream))
    return out


def tg_bias_gelu(C: int, bias: int | None, M: int, N: int, epilogue: int, stream: int | None) -> None:
    _check(_lib.tg_bias_gelu(C, bias, M, N, epilogue, stream))


def bias_gelu_(C, bias=None, gelu: bool = True, stream=None):
    """In place C = epi(C + bias) on a CUDA float16 matrix (the unfused epilogue pass)."""
    M, N = C.shape
    tg_bias_gelu(_dev_fp16(C, "C"), _dev_fp16(bias, "bias") if bias is not None else None, M, N,
                 EPI_GELU if gelu else EPI_NONE, _stream_handle(stream))
    return C


def tg_rope(*args) -> None:
    """The C entry point's arguments in its order (include/tg_gemm.h)."""
    _check(_lib.tg_rope(*args))


def tg_kv_append(*args) -> None:
    """The C entry point's arguments in its order (include/tg_gemm.h)."""
    _check(_lib.tg_kv_append(*args))


def tg_kv_read(*args) -> None:
    """The C entry point's arguments in its order (include/tg_gemm.h)."""
    _check(_lib.tg_kv_read(*args))


def tg_attention_kv_workspace(kv_heads: int, page: int, dim: int, fmt: int, heads: int, batch: int, total: int,
                              max_new: int, max_len: int, window: int, dtype: int) -> int:
    """Bytes of workspace that tg_attention_kv needs for these sizes."""
    n = _i64()
    _check(_lib.tg_attention_kv_workspace(kv_heads, page, dim, fmt, heads, batch, total, max_new, max_len, window,
                                          dtype, ctypes.byref(n)))
    return n.value


def tg_attention_kv(*args) -> None:
    """The C entry point's arguments in its order (include/tg_gemm.h)."""
    _check(_lib.tg_attention_kv(*args))


def tg_device_status(stream: int | None) -> tuple[int, int]:
    where = _int(0)
    st = _lib.tg_device_status(stream, ctypes.byref(where))
    return st, where.value


def tg_debug_status(stream: int | None) -> int:
    """Synchronises `stream` and returns (and clears) the kernels' watchdog status."""
    return _lib.tg_debug_status(stream)


def tg_set_watchdog_ns(ns: int) -> None:
    _check(_lib.tg_set_watchdog_ns(ns))


def tg_debug_skip_first_arrive(on: bool) -> None:
    _check(_lib.tg_debug_skip_first_arrive(1 if on else 0))


def tg_debug_bounds_limit(floats: int) -> None:
    """Debug builds: make the device-side bounds checks treat scratch as `floats` long (0: real size)."""
    _check(_lib.tg_debug_bounds_limit(floats))


def tg_debug_build() -> int:
    """1 if the loaded library was compiled with its device-side bounds checks, else 0."""
    return _lib.tg_debug_build()


def tg_status_string(status: int) -> str:
    return _lib.tg_status_string(status).decode()


def tg_last_error() -> str:
    return _lib.tg_last_error().decode()


def tg_version() -> int:
    return _lib.tg_version()


def tg_ring_bytes(kernel: int) -> int:
    return _lib.tg_ring_bytes(kernel)


def tg_shutdown() -> None:
    _lib.tg_shutdown()


# ---------------------------------------------------------------- torch form

def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _dev_fp16(t, name):
    if t.dtype.__repr__() != "torch.float16":
        raise TypeError(f"{name} must be float16, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")
    return t.data_ptr()


def gemm(A, B, bias=None, gelu: bool = False, out=None, kernel: int = KERNEL_AUTO, split_k: int = 0,
         stream=None):
    """C = epi(A @ B + bias) for CUDA float16 tensors A (M, K), B (K, N), bias (N,).

    Runs on ``stream`` (default: torch's current stream) and returns ``out``
    (allocated with torch when not given). Asynchronous like any CUDA op.
    """
    import torch
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[0]:
        raise ValueError(f"shape mismatch {tuple(A.shape)} @ {tuple(B.shape)}")
    M, K = A.shape
    N = B.shape[1]
    if bias is not None and tuple(bias.shape) != (N,):
        raise ValueError(f"bias must have shape ({N},)")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=A.device)
    elif tuple(out.shape) != (M, N):
        raise ValueError("out has the wrong shape")
    pa = _dev_fp16(A, "A") if A.numel() else None
    pb = _dev_fp16(B, "B") if B.numel() else None
    pbias = _dev_fp16(bias, "bias") if bias is not None else None
    pc = _dev_fp16(out, "out") if out.numel() else None
    tg_gemm_ex(pa, pb, pbias, pc, M, N, K, EPI_GELU if gelu else EPI_NONE, kernel, split_k,
               _stream_handle(stream))
    return out


def gemm_w4(A, Bq, scales, bias=None, gelu: bool = False, out=None, split_k: int = 0, stream=None,
            fmt: int = W4_INT4, kernel: int = W4_KERNEL_AUTO):
    """C = epi(A @ W + bias) with 4-bit weights: A (M, K) float16, Bq (N, K/2)
    uint8 (low nibble = even k; two's complement for W4_INT4, E2M1 codes for
    W4_FP4_E2M1), scales (K/128, N) float16, W[k, n] = fp16(value(q[k, n]) *
    scales[k // 128, n]). CUDA tensors, contiguous. `kernel`: W4_KERNEL_AUTO,
    W4_KERNEL_TMEM or W4_KERNEL_REG (M <= 16, one K slice)."""
    import torch
    if A.dim() != 2 or Bq.dim() != 2 or scales.dim() != 2:
        raise ValueError("A, Bq and scales must be matrices")
    M, K = A.shape
    N = Bq.shape[0]
    if 2 * Bq.shape[1] != K:
        raise ValueError(f"Bq must have shape ({N}, {K // 2}), got {tuple(Bq.shape)}")
    if tuple(scales.shape) != (K // 128, N):
        raise ValueError(f"scales must have shape ({K // 128}, {N}), got {tuple(scales.shape)}")
    if Bq.dtype != torch.uint8 or not Bq.is_cuda or not Bq.is_contiguous():
        raise TypeError("Bq must be a contiguous CUDA uint8 tensor")
    if bias is not None and tuple(bias.shape) != (N,):
        raise ValueError(f"bias must have shape ({N},)")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=A.device)
    elif tuple(out.shape) != (M, N):
        raise ValueError("out has the wrong shape")
    tg_gemm_w4_kernel(_dev_fp16(A, "A") if A.numel() else None, Bq.data_ptr() if Bq.numel() else None,
                      _dev_fp16(scales, "scales") if scales.numel() else None,
                      _dev_fp16(bias, "bias") if bias is not None else None,
                      _dev_fp16(out, "out") if out.numel() else None, M, N, K, EPI_GELU if gelu else EPI_NONE, fmt,
                      kernel, split_k, _stream_handle(stream))
    return out


def gemm_staged(hA, hB, hbias, hC, dA, dB, dbias, dC, gelu: bool = False, stream=None) -> None:
    """End-to-end form: host (pinned) tensors hA, hB, hbias are copied into the
    device tensors dA, dB, dbias, the GEMM runs, and the result is copied from dC
    into host hC, all on ``stream``."""
    M, K = hA.shape
    N = hB.shape[1]
    tg_gemm_staged(hA.data_ptr(), hB.data_ptr(), hbias.data_ptr() if hbias is not None else None,
                   hC.data_ptr(), dA.data_ptr(), dB.data_ptr(),
                   dbias.data_ptr() if dbias is not None else None, dC.data_ptr(), M, N, K,
                   EPI_GELU if gelu else EPI_NONE, _stream_handle(stream))


def ring_bytes(block_M: int, block_N: int, block_K: int, num_stages: int, elem_bytes: int = 2) -> int:
    """Shared memory a pipelined tile ring needs: every stage holds one
    block_M x block_K tile of A and one block_K x block_N tile of B
    ("TileLang: you write the dataflow, the compiler owns the schedule",
    section "What a tile costs, exactly")."""
    return num_stages * (block_M * block_K + block_K * block_N) * elem_bytes


# ---------------------------------------------------------------- rotary positions and the 8-bit cache

_fast = None


def _binding():
    """The module of the tensor forms below (csrc/tg_torch.cpp), loaded with torch on first use."""
    global _fast
    if _fast is None:
        import torch  # noqa: F401  its libraries, which the module needs
        try:
            from . import _tg_torch
        except ImportError as e:
            raise ImportError("the module of the tensor forms (_tg_torch.so) cannot be loaded: build again with this torch") from e
        _fast = _tg_torch
    return _fast


def _answer(result):
    """A tensor form's result, or the library's refusal as an error."""
    if type(result) is int:
        _check(result)
    return result


def rope_frequencies(rotary: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     trained: int = 4096, fast: float = 32.0, slow: float = 1.0, device="cuda"):
    """(inv_freq, amplitude) for ``rope`` and ``kv_append``: base ** (-2 j / rotary) radians per
    position for pair j, in float64, scaled for contexts beyond the ``trained`` length:

    "none"    as they are;
    "linear"  every frequency divided by ``factor`` (positions interpolated);
    "ntk"     the base raised to base * factor ** (rotary / (rotary - 2)), which divides the
              slowest frequency by ``factor`` and leaves the fastest;
    "yarn"    pairs that turn more than ``fast`` times within ``trained`` positions kept, those
              that turn less than ``slow`` times divided by ``factor``, a linear ramp over the
              pair index between, and the amplitude 0.1 ln(factor) + 1.
    """
    import math

    import torch
    if rotary < 2 or rotary % 2:
        raise ValueError(f"rotary must be even and at least 2, got {rotary}")
    if scaling not in ("none", "linear", "ntk", "yarn"):
        raise ValueError(f"scaling must be none, linear, ntk or yarn, got {scaling!r}")
    if not factor >= 1.0 or not base > 1.0 or trained < 1:
        raise ValueError("factor must be at least 1, base above 1 and trained at least 1")
    if scaling == "ntk":
        if rotary < 4:
            raise ValueError("ntk scaling needs rotary of at least 4")
        base = base * factor ** (rotary / (rotary - 2))
    freq = base ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)
    amplitude = 1.0
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        def pair(turns):  # the pair that turns so often within the trained length
            return rotary * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rotary - 1)
        keep = 1 - ((torch.arange(rotary // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
        freq = freq * keep + freq / factor * (1 - keep)
        amplitude = 0.1 * math.log(factor) + 1.0
    return freq.to(device), amplitude


_rope_function = None


def _rope_with_gradient(*args):
    """rope as a step of torch's graph: its gradient is the transposed rotation, with the same positions."""
    global _rope_function
    import torch
    if _rope_function is None:
        class Rope(torch.autograd.Function):
            @staticmethod
            def forward(ctx, X, positions, inv_freq, amplitude, layout, backward):
                ctx.save_for_backward(positions, inv_freq)
                ctx.how = amplitude, layout, backward
                return _answer((_fast or _binding()).rope(X, positions, inv_freq, amplitude, layout, backward, None, None))

            @staticmethod
            def backward(ctx, dY):
                positions, inv_freq = ctx.saved_tensors
                amplitude, layout, backward = ctx.how
                # a gradient may be spread over its last dimension (that of a sum is one value)
                dY = dY if dY.stride(-1) == 1 else dY.contiguous()
                return rope(dY, positions, inv_freq, amplitude, layout, not backward), None, None, None, None, None
        _rope_function = Rope
    *args, out, stream = args
    if out is not None:
        raise RuntimeError("rope with out= has no gradient, but X requires one: leave out out=, or call it under torch.no_grad()")
    with torch.cuda.stream(stream):  # None: the current one. The graph takes the gradient on the same stream
        return _rope_function.apply(*args)


def rope(X, positions, inv_freq, amplitude: float = 1.0, layout: int = ROPE_HALF, backward: bool = False, out=None,
         stream=None):
    """Rotary positions on X (tokens, heads, dim), float16 or bfloat16: the first 2 * len(inv_freq)
    values of each head turned in pairs by positions[token] * inv_freq[pair] and multiplied by
    ``amplitude``, the others copied. ``positions`` int32, ``inv_freq`` float64 (see
    ``rope_frequencies``). ``backward``: the transposed map, which takes the output's gradient to
    the input's. ``out`` may be X. X and out may be slices (contiguous in dim). Where X requires a gradient it gets
    one, by the transposed map (not with ``out``)."""
    if getattr(X, "requires_grad", False):
        import torch
        if torch.is_grad_enabled():
            return _rope_with_gradient(X, positions, inv_freq, amplitude, layout, backward, out, stream)
    return _answer((_fast or _binding()).rope(X, positions, inv_freq, amplitude, layout, backward, out, stream))


class KvCache:
    """A paged key/value cache held in 8 bits: codes k, v (pages, kv_heads, page, dim), float8_e4m3fn
    or int8, and one float32 scale for each (page, kv_head) in k_scale, v_scale (pages, kv_heads).
    Pages hold 16, 32, 64 or 128 tokens; dim is 64 or 128. ``KvCache.empty`` allocates one. A cache keeps
    its four tensors for good (for others, make another cache); what they hold, where and in which shape, is
    looked at in every call."""

    __slots__ = ("args",)

    def __init__(self, k, v, k_scale, v_scale):
        object.__setattr__(self, "args", (_fast or _binding()).cache_args(k, v, k_scale, v_scale))

    def __setattr__(self, name, value):
        raise AttributeError(f"a KvCache's {name} cannot be set: make another KvCache")

    def __delattr__(self, name):
        raise AttributeError(f"a KvCache's {name} cannot be deleted")

    def __reduce__(self):  # copies are made from the tensors
        return KvCache, self.args

    k = property(lambda self: self.args[0])
    v = property(lambda self: self.args[1])
    k_scale = property(lambda self: self.args[2])
    v_scale = property(lambda self: self.args[3])
    pages = property(lambda self: self.k.shape[0])
    kv_heads = property(lambda self: self.k.shape[1])
    page = property(lambda self: self.k.shape[2])
    dim = property(lambda self: self.k.shape[3])
    fmt = property(lambda self: KV_INT8 if str(self.k.dtype) == "torch.int8" else KV_E4M3)

    @classmethod
    def empty(cls, pages: int, kv_heads: int, page: int = 64, dim: int = 128, dtype=None, device="cuda"):
        import torch
        dtype = torch.float8_e4m3fn if dtype is None else dtype
        k, v = (torch.zeros((pages, kv_heads, page, dim), dtype=torch.uint8, device=device).view(dtype) for _ in range(2))
        return cls(k, v, *(torch.zeros((pages, kv_heads), device=device) for _ in range(2)))


def kv_append(cache, K, V, table, lens, cu=None, max_new: int = 1, Q=None, inv_freq=None, amplitude: float = 1.0,
              layout: int = ROPE_HALF, out=None, stream=None):
    """Writes new keys and values K, V (total, kv_heads, dim), float16 or bfloat16, into ``cache``,
    quantised on the way: sequence i's rows cu[i] .. cu[i + 1] - 1 (cu None: one row a sequence) go to
    positions lens[i] .. of the pages in its row of ``table``. lens: int32 tokens held before the call;
    max_new: no sequence has more rows (one that does is left out, and ``tg_device_status`` says so). With ``inv_freq`` the keys are rotated first by their
    positions (see ``rope``), and the queries Q (total, heads, dim), if given, too: returns them
    (``out``, which may be Q; rows that no sequence has as they are), else None. No gradient is recorded. The scales and roundings are in include/tg_gemm.h."""
    return _answer((_fast or _binding()).kv_append(cache.args, K, V, table, lens, cu, max_new, Q, inv_freq, amplitude,
                                                   layout, out, stream))


def kv_read(cache, table, first, cu, total: int, dtype=None, out=None, stream=None):
    """(K, V), each (total, kv_heads, dim), of positions first[i] .. first[i] + (cu[i + 1] - cu[i]) - 1 of
    every sequence, packed at rows cu[i] .. (cu None: one row a sequence; rows that no sequence has are
    zeros): code * scale, rounded once to ``dtype`` (float16, the default, or bfloat16). ``out``: a pair of contiguous tensors."""
    import torch
    K, V = out if out is not None else (None, None)
    if dtype is None:
        dtype = K.dtype if K is not None else torch.float16
    if dtype is not torch.float16 and dtype is not torch.bfloat16:
        raise TypeError(f"dtype must be float16 or bfloat16, got {dtype}")
    return _answer((_fast or _binding()).kv_read(cache.args, table, first, cu, total,
                                                 dtype is torch.bfloat16, K, V, stream))


def attention_kv(Q, cache, table, lens, cu=None, max_new: int = 1, max_len: int | None = None, causal: bool = True,
                 window: int = 0, scale: float | None = None, return_lse: bool = False, out=None, stream=None):
    """Attention of the new tokens' queries Q (total, heads, dim), float16 or bfloat16, over ``cache``;
    heads is a multiple of the cache's kv_heads. lens: int32 lengths with the new tokens, which are
    each sequence's last. ``causal``: a token sees positions up to its own, with ``window`` only the
    last so many. max_new and max_len bound the rows and the length of a sequence (max_len None: what
    the table can hold). scale None: 1 / sqrt(dim). Rows that see nothing, and rows that no sequence has,
    give zeros; so do those of a sequence beyond either bound, and ``tg_device_status`` says so. Returns O (total,
    heads, dim), with ``return_lse`` also the float32 log of each row's sum (total, heads). No gradient is
    recorded."""
    return _answer((_fast or _binding()).attention_kv(Q, cache.args, table, lens, cu, max_new, max_len, causal, window,
                                                      scale, return_lse, out, stream))
