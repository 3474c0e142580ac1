"""ctypes binding of libqlora_nf4.so (the C ABI in include/qlora_nf4.h).

Argument marshalling only: every function here checks that tensors are
contiguous and on the GPU, turns them into raw pointers and calls the C entry
point of the same name on torch's current stream.  All computation happens in
the library's HIP kernels.  There is no fallback: if the library is missing,
importing this module raises.
"""

from __future__ import annotations

import ctypes
import os
from pathlib import Path

PKG = Path(__file__).resolve().parent
LIB_PATH = Path(os.environ.get("QLORA_NF4_LIB", PKG / "libqlora_nf4.so"))

QLORA_OK = 0
QLORA_ERR_INVALID_ARG = 1
QLORA_ERR_UNSUPPORTED_DTYPE = 2
QLORA_ERR_WORKSPACE_TOO_SMALL = 3
QLORA_ERR_HIP = 4
QLORA_F32 = 0
QLORA_BF16 = 1
QLORA_F16 = 2

EXPORTS = ("qlora_nf4_sizes", "qlora_nf4_quantize", "qlora_dequantize", "qlora_linear_fwd",
           "qlora_linear_bwd", "qlora_nf4_codebook", "qlora_status_string", "qlora_last_error",
           "qlora_time_next_launch", "qlora_adamw_step", "qlora_merge_lora",
           "qlora_quantize_format", "qlora_dequantize_format", "qlora_gemv_format",
           "qlora_linear_fwd_ex", "qlora_linear_bwd_ex", "qlora_linear_fwd_noalloc",
           "qlora_bench_mfma_peak", "qlora_bench_copy", "qlora_bench_wall_clock_khz",
           "qlora_adapters_sizes", "qlora_adapters_plan", "qlora_adapters_fwd", "qlora_adapters_bwd",
           "qlora_distill_fwd", "qlora_distill_bwd", "qlora_logprobs_fwd", "qlora_logprobs_bwd",
           "qlora_dropout_linear_sizes", "qlora_dropout_linear_fwd", "qlora_dropout_linear_bwd",
           "qlora_gated_sizes", "qlora_gated_fwd", "qlora_gated_bwd")

QLORA_KERNEL_NONE = 0
QLORA_KERNEL_FWD_GEMM = 1
QLORA_KERNEL_DX_GEMM = 2
QLORA_KERNEL_GEMV = 3
QLORA_KERNEL_QUANTIZE = 4
QLORA_KERNEL_ADAMW = 5
QLORA_KERNEL_MERGE = 6
QLORA_KERNEL_FORMAT_GEMV = 7
QLORA_FMT_NF4 = 1
QLORA_FMT_INT4 = 2
QLORA_FMT_INT8 = 3
FORMATS = {"nf4": QLORA_FMT_NF4, "int4": QLORA_FMT_INT4, "int8": QLORA_FMT_INT8}
QLORA_ACT_SILU = 1
QLORA_ACT_GELU_TANH = 2
ACTIVATIONS = {"silu": QLORA_ACT_SILU, "gelu_tanh": QLORA_ACT_GELU_TANH}
QLORA_ADAMW_MAX_TENSORS = 8
QLORA_ADAPTERS_MAX = 1024
QLORA_LOGPROBS_MAX_TOP = 256


class QloraError(RuntimeError):
    def __init__(self, status: int, text: str):
        super().__init__(f"status {status}: {text}")
        self.status = status


class qlora_nf4_t(ctypes.Structure):
    _fields_ = [("n_rows", ctypes.c_int64), ("n_cols", ctypes.c_int64),
                ("codes", ctypes.c_void_p), ("absmax_e4m3", ctypes.c_void_p),
                ("dq_scale", ctypes.c_void_p), ("dq_mean", ctypes.c_void_p)]


class qlora_sizes_t(ctypes.Structure):
    _fields_ = [("codes_bytes", ctypes.c_size_t), ("absmax_bytes", ctypes.c_size_t),
                ("scale_bytes", ctypes.c_size_t), ("mean_bytes", ctypes.c_size_t),
                ("quantize_ws_bytes", ctypes.c_size_t), ("fwd_ws_bytes", ctypes.c_size_t),
                ("bwd_ws_bytes", ctypes.c_size_t)]


class qlora_adamw_tensor_t(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("n", ctypes.c_int64)]


class qlora_qtensor_t(ctypes.Structure):
    _fields_ = [("n_rows", ctypes.c_int64), ("n_cols", ctypes.c_int64), ("format", ctypes.c_int32),
                ("codes", ctypes.c_void_p), ("absmax", ctypes.c_void_p)]


class qlora_adapters_t(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("B", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("count", ctypes.c_int32), ("r", ctypes.c_int32)]


class qlora_adapters_sizes_t(ctypes.Structure):
    _fields_ = [("plan_bytes", ctypes.c_size_t), ("fwd_ws_bytes", ctypes.c_size_t),
                ("bwd_ws_bytes", ctypes.c_size_t)]


class qlora_dropout_t(ctypes.Structure):
    _fields_ = [("p", ctypes.c_float), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("step", ctypes.c_void_p)]


class qlora_block_sizes_t(ctypes.Structure):
    _fields_ = [("fwd_ws_bytes", ctypes.c_size_t), ("bwd_ws_bytes", ctypes.c_size_t)]


class qlora_gated_adapters_t(ctypes.Structure):
    _fields_ = [("A_gate", ctypes.c_void_p), ("B_gate", ctypes.c_void_p), ("A_up", ctypes.c_void_p),
                ("B_up", ctypes.c_void_p), ("r", ctypes.c_int32), ("alpha", ctypes.c_float)]


def _load():
    # The library must share torch's HIP runtime: it is handed torch's device
    # pointers, streams and events.  torch ships its own libamdhip64 with the
    # same soname, so loading torch first makes the dynamic loader bind this
    # library to that copy; loading this library first would map a second,
    # separate HIP runtime into the process.
    import torch  # noqa: F401

    if not LIB_PATH.exists():
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python quantized_fine_tuning_amd/build.py` (hipcc, gfx950)")
    lib = ctypes.CDLL(str(LIB_PATH))
    i64, i32, vp, sz, f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
    P = ctypes.POINTER
    lib.qlora_nf4_sizes.argtypes = [i64, i64, i64, i32, P(qlora_sizes_t)]
    lib.qlora_nf4_quantize.argtypes = [vp, i32, i64, i64, P(qlora_nf4_t), vp, sz, vp]
    lib.qlora_dequantize.argtypes = [P(qlora_nf4_t), vp, i32, vp]
    lib.qlora_linear_fwd.argtypes = [P(qlora_nf4_t), vp, i64, vp, vp, i32, f32, vp, i32, vp, vp,
                                     sz, vp]
    lib.qlora_linear_bwd.argtypes = [P(qlora_nf4_t), vp, vp, i64, vp, vp, i32, f32, vp, vp, i32,
                                     vp, vp, vp, sz, vp]
    for name in ("qlora_nf4_sizes", "qlora_nf4_quantize", "qlora_dequantize",
                 "qlora_linear_fwd", "qlora_linear_bwd"):
        getattr(lib, name).restype = i32
    lib.qlora_nf4_codebook.argtypes = [P(ctypes.c_float)]
    lib.qlora_nf4_codebook.restype = None
    lib.qlora_status_string.argtypes = [i32]
    lib.qlora_status_string.restype = ctypes.c_char_p
    lib.qlora_last_error.argtypes = []
    lib.qlora_last_error.restype = ctypes.c_char_p
    lib.qlora_time_next_launch.argtypes = [i32, vp, vp]
    lib.qlora_time_next_launch.restype = i32
    lib.qlora_adamw_step.argtypes = [P(qlora_adamw_tensor_t), i32, i32, f32, f32, f32, f32, f32, i64, vp]
    lib.qlora_adamw_step.restype = i32
    lib.qlora_merge_lora.argtypes = [P(qlora_nf4_t), vp, vp, i32, f32, vp, i32, vp]
    lib.qlora_merge_lora.restype = i32
    lib.qlora_linear_fwd_ex.argtypes = [P(qlora_nf4_t), vp, i64, vp, vp, i32, f32, vp, i32, vp, vp,
                                        sz, i32, vp]
    lib.qlora_linear_bwd_ex.argtypes = [P(qlora_nf4_t), vp, vp, i64, vp, vp, i32, f32, vp, vp, i32,
                                        vp, vp, vp, sz, i32, vp]
    lib.qlora_linear_fwd_ex.restype = i32
    lib.qlora_linear_fwd_noalloc.argtypes = [P(qlora_nf4_t), vp, i64, vp, vp, i32, f32, vp, i32, vp, vp]
    lib.qlora_linear_fwd_noalloc.restype = i32
    lib.qlora_bench_mfma_peak.argtypes = [i64, vp, P(i64), vp]
    lib.qlora_bench_mfma_peak.restype = i32
    lib.qlora_bench_copy.argtypes = [vp, vp, i64, vp]
    lib.qlora_bench_copy.restype = i32
    lib.qlora_bench_wall_clock_khz.argtypes = [P(i32)]
    lib.qlora_bench_wall_clock_khz.restype = i32
    lib.qlora_linear_bwd_ex.restype = i32
    lib.qlora_quantize_format.argtypes = [vp, i32, i64, i64, P(qlora_qtensor_t), vp]
    lib.qlora_dequantize_format.argtypes = [P(qlora_qtensor_t), vp, i32, vp]
    lib.qlora_gemv_format.argtypes = [P(qlora_qtensor_t), vp, i64, vp, i32, vp]
    for name in ("qlora_quantize_format", "qlora_dequantize_format", "qlora_gemv_format"):
        getattr(lib, name).restype = i32
    lib.qlora_adapters_sizes.argtypes = [i64, i64, i64, i32, i32, P(qlora_adapters_sizes_t)]
    lib.qlora_adapters_plan.argtypes = [vp, i64, i32, vp, sz, vp]
    lib.qlora_adapters_fwd.argtypes = [P(qlora_nf4_t), vp, i64, P(qlora_adapters_t), vp, sz, vp, i32, vp, vp, sz, vp]
    lib.qlora_adapters_bwd.argtypes = [P(qlora_nf4_t), vp, vp, i64, P(qlora_adapters_t), vp, sz, vp, vp, i32, vp, vp,
                                       vp, sz, vp]
    lib.qlora_distill_fwd.argtypes = [vp, i32, i64, i64, i64, vp, i32, vp, i32, f32, vp, vp, vp, vp, vp]
    lib.qlora_distill_bwd.argtypes = [vp, i32, i64, i64, i64, vp, i32, vp, i32, f32, vp, vp, vp, vp]
    lib.qlora_logprobs_fwd.argtypes = [vp, i32, i64, i64, i64, vp, f32, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp]
    lib.qlora_logprobs_bwd.argtypes = [vp, i32, i64, i64, i64, vp, f32, vp, vp, vp, vp, vp, vp]
    nf4, drop, gated = P(qlora_nf4_t), P(qlora_dropout_t), P(qlora_gated_adapters_t)
    lib.qlora_dropout_linear_sizes.argtypes = [i64, i64, i64, i32, P(qlora_block_sizes_t)]
    lib.qlora_gated_sizes.argtypes = [i64, i64, i64, i32, P(qlora_block_sizes_t)]
    lib.qlora_dropout_linear_fwd.argtypes = [nf4, vp, i64, vp, vp, i32, f32, drop, vp, i32, vp, vp, sz, vp]
    lib.qlora_dropout_linear_bwd.argtypes = [nf4, vp, vp, i64, vp, vp, i32, f32, drop, vp, vp, i32, vp, vp, vp, sz, vp]
    lib.qlora_gated_fwd.argtypes = [nf4, nf4, vp, i64, gated, i32, drop, vp, vp, vp, vp, vp, sz, vp]
    lib.qlora_gated_bwd.argtypes = [nf4, nf4, vp, vp, vp, vp, i64, gated, i32, drop, vp, vp, i32, vp, vp, vp, vp, vp,
                                    sz, vp]
    for name in ("qlora_adapters_sizes", "qlora_adapters_plan", "qlora_adapters_fwd", "qlora_adapters_bwd",
                 "qlora_distill_fwd", "qlora_distill_bwd", "qlora_logprobs_fwd", "qlora_logprobs_bwd",
                 "qlora_dropout_linear_sizes", "qlora_dropout_linear_fwd", "qlora_dropout_linear_bwd",
                 "qlora_gated_sizes", "qlora_gated_fwd", "qlora_gated_bwd"):
        getattr(lib, name).restype = i32
    return lib


lib = _load()


def _check(status: int):
    if status != QLORA_OK:
        raise QloraError(status, lib.qlora_last_error().decode())


# ---------------------------------------------------------------------------
# torch marshalling
# ---------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def _ptr(t, name: str):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _expect(t, name: str, shape, dtypes):
    """Host-side check of a tensor's shape and dtype before its pointer goes to
    the library (a wrong shape would otherwise become an out-of-bounds device
    access or silently reinterpreted data)."""
    if t is None:
        raise ValueError(f"{name} is None")
    if tuple(t.shape) != tuple(int(x) for x in shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(int(x) for x in shape)}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected one of {[str(d) for d in dtypes]}")


def _expect_numel(t, name: str, n: int, dtype):
    if t is None:
        raise ValueError(f"{name} is None")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.dim() != 1 or t.numel() < n:
        raise ValueError(f"{name}: needs a 1-d tensor of at least {n} elements, got shape {tuple(t.shape)}")


def _bytes(t, name: str) -> int:
    if t is None:
        raise ValueError(f"{name} is None")
    return t.numel() * t.element_size()


def _dtype(t, name: str) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return QLORA_F32
    if t.dtype == torch.bfloat16:
        return QLORA_BF16
    if t.dtype == torch.float16:
        return QLORA_F16  # (accepted by qlora_merge_lora's output only)
    raise ValueError(f"{name}: dtype {t.dtype} is not float32, bfloat16 or float16")


def _stream(stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


class Nf4Tensor:
    """The four device arrays of one quantized weight [N, K] (torch tensors)."""

    def __init__(self, n_rows: int, n_cols: int, codes, absmax_e4m3, dq_scale, dq_mean):
        self.n_rows, self.n_cols = int(n_rows), int(n_cols)
        self.codes, self.absmax_e4m3 = codes, absmax_e4m3
        self.dq_scale, self.dq_mean = dq_scale, dq_mean

    @classmethod
    def empty(cls, n_rows: int, n_cols: int, device="cuda"):
        torch = _torch()
        s = qlora_nf4_sizes(n_rows, n_cols, 0, 1)
        u8 = torch.uint8
        return cls(n_rows, n_cols,
                   torch.empty(s["codes_bytes"], dtype=u8, device=device),
                   torch.empty(s["absmax_bytes"], dtype=u8, device=device),
                   torch.empty(s["scale_bytes"] // 4, dtype=torch.float32, device=device),
                   torch.empty(1, dtype=torch.float32, device=device))

    def c_struct(self) -> qlora_nf4_t:
        torch = _torch()
        nb = self.n_rows * self.n_cols // 64
        _expect_numel(self.codes, "codes", self.n_rows * self.n_cols // 2, torch.uint8)
        _expect_numel(self.absmax_e4m3, "absmax_e4m3", nb, torch.uint8)
        _expect_numel(self.dq_scale, "dq_scale", (nb + 255) // 256, torch.float32)
        _expect_numel(self.dq_mean, "dq_mean", 1, torch.float32)
        return qlora_nf4_t(self.n_rows, self.n_cols, _ptr(self.codes, "codes"),
                           _ptr(self.absmax_e4m3, "absmax_e4m3"), _ptr(self.dq_scale, "dq_scale"),
                           _ptr(self.dq_mean, "dq_mean"))


def _weight_on(W: Nf4Tensor, dev: int) -> qlora_nf4_t:
    torch = _torch()
    n, k = W.n_rows, W.n_cols
    nb = n * k // 64
    return qlora_nf4_t(n, k, _address_1d(W.codes, "codes", 32 * nb, torch.uint8, dev),
                       _address_1d(W.absmax_e4m3, "absmax_e4m3", nb, torch.uint8, dev),
                       _address_1d(W.dq_scale, "dq_scale", (nb + 255) // 256, torch.float32, dev),
                       _address_1d(W.dq_mean, "dq_mean", 1, torch.float32, dev))


def workspace(nbytes: int, device="cuda"):
    torch = _torch()
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------------------
# entry points (same names as the C ABI)
# ---------------------------------------------------------------------------

def qlora_nf4_sizes(N: int, K: int, M_max: int, r: int) -> dict:
    out = qlora_sizes_t()
    _check(lib.qlora_nf4_sizes(N, K, M_max, r, ctypes.byref(out)))
    return {name: int(getattr(out, name)) for name, _ in qlora_sizes_t._fields_}


def qlora_nf4_codebook() -> list:
    buf = (ctypes.c_float * 16)()
    lib.qlora_nf4_codebook(buf)
    return list(buf)


def qlora_nf4_quantize(W, out: Nf4Tensor, ws, stream=None) -> None:
    torch = _torch()
    if W.dim() != 2:
        raise ValueError("W must be [N, K]")
    N, K = W.shape
    _expect(W, "W", (out.n_rows, out.n_cols), (torch.float32, torch.bfloat16))
    st = out.c_struct()
    _check(lib.qlora_nf4_quantize(_ptr(W, "W"), _dtype(W, "W"), N, K, ctypes.byref(st),
                                  _ptr(ws, "ws"), ws.numel() * ws.element_size(),
                                  _stream(stream)))


def qlora_dequantize(q: Nf4Tensor, out, stream=None) -> None:
    torch = _torch()
    _expect(out, "out", (q.n_rows, q.n_cols), (torch.bfloat16, torch.float16))
    st = q.c_struct()
    _check(lib.qlora_dequantize(ctypes.byref(st), _ptr(out, "out"), _dtype(out, "out"),
                                _stream(stream)))


def qlora_linear_fwd(W: Nf4Tensor, X, A, B, r: int, alpha: float, Y, T_save, ws,
                     stream=None) -> None:
    """Forward in the compute format of X (bf16 or fp16: qlora_linear_fwd_ex)."""
    qlora_linear_fwd_ex(W, X, A, B, r, alpha, Y, T_save, ws, _dtype(X, "X"), stream)


def _compute_torch_dtype(compute_dtype: int):
    torch = _torch()
    if compute_dtype == QLORA_BF16:
        return torch.bfloat16
    if compute_dtype == QLORA_F16:
        return torch.float16
    raise ValueError(f"compute_dtype {compute_dtype}: QLORA_BF16 or QLORA_F16")


def _check_fwd(W: Nf4Tensor, X, A, B, r: int, Y, T_save, cdt):
    torch = _torch()
    if X is None or X.dim() != 2:
        raise ValueError("X must be [M, K]")
    M = X.shape[0]
    N, K = W.n_rows, W.n_cols
    _expect(X, "X", (M, K), (cdt,))
    _expect(A, "A", (r, K), (cdt,))
    _expect(B, "B", (N, r), (cdt,))
    _expect(Y, "Y", (M, N), (torch.float32, cdt))
    if T_save is not None:
        _expect(T_save, "T_save", (M, r), (torch.float32,))
    return M


def qlora_linear_fwd_ex(W: Nf4Tensor, X, A, B, r: int, alpha: float, Y, T_save, ws, compute_dtype: int,
                        stream=None) -> None:
    M = _check_fwd(W, X, A, B, r, Y, T_save, _compute_torch_dtype(compute_dtype))
    st = W.c_struct()
    _check(lib.qlora_linear_fwd_ex(ctypes.byref(st), _ptr(X, "X"), M, _ptr(A, "A"), _ptr(B, "B"),
                                   r, float(alpha), _ptr(Y, "Y"), _dtype(Y, "Y"),
                                   _ptr(T_save, "T_save"), _ptr(ws, "ws"),
                                   _bytes(ws, "ws"), compute_dtype, _stream(stream)))


def qlora_linear_fwd_noalloc(W: Nf4Tensor, X, A, B, r: int, alpha: float, Y, T_save=None,
                             stream=None) -> None:
    """The bf16 forward with the library's static scratch instead of a
    workspace (for callers that cannot allocate).  Calls that overlap on one
    GPU race: order them."""
    M = _check_fwd(W, X, A, B, r, Y, T_save, _torch().bfloat16)
    st = W.c_struct()
    _check(lib.qlora_linear_fwd_noalloc(ctypes.byref(st), _ptr(X, "X"), M, _ptr(A, "A"), _ptr(B, "B"),
                                        r, float(alpha), _ptr(Y, "Y"), _dtype(Y, "Y"),
                                        _ptr(T_save, "T_save"), _stream(stream)))


def qlora_linear_bwd(W: Nf4Tensor, X, dY, A, B, r: int, alpha: float, T_saved, dX, dA, dB, ws,
                     stream=None) -> None:
    """Backward in the compute format of X (bf16 or fp16: qlora_linear_bwd_ex)."""
    qlora_linear_bwd_ex(W, X, dY, A, B, r, alpha, T_saved, dX, dA, dB, ws, _dtype(X, "X"), stream)


def qlora_linear_bwd_ex(W: Nf4Tensor, X, dY, A, B, r: int, alpha: float, T_saved, dX, dA, dB, ws,
                        compute_dtype: int, stream=None) -> None:
    torch = _torch()
    cdt = _compute_torch_dtype(compute_dtype)
    if X is None or X.dim() != 2:
        raise ValueError("X must be [M, K]")
    M = X.shape[0]
    N, K = W.n_rows, W.n_cols
    _expect(X, "X", (M, K), (cdt,))
    _expect(dY, "dY", (M, N), (cdt,))
    _expect(A, "A", (r, K), (cdt,))
    _expect(B, "B", (N, r), (cdt,))
    if T_saved is not None:
        _expect(T_saved, "T_saved", (M, r), (torch.float32,))
    _expect(dX, "dX", (M, K), (torch.float32, cdt))
    _expect(dA, "dA", (r, K), (torch.float32,))
    _expect(dB, "dB", (N, r), (torch.float32,))
    st = W.c_struct()
    _check(lib.qlora_linear_bwd_ex(ctypes.byref(st), _ptr(X, "X"), _ptr(dY, "dY"), M, _ptr(A, "A"),
                                   _ptr(B, "B"), r, float(alpha), _ptr(T_saved, "T_saved"),
                                   _ptr(dX, "dX"), _dtype(dX, "dX"), _ptr(dA, "dA"), _ptr(dB, "dB"),
                                   _ptr(ws, "ws"), _bytes(ws, "ws"), compute_dtype,
                                   _stream(stream)))


def qlora_bench_mfma_peak(iters: int, sink, stream=None) -> int:
    """Launches the MFMA reference loop; returns its FLOP count.  sink: 2056
    float32 on the device; sink[2048:].view(int64) receives the shader and
    real-time clock counters of workgroup 0 (start, end, start, end)."""
    torch = _torch()
    _expect_numel(sink, "sink", 2056, torch.float32)
    flop = ctypes.c_int64(0)
    _check(lib.qlora_bench_mfma_peak(int(iters), _ptr(sink, "sink"), ctypes.byref(flop), _stream(stream)))
    return int(flop.value)


def qlora_bench_wall_clock_khz() -> int:
    """Rate of the device's real-time counter, kHz."""
    khz = ctypes.c_int32(0)
    _check(lib.qlora_bench_wall_clock_khz(ctypes.byref(khz)))
    return int(khz.value)


def qlora_bench_copy(src, dst, stream=None) -> None:
    """Streaming copy of src into dst (same number of bytes)."""
    if _bytes(src, "src") != _bytes(dst, "dst"):
        raise ValueError("src and dst sizes differ")
    _check(lib.qlora_bench_copy(_ptr(src, "src"), _ptr(dst, "dst"), _bytes(src, "src"), _stream(stream)))


def qlora_time_next_launch(kernel_id: int, start_event=None, stop_event=None) -> None:
    """Bracket the next launch of `kernel_id` with two torch.cuda.Event objects
    (each must have been recorded once so that its HIP event exists)."""
    s = ctypes.c_void_p(start_event.cuda_event) if start_event is not None else None
    e = ctypes.c_void_p(stop_event.cuda_event) if stop_event is not None else None
    _check(lib.qlora_time_next_launch(kernel_id, s, e))


def qlora_adamw_step(tensors, lr: float, beta1: float, beta2: float, eps: float,
                     weight_decay: float, step: int, stream=None) -> None:
    """One AdamW step on up to QLORA_ADAMW_MAX_TENSORS tensors in one launch.
    tensors: sequence of (param, grad, exp_avg, exp_avg_sq); every param is
    bf16 or every param is fp32; grad and the moments are fp32 of the same
    number of elements; all updated in place."""
    tensors = list(tensors)
    arr = (qlora_adamw_tensor_t * max(1, len(tensors)))()
    dt = None
    torch = _torch()
    for i, (p, g, m, v) in enumerate(tensors):
        d = _dtype(p, f"tensors[{i}].param")
        if d not in (QLORA_BF16, QLORA_F32):
            raise ValueError(f"tensors[{i}].param: bf16 or fp32")
        for t_, nm in ((g, "grad"), (m, "exp_avg"), (v, "exp_avg_sq")):
            if t_.dtype != torch.float32:
                raise ValueError(f"tensors[{i}].{nm}: dtype {t_.dtype}, expected float32")
        if dt is not None and d != dt:
            raise ValueError("every param must have the same dtype")
        dt = d
        n = p.numel()
        if not (g.numel() == m.numel() == v.numel() == n):
            raise ValueError(f"tensors[{i}]: element counts differ")
        arr[i] = qlora_adamw_tensor_t(_ptr(p, "param"), _ptr(g, "grad"), _ptr(m, "exp_avg"),
                                      _ptr(v, "exp_avg_sq"), n)
    _check(lib.qlora_adamw_step(arr, len(tensors), QLORA_BF16 if dt is None else dt, float(lr),
                                float(beta1), float(beta2), float(eps), float(weight_decay),
                                int(step), _stream(stream)))


def qlora_merge_lora(W: Nf4Tensor, A, B, r: int, alpha: float, out, stream=None) -> None:
    """out [N, K] (bf16 or fp16) = Ŵ + (alpha / r)·B·A, rounded once."""
    torch = _torch()
    _expect(A, "A", (r, W.n_cols), (torch.bfloat16,))
    _expect(B, "B", (W.n_rows, r), (torch.bfloat16,))
    _expect(out, "out", (W.n_rows, W.n_cols), (torch.bfloat16, torch.float16))
    st = W.c_struct()
    _check(lib.qlora_merge_lora(ctypes.byref(st), _ptr(A, "A"), _ptr(B, "B"), r, float(alpha),
                                _ptr(out, "out"), _dtype(out, "out"), _stream(stream)))


# The entry points below are called once per layer and token by serving loops,
# so their checks are written for the case that passes: one comparison each,
# the message built only when one fails.

def _launch_stream(stream, dev: int) -> int:
    """The given stream, or torch's current one, as a raw pointer; the tensors'
    device has to be the current one and the stream's."""
    torch = _torch()
    if dev < 0:
        raise ValueError("the tensors must be GPU tensors")
    if torch.cuda.current_device() != dev:
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    on = getattr(stream, "device", None)
    if on is not None and on.index != dev:
        raise ValueError(f"stream is on {on}, the tensors on cuda:{dev}")
    return stream.cuda_stream


def _address(t, name: str, shape, dtypes, dev: int) -> int:
    """data_ptr of a contiguous tensor of this shape and one of these dtypes on
    this device."""
    if t is None or t.shape != shape or t.dtype not in dtypes:
        _expect(t, name, shape, dtypes)
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, " + (f"others on cuda:{dev}" if dev >= 0 else "others on the CPU"))
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _address_1d(t, name: str, n: int, dtype, dev: int) -> int:
    """The same for a 1-d tensor of at least n elements."""
    if t is None or t.dtype != dtype or t.dim() != 1 or t.numel() < n:
        _expect_numel(t, name, n, dtype)
    if t.get_device() != dev or not t.is_contiguous():
        _address(t, name, t.shape, (dtype,), dev)
    return t.data_ptr()


def _scratch(t, name: str, dev: int):
    """(address, bytes) of a workspace or plan buffer."""
    if t is None:
        raise ValueError(f"{name} is None")
    return _address(t, name, t.shape, (t.dtype,), dev), t.numel() * t.element_size()


class AdapterPool:
    """`count` low-rank adapters of one width r: A bf16 [count, r, K], B bf16
    [count, N, r], scale fp32 [count] (alpha / rank of each).  r is a multiple
    of 8; an adapter of a smaller rank is padded with zero rows of A and zero
    columns of B."""

    def __init__(self, A, B, scale):
        torch = _torch()
        if A is None or A.dim() != 3 or B is None or B.dim() != 3:
            raise ValueError("A must be [count, r, K] and B [count, N, r]")
        self.count, self.r, self.n_cols = (int(x) for x in A.shape)
        self.n_rows = int(B.shape[1])
        _expect(A, "A", (self.count, self.r, self.n_cols), (torch.bfloat16,))
        _expect(B, "B", (self.count, self.n_rows, self.r), (torch.bfloat16,))
        _expect(scale, "scale", (self.count,), (torch.float32,))
        self.A, self.B, self.scale = A, B, scale

    def _struct_on(self, dev: int) -> qlora_adapters_t:
        torch = _torch()
        c, r, n, k = self.count, self.r, self.n_rows, self.n_cols
        return qlora_adapters_t(_address(self.A, "A", (c, r, k), (torch.bfloat16,), dev),
                                _address(self.B, "B", (c, n, r), (torch.bfloat16,), dev),
                                _address(self.scale, "scale", (c,), (torch.float32,), dev), c, r)


class AdapterPlan:
    """The tokens of one batch sorted by adapter (qlora_adapters_plan): a
    device buffer for M tokens and a pool of `count` adapters.  One plan serves
    both passes of every linear layer of a step."""

    def __init__(self, M: int, count: int, buffer):
        self.M, self.count, self.buffer = int(M), int(count), buffer

    @classmethod
    def empty(cls, M: int, count: int, device="cuda"):
        torch = _torch()
        n = qlora_adapters_sizes(8, 64, M, 8, count)["plan_bytes"]
        return cls(M, count, torch.empty(n, dtype=torch.uint8, device=device))


def qlora_adapters_sizes(N: int, K: int, M_max: int, r: int, count: int) -> dict:
    out = qlora_adapters_sizes_t()
    _check(lib.qlora_adapters_sizes(N, K, M_max, r, count, ctypes.byref(out)))
    return {name: int(getattr(out, name)) for name, _ in qlora_adapters_sizes_t._fields_}


def qlora_adapters_plan(index, plan: AdapterPlan, stream=None) -> None:
    """index int32 [M]: the adapter of every token; outside [0, count): none."""
    dev = plan.buffer.get_device()
    at = _address(index, "index", (plan.M,), (_torch().int32,), dev)
    buf, size = _scratch(plan.buffer, "plan", dev)
    raw = _launch_stream(stream, dev)
    _check(lib.qlora_adapters_plan(at, plan.M, plan.count, buf, size, raw))


def _check_adapters(W: Nf4Tensor, X, pool: AdapterPool, plan: AdapterPlan):
    if X is None or X.dim() != 2:
        raise ValueError("X must be [M, K]")
    if pool.n_rows != W.n_rows or pool.n_cols != W.n_cols:
        raise ValueError(f"the adapters are for a [{pool.n_rows}, {pool.n_cols}] weight, W is "
                         f"[{W.n_rows}, {W.n_cols}]")
    M = X.shape[0]
    if plan.M != M or plan.count != pool.count:
        raise ValueError(f"the plan is for {plan.M} tokens and {plan.count} adapters, the call has {M} and "
                         f"{pool.count}")
    return M


def qlora_adapters_fwd(W: Nf4Tensor, X, pool: AdapterPool, plan: AdapterPlan, Y, T_save, ws, stream=None) -> None:
    """Y[m] = X[m]·Ŵᵀ + s_a·(X[m]·A_aᵀ)·B_aᵀ, a the adapter of token m in the plan."""
    torch = _torch()
    f32, bf16 = torch.float32, torch.bfloat16
    M = _check_adapters(W, X, pool, plan)
    dev = X.get_device()
    x = _address(X, "X", (M, W.n_cols), (bf16,), dev)
    y = _address(Y, "Y", (M, W.n_rows), (f32, bf16), dev)
    t = None if T_save is None else _address(T_save, "T_save", (M, pool.r), (f32,), dev)
    buf, size = _scratch(plan.buffer, "plan", dev)
    w, nbytes = _scratch(ws, "ws", dev)
    wd, ad = _weight_on(W, dev), pool._struct_on(dev)
    _check(lib.qlora_adapters_fwd(ctypes.byref(wd), x, M, ctypes.byref(ad), buf, size, y,
                                  QLORA_BF16 if Y.dtype == bf16 else QLORA_F32, t, w, nbytes,
                                  _launch_stream(stream, dev)))


def qlora_adapters_bwd(W: Nf4Tensor, X, dY, pool: AdapterPool, plan: AdapterPlan, T_saved, dX, dA, dB, ws,
                       stream=None) -> None:
    """dX, and dA, dB of every adapter of the pool (zeros without tokens)."""
    torch = _torch()
    f32, bf16 = torch.float32, torch.bfloat16
    M = _check_adapters(W, X, pool, plan)
    N, K, r, count = W.n_rows, W.n_cols, pool.r, pool.count
    dev = X.get_device()
    x, dy = _address(X, "X", (M, K), (bf16,), dev), _address(dY, "dY", (M, N), (bf16,), dev)
    t = None if T_saved is None else _address(T_saved, "T_saved", (M, r), (f32,), dev)
    dx = _address(dX, "dX", (M, K), (f32, bf16), dev)
    da, db = _address(dA, "dA", (count, r, K), (f32,), dev), _address(dB, "dB", (count, N, r), (f32,), dev)
    buf, size = _scratch(plan.buffer, "plan", dev)
    w, nbytes = _scratch(ws, "ws", dev)
    wd, ad = _weight_on(W, dev), pool._struct_on(dev)
    _check(lib.qlora_adapters_bwd(ctypes.byref(wd), x, dy, M, ctypes.byref(ad), buf, size, t, dx,
                                  QLORA_BF16 if dX.dtype == bf16 else QLORA_F32, da, db, w, nbytes,
                                  _launch_stream(stream, dev)))


class Dropout:
    """Dropout of an adapter's input: each element dropped with probability p (in
    steps of 2^-16), by a generator that knows the element's index, `seed` and
    `offset` alone.  The backward pass takes the forward pass's; every layer and
    step takes a seed or an offset of its own.  step: None, or an int64 tensor [1]
    that is added to the offset when the kernels run, so that a captured step draws
    another mask in every replay once it is raised."""

    def __init__(self, p: float, seed: int, offset: int = 0, step=None):
        for name, v in (("seed", seed), ("offset", offset)):
            if not 0 <= v < 2 ** 64:
                raise ValueError(f"{name}={v} outside [0, 2^64)")
        self.p, self.seed, self.offset, self.step = float(p), int(seed), int(offset), step


def _drop_ref(drop, dev: int):
    if drop is None:
        return None
    step = None if drop.step is None else _address(drop.step, "step", (1,), (_torch().int64,), dev)
    return ctypes.byref(qlora_dropout_t(drop.p, drop.seed, drop.offset, step))


def _block_sizes(call, N: int, K: int, M_max: int, r: int) -> dict:
    out = qlora_block_sizes_t()
    _check(call(N, K, M_max, r, ctypes.byref(out)))
    return {name: int(getattr(out, name)) for name, _ in qlora_block_sizes_t._fields_}


def qlora_dropout_linear_sizes(N: int, K: int, M_max: int, r: int) -> dict:
    return _block_sizes(lib.qlora_dropout_linear_sizes, N, K, M_max, r)


def qlora_gated_sizes(N: int, K: int, M_max: int, r: int) -> dict:
    return _block_sizes(lib.qlora_gated_sizes, N, K, M_max, r)


def _tokens(X) -> int:
    if X is None or X.dim() != 2:
        raise ValueError("X must be [M, K]")
    return X.shape[0]


def qlora_dropout_linear_fwd(W: Nf4Tensor, X, A, B, r: int, alpha: float, drop, Y, T_save, ws, stream=None) -> None:
    """Y = X·Ŵᵀ + (alpha / r)·(D(X)·Aᵀ)·Bᵀ, D the Dropout `drop` (None: no dropout)."""
    torch = _torch()
    f32, bf16 = torch.float32, torch.bfloat16
    M, N, K = _tokens(X), W.n_rows, W.n_cols
    dev = X.get_device()
    x, a = _address(X, "X", (M, K), (bf16,), dev), _address(A, "A", (r, K), (bf16,), dev)
    b, y = _address(B, "B", (N, r), (bf16,), dev), _address(Y, "Y", (M, N), (f32, bf16), dev)
    t = None if T_save is None else _address(T_save, "T_save", (M, r), (f32,), dev)
    w, nbytes = _scratch(ws, "ws", dev)
    wd = _weight_on(W, dev)
    _check(lib.qlora_dropout_linear_fwd(ctypes.byref(wd), x, M, a, b, r, alpha, _drop_ref(drop, dev), y,
                                        QLORA_BF16 if Y.dtype == bf16 else QLORA_F32, t, w, nbytes,
                                        _launch_stream(stream, dev)))


def qlora_dropout_linear_bwd(W: Nf4Tensor, X, dY, A, B, r: int, alpha: float, drop, T_saved, dX, dA, dB, ws,
                             stream=None) -> None:
    """dX, dA and dB of qlora_dropout_linear_fwd; drop is the forward pass's."""
    torch = _torch()
    f32, bf16 = torch.float32, torch.bfloat16
    M, N, K = _tokens(X), W.n_rows, W.n_cols
    dev = X.get_device()
    x, dy = _address(X, "X", (M, K), (bf16,), dev), _address(dY, "dY", (M, N), (bf16,), dev)
    a, b = _address(A, "A", (r, K), (bf16,), dev), _address(B, "B", (N, r), (bf16,), dev)
    t = None if T_saved is None else _address(T_saved, "T_saved", (M, r), (f32,), dev)
    dx = _address(dX, "dX", (M, K), (f32, bf16), dev)
    da, db = _address(dA, "dA", (r, K), (f32,), dev), _address(dB, "dB", (N, r), (f32,), dev)
    w, nbytes = _scratch(ws, "ws", dev)
    wd = _weight_on(W, dev)
    _check(lib.qlora_dropout_linear_bwd(ctypes.byref(wd), x, dy, M, a, b, r, alpha, _drop_ref(drop, dev), t, dx,
                                        QLORA_BF16 if dX.dtype == bf16 else QLORA_F32, da, db, w, nbytes,
                                        _launch_stream(stream, dev)))


class GatedAdapters:
    """The adapters of a gated block's two layers: A_* bf16 [r, K], B_* bf16 [N, r],
    one rank (a multiple of 8) and one alpha."""

    def __init__(self, A_gate, B_gate, A_up, B_up, alpha: float):
        torch = _torch()
        if A_gate is None or A_gate.dim() != 2 or B_gate is None or B_gate.dim() != 2:
            raise ValueError("A_gate must be [r, K] and B_gate [N, r]")
        self.r, self.n_cols = (int(x) for x in A_gate.shape)
        self.n_rows = int(B_gate.shape[0])
        for t, name, shape in self._tensors(A_gate, B_gate, A_up, B_up):
            _expect(t, name, shape, (torch.bfloat16,))
        self.A_gate, self.B_gate, self.A_up, self.B_up, self.alpha = A_gate, B_gate, A_up, B_up, float(alpha)

    def _tensors(self, A_gate, B_gate, A_up, B_up):
        a, b = (self.r, self.n_cols), (self.n_rows, self.r)
        return ((A_gate, "A_gate", a), (B_gate, "B_gate", b), (A_up, "A_up", a), (B_up, "B_up", b))

    def _struct_on(self, dev: int) -> qlora_gated_adapters_t:
        bf16 = (_torch().bfloat16,)
        at = [_address(t, name, shape, bf16, dev)
              for t, name, shape in self._tensors(self.A_gate, self.B_gate, self.A_up, self.B_up)]
        return qlora_gated_adapters_t(*at, self.r, self.alpha)


def _check_gated(gate: Nf4Tensor, up: Nf4Tensor, X, adapters: GatedAdapters, act: str):
    """(M, N, K, the activation's number)"""
    N, K = adapters.n_rows, adapters.n_cols
    for name, W in (("gate", gate), ("up", up)):
        if W.n_rows != N or W.n_cols != K:
            raise ValueError(f"{name} is [{W.n_rows}, {W.n_cols}], the adapters are for [{N}, {K}]")
    if act not in ACTIVATIONS:
        raise ValueError(f"act {act!r}: one of {sorted(ACTIVATIONS)}")
    return _tokens(X), N, K, ACTIVATIONS[act]


def qlora_gated_fwd(gate: Nf4Tensor, up: Nf4Tensor, X, adapters: GatedAdapters, act: str, drop, H, G_save, U_save,
                    T_save, ws, stream=None) -> None:
    """H = act(G)*U with G and U the two layers of X; act "silu" or "gelu_tanh"; drop
    a Dropout or None; G_save, U_save, T_save (fp32 [2, M, r]) for the backward pass
    or None."""
    torch = _torch()
    f32, bf16 = (torch.float32,), (torch.bfloat16,)
    M, N, K, a = _check_gated(gate, up, X, adapters, act)
    dev = X.get_device()
    x, h = _address(X, "X", (M, K), bf16, dev), _address(H, "H", (M, N), bf16, dev)
    g = None if G_save is None else _address(G_save, "G_save", (M, N), bf16, dev)
    u = None if U_save is None else _address(U_save, "U_save", (M, N), bf16, dev)
    t = None if T_save is None else _address(T_save, "T_save", (2, M, adapters.r), f32, dev)
    w, nbytes = _scratch(ws, "ws", dev)
    w0, w1, ad = _weight_on(gate, dev), _weight_on(up, dev), adapters._struct_on(dev)
    _check(lib.qlora_gated_fwd(ctypes.byref(w0), ctypes.byref(w1), x, M, ctypes.byref(ad), a, _drop_ref(drop, dev), h, g, u,
                               t, w, nbytes, _launch_stream(stream, dev)))


def qlora_gated_bwd(gate: Nf4Tensor, up: Nf4Tensor, X, dH, G, U, adapters: GatedAdapters, act: str, drop, T_saved, dX,
                    dA_gate, dB_gate, dA_up, dB_up, ws, stream=None) -> None:
    """dX and the adapters' gradients of qlora_gated_fwd from its G, U (and T, or
    None to recompute it); drop is the forward pass's."""
    torch = _torch()
    f32, bf16 = (torch.float32,), (torch.bfloat16,)
    M, N, K, a = _check_gated(gate, up, X, adapters, act)
    r = adapters.r
    dev = X.get_device()
    x, dh = _address(X, "X", (M, K), bf16, dev), _address(dH, "dH", (M, N), bf16, dev)
    g, u = _address(G, "G", (M, N), bf16, dev), _address(U, "U", (M, N), bf16, dev)
    t = None if T_saved is None else _address(T_saved, "T_saved", (2, M, r), f32, dev)
    dx = _address(dX, "dX", (M, K), f32 + bf16, dev)
    out = [_address(dA_gate, "dA_gate", (r, K), f32, dev), _address(dB_gate, "dB_gate", (N, r), f32, dev),
           _address(dA_up, "dA_up", (r, K), f32, dev), _address(dB_up, "dB_up", (N, r), f32, dev)]
    w, nbytes = _scratch(ws, "ws", dev)
    w0, w1, ad = _weight_on(gate, dev), _weight_on(up, dev), adapters._struct_on(dev)
    _check(lib.qlora_gated_bwd(ctypes.byref(w0), ctypes.byref(w1), x, dh, g, u, M, ctypes.byref(ad), a, _drop_ref(drop, dev),
                               t, dx, QLORA_BF16 if dX.dtype == torch.bfloat16 else QLORA_F32, *out, w, nbytes,
                               _launch_stream(stream, dev)))


def _distill_args(Z, top, top_index, weight, dZ, vocab):
    """(device, the C arguments from Z to k, the weight's and the gradient's
    address)."""
    torch = _torch()
    floats = (torch.float32, torch.bfloat16, torch.float16)
    if Z is None or Z.dim() != 2 or top is None or top.dim() != 2:
        raise ValueError("Z must be [M, ldz] and top [M, k]")
    M, ldz = shape = Z.shape
    dev = Z.get_device()
    k = top.shape[1]
    z = _address(Z, "Z", shape, floats, dev)
    t = _address(top, "top", (M, k), floats, dev)
    at = _address(top_index, "top_index", (M, k), (torch.int32,), dev)
    w = None if weight is None else _address(weight, "weight", (M,), (torch.float32,), dev)
    d = None if dZ is None else _address(dZ, "dZ", shape, (Z.dtype,), dev)
    return dev, (z, _dtype(Z, "Z"), M, ldz if vocab is None else int(vocab), ldz, t, _dtype(top, "top"), at, k), w, d


def qlora_distill_fwd(Z, top, top_index, tau: float, weight, loss, lse=None, dZ=None, vocab=None, stream=None) -> None:
    """loss[m] = w·tau²·KL(softmax(top / tau) || softmax(Z / tau)) per token,
    its log-sum-exp and, if dZ is given (it may be Z), the gradient of their
    sum.  vocab: the columns of Z that count (all of them by default)."""
    dev, args, w, d = _distill_args(Z, top, top_index, weight, dZ, vocab)
    f32 = (_torch().float32,)
    out = _address(loss, "loss", (args[2],), f32, dev)
    norm = None if lse is None else _address(lse, "lse", (args[2],), f32, dev)
    _check(lib.qlora_distill_fwd(*args, tau, w, out, norm, d, _launch_stream(stream, dev)))


def qlora_distill_bwd(Z, top, top_index, tau: float, lse, weight, dZ, vocab=None, stream=None) -> None:
    """The gradient alone, from the lse of qlora_distill_fwd; dZ may be Z."""
    if dZ is None:
        raise ValueError("dZ is None")
    dev, args, w, d = _distill_args(Z, top, top_index, weight, dZ, vocab)
    norm = _address(lse, "lse", (args[2],), (_torch().float32,), dev)
    _check(lib.qlora_distill_bwd(*args, tau, norm, w, d, _launch_stream(stream, dev)))


def _logprobs_args(Z, target, d_logp, d_entropy, dZ, vocab):
    """(device, the C arguments from Z to target, the addresses of the two incoming
    gradients and of dZ)."""
    torch = _torch()
    f32 = (torch.float32,)
    if Z is None or Z.dim() != 2:
        raise ValueError("Z must be [M, ldz]")
    M, ldz = shape = Z.shape
    dev = Z.get_device()
    z = _address(Z, "Z", shape, (torch.float32, torch.bfloat16, torch.float16), dev)
    at = _address(target, "target", (M,), (torch.int32,), dev)
    g = None if d_logp is None else _address(d_logp, "d_logp", (M,), f32, dev)
    h = None if d_entropy is None else _address(d_entropy, "d_entropy", (M,), f32, dev)
    d = None if dZ is None else _address(dZ, "dZ", shape, (Z.dtype,), dev)
    return dev, (z, _dtype(Z, "Z"), M, ldz if vocab is None else int(vocab), ldz, at), g, h, d


def qlora_logprobs_fwd(Z, target, tau: float, logp, lse=None, entropy=None, top_logp=None, top_index=None, d_logp=None,
                       d_entropy=None, dZ=None, vocab=None, stream=None) -> None:
    """logp[m] = log softmax(Z / tau)[target[m]] per token (0 for a target that is no
    column), the log-sum-exp, the entropy, the top_logp.shape[1] most likely
    columns, and, if dZ is given (it may be Z), the gradient of
    Σ d_logp·logp + d_entropy·entropy.  vocab: the columns of Z that count (all
    of them by default)."""
    torch = _torch()
    f32 = (torch.float32,)
    dev, args, g, h, d = _logprobs_args(Z, target, d_logp, d_entropy, dZ, vocab)
    M = args[2]
    out = _address(logp, "logp", (M,), f32, dev)
    norm = None if lse is None else _address(lse, "lse", (M,), f32, dev)
    ent = None if entropy is None else _address(entropy, "entropy", (M,), f32, dev)
    k, tl, ti = 0, None, None
    if top_logp is not None or top_index is not None:
        if top_logp is None or top_logp.dim() != 2:
            raise ValueError("top_logp and top_index must be [M, k]")
        k = top_logp.shape[1]
        tl = _address(top_logp, "top_logp", (M, k), f32, dev)
        ti = _address(top_index, "top_index", (M, k), (torch.int32,), dev)
    _check(lib.qlora_logprobs_fwd(*args, tau, out, norm, ent, k, tl, ti, g, h, d, _launch_stream(stream, dev)))


def qlora_logprobs_bwd(Z, target, tau: float, lse, d_logp, dZ, entropy=None, d_entropy=None, vocab=None,
                       stream=None) -> None:
    """The gradient alone, from the lse (and, with d_entropy, the entropy) of
    qlora_logprobs_fwd; dZ may be Z."""
    f32 = (_torch().float32,)
    if dZ is None:
        raise ValueError("dZ is None")
    dev, args, g, h, d = _logprobs_args(Z, target, d_logp, d_entropy, dZ, vocab)
    norm = _address(lse, "lse", (args[2],), f32, dev)
    ent = None if entropy is None else _address(entropy, "entropy", (args[2],), f32, dev)
    _check(lib.qlora_logprobs_bwd(*args, tau, norm, ent, g, h, d, _launch_stream(stream, dev)))


class QTensor:
    """A weight in one of the comparison formats ("nf4", "int4", "int8"):
    codes (uint8) and one fp32 absmax per 64-block, device tensors."""

    def __init__(self, n_rows: int, n_cols: int, fmt: str, codes, absmax):
        self.n_rows, self.n_cols, self.fmt = n_rows, n_cols, fmt
        self.codes, self.absmax = codes, absmax

    @classmethod
    def empty(cls, n_rows: int, n_cols: int, fmt: str, device="cuda"):
        torch = _torch()
        nbytes = n_rows * n_cols if fmt == "int8" else n_rows * n_cols // 2
        return cls(n_rows, n_cols, fmt, torch.empty(nbytes, dtype=torch.uint8, device=device),
                   torch.empty(n_rows * n_cols // 64, dtype=torch.float32, device=device))

    def c_struct(self) -> qlora_qtensor_t:
        torch = _torch()
        if self.fmt not in FORMATS:
            raise ValueError(f"format {self.fmt!r}: one of {sorted(FORMATS)}")
        nbytes = self.n_rows * self.n_cols * (2 if self.fmt == "int8" else 1) // 2
        _expect_numel(self.codes, "codes", nbytes, torch.uint8)
        _expect_numel(self.absmax, "absmax", self.n_rows * self.n_cols // 64, torch.float32)
        return qlora_qtensor_t(self.n_rows, self.n_cols, FORMATS[self.fmt], _ptr(self.codes, "codes"),
                               _ptr(self.absmax, "absmax"))


def qlora_quantize_format(W, out: QTensor, stream=None) -> None:
    torch = _torch()
    _expect(W, "W", (out.n_rows, out.n_cols), (torch.float32, torch.bfloat16))
    N, K = W.shape
    st = out.c_struct()
    _check(lib.qlora_quantize_format(_ptr(W, "W"), _dtype(W, "W"), N, K, ctypes.byref(st), _stream(stream)))


def qlora_dequantize_format(q: QTensor, out, stream=None) -> None:
    torch = _torch()
    _expect(out, "out", (q.n_rows, q.n_cols), (torch.bfloat16,))
    st = q.c_struct()
    _check(lib.qlora_dequantize_format(ctypes.byref(st), _ptr(out, "out"), _dtype(out, "out"), _stream(stream)))


def qlora_gemv_format(q: QTensor, X, Y, stream=None) -> None:
    torch = _torch()
    if X is None or X.dim() != 2:
        raise ValueError("X must be [M, K]")
    _expect(X, "X", (X.shape[0], q.n_cols), (torch.bfloat16,))
    _expect(Y, "Y", (X.shape[0], q.n_rows), (torch.float32, torch.bfloat16))
    st = q.c_struct()
    _check(lib.qlora_gemv_format(ctypes.byref(st), _ptr(X, "X"), X.shape[0], _ptr(Y, "Y"), _dtype(Y, "Y"),
                                 _stream(stream)))
