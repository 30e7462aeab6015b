"""Python binding of libfp8mp, the GB300 FP8 delayed-scaling linear layer.

Argument marshalling only: every function below forwards to the C entry
point of the same name in ``libfp8mp.so`` (declared in ``include/fp8mp.h``),
passing device pointers, sizes and the CUDA stream. All computation runs in
the library's CUDA kernels. torch is used for device memory and streams.
If the library has not been built, ``load()`` raises: there is no fallback.
"""

from __future__ import annotations

import ctypes
import os

import torch

E4M3, E5M2 = 0, 1
F32, BF16 = 0, 1
AMAX_MAX, AMAX_MOST_RECENT = 0, 1
SILU, GELU_TANH = 0, 1
MAX_HISTORY = 8192
FMT_MAX = {E4M3: 448.0, E5M2: 57344.0}

OK, ERR_INVALID, ERR_DEVICE, ERR_LAUNCH, ERR_TIMEOUT = 0, -1, -2, -3, -4

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8mp.so")
EXPORTS = ("fp8_quantize", "fp8_quantize_ex", "fp8_quantize_current", "fp8_quantize_dbias",
           "fp8_quantize_dbias_workspace_bytes", "fp8_quantize_dbias_noalloc", "fp8_linear_fwd", "fp8_linear_fwd_fp8out", "fp8_linear_dgrad", "fp8_linear_wgrad",
           "fp8_linear_bwd", "fp8_linear_bwd_rowmajor", "fp8_linear_bwd_rowmajor_ex", "delayed_scaling_update",
           "delayed_scaling_update_ex", "mp_master_step", "mp_master_step_adam", "mp_master_step_prescanned", "mp_master_step_adam_prescanned",
           "mp_master_step_prescanned_ex", "mp_master_step_adam_prescanned_ex",
           "mp_master_step_prescanned_scaling_ex", "mp_master_step_adam_prescanned_scaling_ex", "fp8_gated_fwd", "fp8_linear_few", "fp8_gated_dgrad", "fp8_gated_bwd",
           "mp_adamw_workspace_bytes", "mp_grad_norm", "mp_adamw_step",
           "fp8_rmsnorm_fwd", "fp8_rmsnorm_bwd", "fp8_rmsnorm_bwd_workspace_bytes", "mp_logprobs_fwd", "mp_logprobs_bwd",
           "mp_embedding_fwd", "mp_embedding_bwd", "mp_embedding_bwd_workspace_bytes",
           "fp8mp_check", "fp8mp_last_error",
           "fp8mp_version", "fp8mp_selftest_timeout", "fp8mp_selftest_barrier_timeout")

_lib = None


class Fp8mpError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libfp8mp error {code}: {msg}")
        self.code = code


class fp8mp_meta(ctypes.Structure):
    """Mirror of the C struct fp8mp_meta (device pointers + two int32)."""

    _fields_ = [("amax_history", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("scale_inv", ctypes.c_void_p), ("cur_amax", ctypes.c_void_p),
                ("history_len", ctypes.c_int32), ("fmt", ctypes.c_int32)]


class fp8mp_adamw_tensor(ctypes.Structure):
    """Mirror of the C struct fp8mp_adamw_tensor."""

    _fields_ = [("grad", ctypes.c_void_p), ("master", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("exp_avg_scale", ctypes.c_void_p),
                ("exp_avg_sq_scale", ctypes.c_void_p), ("copy", ctypes.c_void_p), ("copy_scale", ctypes.c_void_p),
                ("copy_amax", ctypes.c_void_p), ("n", ctypes.c_int64), ("weight_decay", ctypes.c_float),
                ("grad_dtype", ctypes.c_int32), ("state_bits", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def build(force: bool = False) -> str:
    from . import buildlib

    return buildlib.build(force=force)


def load(path: str | None = None):
    """Loads libfp8mp.so (raises if it is missing) and declares the signatures."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise Fp8mpError(ERR_LAUNCH, f"{path} is missing: build it with "
                         "fp8_mixed_precision_reduce_gb300.build() (no CPU fallback exists)")
    L = ctypes.CDLL(path)
    P, I64, I32, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    L.fp8_quantize.argtypes = [P, I32, I64, I64, I32, P, P, P, P, P]
    L.fp8_quantize_ex.argtypes = [P, I32, I64, I64, I32, P, P, P, P, ctypes.c_uint32, P]
    L.fp8_quantize_current.argtypes = [P, I32, I64, I64, I32, I32, P, P, P, P, P, P]
    L.fp8_quantize_dbias.argtypes = [P, I32, I64, I64, I32, P, P, P, P, P, I32, P, I64, P]
    L.fp8_quantize_dbias_noalloc.argtypes = [P, I32, I64, I64, I32, P, P, P, P, P, I32, P]
    L.fp8_quantize_dbias_workspace_bytes.argtypes = [I64, I64]
    L.fp8_quantize_dbias_workspace_bytes.restype = I64
    L.fp8_linear_fwd.argtypes = [P, P, I64, I64, I64, P, P, P, I32, P, I32, P, P]
    L.fp8_linear_fwd_fp8out.argtypes = [P, P, I64, I64, I64, P, P, P, I32, P, I32, P, P, P]
    L.fp8_linear_dgrad.argtypes = [P, P, I64, I64, I64, I32, P, P, P, I32, P]
    L.fp8_linear_wgrad.argtypes = [P, P, I64, I64, I64, I32, P, P, P, I32, P]
    L.fp8_linear_bwd.argtypes = [P, P, P, P, I64, I64, I64, I32, P, P, P, P, I32, P, I32, P]
    L.fp8_linear_bwd_rowmajor.argtypes = [P, P, P, I64, I64, I64, I32, P, P, P, P, I32, P, I32, P, P]
    L.fp8_linear_bwd_rowmajor_ex.argtypes = [P, P, P, I64, I64, I64, I32, P, P, P, P, I32, P, I32, P,
                                             ctypes.c_uint32, P]
    L.delayed_scaling_update.argtypes = [ctypes.POINTER(fp8mp_meta), I32, I32, I32, P]
    L.delayed_scaling_update_ex.argtypes = [ctypes.POINTER(fp8mp_meta), I32, I32, I32, P, P]
    L.mp_master_step.argtypes = [P, I64, P, P, P, P, P, P, P, P, F, F, F, F, I32, P]
    L.mp_master_step_adam.argtypes = [P, I64, P, P, P, P, P, P, P, P, P, P, F, F, F, F, F, F, I32, P]
    L.mp_master_step_prescanned.argtypes = [P, I64, P, P, P, P, P, P, P, P, P, F, F, F, F, I32, P]
    L.mp_master_step_adam_prescanned.argtypes = [P, I64, P, P, P, P, P, P, P, P, P, P, P, F, F, F, F, F, F, I32, P]
    U32 = ctypes.c_uint32
    L.mp_master_step_prescanned_ex.argtypes = [P, I64, P, P, P, P, P, P, P, P, P, P, F, F, F, F, I32, U32, P]
    L.mp_master_step_adam_prescanned_ex.argtypes = [P, I64, P, P, P, P, P, P, P, P, P, P, P, P, F, F, F, F, F, F,
                                                    I32, U32, P]
    M = ctypes.POINTER(fp8mp_meta)
    L.mp_master_step_prescanned_scaling_ex.argtypes = [P, I64, P, P, P, P, P, P, P, P, P, P, F, F, F, F, I32,
                                                       M, I32, I32, I32, U32, P]
    L.mp_master_step_adam_prescanned_scaling_ex.argtypes = [P, I64, P, P, P, P, P, P, P, P, P, P, P, P, F, F, F,
                                                            F, F, F, I32, M, I32, I32, I32, U32, P]
    L.fp8_gated_fwd.argtypes = [P, P, I64, I64, I64, I32, P, P, P, P, P, P, P]
    L.fp8_gated_dgrad.argtypes = [P, P, P, I64, I64, I64, I32, I32, P, P, P, P, P, P]
    L.fp8_gated_bwd.argtypes = [P, I32, P, P, P, I64, I64, I64, I32, P, P, P, P, P, P, P, I32, P, I32, P, P]
    L.fp8_linear_few.argtypes = [P, P, I64, I64, I64, P, P, P, I32, P, I32, P, P]
    for name in ("fp8_gated_fwd", "fp8_linear_few", "fp8_gated_dgrad", "fp8_gated_bwd"):
        getattr(L, name).restype = ctypes.c_int
    A = ctypes.POINTER(fp8mp_adamw_tensor)
    L.mp_adamw_workspace_bytes.argtypes = []
    L.mp_adamw_workspace_bytes.restype = I64
    L.mp_grad_norm.argtypes = [A, I32, P, P, P, I64, P]
    L.mp_grad_norm.restype = ctypes.c_int
    L.mp_adamw_step.argtypes = [A, I32, P, P, P, P, P, P, F, F, F, F, F, F, F, I32, P, I64, P]
    L.mp_adamw_step.restype = ctypes.c_int
    L.fp8_rmsnorm_fwd.argtypes = [P, I32, P, P, I32, I64, I64, P, I32, F, P, P, I32, P, P, P]
    L.fp8_rmsnorm_bwd.argtypes = [P, I32, P, P, I32, P, I64, I64, P, I32, P, P, P, I32, P, I64, P]
    L.fp8_rmsnorm_bwd_workspace_bytes.argtypes = [I64, I64]
    L.mp_logprobs_fwd.argtypes = [P, I32, I64, I64, I64, P, P, P, P, P, P, I32, P]
    L.mp_logprobs_bwd.argtypes = [P, I32, I64, I64, I64, P, P, P, P, P, P, P, P, P]
    L.mp_embedding_fwd.argtypes = [P, I64, P, I32, I64, I64, P, F, P, I32, P]
    L.mp_embedding_bwd.argtypes = [P, I64, P, I32, I64, I64, F, P, I32, P, I64, P]
    L.mp_embedding_bwd_workspace_bytes.argtypes = [I64, I64, I64]
    for name in ("fp8_rmsnorm_fwd", "fp8_rmsnorm_bwd", "mp_logprobs_fwd", "mp_logprobs_bwd", "mp_embedding_fwd",
                 "mp_embedding_bwd"):
        getattr(L, name).restype = ctypes.c_int
    for name in ("fp8_rmsnorm_bwd_workspace_bytes", "mp_embedding_bwd_workspace_bytes"):
        getattr(L, name).restype = I64
    L.fp8mp_check.argtypes = [P]
    L.fp8mp_selftest_timeout.argtypes = [P]
    L.fp8mp_selftest_barrier_timeout.argtypes = [P]
    L.fp8mp_last_error.restype = ctypes.c_char_p
    L.fp8mp_version.restype = I32
    for name in ("fp8_quantize", "fp8_quantize_ex", "fp8_quantize_current", "fp8_quantize_dbias", "fp8_quantize_dbias_noalloc",
                 "fp8_linear_fwd", "fp8_linear_fwd_fp8out", "fp8_linear_dgrad", "fp8_linear_wgrad",
                 "fp8_linear_bwd", "fp8_linear_bwd_rowmajor", "fp8_linear_bwd_rowmajor_ex", "delayed_scaling_update",
                 "delayed_scaling_update_ex", "mp_master_step", "mp_master_step_adam", "mp_master_step_prescanned", "mp_master_step_adam_prescanned",
                 "mp_master_step_prescanned_ex", "mp_master_step_adam_prescanned_ex", "fp8mp_check",
                 "fp8mp_selftest_timeout", "fp8mp_selftest_barrier_timeout"):
        getattr(L, name).restype = ctypes.c_int
    _lib = L
    return L


def last_error() -> str:
    return load().fp8mp_last_error().decode()


def _check(rc: int) -> None:
    if rc != OK:
        raise Fp8mpError(rc, last_error())


def _ptr(t) -> int | None:
    if t is None or isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:  # the current device's current stream
        try:  # (not torch's public calls, but 3 us faster)
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        except AttributeError:
            return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _rows_cols(t: torch.Tensor):
    if t.dim() == 2:
        return t.shape[0], t.shape[1]
    return 1, t.numel()


# ------------------------------------------------------------- entry points


def fp8_quantize(x: torch.Tensor, fmt: int, scale: torch.Tensor, out: torch.Tensor,
                 out_t: torch.Tensor | None = None, amax: torch.Tensor | None = None,
                 stream=None) -> None:
    """out = sat_rne(x * scale) as FP8 codes (uint8), out_t its transpose,
    amax = max(amax, max|x|). x is 2-D (rows, cols) or flat, contiguous."""
    rows, cols = _rows_cols(x)
    _check(load().fp8_quantize(_ptr(x), _dtype_code(x), rows, cols, fmt, _ptr(scale), _ptr(out),
                               _ptr(out_t), _ptr(amax), _stream(stream)))


OVERLAP_PREVIOUS = 1  # FP8MP_OVERLAP_PREVIOUS: fp8_quantize_ex, mp_master_step(_adam) with w8_in
SIGNAL_DW_DONE = 2  # FP8MP_SIGNAL_DW_DONE: fp8_linear_bwd_rowmajor
WAIT_DW_DONE = 4  # FP8MP_WAIT_DW_DONE: mp_master_step(_adam) with grad_nonfinite and OVERLAP_PREVIOUS


def fp8_quantize_ex(x: torch.Tensor, fmt: int, scale: torch.Tensor, out: torch.Tensor,
                    out_t: torch.Tensor | None = None, amax: torch.Tensor | None = None, flags: int = 0,
                    stream=None) -> None:
    """fp8_quantize with flags. OVERLAP_PREVIOUS: the caller guarantees that the
    work enqueued before this call neither writes nor reads x, out, out_t or
    amax, so the cast may run while the previous kernel is still running; the
    call still completes after it."""
    rows, cols = _rows_cols(x)
    _check(load().fp8_quantize_ex(_ptr(x), _dtype_code(x), rows, cols, fmt, _ptr(scale), _ptr(out),
                                  _ptr(out_t), _ptr(amax), flags, _stream(stream)))


def fp8_quantize_current(x: torch.Tensor, fmt: int, scale: torch.Tensor, scale_inv: torch.Tensor,
                         amax: torch.Tensor, out: torch.Tensor, out_t: torch.Tensor | None = None,
                         margin: int = 0, stream=None) -> None:
    """Just-in-time scaling: amax = max|x|, scale from it (kept when the amax
    is 0 / not finite), then out = sat_rne(x * scale) and its transpose."""
    rows, cols = _rows_cols(x)
    _check(load().fp8_quantize_current(_ptr(x), _dtype_code(x), rows, cols, fmt, margin, _ptr(scale),
                                       _ptr(scale_inv), _ptr(amax), _ptr(out), _ptr(out_t), _stream(stream)))


def fp8_quantize_dbias_workspace_bytes(rows: int, cols: int) -> int:
    return int(load().fp8_quantize_dbias_workspace_bytes(rows, cols))


def fp8_quantize_dbias(dy: torch.Tensor, fmt: int, scale: torch.Tensor, out: torch.Tensor,
                       out_t: torch.Tensor | None, dbias: torch.Tensor, workspace: torch.Tensor,
                       amax: torch.Tensor | None = None, stream=None) -> None:
    """Cast of an output gradient (+ optional transposed copy, + amax) that
    also writes the bias gradient dbias = column sums of dy, in one launch.
    `workspace` is a device buffer of at least
    fp8_quantize_dbias_workspace_bytes(rows, cols) bytes, zero-filled before
    its first use; every call leaves it zero again."""
    rows, cols = _rows_cols(dy)
    _check(load().fp8_quantize_dbias(_ptr(dy), _dtype_code(dy), rows, cols, fmt, _ptr(scale), _ptr(out),
                                     _ptr(out_t), _ptr(amax), _ptr(dbias), _dtype_code(dbias),
                                     _ptr(workspace), workspace.numel() * workspace.element_size(),
                                     _stream(stream)))


NOALLOC_DBIAS_SCRATCH_FLOATS = 1 << 20


def fp8_quantize_dbias_noalloc(dy: torch.Tensor, fmt: int, scale: torch.Tensor, out: torch.Tensor,
                               out_t: torch.Tensor, dbias: torch.Tensor, amax: torch.Tensor | None = None,
                               stream=None) -> None:
    """fp8_quantize_dbias without a workspace, for callers that cannot
    allocate device memory: the partial sums and counters live in a fixed
    4 MiB array in the library (fp8_quantize_dbias_workspace_bytes(rows, cols)
    <= 4 MiB). The first call on a device looks up that array's address;
    calls that overlap on the GPU race on it."""
    rows, cols = _rows_cols(dy)
    _check(load().fp8_quantize_dbias_noalloc(_ptr(dy), _dtype_code(dy), rows, cols, fmt, _ptr(scale), _ptr(out),
                                             _ptr(out_t), _ptr(amax), _ptr(dbias), _dtype_code(dbias),
                                             _stream(stream)))


def fp8_linear_fwd(x8: torch.Tensor, w8: torch.Tensor, sinv_x: torch.Tensor, sinv_w: torch.Tensor,
                   y: torch.Tensor, bias: torch.Tensor | None = None,
                   y_amax: torch.Tensor | None = None, stream=None) -> None:
    """y[M, N] = (x8[M, K] . w8[N, K]^T) * sinv_x * sinv_w + bias."""
    M, K = x8.shape
    N = w8.shape[0]
    _check(load().fp8_linear_fwd(_ptr(x8), _ptr(w8), M, N, K, _ptr(sinv_x), _ptr(sinv_w), _ptr(bias),
                                 _dtype_code(bias) if bias is not None else F32, _ptr(y), _dtype_code(y),
                                 _ptr(y_amax), _stream(stream)))


def fp8_linear_fwd_fp8out(x8: torch.Tensor, w8: torch.Tensor, sinv_x: torch.Tensor, sinv_w: torch.Tensor,
                          y_scale: torch.Tensor, y8: torch.Tensor, y_fmt: int = E4M3,
                          bias: torch.Tensor | None = None, y_amax: torch.Tensor | None = None,
                          stream=None) -> None:
    """y8 = FP8 codes of ((x8 . w8^T) * sinv_x * sinv_w + bias) * y_scale."""
    M, K = x8.shape
    N = w8.shape[0]
    _check(load().fp8_linear_fwd_fp8out(_ptr(x8), _ptr(w8), M, N, K, _ptr(sinv_x), _ptr(sinv_w), _ptr(bias),
                                        _dtype_code(bias) if bias is not None else F32, _ptr(y_scale), y_fmt,
                                        _ptr(y8), _ptr(y_amax), _stream(stream)))


def fp8_linear_dgrad(dy8: torch.Tensor, w8t: torch.Tensor, sinv_dy: torch.Tensor,
                     sinv_w: torch.Tensor, dx: torch.Tensor, dy_fmt: int = E5M2, stream=None) -> None:
    """dx[M, K] = (dy8[M, N] . w8t[K, N]^T) * sinv_dy * sinv_w."""
    M, N = dy8.shape
    K = w8t.shape[0]
    _check(load().fp8_linear_dgrad(_ptr(dy8), _ptr(w8t), M, N, K, dy_fmt, _ptr(sinv_dy), _ptr(sinv_w),
                                   _ptr(dx), _dtype_code(dx), _stream(stream)))


def fp8_linear_wgrad(dy8t: torch.Tensor, x8t: torch.Tensor, sinv_dy: torch.Tensor,
                     sinv_x: torch.Tensor, dw: torch.Tensor, dy_fmt: int = E5M2, stream=None) -> None:
    """dw[N, K] = (dy8t[N, M] . x8t[K, M]^T) * sinv_dy * sinv_x."""
    N, M = dy8t.shape
    K = x8t.shape[0]
    _check(load().fp8_linear_wgrad(_ptr(dy8t), _ptr(x8t), M, N, K, dy_fmt, _ptr(sinv_dy), _ptr(sinv_x),
                                   _ptr(dw), _dtype_code(dw), _stream(stream)))


def fp8_linear_bwd(dy8: torch.Tensor, dy8t: torch.Tensor, w8t: torch.Tensor, x8t: torch.Tensor,
                   sinv_dy: torch.Tensor, sinv_w: torch.Tensor, sinv_x: torch.Tensor, dx: torch.Tensor,
                   dw: torch.Tensor, dy_fmt: int = E5M2, stream=None) -> None:
    """fp8_linear_dgrad and fp8_linear_wgrad in one launch:
    dx[M, K] = (dy8 . w8t^T) * sinv_dy * sinv_w, dw[N, K] = (dy8t . x8t^T) * sinv_dy * sinv_x."""
    M, N = dy8.shape
    K = w8t.shape[0]
    _check(load().fp8_linear_bwd(_ptr(dy8), _ptr(dy8t), _ptr(w8t), _ptr(x8t), M, N, K, dy_fmt, _ptr(sinv_dy),
                                 _ptr(sinv_w), _ptr(sinv_x), _ptr(dx), _dtype_code(dx), _ptr(dw), _dtype_code(dw),
                                 _stream(stream)))


def fp8_linear_bwd_rowmajor(dy8: torch.Tensor, w8: torch.Tensor | None, x8: torch.Tensor | None,
                            sinv_dy: torch.Tensor, sinv_w: torch.Tensor | None, sinv_x: torch.Tensor | None,
                            dx: torch.Tensor | None, dw: torch.Tensor | None, dy_fmt: int = E5M2,
                            dw_nonfinite: torch.Tensor | None = None, stream=None, flags: int = 0) -> None:
    """Both backward GEMMs from the forward's row-major FP8 copies, one launch:
    dx[M, K] = (dy8 . w8) * sinv_dy * sinv_w, dw[N, K] = (dy8^T . x8) * sinv_dy * sinv_x.
    dx or dw may be None to skip that gradient. dw_nonfinite (int32[1] on the
    device) gets 1 OR-ed in when a stored element of dw is Inf or NaN. flags
    (SIGNAL_DW_DONE) selects fp8_linear_bwd_rowmajor_ex."""
    M, N = dy8.shape
    K = (w8 if w8 is not None else x8).shape[1]
    args = (_ptr(dy8), _ptr(w8), _ptr(x8), M, N, K, dy_fmt, _ptr(sinv_dy), _ptr(sinv_w), _ptr(sinv_x), _ptr(dx),
            _dtype_code(dx) if dx is not None else F32, _ptr(dw), _dtype_code(dw) if dw is not None else F32,
            _ptr(dw_nonfinite))
    if flags:
        _check(load().fp8_linear_bwd_rowmajor_ex(*args, int(flags), _stream(stream)))
    else:
        _check(load().fp8_linear_bwd_rowmajor(*args, _stream(stream)))


class Meta:
    """One tensor's delayed-scaling state in device memory (fp32)."""

    def __init__(self, history_len: int, fmt: int, device="cuda"):
        self.fmt = fmt
        self.history_len = history_len
        self.amax_history = torch.zeros(history_len, dtype=torch.float32, device=device)
        self.scale = torch.ones(1, dtype=torch.float32, device=device)
        self.scale_inv = torch.ones(1, dtype=torch.float32, device=device)
        self.cur_amax = torch.zeros(1, dtype=torch.float32, device=device)

    def c_struct(self) -> fp8mp_meta:
        return fp8mp_meta(self.amax_history.data_ptr(), self.scale.data_ptr(),
                          self.scale_inv.data_ptr(), self.cur_amax.data_ptr(),
                          self.history_len, self.fmt)


def delayed_scaling_update(metas, algo: int, margin: int = 0, stream=None,
                           prev_scale_inv: torch.Tensor | None = None) -> None:
    """Rolls each meta's history, picks the amax and refreshes scale/scale_inv.
    With prev_scale_inv (fp32[len(metas)] on the device) each meta's
    scale_inv from before the update is kept there (delayed_scaling_update_ex)."""
    metas = list(metas)
    arr = (fp8mp_meta * max(1, len(metas)))(*[m.c_struct() for m in metas])
    if prev_scale_inv is not None:
        if prev_scale_inv.numel() < len(metas) or prev_scale_inv.dtype != torch.float32:
            raise Fp8mpError(ERR_INVALID, "prev_scale_inv must be float32 with one entry per meta")
        _check(load().delayed_scaling_update_ex(arr, len(metas), algo, margin, _ptr(prev_scale_inv),
                                                _stream(stream)))
        return
    _check(load().delayed_scaling_update(arr, len(metas), algo, margin, _stream(stream)))


def mp_master_step(grad_bf16: torch.Tensor, master: torch.Tensor, momentum: torch.Tensor,
                   w8: torch.Tensor, scale_w: torch.Tensor, amax_w: torch.Tensor,
                   loss_scale: torch.Tensor, growth_tracker: torch.Tensor, found_inf: torch.Tensor,
                   lr: float, momentum_coef: float, backoff: float = 0.5, growth_factor: float = 2.0,
                   growth_interval: int = 2000, stream=None, grad_nonfinite: torch.Tensor | None = None,
                   w8_in: torch.Tensor | None = None, flags: int = 0, metas=None, amax_algo: int = AMAX_MOST_RECENT,
                   margin: int = 0) -> None:
    """Unscale, overflow skip, FP32 SGD-momentum update and E4M3 re-cast, in place.
    With grad_nonfinite (int32[1] on the device holding 0 or 1, set by the
    gradients' producer, e.g. fp8_linear_bwd_rowmajor's dw_nonfinite) the step
    reads that flag instead of scanning the gradients, writes it to found_inf
    and resets it to 0. With it, w8_in (the current E4M3 copy; the new one goes
    to w8, which a skipped step fills with w8_in) and flags
    (OVERLAP_PREVIOUS) select mp_master_step_prescanned_ex; metas (with
    amax_algo, margin; flags OVERLAP_PREVIOUS | WAIT_DW_DONE) select
    mp_master_step_prescanned_scaling_ex, which also runs the metas'
    delayed-scaling update."""
    n = grad_bf16.numel()
    if metas is not None:
        if grad_nonfinite is None:
            raise Fp8mpError(ERR_INVALID, "metas need grad_nonfinite (the prescanned step)")
        metas = list(metas)
        arr = (fp8mp_meta * max(1, len(metas)))(*[m.c_struct() for m in metas])
        _check(load().mp_master_step_prescanned_scaling_ex(
            _ptr(grad_bf16), n, _ptr(master), _ptr(momentum), _ptr(w8_in), _ptr(w8), _ptr(scale_w), _ptr(amax_w),
            _ptr(loss_scale), _ptr(growth_tracker), _ptr(found_inf), _ptr(grad_nonfinite), float(lr),
            float(momentum_coef), float(backoff), float(growth_factor), int(growth_interval), arr, len(metas),
            int(amax_algo), int(margin), int(flags), _stream(stream)))
        return
    if w8_in is not None or flags:
        if grad_nonfinite is None:
            raise Fp8mpError(ERR_INVALID, "w8_in and flags need grad_nonfinite (the prescanned step)")
        _check(load().mp_master_step_prescanned_ex(
            _ptr(grad_bf16), n, _ptr(master), _ptr(momentum), _ptr(w8_in), _ptr(w8), _ptr(scale_w), _ptr(amax_w),
            _ptr(loss_scale), _ptr(growth_tracker), _ptr(found_inf), _ptr(grad_nonfinite), float(lr),
            float(momentum_coef), float(backoff), float(growth_factor), int(growth_interval), int(flags),
            _stream(stream)))
        return
    if grad_nonfinite is not None:
        _check(load().mp_master_step_prescanned(_ptr(grad_bf16), n, _ptr(master), _ptr(momentum), _ptr(w8),
                                                _ptr(scale_w), _ptr(amax_w), _ptr(loss_scale), _ptr(growth_tracker),
                                                _ptr(found_inf), _ptr(grad_nonfinite), float(lr),
                                                float(momentum_coef), float(backoff), float(growth_factor),
                                                int(growth_interval), _stream(stream)))
        return
    _check(load().mp_master_step(_ptr(grad_bf16), n, _ptr(master), _ptr(momentum), _ptr(w8),
                                 _ptr(scale_w), _ptr(amax_w), _ptr(loss_scale), _ptr(growth_tracker),
                                 _ptr(found_inf), float(lr), float(momentum_coef), float(backoff),
                                 float(growth_factor), int(growth_interval), _stream(stream)))


def mp_master_step_adam(grad_bf16: torch.Tensor, master: torch.Tensor, exp_avg: torch.Tensor,
                        exp_avg_sq: torch.Tensor, w8: torch.Tensor, scale_w: torch.Tensor, amax_w: torch.Tensor,
                        loss_scale: torch.Tensor, growth_tracker: torch.Tensor, found_inf: torch.Tensor,
                        beta_pows: torch.Tensor, lr: float, beta1: float = 0.9, beta2: float = 0.999,
                        eps: float = 1e-8, backoff: float = 0.5, growth_factor: float = 2.0,
                        growth_interval: int = 2000, stream=None, grad_nonfinite: torch.Tensor | None = None,
                        w8_in: torch.Tensor | None = None, flags: int = 0, metas=None, amax_algo: int = AMAX_MOST_RECENT,
                        margin: int = 0) -> None:
    """Unscale, overflow skip, FP32 Adam update and E4M3 re-cast, in place
    (grad_nonfinite, w8_in, flags, metas, amax_algo, margin: as mp_master_step)."""
    n = grad_bf16.numel()
    if metas is not None:
        if grad_nonfinite is None:
            raise Fp8mpError(ERR_INVALID, "metas need grad_nonfinite (the prescanned step)")
        metas = list(metas)
        arr = (fp8mp_meta * max(1, len(metas)))(*[m.c_struct() for m in metas])
        _check(load().mp_master_step_adam_prescanned_scaling_ex(
            _ptr(grad_bf16), n, _ptr(master), _ptr(exp_avg), _ptr(exp_avg_sq), _ptr(w8_in), _ptr(w8),
            _ptr(scale_w), _ptr(amax_w), _ptr(loss_scale), _ptr(growth_tracker), _ptr(found_inf),
            _ptr(grad_nonfinite), _ptr(beta_pows), float(lr), float(beta1), float(beta2), float(eps),
            float(backoff), float(growth_factor), int(growth_interval), arr, len(metas), int(amax_algo),
            int(margin), int(flags), _stream(stream)))
        return
    if w8_in is not None or flags:
        if grad_nonfinite is None:
            raise Fp8mpError(ERR_INVALID, "w8_in and flags need grad_nonfinite (the prescanned step)")
        _check(load().mp_master_step_adam_prescanned_ex(
            _ptr(grad_bf16), n, _ptr(master), _ptr(exp_avg), _ptr(exp_avg_sq), _ptr(w8_in), _ptr(w8),
            _ptr(scale_w), _ptr(amax_w), _ptr(loss_scale), _ptr(growth_tracker), _ptr(found_inf),
            _ptr(grad_nonfinite), _ptr(beta_pows), float(lr), float(beta1), float(beta2), float(eps),
            float(backoff), float(growth_factor), int(growth_interval), int(flags), _stream(stream)))
        return
    if grad_nonfinite is not None:
        _check(load().mp_master_step_adam_prescanned(
            _ptr(grad_bf16), n, _ptr(master), _ptr(exp_avg), _ptr(exp_avg_sq), _ptr(w8), _ptr(scale_w),
            _ptr(amax_w), _ptr(loss_scale), _ptr(growth_tracker), _ptr(found_inf), _ptr(grad_nonfinite),
            _ptr(beta_pows), float(lr), float(beta1), float(beta2), float(eps), float(backoff), float(growth_factor),
            int(growth_interval), _stream(stream)))
        return
    _check(load().mp_master_step_adam(_ptr(grad_bf16), n, _ptr(master), _ptr(exp_avg), _ptr(exp_avg_sq), _ptr(w8),
                                      _ptr(scale_w), _ptr(amax_w), _ptr(loss_scale), _ptr(growth_tracker),
                                      _ptr(found_inf), _ptr(beta_pows), float(lr), float(beta1), float(beta2),
                                      float(eps), float(backoff), float(growth_factor), int(growth_interval),
                                      _stream(stream)))


def _shape(t: torch.Tensor, name: str, shape: tuple, *dtypes: torch.dtype) -> None:
    if t.shape != shape or t.dtype not in dtypes or not t.is_contiguous():
        raise Fp8mpError(ERR_INVALID, f"{name} must be a dense {tuple(shape)} of {' or '.join(map(str, dtypes))}, got "
                         f"{t.dtype} {tuple(t.shape)}")


def fp8_gated_fwd(x8: torch.Tensor, w8: torch.Tensor, sinv_x: torch.Tensor, sinv_w: torch.Tensor, h: torch.Tensor,
                  act: int = SILU, h_scale: torch.Tensor | None = None, h_amax: torch.Tensor | None = None,
                  gu: torch.Tensor | None = None, stream=None) -> None:
    """h[M, F] = act(x8 . wg^T) * (x8 . wu^T) with wg = w8[:F], wu = w8[F:] (w8
    is [2F, K]), both products times sinv_x * sinv_w: E4M3 codes (uint8) under
    h_scale, or bf16 without it. h_amax = max(h_amax, max|h|); gu [M, 2F] bf16
    receives the pre-activations for the backward pass. Any M."""
    M, K = x8.shape
    F = w8.shape[0] // 2
    _shape(x8, "x8", (M, K), torch.uint8)
    _shape(w8, "w8", (2 * F, K), torch.uint8)
    _shape(h, "h", (M, F), torch.uint8 if h_scale is not None else torch.bfloat16)
    if gu is not None:
        _shape(gu, "gu", (M, 2 * F), torch.bfloat16)
    _check(load().fp8_gated_fwd(_ptr(x8), _ptr(w8), M, F, K, act, _ptr(sinv_x), _ptr(sinv_w), _ptr(h_scale), _ptr(h),
                                _ptr(h_amax), _ptr(gu), _stream(stream)))


FEW_TOKENS = 128  # FP8MP_FEW_TOKENS: most tokens of fp8_linear_few


def fp8_linear_few(x8: torch.Tensor, w8: torch.Tensor, sinv_x: torch.Tensor, sinv_w: torch.Tensor, y: torch.Tensor,
                   bias: torch.Tensor | None = None, y_amax: torch.Tensor | None = None, stream=None) -> None:
    """fp8_linear_fwd for 0 to FEW_TOKENS tokens, any number of them:
    y[M, N] = (x8[M, K] . w8[N, K]^T) * sinv_x * sinv_w + bias."""
    M, K = x8.shape
    N = w8.shape[0]
    _shape(x8, "x8", (M, K), torch.uint8)
    _shape(w8, "w8", (N, K), torch.uint8)
    _shape(y, "y", (M, N), torch.bfloat16, torch.float32)
    if bias is not None:
        _shape(bias, "bias", (N,), torch.bfloat16, torch.float32)
    _check(load().fp8_linear_few(_ptr(x8), _ptr(w8), M, N, K, _ptr(sinv_x), _ptr(sinv_w), _ptr(bias),
                                 _dtype_code(bias) if bias is not None else F32, _ptr(y), _dtype_code(y),
                                 _ptr(y_amax), _stream(stream)))


def fp8_gated_dgrad(dy8: torch.Tensor, wd8: torch.Tensor, gu: torch.Tensor, sinv_dy: torch.Tensor,
                    sinv_wd: torch.Tensor, dgu_scale: torch.Tensor, dgu8: torch.Tensor, act: int = SILU,
                    dgu_amax: torch.Tensor | None = None, dy_fmt: int = E5M2, stream=None) -> None:
    """dgu8[M, 2F] = E5M2 codes of [dh u act'(g) | dh act(g)] under dgu_scale,
    with dh = (dy8 . wd8) * sinv_dy * sinv_wd from the output gradient's codes
    and the down projection's weight wd8 [N, F]."""
    M, N = dy8.shape
    F = wd8.shape[1]
    _shape(dy8, "dy8", (M, N), torch.uint8)
    _shape(wd8, "wd8", (N, F), torch.uint8)
    _shape(gu, "gu", (M, 2 * F), torch.bfloat16)
    _shape(dgu8, "dgu8", (M, 2 * F), torch.uint8)
    _check(load().fp8_gated_dgrad(_ptr(dy8), _ptr(wd8), _ptr(gu), M, F, N, act, dy_fmt, _ptr(sinv_dy), _ptr(sinv_wd),
                                  _ptr(dgu_scale), _ptr(dgu8), _ptr(dgu_amax), _stream(stream)))


def fp8_gated_bwd(dh: torch.Tensor | None, gu: torch.Tensor | None, x8: torch.Tensor, w8: torch.Tensor,
                  sinv_x: torch.Tensor, sinv_w: torch.Tensor, dgu_scale: torch.Tensor | None, dgu_sinv: torch.Tensor,
                  dgu8: torch.Tensor, dx: torch.Tensor | None, dw: torch.Tensor | None, act: int = SILU,
                  dgu_amax: torch.Tensor | None = None, dw_nonfinite: torch.Tensor | None = None, stream=None) -> None:
    """Backward pass of fp8_gated_fwd: dgu8 [M, 2F] from dh [M, F] (bf16 or
    fp32) and gu, unless dh is None (dgu8 holds fp8_gated_dgrad's codes); then
    dx[M, K] = (dgu8 . w8) * dgu_sinv * sinv_w and
    dw[2F, K] = (dgu8^T . x8) * dgu_sinv * sinv_x, either of which may be None."""
    M, K = x8.shape
    F = w8.shape[0] // 2
    _shape(x8, "x8", (M, K), torch.uint8)
    _shape(w8, "w8", (2 * F, K), torch.uint8)
    _shape(dgu8, "dgu8", (M, 2 * F), torch.uint8)
    high = (torch.bfloat16, torch.float32)
    if dh is not None:
        _shape(dh, "dh", (M, F), *high)
        if gu is None or dgu_scale is None:
            raise Fp8mpError(ERR_INVALID, "dh needs gu and dgu_scale")
        _shape(gu, "gu", (M, 2 * F), torch.bfloat16)
    for t, name, shape in ((dx, "dx", (M, K)), (dw, "dw", (2 * F, K))):
        if t is not None:
            _shape(t, name, shape, *high)
    _check(load().fp8_gated_bwd(_ptr(dh), _dtype_code(dh) if dh is not None else F32, _ptr(gu), _ptr(x8), _ptr(w8),
                                M, F, K, act, _ptr(sinv_x), _ptr(sinv_w), _ptr(dgu_scale), _ptr(dgu_sinv),
                                _ptr(dgu8), _ptr(dgu_amax), _ptr(dx), _dtype_code(dx) if dx is not None else F32,
                                _ptr(dw), _dtype_code(dw) if dw is not None else F32, _ptr(dw_nonfinite),
                                _stream(stream)))


class AdamWTensors:
    """The tensors of mp_grad_norm and mp_adamw_step: add each one once, keep
    the object over the steps. It holds references to every tensor it was
    given; set_grads replaces the gradients when a step has new ones, and
    release_grads lets go of them in between."""

    def __init__(self):
        self._rows, self._keep, self._sizes, self._array, self._released = [], [], [], None, False

    def __len__(self) -> int:
        return len(self._rows)

    def add(self, grad: torch.Tensor, master: torch.Tensor | None = None, exp_avg: torch.Tensor | None = None,
            exp_avg_sq: torch.Tensor | None = None, exp_avg_scale: torch.Tensor | None = None,
            exp_avg_sq_scale: torch.Tensor | None = None, copy: torch.Tensor | None = None,
            copy_scale: torch.Tensor | None = None, copy_amax: torch.Tensor | None = None,
            weight_decay: float = 0.0) -> None:
        """One tensor. grad: bf16 or fp32; master: fp32. Moments: fp32, or int8
        and uint8 codes with exp_avg_scale and exp_avg_sq_scale (fp32, one for
        each 256 elements). copy: uint8 (E4M3 codes under copy_scale, |w| into
        copy_amax), bf16, or None. For mp_grad_norm alone grad is enough."""
        n = grad.numel()
        bits = 32
        if master is not None:
            if exp_avg is None or exp_avg_sq is None:
                raise Fp8mpError(ERR_INVALID, "a master weight needs exp_avg and exp_avg_sq")
            bits = 8 if exp_avg.dtype == torch.int8 else 32
            state = (torch.int8, torch.uint8) if bits == 8 else (torch.float32, torch.float32)
            blocks = (n + 255) // 256
            _expect(master, "master", torch.float32, n)
            _expect(exp_avg, "exp_avg", state[0], n)
            _expect(exp_avg_sq, "exp_avg_sq", state[1], n)
            if bits == 8:
                if exp_avg_scale is None or exp_avg_sq_scale is None:
                    raise Fp8mpError(ERR_INVALID, "8-bit moments need exp_avg_scale and exp_avg_sq_scale")
                _expect(exp_avg_scale, "exp_avg_scale", torch.float32, blocks)
                _expect(exp_avg_sq_scale, "exp_avg_sq_scale", torch.float32, blocks)
            if copy is not None:
                _expect(copy, "copy", torch.bfloat16 if copy_scale is None else torch.uint8, n)
        dtype = self._checked(len(self._rows), n, grad)
        self._rows.append(fp8mp_adamw_tensor(
            grad.data_ptr(), _ptr(master), _ptr(exp_avg), _ptr(exp_avg_sq), _ptr(exp_avg_scale), _ptr(exp_avg_sq_scale),
            _ptr(copy), _ptr(copy_scale), _ptr(copy_amax), n, float(weight_decay), dtype, bits, 0))
        self._keep.append([grad, master, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, copy, copy_scale,
                           copy_amax])
        self._sizes.append(n)
        self._array = None

    @staticmethod
    def _checked(i: int, n: int, grad: torch.Tensor) -> int:
        """The type of a gradient that fits row i."""
        if grad.numel() != n or not grad.is_contiguous():
            raise Fp8mpError(ERR_INVALID, f"gradient {i} must be dense with {n} elements")
        return _dtype_code(grad)

    def set_grads(self, grads) -> None:
        """This step's gradients, one for each tensor, in the order of add."""
        grads = list(grads)
        if len(grads) != len(self._rows):
            raise Fp8mpError(ERR_INVALID, f"{len(grads)} gradients for {len(self._rows)} tensors")
        self._rows_array()
        dtypes = [self._checked(i, n, g) for i, (n, g) in enumerate(zip(self._sizes, grads))]
        for row, keep, g, dtype in zip(self._rows, self._keep, grads, dtypes):
            row.grad, row.grad_dtype = g.data_ptr(), dtype
            keep[0] = g
        self._released = False

    def release_grads(self) -> None:
        """Lets go of the gradients: set_grads has to give new ones before the next call."""
        for keep in self._keep:
            keep[0] = None
        self._released = bool(self._keep)

    def c_array(self):
        if self._released:
            raise Fp8mpError(ERR_INVALID, "the gradients were released: set_grads first")
        return self._rows_array()

    def _rows_array(self):
        if self._array is None:
            self._array = (fp8mp_adamw_tensor * max(1, len(self._rows)))(*self._rows)
            self._rows = [self._array[i] for i in range(len(self._rows))]
        return self._array


def _expect(t: torch.Tensor, name: str, dtype: torch.dtype, n: int) -> None:
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise Fp8mpError(ERR_INVALID, f"{name} must be dense {dtype} with {n} elements, got {t.dtype} with {t.numel()}")


def mp_adamw_workspace_bytes() -> int:
    return int(load().mp_adamw_workspace_bytes())


def _workspace(workspace: torch.Tensor):
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def mp_grad_norm(tensors: AdamWTensors, norm: torch.Tensor, found_inf: torch.Tensor, workspace: torch.Tensor,
                 stream=None) -> None:
    """norm = the 2-norm of all the tensors' gradients (under the loss scale),
    found_inf = 1 if their sum of squares is not finite in fp32, else 0. workspace: at
    least mp_adamw_workspace_bytes() bytes, zero-filled before its first use."""
    _check(load().mp_grad_norm(tensors.c_array(), len(tensors), _ptr(norm), _ptr(found_inf), *_workspace(workspace),
                               _stream(stream)))


def mp_adamw_step(tensors: AdamWTensors, loss_scale: torch.Tensor, growth_tracker: torch.Tensor,
                  found_inf: torch.Tensor, beta_pows: torch.Tensor, workspace: torch.Tensor, lr: float,
                  beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, seed: torch.Tensor | None = None,
                  grad_norm: torch.Tensor | None = None, max_norm: float = 0.0, backoff: float = 0.5,
                  growth_factor: float = 2.0, growth_interval: int = 2000, stream=None) -> None:
    """One AdamW step over all the tensors, in place: unscale, skip when
    found_inf is set, clip to max_norm by grad_norm (mp_grad_norm's), moments,
    weights, weight copies, then the loss scale. seed (int32[1], advanced by
    every step taken) is what 8-bit moments are rounded with."""
    _check(load().mp_adamw_step(tensors.c_array(), len(tensors), _ptr(loss_scale), _ptr(growth_tracker),
                                _ptr(found_inf), _ptr(beta_pows), _ptr(seed), _ptr(grad_norm), float(max_norm),
                                float(lr), float(beta1), float(beta2), float(eps), float(backoff),
                                float(growth_factor), int(growth_interval), *_workspace(workspace), _stream(stream)))


_HIGH = (torch.bfloat16, torch.float32)
_F32, _I64, _U8 = (torch.float32,), (torch.int64,), (torch.uint8,)
_CODE = {torch.float32: F32, torch.bfloat16: BF16}
MAX_NORM_COLS = 16384  # FP8MP_MAX_NORM_COLS
MAX_TOP = 32  # FP8MP_MAX_TOP


def _addresses(rows, stream):
    """The tensors' addresses (None for None) and the stream. rows: (tensor, name,
    shape or None, types); all must be dense and on the current CUDA device."""
    device, out = None, []
    for t, name, shape, dtypes in rows:
        if t is None:
            out.append(None)
            continue
        if t.dtype not in dtypes or not t.is_contiguous() or (shape is not None and t.shape != shape):
            raise Fp8mpError(ERR_INVALID, f"{name} must be a dense {shape if shape is not None else 'tensor'} of "
                             f"{' or '.join(map(str, dtypes))}, got {t.dtype} {tuple(t.shape)}")
        if device is None:
            device = t.get_device()
        elif t.get_device() != device:
            raise Fp8mpError(ERR_INVALID, f"{name} is on {t.device}, the others are not")
        out.append(t.data_ptr())
    if device is None or device < 0 or device != torch.cuda.current_device():
        raise Fp8mpError(ERR_INVALID, "the tensors must be on the current CUDA device")
    out.append(_stream(stream))
    return out


def fp8_rmsnorm_fwd(x: torch.Tensor, w: torch.Tensor, y: torch.Tensor, rstd: torch.Tensor, eps: float = 1e-6,
                    residual: torch.Tensor | None = None, total: torch.Tensor | None = None,
                    y_scale: torch.Tensor | None = None, y_amax: torch.Tensor | None = None, stream=None) -> None:
    """total = x + residual (x alone without one), rstd[m] = 1 / sqrt(mean(total^2) + eps),
    y[M, K] = total * rstd * w: E4M3 codes (uint8) under y_scale, or bf16 / fp32
    without it. y_amax = max(y_amax, max|y|). total may be residual itself."""
    shape = x.shape
    if len(shape) != 2:
        raise Fp8mpError(ERR_INVALID, f"x must be [M, K], got {tuple(shape)}")
    M, K = shape
    if (residual is None) != (total is None):
        raise Fp8mpError(ERR_INVALID, "residual and total come together")
    px, pw, py, pr, pres, ptot, ps, pa, st = _addresses((
        (x, "x", None, _HIGH), (w, "w", (K,), _HIGH), (y, "y", shape, _HIGH if y_scale is None else _U8),
        (rstd, "rstd", (M,), _F32), (residual, "residual", shape, _HIGH),
        (total, "total", shape, _HIGH if residual is None else (residual.dtype,)), (y_scale, "y_scale", (1,), _F32),
        (y_amax, "y_amax", (1,), _F32)), stream)
    _check(load().fp8_rmsnorm_fwd(px, _CODE[x.dtype], pres, ptot, F32 if residual is None else _CODE[residual.dtype], M, K,
                                  pw, _CODE[w.dtype], eps, ps, py, F32 if y_scale is not None else _CODE[y.dtype], pa, pr,
                                  st))


def fp8_rmsnorm_bwd_workspace_bytes(M: int, K: int) -> int:
    return int(load().fp8_rmsnorm_bwd_workspace_bytes(M, K))


def fp8_rmsnorm_bwd(dy: torch.Tensor, total: torch.Tensor, w: torch.Tensor, rstd: torch.Tensor,
                    dresidual: torch.Tensor, dw: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    dtotal: torch.Tensor | None = None, dx: torch.Tensor | None = None, stream=None) -> None:
    """Backward pass of fp8_rmsnorm_fwd: dresidual = the gradient of x and of the
    residual, from dy and the stream's own gradient dtotal (which dresidual may be
    itself); dx the same in dy's type; dw the weight's, which needs a workspace (uint8)
    of fp8_rmsnorm_bwd_workspace_bytes(M, K). total: x itself without a residual."""
    shape = dy.shape
    if len(shape) != 2:
        raise Fp8mpError(ERR_INVALID, f"dy must be [M, K], got {tuple(shape)}")
    M, K = shape
    if dw is not None and workspace is None:
        raise Fp8mpError(ERR_INVALID, "dw needs a workspace")
    like = (total.dtype,)
    pdy, pt, pw, pr, pdr, pdw, pws, pdt, pdx, st = _addresses((
        (dy, "dy", None, _HIGH), (total, "total", shape, _HIGH), (w, "w", (K,), _HIGH), (rstd, "rstd", (M,), _F32),
        (dresidual, "dresidual", shape, like), (dw, "dw", (K,), _HIGH), (workspace, "workspace", None, _U8),
        (dtotal, "dtotal", shape, like), (dx, "dx", shape, (dy.dtype,))), stream)
    _check(load().fp8_rmsnorm_bwd(pdy, _CODE[dy.dtype], pdt, pt, _CODE[total.dtype], pr, M, K, pw, _CODE[w.dtype], pdr, pdx,
                                  pdw, F32 if dw is None else _CODE[dw.dtype], pws,
                                  0 if workspace is None else workspace.numel(), st))


def _logits(logits: torch.Tensor, vocab: int | None):
    if logits.dim() != 2:
        raise Fp8mpError(ERR_INVALID, f"logits must be [M, columns], got {tuple(logits.shape)}")
    M, ld = logits.shape
    V = ld if vocab is None else int(vocab)
    if not 1 <= V <= ld:
        raise Fp8mpError(ERR_INVALID, f"vocab must lie in 1..{ld}, got {V}")
    return M, V, ld


def mp_logprobs_fwd(logits: torch.Tensor, targets: torch.Tensor | None, logprob: torch.Tensor | None,
                    stats: torch.Tensor, entropy: torch.Tensor | None = None, top_logprob: torch.Tensor | None = None,
                    top_id: torch.Tensor | None = None, vocab: int | None = None, stream=None) -> None:
    """logprob[m] = log p of targets[m] (int64; 0 where it is not in 0..V-1) under
    logits [M, columns], of which the first `vocab` (all, if None) count; stats [M, 2]
    = (largest logit, log of the sum of exp(logit - largest)); entropy [M]; the
    top_id.shape[1] (at most MAX_TOP) most probable tokens and their log p, of equal
    logits the lower index first."""
    M, V, ld = _logits(logits, vocab)
    if (targets is None) != (logprob is None) or (top_logprob is None) != (top_id is None):
        raise Fp8mpError(ERR_INVALID, "targets and logprob, top_logprob and top_id come together")
    top = 0
    if top_id is not None:
        top = top_id.shape[-1] if top_id.dim() == 2 else -1
        if not 0 <= top <= min(MAX_TOP, V):
            raise Fp8mpError(ERR_INVALID, f"top_id must be [M, 0..{min(MAX_TOP, V)}], got {tuple(top_id.shape)}")
    row = (M,)
    px, pt, pl, ps, pe, pv, pi, st = _addresses((
        (logits, "logits", None, _HIGH), (targets, "targets", row, _I64), (logprob, "logprob", row, _F32),
        (stats, "stats", (M, 2), _F32), (entropy, "entropy", row, _F32), (top_logprob, "top_logprob", (M, top), _F32),
        (top_id, "top_id", (M, top), _I64)), stream)
    _check(load().mp_logprobs_fwd(px, _CODE[logits.dtype], M, V, ld, pt, pl, ps, pe, pv, pi, top, st))


def mp_logprobs_bwd(logits: torch.Tensor, targets: torch.Tensor, stats: torch.Tensor, dlogprob: torch.Tensor,
                    dlogits: torch.Tensor, entropy: torch.Tensor | None = None, dentropy: torch.Tensor | None = None,
                    scale: torch.Tensor | None = None, amax: torch.Tensor | None = None, vocab: int | None = None,
                    stream=None) -> None:
    """The logits' gradient from those of logprob and entropy (with mp_logprobs_fwd's
    stats and entropy): dlogits [M, columns] in the logits' type, which may be logits
    itself, or E5M2 codes (uint8) under scale, with amax = max(amax, max|gradient|).
    Columns from `vocab` on get 0."""
    M, V, ld = _logits(logits, vocab)
    if (entropy is None) != (dentropy is None):
        raise Fp8mpError(ERR_INVALID, "entropy and dentropy come together")
    row = (M,)
    px, pt, ps, pa, pd, pe, pb, pc, pm, st = _addresses((
        (logits, "logits", None, _HIGH), (targets, "targets", row, _I64), (stats, "stats", (M, 2), _F32),
        (dlogprob, "dlogprob", row, _F32), (dlogits, "dlogits", (M, ld), (logits.dtype,) if scale is None else _U8),
        (entropy, "entropy", row, _F32), (dentropy, "dentropy", row, _F32), (scale, "scale", (1,), _F32),
        (amax, "amax", (1,), _F32)), stream)
    _check(load().mp_logprobs_bwd(px, _CODE[logits.dtype], M, V, ld, pt, ps, pa, pe, pb, pc, pd, pm, st))


def _table(ids: torch.Tensor, table: torch.Tensor, name: str):
    if table.dim() != 2 or ids.dim() != 1:
        raise Fp8mpError(ERR_INVALID, f"{name} must be [V, K] and ids [M], got {tuple(table.shape)}, {tuple(ids.shape)}")
    return ids.shape[0], *table.shape


def mp_embedding_fwd(ids: torch.Tensor, table: torch.Tensor, out: torch.Tensor, scale: float = 1.0,
                     sinv: torch.Tensor | None = None, stream=None) -> None:
    """out[m] = table[ids[m]] * scale (ids int64 [M]; zeros where an id is not in
    0..V-1). table [V, K]: bf16, fp32, or E4M3 codes (uint8) whose values sinv scales."""
    M, V, K = _table(ids, table, "table")
    pi, pt, po, ps, st = _addresses((
        (ids, "ids", None, _I64), (table, "table", None, _HIGH if sinv is None else _U8), (out, "out", (M, K), _HIGH),
        (sinv, "sinv", (1,), _F32)), stream)
    _check(load().mp_embedding_fwd(pi, M, pt, F32 if sinv is not None else _CODE[table.dtype], V, K, ps, scale, po,
                                   _CODE[out.dtype], st))


def mp_embedding_bwd_workspace_bytes(M: int, V: int, K: int) -> int:
    return int(load().mp_embedding_bwd_workspace_bytes(M, V, K))


def mp_embedding_bwd(ids: torch.Tensor, dy: torch.Tensor, dtable: torch.Tensor, workspace: torch.Tensor,
                     scale: float = 1.0, stream=None) -> None:
    """dtable[v] = scale * (sum of the dy[m] with ids[m] == v), for every row v of
    dtable [V, K]; the same bits at every call. workspace (uint8): at least
    mp_embedding_bwd_workspace_bytes(M, V, K)."""
    M, V, K = _table(ids, dtable, "dtable")
    pi, pd, pt, pw, st = _addresses((
        (ids, "ids", None, _I64), (dy, "dy", (M, K), _HIGH), (dtable, "dtable", None, _HIGH),
        (workspace, "workspace", None, _U8)), stream)
    _check(load().mp_embedding_bwd(pi, M, pd, _CODE[dy.dtype], V, K, scale, pt, _CODE[dtable.dtype], pw, workspace.numel(),
                                   st))


def fp8mp_check(stream=None) -> int:
    """Synchronises the stream and returns the library's check code (0 = OK)."""
    return int(load().fp8mp_check(_stream(stream)))


def fp8mp_selftest_timeout(stream=None) -> None:
    """Enqueues the kernel whose bounded wait runs out (about 2 s); the next
    fp8mp_check() on the stream then returns ERR_TIMEOUT."""
    _check(load().fp8mp_selftest_timeout(_stream(stream)))


def fp8mp_selftest_barrier_timeout(stream=None) -> None:
    """Enqueues the one-block kernel whose grid-barrier wait (the master
    step's) runs out (about 2 s); the next fp8mp_check() returns ERR_TIMEOUT."""
    _check(load().fp8mp_selftest_barrier_timeout(_stream(stream)))


def fp8mp_version() -> int:
    return int(load().fp8mp_version())
