"""SmoothQuant W8A8 linear layer for NVIDIA B200 (sm_100a) -- Python binding.

A thin ctypes layer over the C ABI in ``include/sq_w8a8.h`` (``libsq_w8a8.so``, built
in-tree by ``build.py``).  The functions keep the C names; they only marshal torch CUDA
tensors (device pointers, sizes, the current stream) and allocate outputs with torch's
allocator.  Every step runs in the library's CUDA kernels; there is no other code path:
if the library cannot be loaded, every call raises.

Pipeline ("4.2 W8A8 量化与 SmoothQuant", sec. 7.1):
  offline:  sq_calib_absmax / sq_calib_ln_absmax -> sq_smooth_factors -> sq_fold_quant_weights
  runtime:  sq_ln_smooth_quant -> sq_w8a8_gemm
FP8 (E4M3) variant of the quantised steps: sq_fold_quant_weights_fp8, sq_ln_smooth_quant_fp8,
sq_w8a8_gemm_fp8.
Weight-only 4-bit variant for a few tokens: sq_fold_quant_weights_w4, sq_w4_gemm, sq_w4_dequant,
and mixture-of-experts layers of such weights: sq_moe_w4, sq_moe_w4_routed.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import build as _build

SQ_F32, SQ_BF16, SQ_I32 = 0, 1, 2
SQ_MAX_K = 133136
SQ_MAX_K_ROW = 65536
_STATUS = {0: "SQ_OK", 1: "SQ_ERR_INVALID_ARG", 2: "SQ_ERR_UNSUPPORTED", 3: "SQ_ERR_ALIGNMENT",
           4: "SQ_ERR_CUDA", 5: "SQ_ERR_WORKSPACE"}

LIB_PATH = _build.LIB


class SQError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} returned {_STATUS.get(status, status)}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded C library (built first if sources are newer).  Raises if unavailable."""
    global _lib
    if _lib is None:
        if not _build.up_to_date():
            _build.build()
        L = ctypes.CDLL(LIB_PATH)
        P, I64, I, F, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        sigs = {
            "sq_calib_absmax": [P, I, I64, I64, I64, I, I, P, P],
            "sq_calib_ln_absmax": [P, I, I64, I64, I64, P, P, F, I, P, P],
            "sq_smooth_factors": [P, P, I64, F, P, P],
            "sq_fold_quant_weights": [P, I, I64, I64, I64, P, P, P, P, P, P, P, P],
            "sq_ln_smooth_quant": [P, I, I64, I64, I64, P, P, P, F, P, P, P],
            "sq_ln_smooth_quant_per_tensor": [P, I, I64, I64, I64, P, P, P, F, I, P, P, P, P],
            "sq_w8a8_gemm": [P, P, P, P, I64, I64, I64, P, I, I64, P, SZ, P],
            "sq_device_error": [P, I, P],
            "sq_fold_quant_weights_fp8": [P, I, I64, I64, I64, P, P, P, P, P, P, P, P],
            "sq_ln_smooth_quant_fp8": [P, I, I64, I64, I64, P, P, P, F, P, P, P],
            "sq_w8a8_gemm_fp8": [P, P, P, P, I64, I64, I64, P, I, I64, P, SZ, P],
            "sq_fold_next_smoothing": [P, P, I64, P, P],
            "sq_fold_kernel_launches": [P, I, I64, I64, I64],
            "sq_alpha_search": [P, I, I64, I64, I64, P, P, F, P, I, I64, I64, P, I, P, P, SZ, P],
            "sq_selfcheck_shared_divisor": [P, I64, P, I64, P, P, P],
            "sq_w8a8_gemm_rowmax": [P, P, P, P, I64, I64, I64, P, I, I64, P, P, SZ, P],
            "sq_quant_codes": [P, I, I64, I64, I64, P, P, P, P],
            "sq_set_wait_limit": [ctypes.c_uint64, P],
            "sq_fold_quant_weights_w4": [P, I, I64, I64, I64, P, P, P, I, P, P, P, P, P, P],
            "sq_w4_dequant": [P, P, P, I64, I64, I, P, I, I64, P],
            "sq_w4_gemm": [P, I, I64, I64, I64, P, P, P, I64, I, P, I, I64, P],
            "sq_moe_w4": [P, I, I64, I64, I64, P, I, I64, I, I, P, P, P, P, P, P, P, P, I64, I, P, I, I64, P, SZ, P],
            "sq_moe_w4_routed": [P, I, I64, I64, I64, P, P, I64, I, P, P, P, P, P, P, I64, I, P, I, I64, P, SZ, P],
        }
        for name, argt in sigs.items():
            fn = getattr(L, name)
            fn.argtypes = argt
            fn.restype = ctypes.c_int
        L.sq_w8a8_gemm_workspace_size.argtypes = [I64, I64, I64]
        L.sq_w8a8_gemm_workspace_size.restype = SZ
        L.sq_alpha_search_workspace_size.argtypes = [I64, I64, I64]
        L.sq_alpha_search_workspace_size.restype = SZ
        L.sq_moe_w4_workspace_size.argtypes = [I64, I64, I64, I64, I]
        L.sq_moe_w4_workspace_size.restype = SZ
        L.sq_w4_row_bytes.argtypes = [I64]
        L.sq_w4_row_bytes.restype = I64
        L.sq_status_string.argtypes = [I]
        L.sq_status_string.restype = ctypes.c_char_p
        L.sq_abi_version.argtypes = []
        L.sq_abi_version.restype = I
        _lib = L
    return _lib


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise SQError(fn, status)


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return SQ_BF16
    if t.dtype == torch.float32:
        return SQ_F32
    raise TypeError(f"expected a bfloat16 or float32 tensor, got {t.dtype}")


def _mat(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    if t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    return t


def _vec(t: torch.Tensor | None, n: int, name: str):
    if t is None:
        return None
    if t.dtype != torch.float32 or not t.is_cuda or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 CUDA vector of {n} elements")
    return t


# ----------------------------------------------------------------------------- the five calls
def sq_calib_absmax(x: torch.Tensor, axis: int, out: torch.Tensor | None = None, accumulate: bool = False,
                    stream=None) -> torch.Tensor:
    """axis 0: out[j] = max_i |x[i, j]|; axis 1: out[i] = max_j |x[i, j]|."""
    x = _mat(x, "x")
    n = x.shape[1] if axis == 0 else x.shape[0]
    if out is None:
        out = torch.empty(n, dtype=torch.float32, device=x.device)
    _vec(out, n, "out")
    _check("sq_calib_absmax", lib().sq_calib_absmax(_ptr(x), _dt(x), x.shape[0], x.shape[1], x.stride(0), axis,
                                                    int(accumulate), _ptr(out), _stream(stream)))
    return out


def sq_calib_ln_absmax(x: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor | None = None, eps: float = 1e-5,
                       out: torch.Tensor | None = None, accumulate: bool = False, stream=None) -> torch.Tensor:
    """out[j] = max_i |LayerNorm(x_i)_j| with gamma, beta (beta may be None)."""
    x = _mat(x, "x")
    K = x.shape[1]
    if out is None:
        out = torch.empty(K, dtype=torch.float32, device=x.device)
    _vec(out, K, "out")
    _vec(gamma, K, "gamma")
    _vec(beta, K, "beta")
    _check("sq_calib_ln_absmax", lib().sq_calib_ln_absmax(_ptr(x), _dt(x), x.shape[0], K, x.stride(0), _ptr(gamma),
                                                          _ptr(beta), float(eps), int(accumulate), _ptr(out),
                                                          _stream(stream)))
    return out


def sq_smooth_factors(ax: torch.Tensor, aw: torch.Tensor, alpha: float, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """s_j = ax_j^alpha / aw_j^(1 - alpha)."""
    K = ax.numel()
    _vec(ax, K, "ax")
    _vec(aw, K, "aw")
    if out is None:
        out = torch.empty(K, dtype=torch.float32, device=ax.device)
    _vec(out, K, "out")
    _check("sq_smooth_factors", lib().sq_smooth_factors(_ptr(ax), _ptr(aw), K, float(alpha), _ptr(out),
                                                        _stream(stream)))
    return out


def sq_fold_quant_weights(W: torch.Tensor, s: torch.Tensor, gamma: torch.Tensor | None = None,
                          beta: torch.Tensor | None = None, wq: torch.Tensor | None = None,
                          sw: torch.Tensor | None = None, gamma_f: torch.Tensor | None = None,
                          beta_f: torch.Tensor | None = None, stream=None):
    """W [K, N] -> (Wq [N, K] int8, sw [N], gamma / s or None, beta / s or None)."""
    W = _mat(W, "W")
    K, N = W.shape
    _vec(s, K, "s")
    _vec(gamma, K, "gamma")
    _vec(beta, K, "beta")
    dev = W.device
    if wq is None:
        wq = torch.empty(N, K, dtype=torch.int8, device=dev)
    if sw is None:
        sw = torch.empty(N, dtype=torch.float32, device=dev)
    gf = bf = None
    if gamma is not None:
        gf = gamma_f if gamma_f is not None else torch.empty(K, dtype=torch.float32, device=dev)
    if beta is not None:
        bf = beta_f if beta_f is not None else torch.empty(K, dtype=torch.float32, device=dev)
    _check("sq_fold_quant_weights",
           lib().sq_fold_quant_weights(_ptr(W), _dt(W), K, N, W.stride(0), _ptr(s), _ptr(gamma), _ptr(beta),
                                       _ptr(wq), _ptr(sw), _ptr(gf), _ptr(bf), _stream(stream)))
    return wq, sw, gf, bf


def sq_fold_next_smoothing(sw: torch.Tensor, s_next: torch.Tensor, out: torch.Tensor | None = None,
                           stream=None) -> torch.Tensor:
    """sw / s_next: this linear's output scales with the next linear's smoothing folded in."""
    N = sw.shape[0]
    _vec(sw, N, "sw")
    _vec(s_next, N, "s_next")
    if out is None:
        out = torch.empty_like(sw)
    _check("sq_fold_next_smoothing", lib().sq_fold_next_smoothing(_ptr(sw), _ptr(s_next), N, _ptr(out),
                                                                  _stream(stream)))
    return out


def sq_ln_smooth_quant(x: torch.Tensor, gamma_f: torch.Tensor | None = None, beta_f: torch.Tensor | None = None,
                       s: torch.Tensor | None = None, eps: float = 1e-5, xq: torch.Tensor | None = None,
                       sx: torch.Tensor | None = None, stream=None):
    """LayerNorm mode (gamma_f given) or plain mode (s given) -> (xq [M, K] int8, sx [M])."""
    x = _mat(x, "x")
    M, K = x.shape
    _vec(gamma_f, K, "gamma_f")
    _vec(beta_f, K, "beta_f")
    _vec(s, K, "s")
    if xq is None:
        xq = torch.empty(M, K, dtype=torch.int8, device=x.device)
    if sx is None:
        sx = torch.empty(M, dtype=torch.float32, device=x.device)
    _check("sq_ln_smooth_quant", lib().sq_ln_smooth_quant(_ptr(x), _dt(x), M, K, x.stride(0), _ptr(gamma_f),
                                                          _ptr(beta_f), _ptr(s), float(eps), _ptr(xq), _ptr(sx),
                                                          _stream(stream)))
    return xq, sx


def sq_ln_smooth_quant_per_tensor(x: torch.Tensor, gamma_f: torch.Tensor | None = None,
                                  beta_f: torch.Tensor | None = None, s: torch.Tensor | None = None,
                                  eps: float = 1e-5, scale: torch.Tensor | None = None, static: bool = False,
                                  xq: torch.Tensor | None = None, sx: torch.Tensor | None = None, stream=None):
    """One scale for the whole tensor: dynamic (max|y|/127, written to `scale`) or static (the
    calibrated value in `scale`).  Returns (xq [M, K] int8, sx [M] = scale, scale [1])."""
    x = _mat(x, "x")
    M, K = x.shape
    _vec(gamma_f, K, "gamma_f")
    _vec(beta_f, K, "beta_f")
    _vec(s, K, "s")
    if scale is None:
        if static:
            raise ValueError("a static per-tensor scale must be given")
        scale = torch.empty(1, dtype=torch.float32, device=x.device)
    _vec(scale, 1, "scale")
    if xq is None:
        xq = torch.empty(M, K, dtype=torch.int8, device=x.device)
    if sx is None:
        sx = torch.empty(M, dtype=torch.float32, device=x.device)
    _check("sq_ln_smooth_quant_per_tensor",
           lib().sq_ln_smooth_quant_per_tensor(_ptr(x), _dt(x), M, K, x.stride(0), _ptr(gamma_f), _ptr(beta_f),
                                               _ptr(s), float(eps), int(static), _ptr(scale), _ptr(xq), _ptr(sx),
                                               _stream(stream)))
    return xq, sx, scale


def sq_fold_kernel_launches(W: torch.Tensor) -> int:
    """Kernels sq_fold_quant_weights(W, ...) launches (1, or 3 on the streaming route)."""
    W = _mat(W, "W")
    K, N = W.shape
    return int(lib().sq_fold_kernel_launches(_ptr(W), _dt(W), K, N, W.stride(0)))


def sq_w8a8_gemm_workspace_size(M: int, N: int, K: int) -> int:
    return int(lib().sq_w8a8_gemm_workspace_size(M, N, K))


_ODT = {torch.bfloat16: SQ_BF16, torch.float32: SQ_F32, torch.int32: SQ_I32}


def sq_w8a8_gemm(xq: torch.Tensor, sx: torch.Tensor | None, wq: torch.Tensor, sw: torch.Tensor | None,
                 out_dtype: torch.dtype = torch.bfloat16, y: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = bf16(((float)(xq @ wq^T) * sx[:, None]) * sw[None, :]) (or f32 / raw int32)."""
    if xq.dtype != torch.int8 or wq.dtype != torch.int8 or not xq.is_contiguous() or not wq.is_contiguous():
        raise ValueError("xq and wq must be contiguous int8 tensors")
    M, K = xq.shape
    N = wq.shape[0]
    if wq.shape[1] != K:
        raise ValueError("xq and wq disagree on K")
    if y is None:
        y = torch.empty(M, N, dtype=out_dtype, device=xq.device)
    ydt = _ODT[y.dtype]
    if ydt != SQ_I32:
        _vec(sx, M, "sx")
        _vec(sw, N, "sw")
    need = sq_w8a8_gemm_workspace_size(M, N, K)
    if workspace is None and need > 0:
        workspace = torch.zeros(need, dtype=torch.uint8, device=xq.device)  # its counters start at zero
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("sq_w8a8_gemm", lib().sq_w8a8_gemm(_ptr(xq), _ptr(sx), _ptr(wq), _ptr(sw), M, N, K, _ptr(y), ydt,
                                              y.stride(0), _ptr(workspace), ws_bytes, _stream(stream)))
    return y


def sq_w8a8_gemm_rowmax(xq: torch.Tensor, sx: torch.Tensor, wq: torch.Tensor, sw: torch.Tensor,
                        out_dtype: torch.dtype = torch.bfloat16, y: torch.Tensor | None = None,
                        rowmax: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """sq_w8a8_gemm that also returns rowmax[m] = max_n |y[m, n]| of the stored outputs (the next
    linear's per-token statistic).  Returns (y, rowmax)."""
    if xq.dtype != torch.int8 or wq.dtype != torch.int8 or not xq.is_contiguous() or not wq.is_contiguous():
        raise ValueError("xq and wq must be contiguous int8 tensors")
    M, K = xq.shape
    N = wq.shape[0]
    if wq.shape[1] != K:
        raise ValueError("xq and wq disagree on K")
    if y is None:
        y = torch.empty(M, N, dtype=out_dtype, device=xq.device)
    if rowmax is None:
        rowmax = torch.empty(M, dtype=torch.float32, device=xq.device)
    _vec(sx, M, "sx")
    _vec(sw, N, "sw")
    _vec(rowmax, M, "rowmax")
    need = sq_w8a8_gemm_workspace_size(M, N, K)
    if workspace is None and need > 0:
        workspace = torch.zeros(need, dtype=torch.uint8, device=xq.device)  # its sums start at zero
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("sq_w8a8_gemm_rowmax", lib().sq_w8a8_gemm_rowmax(_ptr(xq), _ptr(sx), _ptr(wq), _ptr(sw), M, N, K, _ptr(y),
                                                            _ODT[y.dtype], y.stride(0), _ptr(rowmax), _ptr(workspace),
                                                            ws_bytes, _stream(stream)))
    return y, rowmax


def sq_quant_codes(x: torch.Tensor, rowmax: torch.Tensor, xq: torch.Tensor | None = None,
                   sx: torch.Tensor | None = None, stream=None):
    """Per-token INT8 codes of x given its row maxima: (xq [M, K] int8, sx [M] = rowmax / 127)."""
    x = _mat(x, "x")
    M, K = x.shape
    _vec(rowmax, M, "rowmax")
    if xq is None:
        xq = torch.empty(M, K, dtype=torch.int8, device=x.device)
    if sx is None:
        sx = torch.empty(M, dtype=torch.float32, device=x.device)
    _check("sq_quant_codes", lib().sq_quant_codes(_ptr(x), _dt(x), M, K, x.stride(0), _ptr(rowmax), _ptr(xq), _ptr(sx),
                                                  _stream(stream)))
    return xq, sx


# ----------------------------------------------------------------------------- alpha search
def alpha_grid(n: int = 20) -> list:
    """n migration strengths evenly covering [0, 1] (both ends included)."""
    return [i / (n - 1) for i in range(n)] if n > 1 else [0.5]


def sq_alpha_search(x: torch.Tensor, W: torch.Tensor, alphas=None, gamma: torch.Tensor | None = None,
                    beta: torch.Tensor | None = None, eps: float = 1e-5, workspace: torch.Tensor | None = None,
                    stream=None):
    """Relative squared layer-output error of the W8A8 layer on the calibration batch x for each
    alpha (default: 20 values over [0, 1]).  Returns (err [n] float64 on the device, alphas)."""
    x = _mat(x, "x")
    W = _mat(W, "W")
    M, K = x.shape
    N = W.shape[1]
    if W.shape[0] != K:
        raise ValueError("x and W disagree on K")
    _vec(gamma, K, "gamma")
    _vec(beta, K, "beta")
    alphas = alpha_grid() if alphas is None else [float(a) for a in alphas]
    arr = (ctypes.c_float * len(alphas))(*alphas)
    err = torch.empty(len(alphas), dtype=torch.float64, device=x.device)
    need = int(lib().sq_alpha_search_workspace_size(M, K, N))
    if need == (1 << 64) - 1:
        raise ValueError("unsupported sizes for the alpha search")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    _check("sq_alpha_search",
           lib().sq_alpha_search(_ptr(x), _dt(x), M, K, x.stride(0), _ptr(gamma), _ptr(beta), float(eps), _ptr(W),
                                 _dt(W), N, W.stride(0), arr, len(alphas), _ptr(err), _ptr(workspace), ws_bytes,
                                 _stream(stream)))
    return err, alphas


# ----------------------------------------------------------------------------- FP8 (E4M3) variant
# Codes are uint8 tensors holding E4M3 bit patterns (view them as torch.float8_e4m3fn if
# wanted); scales are max / 448.
def sq_fold_quant_weights_fp8(W: torch.Tensor, s: torch.Tensor, gamma: torch.Tensor | None = None,
                              beta: torch.Tensor | None = None, wq: torch.Tensor | None = None,
                              sw: torch.Tensor | None = None, gamma_f: torch.Tensor | None = None,
                              beta_f: torch.Tensor | None = None, stream=None):
    """W [K, N] -> (Wq [N, K] E4M3 codes (uint8), sw [N], gamma / s or None, beta / s or None)."""
    W = _mat(W, "W")
    K, N = W.shape
    _vec(s, K, "s")
    _vec(gamma, K, "gamma")
    _vec(beta, K, "beta")
    dev = W.device
    if wq is None:
        wq = torch.empty(N, K, dtype=torch.uint8, device=dev)
    if sw is None:
        sw = torch.empty(N, dtype=torch.float32, device=dev)
    gf = bf = None
    if gamma is not None:
        gf = gamma_f if gamma_f is not None else torch.empty(K, dtype=torch.float32, device=dev)
    if beta is not None:
        bf = beta_f if beta_f is not None else torch.empty(K, dtype=torch.float32, device=dev)
    _check("sq_fold_quant_weights_fp8",
           lib().sq_fold_quant_weights_fp8(_ptr(W), _dt(W), K, N, W.stride(0), _ptr(s), _ptr(gamma), _ptr(beta),
                                           _ptr(wq), _ptr(sw), _ptr(gf), _ptr(bf), _stream(stream)))
    return wq, sw, gf, bf


def sq_ln_smooth_quant_fp8(x: torch.Tensor, gamma_f: torch.Tensor | None = None, beta_f: torch.Tensor | None = None,
                           s: torch.Tensor | None = None, eps: float = 1e-5, xq: torch.Tensor | None = None,
                           sx: torch.Tensor | None = None, stream=None):
    """LayerNorm mode (gamma_f given) or plain mode (s given) -> (xq [M, K] E4M3 codes, sx [M])."""
    x = _mat(x, "x")
    M, K = x.shape
    _vec(gamma_f, K, "gamma_f")
    _vec(beta_f, K, "beta_f")
    _vec(s, K, "s")
    if xq is None:
        xq = torch.empty(M, K, dtype=torch.uint8, device=x.device)
    if sx is None:
        sx = torch.empty(M, dtype=torch.float32, device=x.device)
    _check("sq_ln_smooth_quant_fp8",
           lib().sq_ln_smooth_quant_fp8(_ptr(x), _dt(x), M, K, x.stride(0), _ptr(gamma_f), _ptr(beta_f), _ptr(s),
                                        float(eps), _ptr(xq), _ptr(sx), _stream(stream)))
    return xq, sx


def sq_w8a8_gemm_fp8(xq: torch.Tensor, sx: torch.Tensor, wq: torch.Tensor, sw: torch.Tensor,
                     out_dtype: torch.dtype = torch.bfloat16, y: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y = bf16((acc * sx[:, None]) * sw[None, :]) with acc = dec(xq) @ dec(wq)^T in fp32 (or f32 y)."""
    if xq.dtype != torch.uint8 or wq.dtype != torch.uint8 or not xq.is_contiguous() or not wq.is_contiguous():
        raise ValueError("xq and wq must be contiguous uint8 tensors of E4M3 codes")
    M, K = xq.shape
    N = wq.shape[0]
    if wq.shape[1] != K:
        raise ValueError("xq and wq disagree on K")
    if y is None:
        y = torch.empty(M, N, dtype=out_dtype, device=xq.device)
    ydt = _ODT[y.dtype]
    _vec(sx, M, "sx")
    _vec(sw, N, "sw")
    need = sq_w8a8_gemm_workspace_size(M, N, K)
    if workspace is None and need > 0:
        workspace = torch.zeros(need, dtype=torch.uint8, device=xq.device)  # its counters start at zero
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check("sq_w8a8_gemm_fp8", lib().sq_w8a8_gemm_fp8(_ptr(xq), _ptr(sx), _ptr(wq), _ptr(sw), M, N, K, _ptr(y), ydt,
                                                      y.stride(0), _ptr(workspace), ws_bytes, _stream(stream)))
    return y


def sq_selfcheck_shared_divisor(a: torch.Tensor, b: torch.Tensor, want_quotients: bool = False, stream=None):
    """Checks the library's shared-divisor quotient against IEEE division for every pair
    (a[j], b[i]).  Returns ([scalar mismatches, packed mismatches, pairs checked] as a CUDA int64
    tensor, quotients [nb, na] or None)."""
    _vec(a, a.numel(), "a")
    _vec(b, b.numel(), "b")
    counts = torch.zeros(3, dtype=torch.int64, device=a.device)
    q = torch.empty(b.numel(), a.numel(), dtype=torch.float32, device=a.device) if want_quotients else None
    _check("sq_selfcheck_shared_divisor", lib().sq_selfcheck_shared_divisor(_ptr(a), a.numel(), _ptr(b), b.numel(),
                                                                            _ptr(q), _ptr(counts), _stream(stream)))
    return counts, q


# ----------------------------------------------------------------------------- 4-bit weights
# A packed weight is (wq [N, sq_w4_row_bytes(K)] uint8, sg [ceil(K / group), N] bfloat16, zp uint8
# like sg or None); experts stack these on a leading dimension.  Calls run on the tensors' own
# device: its current stream is taken unless `stream` is given, and what a call allocates (outputs,
# a workspace and its zeros) belongs to the stream it runs on.  In decode a call's host time
# counts, so the checks are few steps where everything is right; what is wrong is found out after.
def sq_w4_row_bytes(K: int) -> int:
    return (K + 127) // 128 * 64


_BF16, _F32, _U8, _I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32
_FDT = {_BF16: SQ_BF16, _F32: SQ_F32}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on(stream, like: torch.Tensor):
    """The context of a call on `stream`: it is the current one while the call allocates and launches."""
    if stream.device_index != like.get_device():
        raise ValueError("the stream belongs to another device than the tensors")
    return torch.cuda.stream(stream)


def _call(fn: str, dev: int, *args):
    """One library call on the current stream of device `dev`, made the current one for it if it is not."""
    f, raw = getattr(_lib or lib(), fn), _raw_stream(dev)
    if dev == _current_device():
        status = f(*args, raw)
    else:
        with torch.cuda.device(dev):
            status = f(*args, raw)
    if status != 0:
        raise SQError(fn, status)


def _float_mat(t: torch.Tensor, name: str) -> int:
    """The library's type of a bfloat16 or float32 matrix with unit column stride."""
    dt = _FDT.get(t.dtype)
    if dt is None or not t.is_cuda or t.dim() != 2 or t.stride(1) != 1:
        _mat(t, name)
        _dt(t)
    return dt


def _same(t, shape: tuple, dtype, dev: int) -> bool:
    return t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()


def _check_packed(name: str, wq, sg, zp, lead: tuple, K: int, group: int, dev: int):
    """Checks one packed weight: codes [*lead, row bytes], scales (and zero points) [.., groups, N]."""
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    codes, scales = (*lead, sq_w4_row_bytes(K)), (*lead[:-1], -(-K // group), lead[-1])
    if dev < 0:
        raise ValueError("expected CUDA tensors")
    if not _same(wq, codes, _U8, dev):
        raise ValueError(f"{name}: codes must be contiguous uint8 {codes} on the input's device")
    if not _same(sg, scales, _BF16, dev):
        raise ValueError(f"{name}: scales must be contiguous bfloat16 {scales} on the input's device")
    if zp is not None and not _same(zp, scales, _U8, dev):
        raise ValueError(f"{name}: zero points must be contiguous uint8 {scales} on the input's device")


def _ptr0(t):
    return None if t is None else t.data_ptr()


def _out(like, y, shape: tuple, dtype):
    """y, or a new tensor on the device of `like`; and the library's type of it."""
    if y is None:
        y = like.new_empty(shape) if dtype is like.dtype else like.new_empty(shape, dtype=dtype)
    elif y.shape != shape or y.device != like.device or y.stride(-1) != 1:
        raise ValueError(f"y must be {shape} with unit column stride, on the input's device")
    dt = _FDT.get(y.dtype)
    if dt is None:
        raise TypeError(f"expected a bfloat16 or float32 output, got {y.dtype}")
    return y, dt


def sq_fold_quant_weights_w4(W: torch.Tensor, s: torch.Tensor | None = None, gamma: torch.Tensor | None = None,
                             beta: torch.Tensor | None = None, group: int = 128, asym: bool = False,
                             wq: torch.Tensor | None = None, sg: torch.Tensor | None = None,
                             zp: torch.Tensor | None = None, stream=None):
    """W [K, N] -> (wq packed, sg, zp or None, gamma / s or None, beta / s or None).  asym: with zero points."""
    if stream is not None:
        with _on(stream, W):
            return sq_fold_quant_weights_w4(W, s, gamma, beta, group, asym, wq, sg, zp)
    dt = _float_mat(W, "W")
    K, N = W.shape
    dev = W.get_device()
    for v, name in ((s, "s"), (gamma, "gamma"), (beta, "beta")):
        if v is not None:
            _vec(v, K, name)
            if v.get_device() != dev:
                raise ValueError(f"{name} must be on W's device")
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128")
    if not asym and zp is not None:
        raise ValueError("zero points are written only with asym=True")
    given = wq is not None or sg is not None or zp is not None
    groups = -(-K // group)
    if wq is None:
        wq = W.new_empty((N, sq_w4_row_bytes(K)), dtype=_U8)
    if sg is None:
        sg = W.new_empty((groups, N), dtype=_BF16)
    if asym and zp is None:
        zp = W.new_empty((groups, N), dtype=_U8)
    if given:
        _check_packed("W", wq, sg, zp, (N,), K, group, dev)
    gf = torch.empty_like(gamma) if gamma is not None else None
    bf = torch.empty_like(beta) if beta is not None else None
    _call("sq_fold_quant_weights_w4", dev, W.data_ptr(), dt, K, N, W.stride(0), _ptr0(s), _ptr0(gamma),
          _ptr0(beta), group, wq.data_ptr(), sg.data_ptr(), _ptr0(zp), _ptr0(gf), _ptr0(bf))
    return wq, sg, zp, gf, bf


def sq_w4_dequant(wq: torch.Tensor, sg: torch.Tensor, zp: torch.Tensor | None = None, *, K: int, group: int = 128,
                  out_dtype: torch.dtype = torch.bfloat16, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values [N, K] that a packed weight stands for: (code - zero) * scale."""
    if stream is not None:
        with _on(stream, wq):
            return sq_w4_dequant(wq, sg, zp, K=K, group=group, out_dtype=out_dtype, y=y)
    if wq.dim() != 2:
        raise ValueError("wq must be 2-D")
    N, dev = wq.shape[0], wq.get_device()
    _check_packed("wq", wq, sg, zp, (N,), K, group, dev)
    y, ydt = _out(sg, y, (N, K), out_dtype)
    _call("sq_w4_dequant", dev, wq.data_ptr(), sg.data_ptr(), _ptr0(zp), K, N, group, y.data_ptr(), ydt,
          y.stride(0))
    return y


def sq_w4_gemm(x: torch.Tensor, wq: torch.Tensor, sg: torch.Tensor, zp: torch.Tensor | None = None, group: int = 128,
               out_dtype: torch.dtype = torch.bfloat16, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [M, N] = x [M, K] @ values(wq, sg, zp) [N, K]^T, for a few tokens."""
    if stream is not None:
        with _on(stream, x):
            return sq_w4_gemm(x, wq, sg, zp, group, out_dtype, y)
    dt = _float_mat(x, "x")
    M, K = x.shape
    N, dev = wq.shape[0], x.get_device()
    _check_packed("wq", wq, sg, zp, (N,), K, group, dev)
    y, ydt = _out(x, y, (M, N), out_dtype)
    _call("sq_w4_gemm", dev, x.data_ptr(), dt, M, K, x.stride(0), wq.data_ptr(), sg.data_ptr(),
          None if zp is None else zp.data_ptr(), N, group, y.data_ptr(), ydt, y.stride(0))
    return y


def sq_moe_w4_workspace_size(T: int, D: int, F: int, E: int, top_k: int) -> int:
    n = int(lib().sq_moe_w4_workspace_size(T, D, F, E, top_k))
    if n == (1 << 64) - 1:
        raise ValueError("sizes outside the mixture-of-experts layer's limits")
    return n


def sq_moe_w4_workspace(T: int, D: int, F: int, E: int, top_k: int, device="cuda") -> torch.Tensor:
    """A workspace for sq_moe_w4 and sq_moe_w4_routed, for these sizes and smaller ones; calls that share it must be
    ordered."""
    return torch.zeros(sq_moe_w4_workspace_size(T, D, F, E, top_k), dtype=torch.uint8, device=device)


def _moe(fn, x, dt, E, k, route, w13, s13, w2, s2, z13, z2, group, out_dtype, y, workspace):
    T, D = x.shape
    dev = x.get_device()
    if w13.dim() != 3 or w13.shape[1] % 2:
        raise ValueError("w13 must be [E, 2 F, row bytes]")
    F = w13.shape[1] // 2
    if (z13 is None) != (z2 is None):
        raise ValueError("zero points are given for both weights or for neither")
    _check_packed("w13", w13, s13, z13, (E, 2 * F), D, group, dev)
    _check_packed("w2", w2, s2, z2, (E, D), F, group, dev)
    y, ydt = _out(x, y, (T, D), out_dtype)
    if workspace is None:
        workspace = sq_moe_w4_workspace(T, D, F, E, k, x.device)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous and on the input's device")
    _call(fn, dev, x.data_ptr(), dt, T, D, x.stride(0), *route, w13.data_ptr(), s13.data_ptr(), _ptr0(z13),
          w2.data_ptr(), s2.data_ptr(), _ptr0(z2), F, group, y.data_ptr(), ydt, y.stride(0), workspace.data_ptr(),
          workspace.nbytes)
    return y


def sq_moe_w4(x: torch.Tensor, wr: torch.Tensor, top_k: int, w13: torch.Tensor, s13: torch.Tensor, w2: torch.Tensor,
              s2: torch.Tensor, z13: torch.Tensor | None = None, z2: torch.Tensor | None = None, group: int = 128,
              renorm: bool = True, out_dtype: torch.dtype = torch.bfloat16, y: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, stream=None):
    """A mixture-of-experts layer for a few tokens: router wr [E, D], the top_k experts of each token (softmax
    weights, divided by their sum if renorm), silu(gate) * up, weighted sum.  Returns (y [T, D], ids [T, top_k]
    int32, weights [T, top_k] float32).  workspace: sq_moe_w4_workspace, made for the call if not given."""
    if stream is not None:
        with _on(stream, x):
            return sq_moe_w4(x, wr, top_k, w13, s13, w2, s2, z13, z2, group, renorm, out_dtype, y, workspace)
    dt, rdt = _float_mat(x, "x"), _float_mat(wr, "wr")
    T, E = x.shape[0], wr.shape[0]
    if wr.shape[1] != x.shape[1] or not wr.is_contiguous() or wr.get_device() != x.get_device():
        raise ValueError("wr must be contiguous [E, D] on the input's device")
    if not 0 < top_k <= E:
        raise ValueError("top_k must be between 1 and the number of experts")
    ids = x.new_empty((T, top_k), dtype=_I32)
    wts = x.new_empty((T, top_k), dtype=_F32)
    y = _moe("sq_moe_w4", x, dt, E, top_k, (wr.data_ptr(), rdt, E, top_k, int(renorm), ids.data_ptr(), wts.data_ptr()),
             w13, s13, w2, s2, z13, z2, group, out_dtype, y, workspace)
    return y, ids, wts


def sq_moe_w4_routed(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, w13: torch.Tensor, s13: torch.Tensor,
                     w2: torch.Tensor, s2: torch.Tensor, z13: torch.Tensor | None = None,
                     z2: torch.Tensor | None = None, group: int = 128, out_dtype: torch.dtype = torch.bfloat16,
                     y: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The experts of sq_moe_w4 for given choices: ids [T, top_k] int32 (outside [0, E): left out) and weights
    [T, top_k] float32."""
    if stream is not None:
        with _on(stream, x):
            return sq_moe_w4_routed(x, ids, weights, w13, s13, w2, s2, z13, z2, group, out_dtype, y, workspace)
    dt = _float_mat(x, "x")
    T, E, k, dev = x.shape[0], w13.shape[0], ids.shape[-1], x.get_device()
    if not _same(ids, (T, k), _I32, dev) or not _same(weights, (T, k), _F32, dev):
        raise ValueError("ids must be contiguous int32 and weights contiguous float32 [T, top_k], on the input's device")
    return _moe("sq_moe_w4_routed", x, dt, E, k, (ids.data_ptr(), weights.data_ptr(), E, k), w13, s13, w2, s2, z13, z2,
                group, out_dtype, y, workspace)


WAIT_LIMIT_DEFAULT_NS = 10 * 1000 * 1000 * 1000


def sq_set_wait_limit(ns: int, stream=None) -> None:
    """Limit of the kernels' bounded waits on this device (0: every wait runs out at once)."""
    _check("sq_set_wait_limit", lib().sq_set_wait_limit(int(ns), _stream(stream)))


def sq_device_error(clear: bool = True, stream=None) -> int:
    """Device error word (non-zero when a kernel gave up on a bounded wait)."""
    code = ctypes.c_uint(0)
    _check("sq_device_error", lib().sq_device_error(ctypes.byref(code), int(clear), _stream(stream)))
    return code.value


def loaded_library_path() -> str:
    return os.path.realpath(LIB_PATH)
