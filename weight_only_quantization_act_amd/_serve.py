"""ctypes binding of the serving operators (include/awq_serve.h): argument marshalling only.

Same rules as the rest of the binding: tensors are checked for dtype, device and layout, raw
device pointers and the current HIP stream go to the C ABI, non-zero status codes raise, and
there is no fallback.  Unlike the rest, row strides are free where the C ABI takes them, so
views into a fused projection's output need no copy.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._lib import _buf, _check, _dev, _i32, _i64, _on_stream, _ptr, _stream_ptr, _sz, _vp
from ._lib import lib as _base_lib

AWQ_FP16, AWQ_BF16 = 0, 1
AWQ_FOLD_DIVIDE, AWQ_FOLD_MULTIPLY = 0, 1

_SIGNATURES = {
    "awq_int8_quantize": (ctypes.c_int, [_vp, _i64, _i64, _i64, _i32, _vp, _i32, _vp, _i64, _vp,
                                         _vp]),
    "awq_int8_matmul_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "awq_int8_matmul": (ctypes.c_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i32,
                                       _vp, _i64, _vp, _sz, _vp]),
    "awq_int8_linear_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "awq_int8_linear": (ctypes.c_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i32,
                                       _vp, _i64, _vp, _sz, _vp]),
}

_BOUND: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    """libawq_act.so with the serving entry points' signatures set."""
    global _BOUND
    if _BOUND is None:
        L = _base_lib()
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _BOUND = L
    return _BOUND


_DTYPES = {torch.float16: AWQ_FP16, torch.bfloat16: AWQ_BF16}


def _dtype(dtype: torch.dtype, name: str) -> int:
    if dtype not in _DTYPES:
        raise TypeError(f"{name} must be torch.float16 or torch.bfloat16, got {dtype}")
    return _DTYPES[dtype]


def _rows(t: torch.Tensor, name: str, dtype: Optional[torch.dtype] = None) -> int:
    """Check a 2-D device tensor with unit stride along its rows; returns the row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device (HIP) tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be contiguous along its rows")
    ld = t.stride(0) if rows > 1 and cols > 0 else cols
    if ld < cols:
        raise ValueError(f"{name} has overlapping rows (stride {ld} for {cols} columns)")
    return ld


def _addr(t: Optional[torch.Tensor], other: torch.Tensor) -> Optional[int]:
    # an empty tensor has no address; the call does not read it, any device pointer serves
    if t is None:
        return None
    return t.data_ptr() or other.data_ptr()


def _round16(k: int) -> int:
    return (k + 15) // 16 * 16


# ------------------------------------------------------------------- rows of 8-bit integers
@_on_stream
def awq_int8_quantize(A: torch.Tensor, s: Optional[torch.Tensor] = None, fold: str = "divide",
                      stream=None):
    """Rows of A (fp16 or bf16 [R, K]) as int8 codes [R, K rounded up to 16] (zeros past K) and
    fp32 steps [R].  With s (fp32 [K]) the values are A / s (fold="divide", activations) or
    A * s (fold="multiply", weights)."""
    lda = _rows(A, "A")
    dt = _dtype(A.dtype, "A")
    if fold not in ("divide", "multiply"):
        raise ValueError('fold must be "divide" or "multiply"')
    R, K = A.shape
    if s is not None:
        _dev(s, torch.float32, "s", (K,))
    codes = torch.empty((R, _round16(K)), dtype=torch.int8, device=A.device)
    steps = torch.empty(R, dtype=torch.float32, device=A.device)
    if R == 0:
        return codes, steps
    st = lib().awq_int8_quantize(_addr(A, steps), R, K, lda, dt, _addr(s, steps),
                                 AWQ_FOLD_MULTIPLY if fold == "multiply" else AWQ_FOLD_DIVIDE,
                                 codes.data_ptr() or _ptr(_buf(256, A.device)), _round16(K),
                                 _ptr(steps), _stream_ptr(stream))
    _check(st, "awq_int8_quantize")
    return codes, steps


def awq_int8_matmul_workspace_bytes(n_tokens: int, out_features: int, in_features: int) -> int:
    return int(lib().awq_int8_matmul_workspace_bytes(n_tokens, out_features, in_features))


def awq_int8_linear_workspace_bytes(n_tokens: int, out_features: int, in_features: int) -> int:
    return int(lib().awq_int8_linear_workspace_bytes(n_tokens, out_features, in_features))


def _out_and_bias(T, M, dtype, bias, out, device):
    if bias is not None:
        _dev(bias, dtype, "bias", (M,))
    if out is None:
        out = torch.empty((T, M), dtype=dtype, device=device)
        return out, M
    ldy = _rows(out, "out", dtype)
    if tuple(out.shape) != (T, M):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {(T, M)}")
    return out, ldy


def _workspace(workspace, need, device):
    if workspace is None:
        return (torch.empty(need, dtype=torch.uint8, device=device), need) if need else (None, 0)
    _dev(workspace, torch.uint8, "workspace")
    return workspace, workspace.numel()


@_on_stream
def awq_int8_matmul(xq: torch.Tensor, xstep: torch.Tensor, wq: torch.Tensor, wstep: torch.Tensor,
                    dtype: torch.dtype = torch.float16, bias: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """y [T, M] = (xq wq^T) xstep wstep (+ bias) for int8 codes xq [T, K], wq [M, K] (K a
    multiple of 16, rows 16-byte aligned) and fp32 steps xstep [T], wstep [M]; y in `dtype`."""
    ldx, ldw = _rows(xq, "xq", torch.int8), _rows(wq, "wq", torch.int8)
    T, K = xq.shape
    M = wq.shape[0]
    if wq.shape[1] != K or K % 16:
        raise ValueError("xq and wq must have the same number of columns, a multiple of 16")
    dt = _dtype(dtype, "dtype")
    _dev(xstep, torch.float32, "xstep", (T,))
    _dev(wstep, torch.float32, "wstep", (M,))
    y, ldy = _out_and_bias(T, M, dtype, bias, out, xq.device)
    if T == 0 or M == 0:
        return y
    ws, nw = _workspace(workspace, awq_int8_matmul_workspace_bytes(T, M, K), xq.device)
    st = lib().awq_int8_matmul(_addr(xq, y), ldx, _ptr(xstep), T, _addr(wq, y), ldw, _ptr(wstep), M,
                               K, _addr(bias, y), dt, _ptr(y), ldy, _addr(ws, y), nw,
                               _stream_ptr(stream))
    _check(st, "awq_int8_matmul")
    return y


@_on_stream
def awq_int8_linear(x: torch.Tensor, wq: torch.Tensor, wstep: torch.Tensor,
                    s: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """y [T, M] in x's type: each token of x (fp16 or bf16 [T, K]) divided by s (fp32 [K], if
    given), quantised to int8 with its own step and multiplied with the int8 weight wq
    [M, K rounded up to 16], wstep [M] (as awq_int8_quantize(W, s, "multiply") makes them)."""
    ldx, ldw = _rows(x, "x"), _rows(wq, "wq", torch.int8)
    dt = _dtype(x.dtype, "x")
    T, K = x.shape
    M = wq.shape[0]
    if wq.shape[1] != _round16(K):
        raise ValueError(f"wq has {wq.shape[1]} columns, expected {_round16(K)}")
    _dev(wstep, torch.float32, "wstep", (M,))
    if s is not None:
        _dev(s, torch.float32, "s", (K,))
    y, ldy = _out_and_bias(T, M, x.dtype, bias, out, x.device)
    if T == 0 or M == 0:
        return y
    ws, nw = _workspace(workspace, awq_int8_linear_workspace_bytes(T, M, K), x.device)
    st = lib().awq_int8_linear(_addr(x, y), ldx, _addr(s, y), T, _addr(wq, y), ldw, _ptr(wstep), M,
                               K, _addr(bias, y), dt, _ptr(y), ldy, _addr(ws, y), nw,
                               _stream_ptr(stream))
    _check(st, "awq_int8_linear")
    return y
