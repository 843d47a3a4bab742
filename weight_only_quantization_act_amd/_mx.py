"""ctypes binding of the MXFP4 operators, the norm and the read-back of 8-bit rows
(include/awq_serve.h): argument marshalling only, by the rules of the serving binding.

Every tensor of a call has to be on one device, which is made the current one for the call if it
is not.

Short calls are at the host's pace, so the usual case (tensors of the current device, outputs allocated,
the current stream) goes through one step of native code, the extension module _calls
(csrc/python/calls.cpp).  What that does not take (it returns None) is checked and called from here.
"""
from __future__ import annotations

import functools
import warnings
from typing import Optional

import torch

from ._lib import _check
from ._serve import (AWQ_FOLD_DIVIDE, AWQ_FOLD_MULTIPLY, AWQ_FP32, _FP32, _I8, _U8, _dtype,
                     _round16, _workspace, lib)

_empty = torch.empty_strided
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream
_C = None
_N = None


def _lib():
    global _C
    _C = lib()
    return _C


class _NoCalls:
    """In the extension module's place: it takes no call."""
    def __getattr__(self, name):
        return lambda *args: None


def _native():
    """The extension module, after the library that it calls."""
    global _N
    lib()
    try:
        from . import _calls
    except ImportError as e:
        warnings.warn(f"the extension module _calls is missing or does not fit ({e}): calls of the norm and of MXFP4 "
                      "take some microseconds more; build it with "
                      "`python -m weight_only_quantization_act_amd.build`", RuntimeWarning, stacklevel=3)
        _calls = _NoCalls()
    _N = _calls
    return _N


def _device(first) -> int:
    """The current device, for a call with this first argument."""
    if not isinstance(first, torch.Tensor):
        raise TypeError("the first argument must be a torch.Tensor")
    if not first.is_cuda:
        raise ValueError("the first argument must be a device (HIP) tensor")
    return _current_device()


def _elsewhere(fn, stream, first, *args, **kwargs):
    """Run an entry point with `stream` (when given) as torch's current stream, or with the device of its
    first argument as the current one, so that what it allocates belongs to the stream that the kernels
    are enqueued on."""
    if stream is not None:
        if stream.device != first.device:
            raise ValueError(f"stream is of {stream.device}, the tensors are on {first.device}")
        with torch.cuda.stream(stream):
            return fn(first, *args, **kwargs)
    with torch.cuda.device(first.device):
        return fn(first, *args, **kwargs)


def _matrix(t: torch.Tensor, name: str, dtype: Optional[torch.dtype], dev: int) -> int:
    """Check a 2-D tensor on the call's device with unit stride along its rows; returns the row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device (HIP) tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on device {t.get_device()}, the call runs on device {dev}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    sr, sc = t.stride()
    if cols > 1 and sc != 1:
        raise ValueError(f"{name} must be contiguous along its rows")
    ld = sr if rows > 1 and cols > 0 else cols
    if ld < cols:
        raise ValueError(f"{name} has overlapping rows (stride {ld} for {cols} columns)")
    return ld


def _vector(t: torch.Tensor, dtype: torch.dtype, name: str, n: int, dev: int) -> int:
    """Check a contiguous vector of n elements on the call's device; returns its address."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.get_device() != dev:
        raise ValueError(f"{name} must be a tensor on device {dev}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous of shape ({n},), got {tuple(t.shape)}")
    return t.data_ptr()


def _blocks(cols: int) -> int:
    return (cols + 31) // 32


def _codes(codes: torch.Tensor, scales: torch.Tensor, names, dev: int):
    """Check MXFP4 codes [R, 16 a block] and scales [blocks / 4, at least R, 4]; returns rows, bytes a
    row and the rows' strides of both (bytes, words)."""
    ld = _matrix(codes, names[0], _U8, dev)
    if not (isinstance(scales, torch.Tensor) and scales.dtype is _U8 and scales.get_device() == dev
            and scales.is_contiguous() and scales.dim() == 3):
        raise TypeError(f"{names[1]} must be contiguous uint8 [column words, rows, 4] on device {dev}")
    rows, nb = codes.shape
    words, lds, four = scales.shape
    if nb % 16 or words != (nb // 16 + 3) // 4 or four != 4 or lds < rows or lds % 4:
        raise ValueError(f"{names[0]} {tuple(codes.shape)} and {names[1]} {tuple(scales.shape)} do not belong "
                         "together: expected [R, 16 B] and [ceil(B / 4), R rounded up to 4, 4]")
    return rows, nb, ld, lds


def _new_codes(rows: int, cols: int, device):
    nb = (cols + 31) // 32 * 16
    lds = (rows + 3) // 4 * 4
    return (_empty((rows, nb), (nb, 1), dtype=_U8, device=device),
            _empty(((cols + 127) // 128, lds, 4), (4 * lds, 4, 1), dtype=_U8, device=device))


def _fold(fold: str) -> int:
    if fold not in ("divide", "multiply"):
        raise ValueError('fold must be "divide" or "multiply"')
    return AWQ_FOLD_MULTIPLY if fold == "multiply" else AWQ_FOLD_DIVIDE


def _out(out: Optional[torch.Tensor], rows: int, cols: int, dtype: torch.dtype, like: torch.Tensor,
         dev: int, name: str = "out"):
    if out is None:
        return _empty((rows, cols), (cols, 1), dtype=dtype, device=like.device), cols
    ld = _matrix(out, name, dtype, dev)
    if tuple(out.shape) != (rows, cols):
        raise ValueError(f"{name} has shape {tuple(out.shape)}, expected {(rows, cols)}")
    return out, ld


# -------------------------------------------------------------------------- rows and values
def awq_int8_dequantize(codes: torch.Tensor, steps: torch.Tensor, cols: int,
                        dtype: torch.dtype = torch.float16, out: Optional[torch.Tensor] = None, *,
                        stream=None):
    """The values [R, cols] in dtype (fp16 or bf16) that 8-bit rows stand for: codes int8 [R, cols rounded
    up to 16] (as awq_int8_quantize and awq_rmsnorm_int8 make them) times steps fp32 [R]."""
    if out is None and stream is None:
        y = (_N or _native()).int8_dequantize(codes, steps, cols, dtype)
        if y is not None:
            return y
    dev = _device(codes)
    if stream is not None or codes.get_device() != dev:
        return _elsewhere(awq_int8_dequantize, stream, codes, steps, cols, dtype, out)
    ld = _matrix(codes, "codes", _I8, dev)
    R, nc = codes.shape
    if cols < 0 or nc != _round16(cols):
        raise ValueError(f"codes has {nc} columns, expected {_round16(cols)}")
    dt = _dtype(dtype, "dtype")
    ps = _vector(steps, _FP32, "steps", R, dev)
    y, ldo = _out(out, R, cols, dtype, codes, dev)
    if R == 0 or cols == 0:
        return y
    st = (_C or _lib()).awq_int8_dequantize(codes.data_ptr(), ld, ps, R, cols, dt, y.data_ptr(), ldo,
                                   _raw_stream(dev))
    if st:
        _check(st, "awq_int8_dequantize")
    return y


def awq_mxfp4_quantize(A: torch.Tensor, s: Optional[torch.Tensor] = None, fold: str = "divide", *,
                       stream=None):
    """Rows of A (fp16 or bf16 [R, K]) in MXFP4: codes uint8 [R, 16 ceil(K / 32)], two columns a byte, and
    scales uint8 [ceil(K / 128), R rounded up to 4, 4] (see awq_serve.h for both).  With s (fp32 [K])
    the values are A / s (fold="divide", activations) or A * s (fold="multiply", weights)."""
    multiply = _fold(fold) == AWQ_FOLD_MULTIPLY
    if stream is None:
        got = (_N or _native()).mxfp4_quantize(A, s, multiply)
        if got is not None:
            return got
    dev = _device(A)
    if stream is not None or A.get_device() != dev:
        return _elsewhere(awq_mxfp4_quantize, stream, A, s, fold)
    lda = _matrix(A, "A", None, dev)
    dt = _dtype(A.dtype, "A")
    f = AWQ_FOLD_MULTIPLY if multiply else AWQ_FOLD_DIVIDE
    R, K = A.shape
    ps = None if s is None else _vector(s, _FP32, "s", K, dev)
    codes, scales = _new_codes(R, K, A.device)
    if R == 0 or K == 0:
        return codes, scales
    st = (_C or _lib()).awq_mxfp4_quantize(A.data_ptr(), R, K, lda, dt, ps, f, codes.data_ptr(), (K + 31) // 32 * 16,
                                  scales.data_ptr(), (R + 3) // 4 * 4, _raw_stream(dev))
    if st:
        _check(st, "awq_mxfp4_quantize")
    return codes, scales


def awq_mxfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, cols: int,
                         dtype: torch.dtype = torch.float16, out: Optional[torch.Tensor] = None, *,
                         stream=None):
    """The values [R, cols] in dtype (fp16 or bf16) that MXFP4 codes and scales stand for."""
    if out is None and stream is None:
        y = (_N or _native()).mxfp4_dequantize(codes, scales, cols, dtype)
        if y is not None:
            return y
    dev = _device(codes)
    if stream is not None or codes.get_device() != dev:
        return _elsewhere(awq_mxfp4_dequantize, stream, codes, scales, cols, dtype, out)
    R, nb, ld, lds = _codes(codes, scales, ("codes", "scales"), dev)
    if cols < 0 or nb != 16 * _blocks(cols):
        raise ValueError(f"codes has {nb} bytes a row, expected {16 * _blocks(cols)}")
    dt = _dtype(dtype, "dtype")
    y, ldo = _out(out, R, cols, dtype, codes, dev)
    if R == 0 or cols == 0:
        return y
    st = (_C or _lib()).awq_mxfp4_dequantize(codes.data_ptr(), ld, scales.data_ptr(), lds, R, cols, dt,
                                    y.data_ptr(), ldo, _raw_stream(dev))
    if st:
        _check(st, "awq_mxfp4_dequantize")
    return y


# ---------------------------------------------------------------------------------- product
@functools.lru_cache(maxsize=4096)
def awq_mxfp4_linear_workspace_bytes(n_tokens: int, out_features: int, in_features: int) -> int:
    return int(lib().awq_mxfp4_linear_workspace_bytes(n_tokens, out_features, in_features))


def awq_mxfp4_matmul(xc: torch.Tensor, xs: torch.Tensor, wc: torch.Tensor, ws: torch.Tensor,
                     dtype: torch.dtype = torch.float16, bias: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, *, stream=None):
    """y [T, M] = x w^T (+ bias) in `dtype` for MXFP4 codes and scales of tokens (xc, xs) and weights
    (wc, ws), as awq_mxfp4_quantize and awq_rmsnorm_mxfp4 make them.  All columns of the codes' blocks count:
    where the last block is not whole, its columns past the last must be zero in one of the two."""
    if out is None and stream is None:
        y = (_N or _native()).mxfp4_matmul(xc, xs, wc, ws, dtype, bias)
        if y is not None:
            return y
    dev = _device(xc)
    if stream is not None or xc.get_device() != dev:
        return _elsewhere(awq_mxfp4_matmul, stream, xc, xs, wc, ws, dtype, bias, out)
    T, nb, ldx, ldxs = _codes(xc, xs, ("xc", "xs"), dev)
    M, nw, ldw, ldws = _codes(wc, ws, ("wc", "ws"), dev)
    if nw != nb:
        raise ValueError(f"xc and wc differ in columns ({nb} and {nw} bytes)")
    dt = _dtype(dtype, "dtype")
    pb = None if bias is None else _vector(bias, dtype, "bias", M, dev)
    y, ldy = _out(out, T, M, dtype, xc, dev)
    if T == 0 or M == 0:
        return y
    py = y.data_ptr()
    # an empty tensor has no address; the call does not read it, any device pointer serves
    st = (_C or _lib()).awq_mxfp4_matmul(xc.data_ptr() or py, ldx, xs.data_ptr() or py, ldxs, T,
                                wc.data_ptr() or py, ldw, ws.data_ptr() or py, ldws, M, 2 * nb, pb, dt,
                                py, ldy, _raw_stream(dev))
    if st:
        _check(st, "awq_mxfp4_matmul")
    return y


def awq_mxfp4_linear(x: torch.Tensor, wc: torch.Tensor, ws: torch.Tensor,
                     s: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, *,
                     stream=None):
    """y [T, M] in x's type: each token of x (fp16 or bf16 [T, K]) divided by s (fp32 [K], if given),
    quantised to MXFP4 and multiplied with the weight's codes and scales wc, ws (as
    awq_mxfp4_quantize(W, s, "multiply") makes them).  out must not overlap x."""
    if out is None and workspace is None and stream is None:
        y = (_N or _native()).mxfp4_linear(x, wc, ws, s, bias)
        if y is not None:
            return y
    dev = _device(x)
    if stream is not None or x.get_device() != dev:
        return _elsewhere(awq_mxfp4_linear, stream, x, wc, ws, s, bias, out, workspace)
    ldx = _matrix(x, "x", None, dev)
    dtype = x.dtype
    dt = _dtype(dtype, "x")
    M, nb, ldw, ldws = _codes(wc, ws, ("wc", "ws"), dev)
    T, K = x.shape
    if nb != 16 * _blocks(K):
        raise ValueError(f"wc has {nb} bytes a row, expected {16 * _blocks(K)}")
    ps = None if s is None else _vector(s, _FP32, "s", K, dev)
    pb = None if bias is None else _vector(bias, dtype, "bias", M, dev)
    y, ldy = _out(out, T, M, dtype, x, dev)
    if T == 0 or M == 0:
        return y
    py = y.data_ptr()
    if py == x.data_ptr():
        raise ValueError("out must not be x: blocks read the tokens when others have stored their results")
    ws_, pws, nws = _workspace(workspace, awq_mxfp4_linear_workspace_bytes(T, M, K), x.device)
    st = (_C or _lib()).awq_mxfp4_linear(x.data_ptr() or py, ldx, (ps or py) if s is not None else None, T,
                                wc.data_ptr() or py, ldw, ws.data_ptr() or py, ldws, M, K, pb, dt, py,
                                ldy, pws, nws, _raw_stream(dev))
    if st:
        _check(st, "awq_mxfp4_linear")
    return y


# ------------------------------------------------------------------------------------- norm
def _norm_args(x, weight, eps, residual, h_out, dev):
    """The leading arguments of the norm's C calls (see awq_rmsnorm), and h."""
    ldx = _matrix(x, "x", None, dev)
    dtype = x.dtype
    dt = _dtype(dtype, "x")
    R, K = shape = x.shape
    if K == 0:
        raise ValueError("x must have columns")
    pw, wt = None, dt
    if weight is not None:
        if isinstance(weight, torch.Tensor) and weight.dtype is _FP32:
            pw, wt = _vector(weight, _FP32, "weight", K, dev), AWQ_FP32
        else:
            pw = _vector(weight, dtype, "weight", K, dev)
    if residual is None:
        if h_out is not None:
            raise ValueError("h_out is written only where a residual is given")
        return (x.data_ptr(), ldx, None, 0, R, K, dt, pw, wt, eps, None, 0), x
    ldr = _matrix(residual, "residual", dtype, dev)
    if residual.shape != shape:
        raise ValueError(f"residual has shape {tuple(residual.shape)}, expected {(R, K)}")
    h, ldh = _out(h_out, R, K, dtype, x, dev, "h_out")
    return (x.data_ptr(), ldx, residual.data_ptr(), ldr, R, K, dt, pw, wt, eps, h.data_ptr(), ldh), h


def awq_rmsnorm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6, *,
                residual: Optional[torch.Tensor] = None, h_out: Optional[torch.Tensor] = None,
                out: Optional[torch.Tensor] = None, stream=None):
    """Root-mean-square norm of the rows of x (fp16 or bf16 [R, K]): returns (y, h) with h = x + residual in
    x's type (x itself without a residual) and y = h weight / sqrt(mean h^2 + eps) in x's type.
    weight [K] is fp32 or of x's type (None: ones); the scales of a search are folded into it (weight
    / s).  h goes to h_out if given, y to out; each may be x or the residual itself, but not both the same."""
    if h_out is None and out is None and stream is None:
        got = (_N or _native()).rmsnorm(x, weight, eps, residual)
        if got is not None:
            return got
    dev = _device(x)
    if stream is not None or x.get_device() != dev:
        return _elsewhere(awq_rmsnorm, stream, x, weight, eps, residual=residual, h_out=h_out, out=out)
    args, h = _norm_args(x, weight, eps, residual, h_out, dev)
    y, ldy = _out(out, args[4], args[5], x.dtype, x, dev)
    if args[4]:
        if residual is not None and y.data_ptr() == h.data_ptr():
            raise ValueError("out and h_out must not be the same")
        st = (_C or _lib()).awq_rmsnorm(*args, y.data_ptr(), ldy, _raw_stream(dev))
        if st:
            _check(st, "awq_rmsnorm")
    return y, h


def awq_rmsnorm_int8(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6, *,
                     residual: Optional[torch.Tensor] = None, h_out: Optional[torch.Tensor] = None,
                     stream=None):
    """The same norm as rows of 8-bit integers: returns (codes, steps, h), codes int8 [R, K rounded up to
    16] and steps fp32 [R] as awq_int8_matmul takes them."""
    if h_out is None and stream is None:
        got = (_N or _native()).rmsnorm_int8(x, weight, eps, residual)
        if got is not None:
            return got
    dev = _device(x)
    if stream is not None or x.get_device() != dev:
        return _elsewhere(awq_rmsnorm_int8, stream, x, weight, eps, residual=residual, h_out=h_out)
    args, h = _norm_args(x, weight, eps, residual, h_out, dev)
    R, nc = args[4], _round16(args[5])
    device = x.device
    codes = _empty((R, nc), (nc, 1), dtype=_I8, device=device)
    steps = _empty((R,), (1,), dtype=_FP32, device=device)
    if R:
        st = (_C or _lib()).awq_rmsnorm_int8(*args, codes.data_ptr(), nc, steps.data_ptr(), _raw_stream(dev))
        if st:
            _check(st, "awq_rmsnorm_int8")
    return codes, steps, h


def awq_rmsnorm_mxfp4(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6, *,
                      residual: Optional[torch.Tensor] = None, h_out: Optional[torch.Tensor] = None,
                      stream=None):
    """The same norm as rows of MXFP4: returns (codes, scales, h), codes and scales as awq_mxfp4_quantize
    gives them and awq_mxfp4_matmul takes them."""
    if h_out is None and stream is None:
        got = (_N or _native()).rmsnorm_mxfp4(x, weight, eps, residual)
        if got is not None:
            return got
    dev = _device(x)
    if stream is not None or x.get_device() != dev:
        return _elsewhere(awq_rmsnorm_mxfp4, stream, x, weight, eps, residual=residual, h_out=h_out)
    args, h = _norm_args(x, weight, eps, residual, h_out, dev)
    R, K = args[4], args[5]
    codes, scales = _new_codes(R, K, x.device)
    if R:
        st = (_C or _lib()).awq_rmsnorm_mxfp4(*args, codes.data_ptr(), (K + 31) // 32 * 16, scales.data_ptr(),
                                              (R + 3) // 4 * 4, _raw_stream(dev))
        if st:
            _check(st, "awq_rmsnorm_mxfp4")
    return codes, scales, h
