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

class awq_kv4_config(ctypes.Structure):
    """Layout of a 4-bit key/value cache: head_dim (64 or 128), kv_heads, page_size (tokens a
    page: 16 .. 256, a power of two), group_size (32, 64, 128) and zero_point (0 or 1)."""
    _fields_ = [("head_dim", _i32), ("kv_heads", _i32), ("page_size", _i32), ("group_size", _i32),
                ("zero_point", _i32)]

    def __init__(self, head_dim: int = 128, kv_heads: int = 8, page_size: int = 64,
                 group_size: int = 64, zero_point: int = 1):
        super().__init__(int(head_dim), int(kv_heads), int(page_size), int(group_size),
                         int(zero_point))


_kvp = ctypes.POINTER(awq_kv4_config)

_SIGNATURES = {
    "awq_int8_quantize": (ctypes.c_int, [_vp, _i64, _i64, _i64, _i32, _vp, _i32, _vp, _i64, _vp,
                                         _vp]),
    "awq_int8_matmul_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "awq_int8_matmul": (ctypes.c_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i32,
                                       _vp, _i64, _vp, _sz, _vp]),
    "awq_int8_linear_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "awq_int8_linear": (ctypes.c_int, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _vp, _i32,
                                       _vp, _i64, _vp, _sz, _vp]),
    "awq_kv4_record_bytes": (_sz, [_kvp]),
    "awq_kv4_append": (ctypes.c_int, [_vp, _i64, _i64, _vp, _i64, _i64, _i64, _i32, _vp, _i64, _vp,
                                      _i64, _i64, _vp, _vp, _kvp, _vp]),
    "awq_kv4_read": (ctypes.c_int, [_vp, _i64, _vp, _i64, _i64, _vp, _vp, _i64, _kvp, _i32, _vp, _vp,
                                    _vp]),
    "awq_kv4_attention_workspace_bytes": (_sz, [_i64, _i64, _i64, _kvp, _i64, _i64]),
    "awq_kv4_attention": (ctypes.c_int, [_vp, _i64, _i64, _i64, _i64, _i32, _vp, _i64, _vp, _i64,
                                         _i64, _vp, _vp, _kvp, _i64, _i64, ctypes.c_float, _i64, _vp,
                                         _vp, _vp, _sz, _vp]),
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


# -------------------------------------------------------------- key/value cache in 4 bits
def awq_kv4_record_bytes(cfg: awq_kv4_config) -> int:
    """Bytes of one page of one head (0 for an invalid configuration)."""
    return int(lib().awq_kv4_record_bytes(ctypes.byref(cfg)))


def awq_kv4_cache(n_pages: int, cfg: awq_kv4_config, device="cuda") -> torch.Tensor:
    """An empty cache: uint8 [n_pages, kv_heads, record], zeroed."""
    rec = awq_kv4_record_bytes(cfg)
    if rec == 0:
        raise ValueError("invalid awq_kv4_config")
    return torch.zeros((n_pages, cfg.kv_heads, rec), dtype=torch.uint8, device=device)


def _kv4_args(cache, table, lens, starts, cfg):
    rec = awq_kv4_record_bytes(cfg)
    if rec == 0:
        raise ValueError("invalid awq_kv4_config")
    _dev(cache, torch.uint8, "cache")
    if cache.dim() != 3 or cache.shape[1] != cfg.kv_heads or cache.shape[2] != rec:
        raise ValueError(f"cache has shape {tuple(cache.shape)}, expected "
                         f"[n_pages, {cfg.kv_heads}, {rec}]")
    _dev(table, torch.int32, "block_table")
    if table.dim() != 2:
        raise ValueError("block_table must be [n_seqs, max_blocks]")
    n = table.shape[0]
    _dev(lens, torch.int32, "seq_lens", (n,))
    _dev(starts, torch.int32, "q_start", (n + 1,))
    return n


def _heads(t, name, heads, dim, dtype=None):
    """Check [tokens, heads, dim] with unit stride in dim; returns token and head strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device (HIP) tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or t.shape[2] != dim or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [tokens, "
                         f"{'heads' if heads is None else heads}, {dim}]")
    if t.stride(2) != 1:
        raise ValueError(f"{name} must be contiguous along head_dim")
    return (t.stride(0) if t.shape[0] > 1 else 0), (t.stride(1) if t.shape[1] > 1 else 0)


@_on_stream
def awq_kv4_append(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                   seq_lens: torch.Tensor, q_start: torch.Tensor, cfg: awq_kv4_config,
                   stream=None) -> None:
    """Quantise the rows k, v (fp16 or bf16 [T, kv_heads, head_dim], any token and head strides
    that are multiples of 8) into the pages of their sequences.  Rows q_start[b] ..
    q_start[b + 1] - 1 are the last tokens of sequence b, whose length with them is seq_lens[b]."""
    n = _kv4_args(cache, block_table, seq_lens, q_start, cfg)
    dt = _dtype(k.dtype, "k")
    kt, kh = _heads(k, "k", cfg.kv_heads, cfg.head_dim)
    vt, vh = _heads(v, "v", cfg.kv_heads, cfg.head_dim, k.dtype)
    if v.shape[0] != k.shape[0]:
        raise ValueError("k and v differ in tokens")
    if k.shape[0] == 0 or n == 0:
        return
    st = lib().awq_kv4_append(_ptr(k), kt, kh, _ptr(v), vt, vh, k.shape[0], dt, _ptr(cache),
                              cache.shape[0], _ptr(block_table), n, block_table.shape[1],
                              _ptr(seq_lens), _ptr(q_start), ctypes.byref(cfg), _stream_ptr(stream))
    _check(st, "awq_kv4_append")


@_on_stream
def awq_kv4_read(cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                 q_start: torch.Tensor, cfg: awq_kv4_config, n_tokens: int,
                 dtype: torch.dtype = torch.float16, stream=None):
    """The stored keys and values of the same rows as awq_kv4_append: two tensors
    [n_tokens, kv_heads, head_dim] of dtype (zeros where no such token exists)."""
    n = _kv4_args(cache, block_table, seq_lens, q_start, cfg)
    dt = _dtype(dtype, "dtype")
    shape = (n_tokens, cfg.kv_heads, cfg.head_dim)
    k = torch.empty(shape, dtype=dtype, device=cache.device)
    v = torch.empty(shape, dtype=dtype, device=cache.device)
    if n_tokens == 0:
        return k, v
    if n == 0:
        return k.zero_(), v.zero_()
    st = lib().awq_kv4_read(_ptr(cache), cache.shape[0], _ptr(block_table), n, block_table.shape[1],
                            _ptr(seq_lens), _ptr(q_start), n_tokens, ctypes.byref(cfg), dt, _ptr(k),
                            _ptr(v), _stream_ptr(stream))
    _check(st, "awq_kv4_read")
    return k, v


def awq_kv4_attention_workspace_bytes(n_tokens: int, n_seqs: int, heads: int, cfg: awq_kv4_config,
                                      max_q: int, max_len: int) -> int:
    return int(lib().awq_kv4_attention_workspace_bytes(n_tokens, n_seqs, heads, ctypes.byref(cfg),
                                                       max_q, max_len))


@_on_stream
def awq_kv4_attention(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                      seq_lens: torch.Tensor, q_start: torch.Tensor, cfg: awq_kv4_config, *,
                      max_q: int, max_len: int, scale: Optional[float] = None, window: int = 0,
                      out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                      stream=None):
    """Causal attention of q (fp16 or bf16 [T, heads, head_dim]) over the cache: returns out
    [T, heads, head_dim] in q's type and lse fp32 [T, heads].  max_q and max_len are host
    bounds on the rows of a sequence and on seq_lens; scale defaults to 1 / sqrt(head_dim);
    window > 0 keeps the last `window` keys of each row.  Rows without keys give 0 and -inf.
    A workspace (see awq_kv4_attention_workspace_bytes) is allocated unless one is passed."""
    n = _kv4_args(cache, block_table, seq_lens, q_start, cfg)
    dt = _dtype(q.dtype, "q")
    qt, qh = _heads(q, "q", None, cfg.head_dim)
    T, H = q.shape[0], q.shape[1]
    if out is None:
        out = torch.empty((T, H, cfg.head_dim), dtype=q.dtype, device=q.device)
    else:
        _dev(out, q.dtype, "out", (T, H, cfg.head_dim))
    lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    if T == 0 or n == 0:
        return out, lse
    ws, nw = _workspace(workspace,
                        awq_kv4_attention_workspace_bytes(T, n, H, cfg, max_q, max_len), q.device)
    st = lib().awq_kv4_attention(_ptr(q), qt, qh, T, H, dt, _ptr(cache), cache.shape[0],
                                 _ptr(block_table), n, block_table.shape[1], _ptr(seq_lens),
                                 _ptr(q_start), ctypes.byref(cfg), max_q, max_len,
                                 float(cfg.head_dim ** -0.5 if scale is None else scale), int(window),
                                 _ptr(out), _ptr(lse), _addr(ws, out), nw, _stream_ptr(stream))
    _check(st, "awq_kv4_attention")
    return out, lse
