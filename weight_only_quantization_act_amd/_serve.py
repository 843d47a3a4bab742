"""ctypes binding of the serving operators (include/awq_serve.h): argument marshalling only.

Same rules as the rest of the binding: tensors are checked for dtype, device and layout, raw
device pointers and the current HIP stream go to the C ABI, non-zero status codes raise, and
there is no fallback.  Unlike the rest, row strides are free where the C ABI takes them, so
views into a fused projection's output need no copy.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from ._lib import _buf, _check, _dev, _i32, _i64, _sz, _vp
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


# A decode step's calls last a few microseconds on the device, so the path to the C ABI is kept
# short: one combined test per tensor (the detailed checks run only to say what is wrong), the
# current stream's handle without a Stream object, workspace sizes remembered by their sizes.
_FP16, _BF16, _FP32, _I8, _U8, _INT32 = (torch.float16, torch.bfloat16, torch.float32, torch.int8,
                                         torch.uint8, torch.int32)
_DTYPES = {_FP16: AWQ_FP16, _BF16: AWQ_BF16}


def _dtype(dtype: torch.dtype, name: str) -> int:
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise TypeError(f"{name} must be torch.float16 or torch.bfloat16, got {dtype}")
    return dt


def _current_stream() -> int:
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _on_stream(fn):
    """Run the wrapper with `stream` (when given) as torch's current stream, so that what it
    allocates belongs to the stream that the kernels are enqueued on."""
    @functools.wraps(fn)
    def wrapper(*args, stream=None, **kwargs):
        if stream is None:
            return fn(*args, **kwargs)
        with torch.cuda.stream(stream):
            return fn(*args, **kwargs)
    return wrapper


def _rows(t: torch.Tensor, name: str, dtype: Optional[torch.dtype] = None) -> int:
    """Check a 2-D device tensor with unit stride along its rows; returns the row stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device (HIP) tensor")
    if dtype is not None and t.dtype != dtype:
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


def _vec(t: torch.Tensor, dtype: torch.dtype, name: str, n: int) -> int:
    """Check a contiguous device vector of n elements; returns its address."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == (n,) and t.is_cuda
            and t.is_contiguous()):
        _dev(t, dtype, name, (n,))
    return t.data_ptr()


def _round16(k: int) -> int:
    return (k + 15) // 16 * 16


# ------------------------------------------------------------------- rows of 8-bit integers
@_on_stream
def awq_int8_quantize(A: torch.Tensor, s: Optional[torch.Tensor] = None, fold: str = "divide"):
    """Rows of A (fp16 or bf16 [R, K]) as int8 codes [R, K rounded up to 16] (zeros past K) and
    fp32 steps [R].  With s (fp32 [K]) the values are A / s (fold="divide", activations) or
    A * s (fold="multiply", weights)."""
    lda = _rows(A, "A")
    dt = _dtype(A.dtype, "A")
    if fold not in ("divide", "multiply"):
        raise ValueError('fold must be "divide" or "multiply"')
    R, K = A.shape
    ps = None if s is None else _vec(s, _FP32, "s", K)
    codes = torch.empty((R, _round16(K)), dtype=_I8, device=A.device)
    steps = torch.empty(R, dtype=_FP32, device=A.device)
    if R == 0:
        return codes, steps
    # an empty tensor has no address; the call does not read it, any device pointer serves
    some = steps.data_ptr()
    st = lib().awq_int8_quantize(A.data_ptr() or some, R, K, lda, dt, ps,
                                 AWQ_FOLD_MULTIPLY if fold == "multiply" else AWQ_FOLD_DIVIDE,
                                 codes.data_ptr() or _buf(256, A.device).data_ptr(), _round16(K),
                                 some, _current_stream())
    _check(st, "awq_int8_quantize")
    return codes, steps


@functools.lru_cache(maxsize=4096)
def awq_int8_matmul_workspace_bytes(n_tokens: int, out_features: int, in_features: int) -> int:
    return int(lib().awq_int8_matmul_workspace_bytes(n_tokens, out_features, in_features))


@functools.lru_cache(maxsize=4096)
def awq_int8_linear_workspace_bytes(n_tokens: int, out_features: int, in_features: int) -> int:
    return int(lib().awq_int8_linear_workspace_bytes(n_tokens, out_features, in_features))


def _out_rows(T, M, dtype, out, like):
    if out is None:
        return like.new_empty((T, M), dtype=dtype), M
    ldy = _rows(out, "out", dtype)
    if tuple(out.shape) != (T, M):
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {(T, M)}")
    return out, ldy


def _workspace(workspace, need, device):
    """(tensor that must live until the call, address or None, bytes)."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=_U8, device=device)
    else:
        _dev(workspace, _U8, "workspace")
    return workspace, workspace.data_ptr() or None, workspace.numel()


@_on_stream
def awq_int8_matmul(xq: torch.Tensor, xstep: torch.Tensor, wq: torch.Tensor, wstep: torch.Tensor,
                    dtype: torch.dtype = torch.float16, bias: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [T, M] = (xq wq^T) xstep wstep (+ bias) for int8 codes xq [T, K], wq [M, K] (K a
    multiple of 16, rows 16-byte aligned) and fp32 steps xstep [T], wstep [M]; y in `dtype`."""
    ldx, ldw = _rows(xq, "xq", _I8), _rows(wq, "wq", _I8)
    T, K = xq.shape
    M = wq.shape[0]
    if wq.shape[1] != K or K % 16:
        raise ValueError("xq and wq must have the same number of columns, a multiple of 16")
    dt = _dtype(dtype, "dtype")
    px, pw = _vec(xstep, _FP32, "xstep", T), _vec(wstep, _FP32, "wstep", M)
    pb = None if bias is None else _vec(bias, dtype, "bias", M)
    y, ldy = _out_rows(T, M, dtype, out, xq)
    if T == 0 or M == 0:
        return y
    py = y.data_ptr()
    ws, pws, nws = _workspace(workspace, awq_int8_matmul_workspace_bytes(T, M, K), xq.device)
    st = lib().awq_int8_matmul(xq.data_ptr() or py, ldx, px, T, wq.data_ptr() or py, ldw, pw, M, K,
                               pb, dt, py, ldy, pws, nws, _current_stream())
    _check(st, "awq_int8_matmul")
    return y


@_on_stream
def awq_int8_linear(x: torch.Tensor, wq: torch.Tensor, wstep: torch.Tensor,
                    s: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [T, M] in x's type: each token of x (fp16 or bf16 [T, K]) divided by s (fp32 [K], if
    given), quantised to int8 with its own step and multiplied with the int8 weight wq
    [M, K rounded up to 16], wstep [M] (as awq_int8_quantize(W, s, "multiply") makes them)."""
    ldx, ldw = _rows(x, "x"), _rows(wq, "wq", _I8)
    dtype = x.dtype
    dt = _dtype(dtype, "x")
    T, K = x.shape
    M = wq.shape[0]
    if wq.shape[1] != _round16(K):
        raise ValueError(f"wq has {wq.shape[1]} columns, expected {_round16(K)}")
    pw = _vec(wstep, _FP32, "wstep", M)
    ps = None if s is None else _vec(s, _FP32, "s", K)
    pb = None if bias is None else _vec(bias, dtype, "bias", M)
    y, ldy = _out_rows(T, M, dtype, out, x)
    if T == 0 or M == 0:
        return y
    py = y.data_ptr()
    ws, pws, nws = _workspace(workspace, awq_int8_linear_workspace_bytes(T, M, K), x.device)
    st = lib().awq_int8_linear(x.data_ptr() or py, ldx, (ps or py) if s is not None else None, T,
                               wq.data_ptr() or py, ldw, pw, M, K, pb, dt, py, ldy, pws, nws,
                               _current_stream())
    _check(st, "awq_int8_linear")
    return y


# -------------------------------------------------------------- key/value cache in 4 bits
def awq_kv4_record_bytes(cfg: awq_kv4_config) -> int:
    """Bytes of one page of one head (0 for an invalid configuration)."""
    return int(lib().awq_kv4_record_bytes(cfg))


def awq_kv4_cache(n_pages: int, cfg: awq_kv4_config, device="cuda") -> torch.Tensor:
    """An empty cache: uint8 [n_pages, kv_heads, record], zeroed."""
    rec = awq_kv4_record_bytes(cfg)
    if rec == 0:
        raise ValueError("invalid awq_kv4_config")
    return torch.zeros((n_pages, cfg.kv_heads, rec), dtype=torch.uint8, device=device)


def _kv4_args(cache, table, lens, starts, cfg):
    """Check the cache and its index tensors; returns the number of sequences."""
    d, p, hk, g = cfg.head_dim, cfg.page_size, cfg.kv_heads, cfg.group_size
    rec = p * (d + 8 * (d // g)) if g > 0 else 0  # the C side refuses what is no configuration
    try:
        cs, ts = cache.shape, table.shape
        n = ts[0]
        if (cache.dtype is _U8 and cs[1] == hk and cs[2] == rec and len(cs) == 3 and cache.is_cuda
                and cache.is_contiguous() and table.dtype is _INT32 and len(ts) == 2 and table.is_cuda
                and table.is_contiguous() and lens.dtype is _INT32 and lens.shape == (n,) and lens.is_cuda
                and lens.is_contiguous() and starts.dtype is _INT32 and starts.shape == (n + 1,)
                and starts.is_cuda and starts.is_contiguous()):
            return n
    except (AttributeError, IndexError, TypeError):
        pass
    _kv4_complain(cache, table, lens, starts, cfg, rec)


def _kv4_complain(cache, table, lens, starts, cfg, rec):
    """Say which of the arguments that _kv4_args refused is wrong."""
    if awq_kv4_record_bytes(cfg) == 0:
        raise ValueError("invalid awq_kv4_config")
    _dev(cache, _U8, "cache")
    if cache.dim() != 3 or tuple(cache.shape[1:]) != (cfg.kv_heads, rec):
        raise ValueError(f"cache has shape {tuple(cache.shape)}, expected [n_pages, {cfg.kv_heads}, {rec}]")
    _dev(table, _INT32, "block_table")
    if table.dim() != 2:
        raise ValueError("block_table must be [n_seqs, max_blocks]")
    _dev(lens, _INT32, "seq_lens", (table.shape[0],))
    _dev(starts, _INT32, "q_start", (table.shape[0] + 1,))
    raise ValueError("invalid cache arguments")


def _heads(t, name, heads, dim, dtype=None):
    """Check [tokens, heads, dim] with unit stride in dim; returns token and head strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device (HIP) tensor")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected [tokens, "
                         f"{'heads' if heads is None else heads}, {dim}]")
    st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name} must be contiguous along head_dim")
    return (st if shape[0] > 1 else 0), (sh if shape[1] > 1 else 0)


@_on_stream
def awq_kv4_append(k: torch.Tensor, v: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                   seq_lens: torch.Tensor, q_start: torch.Tensor, cfg: awq_kv4_config) -> None:
    """Quantise the rows k, v (fp16 or bf16 [T, kv_heads, head_dim], any token and head strides
    that are multiples of 8) into the pages of their sequences.  Rows q_start[b] ..
    q_start[b + 1] - 1 are the last tokens of sequence b, whose length with them is seq_lens[b]."""
    n = _kv4_args(cache, block_table, seq_lens, q_start, cfg)
    dt = _dtype(k.dtype, "k")
    hk, d = cfg.kv_heads, cfg.head_dim
    kt, kh = _heads(k, "k", hk, d)
    vt, vh = _heads(v, "v", hk, d, k.dtype)
    T = k.shape[0]
    if v.shape[0] != T:
        raise ValueError("k and v differ in tokens")
    if T == 0 or n == 0:
        return
    st = lib().awq_kv4_append(k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, T, dt, cache.data_ptr(),
                              cache.shape[0], block_table.data_ptr(), n, block_table.shape[1],
                              seq_lens.data_ptr(), q_start.data_ptr(), cfg, _current_stream())
    _check(st, "awq_kv4_append")


@_on_stream
def awq_kv4_read(cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                 q_start: torch.Tensor, cfg: awq_kv4_config, n_tokens: int,
                 dtype: torch.dtype = torch.float16):
    """The stored keys and values of the same rows as awq_kv4_append: two tensors
    [n_tokens, kv_heads, head_dim] of dtype (zeros where no such token exists)."""
    n = _kv4_args(cache, block_table, seq_lens, q_start, cfg)
    dt = _dtype(dtype, "dtype")
    shape = (n_tokens, cfg.kv_heads, cfg.head_dim)
    k = cache.new_empty(shape, dtype=dtype)
    v = torch.empty_like(k)
    if n_tokens == 0:
        return k, v
    if n == 0:
        return k.zero_(), v.zero_()
    st = lib().awq_kv4_read(cache.data_ptr(), cache.shape[0], block_table.data_ptr(), n,
                            block_table.shape[1], seq_lens.data_ptr(), q_start.data_ptr(), n_tokens,
                            cfg, dt, k.data_ptr(), v.data_ptr(), _current_stream())
    _check(st, "awq_kv4_read")
    return k, v


@functools.lru_cache(maxsize=4096)
def _attention_workspace(T, n, H, d, hk, p, g, max_q, max_len):
    cfg = awq_kv4_config(d, hk, p, g, 0)
    return int(lib().awq_kv4_attention_workspace_bytes(T, n, H, cfg, max_q, max_len))


def awq_kv4_attention_workspace_bytes(n_tokens: int, n_seqs: int, heads: int, cfg: awq_kv4_config,
                                      max_q: int, max_len: int) -> int:
    return int(lib().awq_kv4_attention_workspace_bytes(n_tokens, n_seqs, heads, cfg, max_q, max_len))


@_on_stream
def awq_kv4_attention(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                      seq_lens: torch.Tensor, q_start: torch.Tensor, cfg: awq_kv4_config, *,
                      max_q: int, max_len: int, scale: Optional[float] = None, window: int = 0,
                      out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Causal attention of q (fp16 or bf16 [T, heads, head_dim]) over the cache: returns out
    [T, heads, head_dim] in q's type and lse fp32 [T, heads].  max_q and max_len are host
    bounds on the rows of a sequence and on seq_lens; scale defaults to 1 / sqrt(head_dim);
    window > 0 keeps the last `window` keys of each row.  Rows without keys give 0 and -inf.
    Rows of no sequence (past q_start[-1]) and rows beyond max_q are not written: without an
    `out` of the caller's they hold anything.
    A workspace (see awq_kv4_attention_workspace_bytes) is allocated unless one is passed."""
    n = _kv4_args(cache, block_table, seq_lens, q_start, cfg)
    dtype = q.dtype
    dt = _dtype(dtype, "q")
    d = cfg.head_dim
    qt, qh = _heads(q, "q", None, d)
    T, H, _ = q.shape
    if out is None:
        out = q.new_empty((T, H, d))
    else:
        _dev(out, dtype, "out", (T, H, d))
    lse = q.new_empty((T, H), dtype=_FP32)
    if T == 0 or n == 0:
        return out, lse
    need = 0 if workspace is not None else _attention_workspace(
        T, n, H, d, cfg.kv_heads, cfg.page_size, cfg.group_size, max_q, max_len)
    ws, pws, nws = _workspace(workspace, need, q.device)
    st = lib().awq_kv4_attention(q.data_ptr(), qt, qh, T, H, dt, cache.data_ptr(), cache.shape[0],
                                 block_table.data_ptr(), n, block_table.shape[1],
                                 seq_lens.data_ptr(), q_start.data_ptr(), cfg, max_q, max_len,
                                 d ** -0.5 if scale is None else scale, window, out.data_ptr(),
                                 lse.data_ptr(), pws, nws, _current_stream())
    _check(st, "awq_kv4_attention")
    return out, lse
