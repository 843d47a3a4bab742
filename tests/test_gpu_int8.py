"""Rows of 8-bit integers and their product on the GPU (through the C ABI) against numpy.

Bars, derived from the kernels' arithmetic:
  - codes and steps are defined by single IEEE fp32 operations, so they are equal bit for bit;
  - the product's sum is exact in int32; its conversion to fp32, the two multiplications and
    the bias addition round once each (relative 2^-24 each of a value that is at most
    |sum| xstep wstep (1 + 2^-22) + |bias|), so before the last rounding the result is within
    2^-22 (|y_product| + |bias|) of the formula in 64 bits, and the rounding to fp16 or bf16
    adds half an ulp of the type (a whole ulp is allowed, for values at a rounding boundary).
"""
import numpy as np
import pytest
import torch

import weight_only_quantization_act_amd as awq
from tests.gpu_util import requires_gpu, say

pytestmark = [pytest.mark.gpu, requires_gpu]

F32, F64 = np.float32, np.float64
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _quantise_ref(x32):
    """codes, steps of fp32 rows (numpy fp32 operations, one rounding each)."""
    amax = np.max(np.abs(x32), axis=1, initial=0.0).astype(F32)
    finite = np.all(np.isfinite(x32), axis=1)
    step = (amax / F32(127)).astype(F32)
    step[step == 0] = 1
    with np.errstate(all="ignore"):
        q = np.clip(np.rint((x32 / step[:, None]).astype(F32)), -127, 127)
    q[~finite] = 0
    step[~finite] = np.nan
    return q.astype(np.int8), step


def _fold_ref(A, s, fold):
    x = A.float().cpu().numpy()
    if s is None:
        return x
    s = s.cpu().numpy()
    with np.errstate(all="ignore"):
        return (x / s if fold == "divide" else x * s).astype(F32)


def _check_rows(A, s, fold, where):
    q, st = awq.awq_int8_quantize(A, s, fold)
    qr, sr = _quantise_ref(_fold_ref(A, s, fold))
    K = A.shape[1]
    assert q.shape == (A.shape[0], (K + 15) // 16 * 16)
    qg = q.cpu().numpy()
    assert np.array_equal(st.cpu().numpy().view(np.uint32)[~np.isnan(sr)],
                          sr.view(np.uint32)[~np.isnan(sr)]), where
    assert np.array_equal(np.isnan(st.cpu().numpy()), np.isnan(sr)), where
    assert np.array_equal(qg[:, :K], qr), where
    assert not qg[:, K:].any(), where


ROWS = [  # rows, columns: one chunk, odd, tails, the register limits and beyond
    (1, 1), (3, 7), (1, 16), (5, 131), (2, 4096), (3, 4097), (2, 16384), (2, 16390), (1, 70001),
    (300, 512),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("fold", [None, "divide", "multiply"])
def test_rows(dtype, fold):
    for R, K in ROWS:
        say(f"int8 rows {R}x{K} {dtype} {fold}")
        g = torch.Generator(device="cuda").manual_seed(R * 7 + K)
        A = torch.randn(R, K, generator=g, device="cuda")
        A[:, ::5] *= 30
        A = A.to(DT[dtype])
        s = torch.exp(torch.randn(K, generator=g, device="cuda")) if fold else None
        _check_rows(A, s, fold or "divide", (R, K, dtype, fold))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_rows_ties_and_extremes(dtype):
    """Exact halves (step a power of two), zero rows, subnormal rows, non-finite rows, and the
    type's largest value."""
    K = 264
    A = torch.zeros(9, K, dtype=torch.float32)
    A[1, :] = (torch.arange(K) % 255 - 127).float() / 2 / 64
    A[1, 0] = 127 / 64.0                                # step 1/64: quotients n + 1/2
    A[2, 3] = torch.finfo(DT[dtype]).tiny / 4           # subnormal of the type
    A[2, 4] = -A[2, 3]
    A[3] = 1.0
    A[3, 100] = float("inf")
    A[4] = -2.0
    A[4, K - 1] = float("nan")
    A[5, 7] = torch.finfo(DT[dtype]).max
    A[5, 8] = 1.0
    A[6] = -0.0
    A[7] = torch.linspace(-3, 3, K)
    A[8] = torch.finfo(DT[dtype]).min
    A = A.to(DT[dtype]).cuda()
    _check_rows(A, None, "divide", dtype)
    s = torch.full((K,), 1e-38, device="cuda")          # the fold overflows: rows become infinite
    _check_rows(A, s, "divide", dtype)
    _check_rows(A, torch.full((K,), 1e-42, device="cuda"), "multiply", dtype)  # subnormal steps


def test_rows_strides():
    """Row strides and bases that rule the 16-byte loads out, and a strided view."""
    base = torch.randn(40, 301, device="cuda").half()
    for A in (base[:, :257], base[:, 1:200], base[::3, 5:299], base[7:8, 2:250]):
        _check_rows(A, None, "divide", tuple(A.shape))


def _product_ref(xq, xs, wq, ws, bias):
    acc = xq.cpu().numpy().astype(F64) @ wq.cpu().numpy().astype(F64).T
    y = acc * xs.cpu().numpy().astype(F64)[:, None] * ws.cpu().numpy().astype(F64)
    b = 0.0 if bias is None else bias.float().cpu().numpy().astype(F64)
    return y, y + b, np.abs(y) + np.abs(b)


def _ulp(v, dtype):
    """The spacing of the output type at |v| (its subnormal spacing below the normal range)."""
    bits, emin = (10, -14) if dtype == torch.float16 else (7, -126)
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** emin)))
    return 2.0 ** (np.maximum(e, emin) - bits)


def _check_product(y, xq, xs, wq, ws, bias, dtype, where):
    _, want, mag = _product_ref(xq, xs, wq, ws, bias)
    got = y.float().cpu().numpy().astype(F64)
    assert got.shape == want.shape and y.dtype == dtype
    E = 2.0 ** -22 * mag
    err = np.abs(got - want)
    bound = E + _ulp(np.abs(want) + E, dtype)
    bad = ~(err <= bound)
    assert not bad.any(), (where, int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


def _random(T, M, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def codes(r):
        return torch.randint(-127, 128, (r, K), generator=g, device="cuda").to(torch.int8)

    xs = torch.rand(T, generator=g, device="cuda") * 0.02 + 1e-4
    ws = torch.rand(M, generator=g, device="cuda") * 1e-3 + 1e-5
    return codes(T), xs, codes(M), ws, torch.randn(M, generator=g, device="cuda")


SHAPES = [  # tokens, outputs, K: one of each, tile edges, odd counts, one stage, many
    (1, 1, 16), (1, 4096, 4096), (2, 257, 512), (3, 33, 48), (5, 1000, 1040), (15, 640, 128),
    (16, 512, 4096), (17, 129, 272), (31, 100, 2048), (33, 300, 5120), (63, 64, 512), (64, 777, 1024),
    (65, 5120, 208), (100, 1000, 13824), (127, 128, 144), (128, 256, 256), (129, 255, 400),
    (255, 300, 4096), (256, 512, 512), (257, 513, 1024), (333, 1111, 656), (1000, 1500, 272),
    (2100, 700, 160), (4, 28672, 256),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_product(dtype):
    for T, M, K in SHAPES:
        say(f"int8 product T={T} M={M} K={K} {dtype}")
        xq, xs, wq, ws, b = _random(T, M, K, T * 31 + M + K)
        bias = b.to(DT[dtype]) if (T + M) % 2 else None
        y = awq.awq_int8_matmul(xq, xs, wq, ws, dtype=DT[dtype], bias=bias)
        _check_product(y, xq, xs, wq, ws, bias, DT[dtype], (T, M, K, dtype))


def test_product_widest_rows():
    """All codes at the ends of the range over the longest rows: the sum nearly fills int32."""
    K = 131056
    for T in (2, 20, 140):
        xq = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
        wq = torch.full((40, K), -128, dtype=torch.int8, device="cuda")
        wq[1::2] = 127
        xs, ws = torch.full((T,), 2.0 ** -16, device="cuda"), torch.full((40,), 2.0 ** -8, device="cuda")
        y = awq.awq_int8_matmul(xq, xs, wq, ws, dtype=torch.bfloat16)
        _check_product(y, xq, xs, wq, ws, None, torch.bfloat16, T)


def test_product_strides_and_empty():
    """Padded rows in every operand, an output view, no tokens, no outputs, no columns."""
    big = torch.randint(-127, 128, (200, 640), device="cuda").to(torch.int8)
    for T in (3, 70):
        xq, wq = big[:T, 16:544], big[60:161, 96:624]
        xs, ws = torch.rand(T, device="cuda"), torch.rand(101, device="cuda") * 1e-3
        base = torch.full((T, 150), 7.0, dtype=torch.float16, device="cuda")
        y = awq.awq_int8_matmul(xq, xs, wq, ws, out=base[:, 3:104])
        _check_product(y, xq, xs, wq, ws, None, torch.float16, T)
        assert (base[:, :3] == 7).all() and (base[:, 104:] == 7).all()
    for T, M, K in ((0, 5, 32), (4, 0, 32), (4, 5, 0)):
        xq = torch.zeros((T, K), dtype=torch.int8, device="cuda")
        wq = torch.zeros((M, K), dtype=torch.int8, device="cuda")
        b = torch.arange(M, device="cuda").half()
        y = awq.awq_int8_matmul(xq, torch.ones(T, device="cuda"), wq, torch.ones(M, device="cuda"),
                                bias=b)
        assert y.shape == (T, M)
        assert torch.equal(y, b.expand(T, M))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("smooth", [False, True])
def test_linear_is_quantise_then_product(dtype, smooth):
    """The linear layer gives the two calls' result bit for bit, whatever path it takes, and a
    row that holds a NaN or an infinity comes out as NaN."""
    for T, M, K in ((1, 4096, 4096), (2, 300, 250), (3, 1000, 8192), (4, 65, 129), (7, 500, 1000),
                    (16, 1024, 4096), (40, 333, 515), (300, 600, 1025), (1, 64, 16384), (1, 70, 40000)):
        say(f"int8 linear T={T} M={M} K={K} {dtype} smooth={smooth}")
        g = torch.Generator(device="cuda").manual_seed(T + M + K)
        x = torch.randn(T, K, generator=g, device="cuda")
        x[:, ::9] *= 20
        x = x.to(DT[dtype])
        if T >= 3:
            x[1, K // 2] = float("nan")
            x[2, K - 1] = float("-inf")
        W = (torch.randn(M, K, generator=g, device="cuda") * 0.02).to(DT[dtype])
        s = torch.exp(torch.randn(K, generator=g, device="cuda") * 0.5) if smooth else None
        wq, ws = awq.awq_int8_quantize(W, s, "multiply")
        bias = torch.randn(M, generator=g, device="cuda").to(DT[dtype]) if M % 2 else None
        y = awq.awq_int8_linear(x, wq, ws, s=s, bias=bias)
        xq, xs = awq.awq_int8_quantize(x, s, "divide")
        y2 = awq.awq_int8_matmul(xq, xs, wq, ws, dtype=DT[dtype], bias=bias)
        assert torch.equal(y.view(torch.int16), y2.view(torch.int16)) or (
            torch.equal(torch.isnan(y), torch.isnan(y2))
            and torch.equal(torch.nan_to_num(y), torch.nan_to_num(y2)))
        if T >= 3:
            assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
        ok = torch.isfinite(xs)
        _check_product(y[ok], xq[ok], xs[ok], wq, ws, bias, DT[dtype], (T, M, K))
        # against the unquantised product: every code stands for its value to within half a step
        # (and three fp32 roundings), so with e_x = step_x / 2, e_w = step_w / 2 the result is
        # within sum |x'| e_w + |w'| e_x + e_x e_w of x' w', x' = x / s and w' = W s
        xf = x[ok].double() if s is None else x[ok].double() / s.double()
        wf = W.double() if s is None else W.double() * s.double()
        ex, ew = (xs[ok].double() * 0.50001)[:, None], ws.double() * 0.50001
        bound = xf.abs().sum(1, keepdim=True) * ew + wf.abs().sum(1) * ex + K * ex * ew
        exact = xf @ wf.t()
        if bias is not None:
            exact = exact + bias.double()
        got = y[ok].double()
        eps = 2.0 ** -10 if DT[dtype] == torch.float16 else 2.0 ** -7
        assert ((got - exact).abs() <= bound + eps * (exact.abs() + bound)).all()


def test_linear_other_stream():
    """Work follows the given stream: inputs made on a side stream are read after it."""
    side = torch.cuda.Stream()
    W = torch.randn(512, 1024, device="cuda").half()
    wq, ws = awq.awq_int8_quantize(W)
    torch.cuda.synchronize()
    for T in (2, 200):
        with torch.cuda.stream(side):
            x = torch.randn(T, 1024, device="cuda").half()
            for _ in range(20):
                x = (x * 1.01).half()
        y = awq.awq_int8_linear(x, wq, ws, stream=side)
        side.synchronize()
        xq, xs = awq.awq_int8_quantize(x)
        assert torch.equal(y, awq.awq_int8_matmul(xq, xs, wq, ws))
