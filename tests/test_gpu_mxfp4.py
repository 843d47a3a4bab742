"""Rows of MXFP4 and their product on the GPU (through the C ABI) against numpy in 64 bits.

Bars, derived from the kernels' arithmetic:
  - codes and scales follow from single fp32 operations and comparisons, so they are equal bit for bit;
    so are the values read back (a power of two times an element, one rounding);
  - the product adds 64 columns at a time to an fp32 sum, each step within 2^-22 of its largest term or
    result, both at most S = sum |x w|: (K / 64 + 1) 2^-22 S; the sums of up to 8 waves are joined,
    8 * 2^-24 S more, and the bias adds 2^-24 (S + |bias|); the output's rounding is half a step of the
    type;
  - where every term is a multiple of 1/4 and S 4 < 2^24 all sums are exact in fp32, whatever their
    order: equal bit for bit.
"""
import numpy as np
import pytest
import torch

import weight_only_quantization_act_amd as awq
from tests import mx_ref
from tests.gpu_util import requires_gpu, say
from tests.mx_forms import SHAPES

pytestmark = [pytest.mark.gpu, requires_gpu]

F32, F64 = np.float32, np.float64
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _fold(A, s, fold):
    x = A.float().cpu().numpy()
    if s is None:
        return x
    s = s.cpu().numpy()
    with np.errstate(all="ignore"):
        return (x / s if fold == "divide" else x * s).astype(F32)


def _to16(v32, dtype):
    return torch.from_numpy(np.ascontiguousarray(v32)).to(dtype)


def _same(a, b):
    """Equal bit for bit, any NaN for any NaN."""
    a, b = a.cpu(), b.cpu()
    return a.shape == b.shape and a.dtype == b.dtype and bool(
        ((a.view(torch.int16) == b.view(torch.int16)) | (a.isnan() & b.isnan())).all())


def _check_rows(A, s=None, fold="divide", where=""):
    codes, scales = awq.awq_mxfp4_quantize(A, s, fold)
    v = _fold(A, s, fold)
    R, K = v.shape
    cr, sr = mx_ref.quantise(v)
    assert codes.shape == cr.shape and scales.shape == sr.shape, where
    assert np.array_equal(scales.cpu().numpy()[:, :R], sr[:, :R]), where
    cg = codes.cpu().numpy()
    assert np.array_equal(cg, cr), (where, np.argwhere(cg != cr)[:4])
    with np.errstate(all="ignore"):
        want = mx_ref.values(cr, sr, K).astype(F32)
    for dt in DT.values():
        assert _same(awq.awq_mxfp4_dequantize(codes, scales, K, dtype=dt), _to16(want, dt)), where
    return codes, scales


ROWS = [  # rows, columns: one value, partial blocks and words, tile edges in both directions
    (1, 1), (3, 31), (1, 32), (5, 33), (2, 127), (4, 128), (7, 129), (16, 512), (17, 513), (33, 1000), (15, 2047),
    (300, 544), (1, 70001), (64, 4096),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("fold", [None, "divide", "multiply"])
def test_rows(dtype, fold):
    for R, K in ROWS:
        say(f"mxfp4 rows {R}x{K} {dtype} {fold}")
        g = torch.Generator(device="cuda").manual_seed(R * 7 + K)
        A = torch.randn(R, K, generator=g, device="cuda")
        A[:, ::5] *= 30
        A = A.to(DT[dtype])
        s = torch.exp(torch.randn(K, generator=g, device="cuda")) if fold else None
        _check_rows(A, s, fold or "divide", (R, K, dtype, fold))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_every_value_against_every_maximum(dtype):
    """All finite numbers of the type, blocks of 32 of them under largest values of every exponent: ties, all
    binades, subnormals, zeros of both signs."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(DT[dtype])
    v = bits[bits.isfinite()]
    v = v[torch.argsort(v.abs().float(), stable=True)]          # neighbours share a block: all ties occur
    n = v.numel() // 31 * 31
    say(f"mxfp4 all values {dtype}")
    _check_rows(v[:v.numel() // 32 * 32].reshape(-1, 32).contiguous().cuda())
    for up in (1, 2, 3, 6):                                     # and under a largest value 2^up above
        rows = v[:n].reshape(-1, 31)
        top = (rows.abs().amax(1, keepdim=True).float() * 2.0 ** up).clamp(max=float(torch.finfo(DT[dtype]).max))
        _check_rows(torch.cat([rows, top.to(DT[dtype])], 1).cuda())


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_rows_not_finite(dtype):
    """NaN and infinities spoil their block and no other; folds that overflow or vanish."""
    A = torch.randn(6, 200)
    A[0, 5] = float("nan")
    A[1, 40] = float("inf")
    A[2, 199] = float("-inf")
    A[3] = 0.0
    A[4] = -0.0
    A[5, 0:32] = torch.finfo(DT[dtype]).max
    A = A.to(DT[dtype]).cuda()
    codes, scales = _check_rows(A)
    bad = scales.cpu().transpose(0, 1).reshape(8, -1)[:6, :7] == 255
    assert bad.nonzero().tolist() == [[0, 0], [1, 1], [2, 6]]
    _check_rows(A, torch.full((200,), 1e-38, device="cuda"), "divide")
    _check_rows(A, torch.full((200,), 1e-42, device="cuda"), "multiply")
    _check_rows(A, torch.full((200,), float("inf"), device="cuda"), "divide")
    _check_rows(A, torch.full((200,), float("nan"), device="cuda"), "multiply")
    s = torch.exp(torch.randn(200, device="cuda") * 30)          # from 1e-30 to 1e30
    s[7] = 0.0
    _check_rows(A, s, "divide")
    _check_rows(A, s, "multiply")


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("R,K", [(3, 640), (40, 3200), (2050, 4096)])
def test_divisions_at_borders(R, K, dtype):
    """Quotients within three fp32 numbers of every border between two elements and of the borders of the scale,
    where one wrong rounding of v / s is another code; scales at the ends of fp32."""
    say(f"mxfp4 divisions {R}x{K} {dtype}")
    rng = np.random.default_rng(R)
    t = torch.from_numpy(rng.uniform(1, 2, (R, K)) * 2.0 ** rng.integers(-3, 4, (R, K))).to(DT[dtype])
    border = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0, 8.0])[rng.integers(0, 9, K)]
    first = t[rng.integers(0, R, K), np.arange(K)].float().numpy()  # the row whose quotient lies at the border
    s = (first / border).astype(F32)
    for n in range(3):
        s = np.where(rng.integers(0, 3, K) == n, np.nextafter(s, F32(rng.choice([0, 1e30]))), s)
    t[:, ::32], s[::32] = 4.0, 1.0                              # scales of 1 or so
    _check_rows(t.cuda(), torch.from_numpy(s).cuda(), "divide")
    if R < 100:
        for k in (-149, -140, -126, -100, 100, 127):
            with np.errstate(all="ignore"):
                far = np.ldexp(s, k).astype(F32)                    # zeros, subnormals and infinities among them
            _check_rows(t.cuda(), torch.from_numpy(far).cuda(), "divide", k)


def test_rows_strides():
    """Row strides and bases that rule the 16-byte loads out, strided views, padded codes."""
    base = torch.randn(40, 301, device="cuda").half()
    for A in (base[:, :257], base[:, 1:200], base[::3, 5:299], base[7:8, 2:250]):
        _check_rows(A, where=tuple(A.shape))
    codes, scales = awq.awq_mxfp4_quantize(base)
    wide = torch.full((40, 301 + 11), 3.0, dtype=torch.bfloat16, device="cuda")
    y = awq.awq_mxfp4_dequantize(codes, scales, 301, dtype=torch.bfloat16, out=wide[:, 5:306])
    assert torch.equal(y, awq.awq_mxfp4_dequantize(codes, scales, 301, dtype=torch.bfloat16))
    assert (wide[:, :5] == 3).all() and (wide[:, 306:] == 3).all()
    pad = torch.zeros(40, codes.shape[1] + 32, dtype=torch.uint8, device="cuda")
    pad[:, 16:-16] = codes
    assert torch.equal(awq.awq_mxfp4_dequantize(pad[:, 16:-16], scales, 301),
                       awq.awq_mxfp4_dequantize(codes, scales, 301))
    assert torch.equal(awq.awq_mxfp4_dequantize(codes[:13], scales, 301),
                       awq.awq_mxfp4_dequantize(codes, scales, 301)[:13])


def test_rows_empty():
    for R, K in ((0, 64), (5, 0)):
        codes, scales = awq.awq_mxfp4_quantize(torch.zeros(R, K, device="cuda").half())
        assert codes.shape == (R, K // 2)
        assert awq.awq_mxfp4_dequantize(codes, scales, K).shape == (R, K)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_int8_values(dtype):
    """The read-back of 8-bit rows: the code times the step, rounded once more to the type."""
    for R, K in ((1, 1), (3, 17), (5, 4096), (37, 1003), (16, 512)):
        say(f"int8 values {R}x{K} {dtype}")
        A = (torch.randn(R, K, device="cuda") * 3).to(DT[dtype])
        if R > 3:
            A[2, K // 2] = float("inf")
        q, st = awq.awq_int8_quantize(A)
        want = _to16((q[:, :K].float() * st[:, None]).cpu().numpy(), DT[dtype])
        assert _same(awq.awq_int8_dequantize(q, st, K, dtype=DT[dtype]), want)
        wide = torch.full((R, K + 9), 3.0, dtype=DT[dtype], device="cuda")
        awq.awq_int8_dequantize(q, st, K, dtype=DT[dtype], out=wide[:, 3:3 + K])
        assert _same(wide[:, 3:3 + K].contiguous(), want) and (wide[:, :3] == 3).all() and (wide[:, 3 + K:] == 3).all()


def test_int8_values_are_rounded_twice():
    """Steps whose products lie so close to a border of fp16 that fp32 rounds them onto it."""
    say("int8 values at borders")
    rng = np.random.default_rng(0)
    steps = rng.uniform(0.001, 1, 1 << 22).astype(F32)
    exact = steps.astype(F64) * 3
    near = exact.astype(np.float16) != exact.astype(F32).astype(np.float16)
    steps = steps[near]
    assert steps.size > 50
    q = torch.zeros(steps.size, 16, dtype=torch.int8, device="cuda")
    q[:, 0], q[:, 15] = 3, -3
    y = awq.awq_int8_dequantize(q, torch.from_numpy(steps).cuda(), 16)
    want = torch.from_numpy((steps * F32(3)).astype(np.float16))
    assert _same(y[:, 0].contiguous(), want) and _same(y[:, 15].contiguous(), -want)


# ---------------------------------------------------------------------------------- product
def _ulp(v, dtype):
    bits, emin = (10, -14) if dtype == torch.float16 else (7, -126)
    e = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** emin)))
    return 2.0 ** (np.maximum(e, emin) - bits)


def _random_rows(R, K, g, spread=3):
    """Codes of all values and scales over a few binades, zeros past K, padding rows of NaN scales."""
    B = (K + 31) // 32
    codes = torch.randint(0, 256, (R, 16 * B), generator=g, device="cuda", dtype=torch.uint8)
    col = 2 * torch.arange(16 * B, device="cuda")
    codes = torch.where(col < K, codes, 0)
    if K % 2:
        codes[:, K // 2] &= 15
    scales = torch.randint(127 - spread, 128 + spread, ((B + 3) // 4, (R + 3) // 4 * 4, 4), generator=g,
                           device="cuda", dtype=torch.uint8)
    scales[:, R:] = 255
    return codes, scales


def _product_ref(xc, xs, wc, ws, K, bias):
    x, w = (mx_ref.values(c.cpu().numpy(), s.cpu().numpy(), K) for c, s in ((xc, xs), (wc, ws)))
    b = 0.0 if bias is None else bias.float().cpu().numpy().astype(F64)
    return x @ w.T + b, np.abs(x) @ np.abs(w).T, np.abs(b)


def _check_product(y, xc, xs, wc, ws, K, bias, where):
    want, S, b = _product_ref(xc, xs, wc, ws, K, bias)
    got = y.float().cpu().numpy().astype(F64)
    assert got.shape == want.shape, where
    E = (K / 64 + 1 + 2 + 1) * 2.0 ** -22 * S + 2.0 ** -24 * b
    bound = E + _ulp(np.abs(want) + E, y.dtype) / 2
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (where, int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_product(shape, dtype):
    form, T, M, K = shape
    say(f"mxfp4 product, form {form}, T={T} M={M} K={K} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(T * 31 + M + K)
    (xc, xs), (wc, ws) = _random_rows(T, K, g), _random_rows(M, K, g)
    xs, ws = xs - 4, ws - 4                                     # (fp16's range; 255 stays a power of two)
    bias = torch.randn(M, generator=g, device="cuda").to(DT[dtype]) if (T + M) % 2 else None
    y = awq.awq_mxfp4_matmul(xc, xs, wc, ws, dtype=DT[dtype], bias=bias)
    _check_product(y, xc, xs, wc, ws, K, bias, (T, M, K, dtype))


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_product_bit_for_bit(shape):
    """Scales of 1 and sums that are exact in fp32: every bit is the formula's."""
    form, T, M, K = shape
    say(f"mxfp4 product, exact, form {form}, T={T} M={M} K={K}")
    g = torch.Generator(device="cuda").manual_seed(T + M + K)
    xc, xs = _random_rows(T, K, g)
    wc, ws = _random_rows(M, K, g)
    xs.fill_(127)
    ws.fill_(127)
    want, S, _ = _product_ref(xc, xs, wc, ws, K, None)
    exact = S.max() * 4 < 2 ** 24
    assert exact or K > 4096
    for dt in DT.values():
        y = awq.awq_mxfp4_matmul(xc, xs, wc, ws, dtype=dt)
        if exact:
            assert _same(y, _to16(want.astype(F32), dt))
        assert torch.equal(y, awq.awq_mxfp4_matmul(xc, xs, wc, ws, dtype=dt))


@pytest.mark.parametrize("T", [1, 5, 16, 20, 40, 100, 300, 3900])
def test_scales_reach_their_blocks(T):
    """One block of a row not zero at a time, with a scale of its own: each block's scale is its own in every
    form (a swapped one would show as a power of two)."""
    M, K = 130, 1120                                            # 35 blocks: odd words and steps
    g = torch.Generator(device="cuda").manual_seed(T)
    xc, xs = _random_rows(T, K, g, 1)
    wc, ws = _random_rows(M, K, g, 1)
    say(f"mxfp4 scales T={T}")
    xs[:, :T] = torch.randint(100, 154, xs[:, :T].shape, generator=g, device="cuda", dtype=torch.uint8)
    block = torch.arange(T, device="cuda") % 35
    keep = torch.arange(xc.shape[1], device="cuda")[None] // 16 == block[:, None]
    xc = torch.where(keep, xc, 0)
    ws[:, :M] = torch.randint(100, 154, ws[:, :M].shape, generator=g, device="cuda", dtype=torch.uint8)
    y = awq.awq_mxfp4_matmul(xc, xs, wc, ws, dtype=torch.bfloat16)
    want, _, _ = _product_ref(xc, xs, wc, ws, K, None)          # 32 terms of one scale: exact in fp32
    assert _same(y, _to16(want.astype(F32), torch.bfloat16))


@pytest.mark.parametrize("T", [1, 7, 16, 30, 60, 200, 3900])
def test_product_nan_scale_spoils_its_row_only(T):
    M, K = 300, 1000
    say(f"mxfp4 product nan T={T}")
    g = torch.Generator(device="cuda").manual_seed(T)
    (xc, xs), (wc, ws) = _random_rows(T, K, g), _random_rows(M, K, g)
    clean = awq.awq_mxfp4_matmul(xc, xs, wc, ws, dtype=torch.bfloat16)
    assert clean.isfinite().all()
    rows, cols = torch.zeros(T, dtype=torch.bool), torch.zeros(M, dtype=torch.bool)
    rows[T // 2] = cols[77] = cols[299] = True
    xs[7, T // 2, 3] = 255                                       # the last block of all (K = 31.25 blocks)
    ws[0, 77, 0] = 255
    ws[3, 299, 2] = 255
    y = awq.awq_mxfp4_matmul(xc, xs, wc, ws, dtype=torch.bfloat16)
    bad = (rows[:, None] | cols[None]).cuda()
    assert torch.equal(y.isnan(), bad)
    assert torch.equal(y[~bad], clean[~bad])


def test_product_strides_and_empty():
    """Padded rows in every operand, an output view, no tokens, no outputs, no columns."""
    g = torch.Generator(device="cuda").manual_seed(1)
    big, bs = _random_rows(200, 1280, g)
    for T in (3, 40, 70, 150):
        xc, wc = big[:T, 16:272], big[30:131, 96:352]
        _, xs = _random_rows(T, 512, g)
        _, ws = _random_rows(101, 512, g)
        base = torch.full((T, 150), 7.0, dtype=torch.bfloat16, device="cuda")
        y = awq.awq_mxfp4_matmul(xc, xs, wc, ws, dtype=torch.bfloat16, out=base[:, 3:104])
        _check_product(y, xc, xs, wc, ws, 512, None, T)
        assert (base[:, :3] == 7).all() and (base[:, 104:] == 7).all()
        # a prefix of more rows, whose scales are those of the whole
        _, more = _random_rows(200, 512, g)
        more[:, :T] = xs[:, :T]
        assert torch.equal(awq.awq_mxfp4_matmul(xc, more, wc, ws, dtype=torch.bfloat16), y)
    for T, M, K in ((0, 5, 32), (4, 0, 32), (4, 5, 0), (40, 5, 0)):
        (xc, xs), (wc, ws) = _random_rows(T, K, g), _random_rows(M, K, g)
        b = torch.arange(M, device="cuda").half()
        y = awq.awq_mxfp4_matmul(xc, xs, wc, ws, bias=b)
        assert y.shape == (T, M) and torch.equal(y, b.expand(T, M))
        if K == 0:
            y = awq.awq_mxfp4_linear(torch.zeros(T, 0, device="cuda").half(), wc, ws, bias=b)
            assert torch.equal(y, b.expand(T, M))


# ----------------------------------------------------------------------------------- linear
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("smooth", [False, True])
def test_linear_is_quantise_then_product(dtype, smooth):
    """The linear layer gives the two calls' result bit for bit, whatever path it takes, leaves the bytes
    behind its workspace, and a row with a NaN or an infinity comes out as NaN."""
    for T, M, K in ((1, 4096, 4096), (1, 70, 40000), (1, 300, 33), (1, 16500, 250), (2, 300, 250), (3, 1000, 8192),
                    (4, 65, 129), (7, 500, 1000), (16, 1024, 4096), (20, 333, 515), (40, 333, 8000),
                    (300, 600, 1025), (200, 128, 9001)):
        say(f"mxfp4 linear T={T} M={M} K={K} {dtype} smooth={smooth}")
        g = torch.Generator(device="cuda").manual_seed(T + M + K)
        x = torch.randn(T, K + 3, generator=g, device="cuda")
        x[:, ::9] *= 20
        x = x.to(DT[dtype])[:, :K] if T % 2 else x.to(DT[dtype])[:, 1:K + 1]
        if T >= 3:
            x[1, K // 2] = float("nan")
            x[2, K - 1] = float("-inf")
        W = (torch.randn(M, K, generator=g, device="cuda") * 0.02).to(DT[dtype])
        s = torch.exp(torch.randn(K, generator=g, device="cuda") * 0.5) if smooth else None
        wc, ws = awq.awq_mxfp4_quantize(W, s, "multiply")
        bias = torch.randn(M, generator=g, device="cuda").to(DT[dtype]) if M % 2 else None
        need = awq.awq_mxfp4_linear_workspace_bytes(T, M, K)
        buf = torch.full((need + (1 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
        y = awq.awq_mxfp4_linear(x, wc, ws, s=s, bias=bias, workspace=buf[:need])
        assert (buf[need:] == 0x5A).all()
        xc, xs = awq.awq_mxfp4_quantize(x, s, "divide")
        assert _same(y, awq.awq_mxfp4_matmul(xc, xs, wc, ws, dtype=DT[dtype], bias=bias))
        assert _same(y, awq.awq_mxfp4_linear(x, wc, ws, s=s, bias=bias))
        if T >= 3:
            assert y[1].isnan().all() and y[2].isnan().all()
        ok = torch.ones(T, dtype=torch.bool, device="cuda")
        if T >= 3:
            ok[1] = ok[2] = False
        some, codes = xs[:, :T][:, ok], xc[ok]
        some = torch.nn.functional.pad(some, (0, 0, 0, -codes.shape[0] % 4)).contiguous()
        _check_product(y[ok], codes, some, wc, ws, K, bias, (T, M, K))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("smooth", [False, True])
@pytest.mark.parametrize("K", [1, 250, 1001, 1024, 4096])
def test_linear_in_one_launch(K, smooth, dtype):
    """Few tokens times few columns: quantised inside the product, in groups of tokens, the last one short."""
    W = torch.randn(70, K, device="cuda").to(DT[dtype])
    s = torch.exp(torch.randn(K, device="cuda")) if smooth else None
    wc, ws = awq.awq_mxfp4_quantize(W, s, "multiply")
    for T in (1, 2, 3, 4, 5, 7, 8, 9, 16):
        if T * K > 16384:
            continue
        say(f"mxfp4 linear in one launch T={T} K={K} {dtype} smooth={smooth}")
        assert awq.awq_mxfp4_linear_workspace_bytes(T, 70, K) == 0
        wide = torch.randn(T, K + 5, device="cuda").to(DT[dtype])
        x = wide[:, 3:3 + K]
        x[T // 2, K // 2] = float("nan") if T % 2 else 1e4
        xc, xs = awq.awq_mxfp4_quantize(x, s, "divide")
        want = awq.awq_mxfp4_matmul(xc, xs, wc, ws, dtype=DT[dtype])
        assert _same(awq.awq_mxfp4_linear(x, wc, ws, s=s), want)
        if T % 2:
            assert want[T // 2].isnan().all() and int(want.isnan().sum()) == 70


def test_linear_on_another_stream():
    """Work follows the given stream: inputs made on a side stream are read after it."""
    side = torch.cuda.Stream()
    W = torch.randn(512, 1024, device="cuda").half()
    wc, ws = awq.awq_mxfp4_quantize(W)
    torch.cuda.synchronize()
    for T in (1, 2, 200):
        say(f"mxfp4 linear on a side stream T={T}")
        with torch.cuda.stream(side):
            x = torch.randn(T, 1024, device="cuda").half()
            for _ in range(20):
                x = (x * 1.01).half()
        y = awq.awq_mxfp4_linear(x, wc, ws, stream=side)
        side.synchronize()
        xc, xs = awq.awq_mxfp4_quantize(x)
        assert torch.equal(y, awq.awq_mxfp4_matmul(xc, xs, wc, ws))


def test_refusals_of_the_binding():
    x = torch.zeros(4, 64, device="cuda").half()
    c, s = awq.awq_mxfp4_quantize(x)
    with pytest.raises(ValueError):
        awq.awq_mxfp4_quantize(x, fold="add")
    with pytest.raises(TypeError):
        awq.awq_mxfp4_quantize(x.float())
    with pytest.raises(ValueError):
        awq.awq_mxfp4_quantize(x.t())
    with pytest.raises(ValueError):
        awq.awq_mxfp4_quantize(x, torch.ones(63, device="cuda"))
    with pytest.raises(ValueError):
        awq.awq_mxfp4_matmul(c, s[:, :3], c, s)
    with pytest.raises(TypeError):
        awq.awq_mxfp4_matmul(c, s.view(torch.int8), c, s)
    with pytest.raises(ValueError):
        awq.awq_mxfp4_matmul(c, s, *awq.awq_mxfp4_quantize(x[:, :32].contiguous()))
    with pytest.raises(ValueError):
        awq.awq_mxfp4_linear(x[:, :32], c, s)
    with pytest.raises(TypeError):
        awq.awq_mxfp4_linear(x, c, s, bias=torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError):
        awq.awq_mxfp4_dequantize(c, s, 32)
    with pytest.raises(ValueError):
        awq.awq_int8_dequantize(c.view(torch.int8), torch.ones(4, device="cuda"), 16)
    need = awq.awq_mxfp4_linear_workspace_bytes(40, 4, 64)
    with pytest.raises(awq.AwqError):
        awq.awq_mxfp4_linear(torch.zeros(40, 64, device="cuda").half(), c, s,
                             workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
