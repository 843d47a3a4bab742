"""MXFP4 rows, products and the norm past the sizes of caches, of 32-bit offsets and of one grid dimension:
what a large call gives is what calls on parts of it give, bit for bit, and products of small integers are
exact."""
import pytest
import torch

import weight_only_quantization_act_amd as awq
from tests.gpu_util import requires_gpu, say

pytestmark = [pytest.mark.gpu, requires_gpu]

NORMS = {"same": awq.awq_rmsnorm, "int8": awq.awq_rmsnorm_int8, "mxfp4": awq.awq_rmsnorm_mxfp4}


def _equal(kind, whole, part, a, b):
    """Outputs of rows a to b of a large call against those of the rows by themselves."""
    if kind == "mxfp4":
        return (torch.equal(whole[0][a:b], part[0]) and torch.equal(whole[1][:, a:b], part[1][:, :b - a])
                and torch.equal(whole[2][a:b], part[2]))
    return all(torch.equal(w[a:b], p) for w, p in zip(whole, part))


def _parts(rows, n=3, size=1100):                                 # (as many rows a wave as the whole has)
    step = (rows - size) // (n - 1)
    return [(i * step, i * step + size) for i in range(n - 1)] + [(rows - size, rows)]


@pytest.mark.parametrize("kind", NORMS)
@pytest.mark.parametrize("rows,cols", [(300001, 500), (40000, 4000), (17000, 8192), (7001, 20004), (4099, 33001)])
def test_norm_of_sums_past_the_caches(rows, cols, kind):
    say(f"norm {kind} {rows} x {cols}")
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.float16)
    r = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.float16)
    w = torch.randn(cols, generator=g, device="cuda")
    want = NORMS[kind](x, w, 1e-6, residual=r)
    for a, b in _parts(rows):
        assert _equal(kind, want, NORMS[kind](x[a:b], w, 1e-6, residual=r[a:b]), a, b)
    assert torch.equal(want[-1], (x.float() + r.float()).half())
    got = NORMS[kind](x, w, 1e-6, residual=r, h_out=r)            # the sum in the residual's place
    assert got[-1] is r
    assert _equal(kind, got, (*want[:-1], want[-1]), 0, rows)


@pytest.mark.parametrize("kind", NORMS)
def test_norm_past_32_bits(kind):
    say(f"norm {kind}, offsets past 32 bits")
    rows, cols, ld = 66001, 101, 66003
    base = torch.empty(rows * ld, device="cuda", dtype=torch.bfloat16)
    x = base.as_strided((rows, cols), (ld, 1))
    r = base.as_strided((rows, cols), (ld, 1), 3001)
    h = base.as_strided((rows, cols), (ld, 1), 9002)
    x.copy_(torch.randn(rows, cols, device="cuda"))
    r.copy_(torch.randn(rows, cols, device="cuda"))
    got = NORMS[kind](x, None, 1e-6, residual=r, h_out=h)
    want = NORMS[kind](x.contiguous(), None, 1e-6, residual=r.contiguous())
    assert _equal(kind, got, want, 0, rows)
    if kind == "same":
        y = base.as_strided((rows, cols), (ld, 1), 20005)
        awq.awq_rmsnorm(x, None, 1e-6, residual=r, h_out=h, out=y)
        assert torch.equal(y, want[0])


def test_rows_past_32_bits():
    say("rows, offsets past 32 bits")
    rows, cols, ld = 66001, 101, 66003
    base = torch.empty(rows * ld, device="cuda", dtype=torch.bfloat16)
    x, back = (base.as_strided((rows, cols), (ld, 1), o) for o in (0, 5001))
    x.copy_(torch.randn(rows, cols, device="cuda"))
    c, s = awq.awq_mxfp4_quantize(x)
    c2, s2 = awq.awq_mxfp4_quantize(x.contiguous())
    assert torch.equal(c, c2) and torch.equal(s[:, :rows], s2[:, :rows])
    awq.awq_mxfp4_dequantize(c, s, cols, torch.bfloat16, out=back)
    assert torch.equal(back, awq.awq_mxfp4_dequantize(c, s, cols, torch.bfloat16))
    # codes far apart
    ldc = (1 << 22) - 16
    wide = torch.empty(1100 * ldc, device="cuda", dtype=torch.uint8).as_strided((1100, 64), (ldc, 1))
    wide.copy_(c[:1100])
    s1 = s[:, :1100].contiguous()
    assert torch.equal(awq.awq_mxfp4_dequantize(wide, s1, cols), awq.awq_mxfp4_dequantize(c[:1100], s1, cols))
    for T in (1, 16, 100, 1100):                                   # both operands of the product
        for M in (1100, 40):
            st, sm = s[:, :(T + 3) // 4 * 4].contiguous(), s[:, :M].contiguous()
            assert torch.equal(awq.awq_mxfp4_matmul(wide[:T], st, wide[:M], sm),
                               awq.awq_mxfp4_matmul(c[:T], st, c[:M], sm))
    q, steps = awq.awq_int8_quantize(x)
    awq.awq_int8_dequantize(q, steps, cols, torch.bfloat16, out=back)
    assert torch.equal(back, awq.awq_int8_dequantize(q, steps, cols, torch.bfloat16))


@pytest.mark.parametrize("T,M,K", [(9000, 16001, 100), (16384, 9000, 64), (40000, 4104, 130), (140001, 1000, 40)])
def test_results_past_the_caches(T, M, K):
    say(f"product {T} {M} {K}")
    g = torch.Generator(device="cuda").manual_seed(K)
    v = torch.tensor([0, 1, 2, 3, 4, 6, -1, -2, -3, -4, -6], device="cuda", dtype=torch.float16)
    x = v[torch.randint(0, 11, (T, K), generator=g, device="cuda")]
    w = v[torch.randint(0, 11, (M, K), generator=g, device="cuda")]
    x[:, ::32], w[:, ::32] = 6, 6                                  # every block's scale is 1
    y = awq.awq_mxfp4_matmul(*awq.awq_mxfp4_quantize(x), *awq.awq_mxfp4_quantize(w), dtype=torch.float16)
    xf, wf = x.float(), w.float().t().contiguous()
    for a in range(0, T, 10000):                                   # sums below 2^24: exact in any order
        assert torch.equal(y[a:a + 10000], torch.mm(xf[a:a + 10000], wf).half())
    del y
    ldy = M + 13                                                   # rows at any address, their gaps kept
    base = torch.full((T, ldy), 7.0, device="cuda", dtype=torch.float16)
    awq.awq_mxfp4_matmul(*awq.awq_mxfp4_quantize(x), *awq.awq_mxfp4_quantize(w), dtype=torch.float16,
                         out=base[:, 3:M + 3])
    for a in range(0, T, 10000):
        assert torch.equal(base[a:a + 10000, 3:M + 3], torch.mm(xf[a:a + 10000], wf).half())
    assert bool((base[:, :3] == 7).all()) and bool((base[:, M + 3:] == 7).all())


def test_results_past_32_bits():
    say("product, results past 32 bits")
    T, M, ldy = 3001, 70, 1500001
    x = torch.randn(T, 200, device="cuda").half()
    w = torch.randn(M, 200, device="cuda").half()
    y = torch.empty(T * ldy, device="cuda", dtype=torch.float16).as_strided((T, M), (ldy, 1))
    wq = awq.awq_mxfp4_quantize(w)
    awq.awq_mxfp4_linear(x, *wq, out=y)
    assert torch.equal(y, awq.awq_mxfp4_linear(x, *wq))


def test_grids_past_32_bits():
    """More threads than 2^32: the launch's grid is split in two dimensions."""
    say("grids past 2^32 threads")
    rows, cols = (1 << 26) + 5, 8
    x = torch.randn(rows, cols, device="cuda", dtype=torch.float16)
    y, _ = awq.awq_rmsnorm(x)
    for a, b in _parts(rows):
        assert torch.equal(y[a:b], awq.awq_rmsnorm(x[a:b])[0])
    assert bool(torch.isfinite(y).all())
    del x, y
    rows, cols = (1 << 27) + 9, 3
    x = torch.randn(rows, cols, device="cuda", dtype=torch.float16)
    c, s = awq.awq_mxfp4_quantize(x)
    for a, b in _parts(rows):
        cp, sp = awq.awq_mxfp4_quantize(x[a:b])
        assert torch.equal(c[a:b], cp) and torch.equal(s[:, a:b], sp[:, :b - a])
    del c, s, x
    rows, cols = (1 << 28) + 17, 2
    q = torch.zeros(rows, 16, device="cuda", dtype=torch.int8)
    q[:, 0], q[:, 1] = 3, -5
    steps = torch.rand(rows, device="cuda")
    y = awq.awq_int8_dequantize(q, steps, cols)
    for a in range(0, rows, 1 << 26):
        part = steps[a:a + (1 << 26)]
        assert torch.equal(y[a:a + (1 << 26), 0], (3 * part).half())
        assert torch.equal(y[a:a + (1 << 26), 1], (-5 * part).half())


def test_longest_rows():
    """The norm over rows of 2^27 columns and more, MXFP4 rows and products over 2^22, the most they take."""
    say("longest rows")
    K = (1 << 27) + 9
    x = torch.full((2, K), 2.0, device="cuda", dtype=torch.float16)
    x[1] = -2
    # the mean is 4 to within fp64's rounding, v fp32's 1
    y, _ = awq.awq_rmsnorm(x, None, 1e-30)
    assert bool((y[0] == 1).all()) and bool((y[1] == -1).all())
    q, st, _ = awq.awq_rmsnorm_int8(x, None, 1e-30)
    assert bool((q[0, :K] == 127).all()) and bool((q[1, :K] == -127).all()) and bool((q[:, K:] == 0).all())
    del x, y, q
    K = 1 << 22
    g = torch.Generator(device="cuda").manual_seed(0)
    for T, M in ((1, 10), (3, 200), (70, 300), (300, 300)):
        x, w = (torch.randint(-40, 41, (n, K), generator=g, device="cuda", dtype=torch.int8) for n in (T, M))
        x, w = (torch.where(a.abs() <= 1, a, 0).half() for a in (x, w))
        x[:, ::32], w[:, ::32] = 4, 0                               # scales of 1 and of 1 / 4 or 0
        xq, wq = awq.awq_mxfp4_quantize(x), awq.awq_mxfp4_quantize(w)
        assert torch.equal(awq.awq_mxfp4_dequantize(*xq, K), x) and torch.equal(awq.awq_mxfp4_dequantize(*wq, K), w)
        y = awq.awq_mxfp4_matmul(*xq, *wq)
        want = torch.mm(x.float(), w.float().t().contiguous())      # sums of a few thousand ones: exact
        assert float(want.abs().max()) < 2048 and torch.equal(y, want.half())
        assert torch.equal(awq.awq_mxfp4_linear(x, *wq), y)
    with pytest.raises(Exception):
        awq.awq_mxfp4_quantize(torch.zeros(1, K + 1, device="cuda", dtype=torch.float16))
