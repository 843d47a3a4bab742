"""MXFP4 products on the GPU at the edges of their operands: what lies behind the last block of a row.

Bars: a product whose operands differ in what it does not look at is the same bit for bit.
"""
import pytest
import torch

import weight_only_quantization_act_amd as awq
from tests.gpu_util import requires_gpu, say
from tests.mx_forms import SHAPES
from tests.test_gpu_mxfp4 import _random_rows

pytestmark = [pytest.mark.gpu, requires_gpu]


def _behind(scales, K, byte):
    """A copy with the bytes behind each row's last block set (tensor or number)."""
    last = (K + 31) // 32 % 4
    scales = scales.clone()
    if last:
        scales[-1, :, last:] = byte
    return scales


@pytest.mark.parametrize("shape", [s for s in SHAPES if (s[3] + 31) // 32 % 4], ids=lambda s: "-".join(map(str, s)))
def test_scales_behind_the_last_block_are_not_looked_at(shape):
    """Scales packed elsewhere may hold anything in a word's bytes past the row's last block, 255 among it."""
    form, T, M, K = shape
    say(f"mxfp4 product, bytes behind the last scale, form {form}, T={T} M={M} K={K}")
    g = torch.Generator(device="cuda").manual_seed(T + 3 * M + K)
    (xc, xs), (wc, ws) = _random_rows(T, K, g), _random_rows(M, K, g)
    xs, ws = (_behind(s, K, 0) for s in (xs, ws))
    want = awq.awq_mxfp4_matmul(xc, xs, wc, ws, dtype=torch.bfloat16)
    assert want.isfinite().all()
    noise = [_behind(s, K, torch.randint(0, 256, (1, s.shape[1], 1), generator=g, device="cuda", dtype=torch.uint8))
             for s in (xs, ws)]
    for x2, w2 in ((_behind(xs, K, 255), ws), (xs, _behind(ws, K, 255)), noise):
        assert torch.equal(awq.awq_mxfp4_matmul(xc, x2, wc, w2, dtype=torch.bfloat16), want)
    # a NaN of the last block itself still is one
    B = (K + 31) // 32
    ws = _behind(ws, K, 255)
    ws[-1, 0, (B - 1) % 4] = 255
    y = awq.awq_mxfp4_matmul(xc, xs, wc, ws, dtype=torch.bfloat16)
    assert y[:, 0].isnan().all() and torch.equal(y[:, 1:], want[:, 1:])


@pytest.mark.parametrize("T", [1, 4, 40, 300])
def test_linear_with_scales_behind_the_last_block(T):
    M, K = 300, 1060                                            # 34 blocks
    say(f"mxfp4 linear, bytes behind the last scale, T={T}")
    x = torch.randn(T, K, device="cuda").half()
    wc, ws = awq.awq_mxfp4_quantize(torch.randn(M, K, device="cuda").half())
    want = awq.awq_mxfp4_linear(x, wc, ws)
    w2 = _behind(ws, K, 255)
    assert torch.equal(awq.awq_mxfp4_linear(x, wc, w2), want)
    assert torch.equal(awq.awq_mxfp4_dequantize(wc, w2, K), awq.awq_mxfp4_dequantize(wc, ws, K))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M,K", [(300, 17632), (4096, 17601), (5000, 7744), (8192, 7001), (33, 11008)])
def test_linear_of_one_token_at_its_longest(M, K, dtype):
    """The most columns that one token is quantised inside the product's launch for: no workspace, the two calls'
    result bit for bit; one block more takes two launches."""
    say(f"mxfp4 linear of one token M={M} K={K} {dtype}")
    assert awq.awq_mxfp4_linear_workspace_bytes(1, M, K) == 0
    most = 17632 if M <= 4096 else 7744
    assert awq.awq_mxfp4_linear_workspace_bytes(1, M, most) == 0
    assert awq.awq_mxfp4_linear_workspace_bytes(1, M, most + 1) > 0
    wc, ws = awq.awq_mxfp4_quantize((torch.randn(M, K, device="cuda") * 0.02).to(dtype))
    s = torch.exp(torch.randn(K, device="cuda") * 0.5)
    x = torch.randn(1, K, device="cuda").to(dtype)
    bias = torch.randn(M, device="cuda").to(dtype)
    for scale in (None, s):
        got = awq.awq_mxfp4_linear(x, wc, ws, s=scale, bias=bias)
        want = awq.awq_mxfp4_matmul(*awq.awq_mxfp4_quantize(x, scale), wc, ws, dtype=dtype, bias=bias)
        assert torch.equal(got, want) and got.isfinite().all()
    x[0, K - 1] = float("nan")
    assert awq.awq_mxfp4_linear(x, wc, ws, s=s).isnan().all()


@pytest.mark.parametrize("K", [64, 1000, 5000, 17000])
@pytest.mark.parametrize("T", [1, 7, 1030])
def test_norm_over_its_inputs(T, K):
    """y in the place of x or of the residual, rows in registers and rows read twice, one wave a row and eight."""
    say(f"norm over its inputs T={T} K={K}")
    x, r = (torch.randn(T, K, device="cuda").half() for _ in range(2))
    w = torch.randn(K, device="cuda")
    alone, (both, h) = awq.awq_rmsnorm(x, w)[0], awq.awq_rmsnorm(x, w, residual=r)
    a, b, c = x.clone(), x.clone(), r.clone()
    assert torch.equal(awq.awq_rmsnorm(a, w, out=a)[0], alone)
    got = awq.awq_rmsnorm(b, w, residual=r, out=b)
    assert torch.equal(b, both) and torch.equal(got[1], h)
    got = awq.awq_rmsnorm(x, w, residual=c, out=c)
    assert torch.equal(c, both) and torch.equal(got[1], h)
    b, c = x.clone(), r.clone()                                  # both results over both inputs, either way round
    awq.awq_rmsnorm(b, w, residual=c, out=b, h_out=c)
    assert torch.equal(b, both) and torch.equal(c, h)
    b, c = x.clone(), r.clone()
    awq.awq_rmsnorm(b, w, residual=c, out=c, h_out=b)
    assert torch.equal(c, both) and torch.equal(b, h)
