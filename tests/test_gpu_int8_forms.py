"""The product in 8-bit integers in each of its forms, bit for bit: the sum is exact, so that the fp32
operations that awq_serve.h writes down, in their order, give the result's every bit."""
import pytest
import torch

import weight_only_quantization_act_amd as awq
from tests.gpu_util import requires_gpu, say
from tests.int8_forms import SHAPES

pytestmark = [pytest.mark.gpu, requires_gpu]

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _want(xq, xs, wq, ws, bias, dtype):
    # 2^14 K < 2^53: exact in any order; one rounding an operation after that
    y = (xq.double() @ wq.double().t()).float() * xs[:, None] * ws
    if bias is not None:
        y = y + bias.float()
    return y.to(dtype)


def _codes(rows, cols, pad, g):
    """int8 [rows, cols] as a view with padded rows (the padding is never to be read: random)."""
    return torch.randint(-127, 128, (rows, cols + pad), generator=g, device="cuda").to(torch.int8)[:, :cols]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_product_bit_for_bit(shape, dtype):
    form, parts, T, M, K = shape
    say(f"int8 form {form} in {parts} parts: T={T} M={M} K={K} {dtype}")
    g = torch.Generator(device="cuda").manual_seed(T + M + K)
    xs = torch.rand(T, generator=g, device="cuda") * 0.02 + 1e-4
    ws = torch.rand(M, generator=g, device="cuda") * 1e-3 + 1e-5
    b = torch.randn(M, generator=g, device="cuda").to(DT[dtype])
    for pad, bias in ((0, None), (48, b)):
        xq, wq = _codes(T, K, pad, g), _codes(M, K, pad, g)
        base = torch.full((T, M + 2 * pad), 3.0, dtype=DT[dtype], device="cuda")
        out = base[:, pad:pad + M]
        y = awq.awq_int8_matmul(xq, xs, wq, ws, dtype=DT[dtype], bias=bias, out=out)
        want = _want(xq, xs, wq, ws, bias, DT[dtype])
        assert torch.equal(y, want), (int((y != want).sum()), (y != want).nonzero()[:3])
        if pad:
            assert (base[:, :pad] == 3).all() and (base[:, pad + M:] == 3).all()


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("M", [100, 16401, 16384 + 32])
def test_fused_token_bit_for_bit(M, dtype):
    """One token with the quantisation fused, 16 and 32 outputs a block, the last block in part."""
    for K in (16, 272, 1000, 4096, 16384):
        say(f"int8 fused M={M} K={K} {dtype}")
        g = torch.Generator(device="cuda").manual_seed(M + K)
        x = torch.randn(1, K, generator=g, device="cuda").to(DT[dtype])
        s = torch.exp(torch.randn(K, generator=g, device="cuda"))
        K16 = (K + 15) // 16 * 16
        wq = torch.randint(-127, 128, (M, K16), generator=g, device="cuda").to(torch.int8)
        ws = torch.rand(M, generator=g, device="cuda") * 1e-3
        bias = torch.randn(M, generator=g, device="cuda").to(DT[dtype])
        for scales, bb in ((None, None), (s, bias)):
            xq, xs = awq.awq_int8_quantize(x, scales)
            y = awq.awq_int8_linear(x, wq, ws, s=scales, bias=bb)
            assert torch.equal(y, _want(xq, xs, wq, ws, bb, DT[dtype]))
