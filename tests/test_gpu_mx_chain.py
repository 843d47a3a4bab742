"""The norm, the MXFP4 rows and the product together, as the layers of a decoder use them: an MLP block on
MXFP4 weights under smoothing scales (norm with the residual's addition into MXFP4, product, linear layer
back, next norm into 8 bits, 8-bit product), as plain calls, on a side stream, and captured into a graph that
is replayed with other inputs.

Bars: what two ways of the same kernels give is equal bit for bit.  Against the block on the values that
the codes stand for (each stage on the GPU's own inputs to it, in 64 bits): the product's bound of
test_gpu_mxfp4.py.  Against the same block on 16-bit weights, derived for unit normal values: an MXFP4
block of 32 has its largest value, 2.3 sigma or so, at 4 to 8 units of its scale, so the scale is 0.29 to
0.58 sigma; most values lie below 4 units, where the steps are 1/2 (up to 2) and 1 (2 to 4), so the error of one
is about 0.3 units, 0.13 sigma (0.115 on the CPU's plain form); the gated values, whose tails are longer, are
rounded by 0.15 of their size.  A sum of products of x with w, both so rounded, is off by sqrt(2) 0.13 = 0.18
of its size, the gate's product of two such by sqrt(2) 0.18 = 0.26, and the way back, whose weights add 0.13, by
sqrt(0.26^2 + 0.15^2 + 0.13^2) = 0.33.  Below 0.4 of the block's contribution.
"""
import numpy as np
import pytest
import torch

import weight_only_quantization_act_amd as awq
from tests import mx_ref
from tests.gpu_util import requires_gpu, say
from tests.test_gpu_mxfp4 import _check_product

pytestmark = [pytest.mark.gpu, requires_gpu]


class Block:
    """norm -> gate and up (one product) -> silu gate -> down -> residual -> norm in 8 bits -> 8-bit head."""

    def __init__(self, hidden, inner, out, dtype, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda")
        self.dtype = dtype
        self.w1, self.w2 = 1 + 0.1 * normal(hidden), (1 + 0.1 * normal(hidden)).to(dtype)
        self.s = torch.exp(0.3 * normal(hidden))               # smoothing scales of gate and up
        self.gate_up = (normal(2 * inner, hidden) * hidden ** -0.5).to(dtype)
        self.down = (normal(hidden, inner) * inner ** -0.5).to(dtype)
        self.head = (normal(out, hidden) * hidden ** -0.5).to(dtype)
        self.gu = awq.awq_mxfp4_quantize(self.gate_up, self.s, fold="multiply")
        self.d = awq.awq_mxfp4_quantize(self.down)
        self.hq = awq.awq_int8_quantize(self.head)
        self.folded = self.w1 / self.s                         # the norm's weight takes 1 / s

    def forward(self, x, r, stream=None):
        kw = {} if stream is None else {"stream": stream}
        xc, xs, h = awq.awq_rmsnorm_mxfp4(x, self.folded, 1e-5, residual=r, **kw)
        gu = awq.awq_mxfp4_matmul(xc, xs, *self.gu, dtype=self.dtype, **kw)
        if stream is None:
            a = self.act(gu)
        else:
            with torch.cuda.stream(stream):
                a = self.act(gu)
        y = awq.awq_mxfp4_linear(a, *self.d, **kw)
        q, st, h2 = awq.awq_rmsnorm_int8(y, self.w2, 1e-5, residual=h, **kw)
        z = awq.awq_int8_matmul(q, st, *self.hq, dtype=self.dtype, **kw)
        return {"xc": xc, "xs": xs, "h": h, "gu": gu, "a": a, "y": y, "q": q, "st": st, "h2": h2, "z": z}

    @staticmethod
    def act(gu):
        g, u = gu.float().chunk(2, 1)
        return (g * torch.sigmoid(g) * u).to(gu.dtype)

    def plain(self, x, r):
        h = x.double() + r.double()

        def norm(v, w):
            return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-5) * w.double()
        gu = norm(h, self.w1).cpu() @ self.gate_up.double().cpu().t()
        g, u = gu.chunk(2, 1)
        y = ((g * torch.sigmoid(g) * u) @ self.down.double().cpu().t()).to(h.device)
        return y, h + y


def _same(a, b):
    return all(torch.equal(a[k][:, :a["h"].shape[0]] if k == "xs" else a[k], b[k][:, :a["h"].shape[0]] if k == "xs" else b[k])
               for k in a)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("T", [1, 5, 16, 70, 400])
def test_block(T, dtype):
    say(f"mxfp4 block T={T} {dtype}")
    b = Block(520, 1000, 300, dtype)
    x, r = (torch.randn(T, 520, device="cuda").to(dtype) for _ in range(2))
    o = b.forward(x, r)
    # each stage against what its inputs stand for
    h, v, sure = mx_ref.norm(x, r, b.folded, 1e-5, dtype)
    assert np.array_equal(o["h"].double().cpu().numpy(), h)
    cr, sr = mx_ref.quantise(v)
    rows = sure.all(1)
    assert np.array_equal(o["xc"].cpu().numpy()[rows], cr[rows])
    _check_product(o["gu"], o["xc"], o["xs"], *b.gu, 520, None, T)
    ac, as_ = awq.awq_mxfp4_quantize(o["a"])
    _check_product(o["y"], ac, as_, *b.d, 1000, None, T)
    h2, v2, sure2 = mx_ref.norm(o["y"], o["h"], b.w2, 1e-5, dtype)
    q, st = mx_ref.int8_rows(v2)
    rows = sure2.all(1)
    assert np.array_equal(o["h2"].double().cpu().numpy(), h2)
    assert np.array_equal(o["q"].cpu().numpy()[rows, :520], q[rows])
    y, _ = b.plain(x, r)
    off = float((o["y"].double() - y).norm() / y.norm())
    say(f"  off the 16-bit block by {off:.3f} of its norm")
    assert off < 0.4


@pytest.mark.parametrize("T", [1, 33, 300])
def test_block_on_a_side_stream(T):
    say(f"mxfp4 block on a side stream T={T}")
    b = Block(520, 1000, 300, torch.bfloat16, seed=1)
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for rep in range(3):
        with torch.cuda.stream(side):
            for _ in range(4):
                big = torch.mm(big, big).clamp_(-1, 1)         # keeps the stream busy
            x = torch.randn(T, 520, device="cuda").bfloat16() + big[0, 0].bfloat16() * 0
            r = torch.randn(T, 520, device="cuda").bfloat16()
        got = b.forward(x, r, stream=side)
        side.synchronize()
        want = b.forward(x, r)
        torch.cuda.synchronize()
        assert _same(got, want), rep


@pytest.mark.parametrize("T", [1, 16, 150])
def test_block_replayed(T):
    """A captured block, replayed with other inputs, beside eager calls of the same operators and a second
    graph: every replay is what plain calls give."""
    say(f"mxfp4 block captured T={T}")
    b = Block(520, 1000, 300, torch.float16, seed=2)
    xs = [torch.zeros(T, 520, device="cuda").half() for _ in range(4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.forward(xs[0], xs[1])
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(b.forward(xs[2 * k], xs[2 * k + 1]))
        graphs.append(g)
    for rep in range(4):
        for t in xs:
            t.copy_(torch.randn(T, 520, device="cuda").half())
        for k in (0, 1):
            graphs[k].replay()
        b.forward(xs[1], xs[0])                                # eager work between
        torch.cuda.synchronize()
        for k in (0, 1):
            want = b.forward(xs[2 * k], xs[2 * k + 1])
            assert _same(outs[k], want), (rep, k)
    del graphs


def test_two_calls_at_once():
    """The same operators on two streams at a time, one workspace each: neither changes the other's."""
    say("mxfp4 two streams")
    b = Block(520, 1000, 300, torch.bfloat16, seed=3)
    ins = [[torch.randn(t, 520, device="cuda").bfloat16() for _ in range(2)] for t in (40, 300)]
    want = [b.forward(*i) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(5):
        got = [None, None]
        for k in (0, 1):
            got[k] = b.forward(*ins[k], stream=streams[k])
        torch.cuda.synchronize()
        for k in (0, 1):
            assert _same(got[k], want[k]), (rep, k)
