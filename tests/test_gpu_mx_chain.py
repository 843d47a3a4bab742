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


def test_calls_from_threads():
    """Threads of one process, a stream each: the short way into the calls frees the interpreter while it
    enqueues."""
    import threading
    say("mxfp4 block from threads")
    b = Block(520, 1000, 300, torch.float16, seed=4)
    ins = [[torch.randn(t, 520, device="cuda").half() for _ in range(2)] for t in (1, 9, 64, 130)]
    want = [b.forward(*i) for i in ins]
    torch.cuda.synchronize()
    bad = []

    def run(k):
        side = torch.cuda.Stream()
        try:
            for rep in range(20):
                with torch.cuda.stream(side):
                    got = b.forward(*ins[k])
                side.synchronize()
                if not _same(got, want[k]):
                    bad.append((k, rep))
        except Exception as e:  # noqa: BLE001  (a thread's error is the test's)
            bad.append((k, repr(e)))

    threads = [threading.Thread(target=run, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_what_a_program_passes():
    """Parameters, views, tensors of another mode, whole numbers for eps: all the same as plain tensors; rows that
    overlap are refused."""
    say("mxfp4 kinds of tensors")
    x = torch.randn(7, 520, device="cuda").half()
    w = (1 + 0.1 * torch.randn(520, device="cuda")).half()
    want = awq.awq_rmsnorm(x, w, 1.0)
    assert want[1] is x
    p = torch.nn.Parameter(w)
    wide = torch.randn(9, 3 * 520, device="cuda").half()
    wide[1:8, 520:1040] = x
    view = wide[1:8, 520:1040]
    for got in (awq.awq_rmsnorm(x, p, 1.0), awq.awq_rmsnorm(x, w, 1), awq.awq_rmsnorm(view, w, 1.0),
                awq.awq_rmsnorm(view, p, 1)):
        assert torch.equal(got[0], want[0]) and not got[0].requires_grad
    with torch.inference_mode():
        got = awq.awq_rmsnorm(x + 0, w, 1.0)
    assert torch.equal(got[0], want[0])
    c, s = awq.awq_mxfp4_quantize(view)
    c1, s1 = awq.awq_mxfp4_quantize(x)
    assert torch.equal(c, c1) and torch.equal(s[:, :7], s1[:, :7])
    one = x[:1].expand(5, 520)
    for call in (lambda: awq.awq_rmsnorm(one), lambda: awq.awq_mxfp4_quantize(one),
                 lambda: awq.awq_mxfp4_linear(one, c1, s1), lambda: awq.awq_rmsnorm_int8(x, residual=one)):
        with pytest.raises(ValueError):
            call()
    # a row by itself, however far its neighbours would be
    assert torch.equal(awq.awq_rmsnorm(wide[3:4, 520:1040], w, 1.0)[0], want[0][2:3])
    # a prefix of the tokens' codes with the scales of all of them
    wc, ws = awq.awq_mxfp4_quantize(torch.randn(33, 520, device="cuda").half())
    y = awq.awq_mxfp4_matmul(c1, s1, wc, ws)
    assert torch.equal(awq.awq_mxfp4_matmul(c1[:3], s1, wc, ws), y[:3])
    assert torch.equal(awq.awq_mxfp4_matmul(c1, s1, wc[:5], ws), y[:, :5])
    # both operands the same tensors
    z = awq.awq_mxfp4_matmul(c1, s1, c1, s1)
    assert torch.equal(z, z.t().contiguous()) and bool(torch.isfinite(z).all())


def test_capture_of_calls_in_place():
    """h written over the residual in a captured graph: each replay adds once more."""
    say("norm in place, captured")
    x = torch.full((5, 264), 0.5, device="cuda", dtype=torch.bfloat16)
    r = torch.zeros(5, 264, device="cuda", dtype=torch.bfloat16)
    awq.awq_rmsnorm_mxfp4(x, residual=r, h_out=r)
    torch.cuda.synchronize()
    r.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c, s, h = awq.awq_rmsnorm_mxfp4(x, residual=r, h_out=r)
    assert h is r
    for rep in range(1, 6):
        g.replay()
        torch.cuda.synchronize()
        assert bool((r == 0.5 * rep).all())
        v = awq.awq_mxfp4_dequantize(c, s, 264)
        # v = h / sqrt(h^2 + 1e-6) = 1 - 5e-7 / h^2 for h up to 2.5: at most 1 - 8e-8, which fp32 (steps of 6e-8 there) keeps
        # below 1, so the scale is 2^(-1 - 2) and v over it lies in (6, 8): the element is 6, the value 6 / 8
        assert bool((v == 0.75).all()), rep
    del g
