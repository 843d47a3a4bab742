"""The norm with the residual's addition on the GPU against numpy in 64 bits.

Bars: h is one fp32 addition and one rounding, so it is equal bit for bit.  v is the formula's
value, formed in fp64 with an error of a few units of 2^-52, rounded to fp32: equal to numpy's wherever
the 64-bit value is further than 2^-46 of itself from the middle between two fp32 numbers (nearly
everywhere; mx_ref.norm says where), and what is made of v (the rounding to 16 bits, the codes, steps and
scales) follows from single operations: equal bit for bit on rows that hold no other value.
"""
import numpy as np
import pytest
import torch

import weight_only_quantization_act_amd as awq
from tests import mx_ref
from tests.gpu_util import requires_gpu, say

pytestmark = [pytest.mark.gpu, requires_gpu]

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def _bits(t):
    return t.contiguous().view(torch.int16).cpu().numpy()


def _check(x, w, eps, r, outs=("same", "int8", "mxfp4"), where=""):
    R, K = x.shape
    h, v, sure = mx_ref.norm(x, r, w, eps, x.dtype)
    rows = sure.all(1)
    assert rows.mean() >= 0.9 or R < 10, where
    for out in outs:
        if out == "same":
            y, hg = awq.awq_rmsnorm(x, w, eps, residual=r)
            want = torch.from_numpy(v).to(x.dtype)
            same = (_bits(y) == _bits(want)) | (np.isnan(v) & y.isnan().cpu().numpy())
            assert y.shape == x.shape and same[rows].all(), (where, np.argwhere(~same)[:4])
        elif out == "int8":
            codes, steps, hg = awq.awq_rmsnorm_int8(x, w, eps, residual=r)
            q, st = mx_ref.int8_rows(v)
            c = codes.cpu().numpy()
            assert c.shape == (R, (K + 15) // 16 * 16) and not c[:, K:].any(), where
            s = steps.cpu().numpy()
            assert np.array_equal(np.isnan(s), np.isnan(st)), where
            ok = rows & ~np.isnan(st)
            assert np.array_equal(s.view(np.uint32)[ok], st.view(np.uint32)[ok]), where
            assert np.array_equal(c[rows, :K], q[rows]), where
        else:
            codes, scales, hg = awq.awq_rmsnorm_mxfp4(x, w, eps, residual=r)
            cr, sr = mx_ref.quantise(v)
            assert codes.shape == cr.shape and scales.shape == sr.shape, where
            assert np.array_equal(scales.cpu().numpy()[:, :R][:, rows], sr[:, :R][:, rows]), where
            assert np.array_equal(codes.cpu().numpy()[rows], cr[rows]), where
        if r is None:
            assert hg is x
        else:
            got = hg.double().cpu().numpy()
            assert np.array_equal(got, h, equal_nan=True), where


SHAPES = [  # rows, columns: one value, partial blocks, each count of registers a thread and beyond
    (1, 1), (3, 7), (2, 33), (5, 127), (1, 128), (4, 1000), (1, 4096), (33, 5120), (2, 4097), (3, 8192), (2, 8200),
    (1, 16384), (2, 16391), (1, 70001), (300, 512), (1000, 64), (17, 2047), (1027, 511), (1025, 129), (1026, 1000),
    (1030, 2001), (1031, 4090), (1025, 5003), (1029, 8191), (1025, 8200),
]


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("weight", [None, "same", "fp32"])
def test_norm(dtype, residual, weight):
    for R, K in SHAPES:
        say(f"norm {R}x{K} {dtype} residual={residual} weight={weight}")
        g = torch.Generator(device="cuda").manual_seed(R * 7 + K)
        x = torch.randn(R, K, generator=g, device="cuda")
        x[:, ::9] *= 20
        x = x.to(DT[dtype])
        r = (4 * torch.randn(R, K, generator=g, device="cuda")).to(DT[dtype]) if residual else None
        w = None if weight is None else 1 + 0.3 * torch.randn(K, generator=g, device="cuda")
        if weight == "same":
            w = w.to(DT[dtype])
        _check(x, w, 1e-6, r, where=(R, K, dtype, residual, weight))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_extremes(dtype):
    """Zero rows, rows at the ends of the type's range, subnormals, sums that overflow, NaN and infinities
    in tokens and weights."""
    info = torch.finfo(DT[dtype])
    K = 300
    x = torch.randn(12, K, device="cuda").to(DT[dtype])
    r = torch.randn(12, K, device="cuda").to(DT[dtype])
    x[0] = 0.0
    r[0] = -0.0
    x[1], r[1] = r[1].clone(), -r[1]                           # the sum vanishes
    x[2] = info.max
    r[2] = 0.0
    x[3], r[3] = info.tiny / 4, 0.0                             # subnormal
    x[4, 7] = float("nan")
    x[5, 299] = float("inf")
    r[6, 0] = float("-inf")
    x[7, 3], r[7, 3] = info.max, info.max                       # overflows to infinity
    x[8, 3], r[8, 3] = float("inf"), float("-inf")
    x[9], r[9] = 0.0, 0.0
    x[9, 31] = 1.0                                              # one value in a row of zeros
    w = 1 + 0.3 * torch.randn(K, device="cuda")
    for eps in (1e-6, 1e-38, 1.0):
        say(f"norm extremes {dtype} eps={eps}")
        eps = max(eps, 2.0 ** -126)
        _check(x, w, eps, r, where=eps)
        _check(x, None, eps, None, where=eps)
    w[5] = 0.0
    w[6] = 1e38
    w[7] = 1e-38
    _check(x, w, 1e-6, r, where="weights")
    for bad in (float("nan"), float("inf")):
        w[40] = bad
        codes, steps, _ = awq.awq_rmsnorm_int8(x, w, residual=r)
        assert steps.isnan().all() and not codes.any()
        codes, scales, _ = awq.awq_rmsnorm_mxfp4(x, w, residual=r)
        nan = scales.transpose(0, 1).reshape(12, -1)[:12, :10] == 255
        assert nan[[2, 3, 10, 11]].nonzero()[:, 1].tolist() == [1] * 4 and nan[4:9].all()


def test_strides_and_places():
    """Row strides and bases that rule the 16-byte loads out; sums written over the residual, over x, into
    a view; rows behind the last stay as they were."""
    base = torch.randn(40, 3 * 301, device="cuda").half()
    w = torch.randn(700, device="cuda")
    for K, at in ((257, 0), (200, 1), (296, 8)):
        x, r = base[:, at:at + K], base[:, 301 + at:301 + at + K]
        for ww in (None, w[:K], w[1:K + 1], w.half()[3:K + 3]):
            _check(x, ww, 1e-5, r, where=(K, at))
        _check(x[::3], None, 1e-5, r[::3], where=(K, at))
    for K in (296, 257, 5000, 17000):
        say(f"norm in place K={K}")
        x = torch.randn(6, K, device="cuda").bfloat16()
        r = torch.randn(6, K, device="cuda").bfloat16()
        ww = torch.randn(K, device="cuda")
        for call in (awq.awq_rmsnorm, awq.awq_rmsnorm_int8, awq.awq_rmsnorm_mxfp4):
            want = call(x, ww, residual=r)
            for over in ("r", "x", "view"):
                x2, r2 = x.clone(), r.clone()
                wide = torch.full((8, K + 16), 3.0, dtype=torch.bfloat16, device="cuda")
                h = {"r": r2, "x": x2, "view": wide[1:7, 8:K + 8]}[over]
                got = call(x2, ww, residual=r2, h_out=h)
                assert got[-1] is h
                for a, b in zip(want, got):
                    a, b = (t[:, :6] if t.dim() == 3 else t for t in (a, b))
                    assert torch.equal(a, b), (K, over)
                if over == "view":
                    assert (wide[0] == 3).all() and (wide[7] == 3).all() and (wide[:, :8] == 3).all()
                    assert (wide[:, K + 8:] == 3).all()
    out = torch.full((8, 320), 3.0, device="cuda").half()
    x = torch.randn(6, 300, device="cuda").half()
    y, _ = awq.awq_rmsnorm(x, out=out[1:7, 9:309])
    assert torch.equal(y, awq.awq_rmsnorm(x)[0])
    assert (out[0] == 3).all() and (out[7] == 3).all() and (out[:, :9] == 3).all() and (out[:, 309:] == 3).all()


def test_no_rows():
    x = torch.zeros(0, 64, device="cuda").half()
    assert awq.awq_rmsnorm(x)[0].shape == (0, 64)
    assert awq.awq_rmsnorm_int8(x, residual=x)[0].shape == (0, 64)
    assert awq.awq_rmsnorm_mxfp4(x)[0].shape == (0, 32)


def test_many_rows_repeat():
    """Enough rows for every compute unit, several times over: each as it is alone, and again."""
    say("norm many rows")
    x = torch.randn(9000, 700, device="cuda").half()
    r = torch.randn(9000, 700, device="cuda").half()
    w = torch.randn(700, device="cuda")
    c, s, h = awq.awq_rmsnorm_mxfp4(x, w, residual=r)
    c2, s2, _ = awq.awq_rmsnorm_mxfp4(x, w, residual=r)
    assert torch.equal(c, c2) and torch.equal(s, s2)
    q, st, _ = awq.awq_rmsnorm_int8(x, w, residual=r)
    y, _ = awq.awq_rmsnorm(x, w, residual=r)
    for at in (0, 1, 4444, 8999):
        one = slice(at, at + 1)
        c1, s1, h1 = awq.awq_rmsnorm_mxfp4(x[one], w, residual=r[one])
        assert torch.equal(c1, c[one]) and torch.equal(s1[:, 0], s[:, at]) and torch.equal(h1, h[one])
        q1, st1, _ = awq.awq_rmsnorm_int8(x[one], w, residual=r[one])
        assert torch.equal(q1, q[one]) and torch.equal(st1, st[one])
        assert torch.equal(awq.awq_rmsnorm(x[one], w, residual=r[one])[0], y[one])


def test_refusals_of_the_binding():
    x = torch.zeros(4, 64, device="cuda").half()
    w = torch.ones(64, device="cuda")
    for call in (awq.awq_rmsnorm, awq.awq_rmsnorm_int8, awq.awq_rmsnorm_mxfp4):
        for bad, err in ((dict(weight=w[:63]), ValueError), (dict(weight=w.bfloat16()), TypeError),
                         (dict(residual=x[:3]), ValueError), (dict(residual=x.bfloat16()), TypeError),
                         (dict(h_out=x), ValueError), (dict(residual=x, h_out=x[:, :32]), ValueError),
                         (dict(eps=0.0), awq.AwqError), (dict(eps=float("nan")), awq.AwqError)):
            with pytest.raises(err):
                call(x, **bad)
        with pytest.raises(ValueError):
            call(x[:, :0])
        with pytest.raises(TypeError):
            call(x.float())
