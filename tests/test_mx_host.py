"""Refusals of the MXFP4 operators, the norm and the read-back of 8-bit rows on the host: bad arguments
get the documented status codes before anything touches the GPU (fake pointers, never dereferenced), and the plain
forms of the tests agree with the format's definition."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import weight_only_quantization_act_amd as awq
from tests import mx_ref
from tests.mx_forms import SHAPES
from weight_only_quantization_act_amd import _serve

OK, NULL, SHAPE, CONFIG, WORKSPACE, DEVICE, ALIGN = 0, 1, 2, 3, 5, 6, 9
P = ctypes.c_void_p(0x10000)
P1, P2, P8 = (ctypes.c_void_p(0x10000 + k) for k in (1, 2, 8))
ROWS = (1 << 29) - 512


@pytest.fixture(scope="module")
def L():
    return _serve.lib()


def _quant(L, A=P, rows=4, cols=100, lda=100, dtype=0, s=None, fold=0, codes=P, ldc=64, scales=P, lds=4):
    return L.awq_mxfp4_quantize(A, rows, cols, lda, dtype, s, fold, codes, ldc, scales, lds, None)


def test_quantize_refusals(L):
    for name in ("A", "codes", "scales"):
        assert _quant(L, **{name: None}) == NULL, name
    assert _quant(L, dtype=2) == CONFIG and _quant(L, dtype=-1) == CONFIG and _quant(L, fold=2) == CONFIG
    for bad in (dict(rows=-1), dict(cols=-1), dict(lda=99), dict(ldc=48), dict(ldc=72), dict(ldc=1 << 22),
                dict(lds=0), dict(lds=6), dict(rows=5, lds=4), dict(rows=ROWS + 1, lds=1 << 29),
                dict(lds=1 << 29), dict(cols=(1 << 22) + 1, lda=1 << 23, ldc=(1 << 22) - 16),
                dict(rows=1 << 28, lds=1 << 28, lda=1 << 20)):
        assert _quant(L, **bad) == SHAPE, bad
    assert _quant(L, A=P1) == ALIGN and _quant(L, s=P2) == ALIGN
    assert _quant(L, codes=P8) == ALIGN and _quant(L, scales=P8) == ALIGN
    assert _quant(L, rows=0) == OK and _quant(L, cols=0) == OK
    assert _quant(L) == DEVICE


def _values(L, codes=P, ldc=64, scales=P, lds=4, rows=4, cols=100, dtype=0, out=P, ldo=100):
    return L.awq_mxfp4_dequantize(codes, ldc, scales, lds, rows, cols, dtype, out, ldo, None)


def test_dequantize_refusals(L):
    for name in ("codes", "scales", "out"):
        assert _values(L, **{name: None}) == NULL, name
    assert _values(L, dtype=2) == CONFIG
    for bad in (dict(rows=-1), dict(cols=-1), dict(ldo=99), dict(ldc=48), dict(ldc=72), dict(lds=6),
                dict(rows=5), dict(rows=ROWS + 1, lds=1 << 29)):
        assert _values(L, **bad) == SHAPE, bad
    assert _values(L, codes=P8) == ALIGN and _values(L, scales=P8) == ALIGN and _values(L, out=P1) == ALIGN
    assert _values(L, rows=0) == OK and _values(L, cols=0) == OK and _values(L) == DEVICE


def _int8(L, codes=P, ldc=112, steps=P, rows=4, cols=100, dtype=0, out=P, ldo=100):
    return L.awq_int8_dequantize(codes, ldc, steps, rows, cols, dtype, out, ldo, None)


def test_int8_dequantize_refusals(L):
    for name in ("codes", "steps", "out"):
        assert _int8(L, **{name: None}) == NULL, name
    assert _int8(L, dtype=2) == CONFIG
    for bad in (dict(rows=-1), dict(cols=-1), dict(ldo=99), dict(ldc=96), dict(ldc=120), dict(rows=1 << 31),
                dict(rows=1 << 30, ldo=1 << 20), dict(rows=(1 << 31) - 512, cols=1 << 16, ldo=1 << 16, ldc=1 << 16)):
        assert _int8(L, **bad) == SHAPE, bad
    assert _int8(L, codes=P8) == ALIGN and _int8(L, steps=P2) == ALIGN and _int8(L, out=P1) == ALIGN
    assert _int8(L, rows=0) == OK and _int8(L, cols=0) == OK and _int8(L) == DEVICE


def _mm(L, xc=P, ldx=64, xs=P, ldxs=4, T=4, wc=P, ldw=64, ws=P, ldws=8, M=8, K=128, bias=None, dtype=0, y=P,
        ldy=8):
    return L.awq_mxfp4_matmul(xc, ldx, xs, ldxs, T, wc, ldw, ws, ldws, M, K, bias, dtype, y, ldy, None)


def _lin(L, x=P, ldx=128, s=None, T=4, wc=P, ldw=64, ws=P, ldws=8, M=8, K=128, bias=None, dtype=0, y=P, ldy=8,
         wsp=P, n=1 << 40):
    return L.awq_mxfp4_linear(x, ldx, s, T, wc, ldw, ws, ldws, M, K, bias, dtype, y, ldy, wsp, n, None)


def test_product_refusals(L):
    for name in ("xc", "xs", "wc", "ws", "y"):
        assert _mm(L, **{name: None}) == NULL, name
    for name in ("x", "wc", "ws", "y"):
        assert _lin(L, **{name: None}) == NULL, name
    for call in (_mm, _lin):
        assert call(L, dtype=2) == CONFIG
        for bad in (dict(T=-1), dict(M=-1), dict(K=-1), dict(ldw=48), dict(ldw=72), dict(ldw=1 << 22),
                    dict(ldws=4), dict(ldws=10), dict(ldy=7), dict(M=ROWS + 1, ldws=1 << 29, ldy=1 << 30),
                    dict(K=(1 << 22) + 1, ldw=(1 << 22) - 16, ldx=1 << 23), dict(T=ROWS + 1, ldxs=1 << 29)
                    if call is _mm else dict(T=ROWS + 1)):
            assert call(L, **bad) == SHAPE, (call, bad)
        for bad in (dict(wc=P8), dict(ws=P8), dict(bias=P1), dict(y=P1)):
            assert call(L, **bad) == ALIGN, (call, bad)
        assert call(L, T=0) == OK and call(L, M=0) == OK and call(L) == DEVICE
    for bad in (dict(ldx=48), dict(ldx=72), dict(ldx=1 << 22), dict(ldxs=0), dict(ldxs=6)):
        assert _mm(L, **bad) == SHAPE, bad
    assert _mm(L, xc=P8) == ALIGN and _mm(L, xs=P8) == ALIGN
    assert _lin(L, ldx=127) == SHAPE and _lin(L, x=P1) == ALIGN and _lin(L, s=P2) == ALIGN


def test_linear_workspaces(L):
    lin = dict(T=64, M=512, K=16384, ldw=8192, ldws=512, ldy=512, ldx=16384)
    need = L.awq_mxfp4_linear_workspace_bytes(64, 512, 16384)
    assert need >= 64 * 8192 + 64 * 512
    assert _lin(L, **lin, wsp=None, n=0) == WORKSPACE and _lin(L, **lin, n=need - 1) == WORKSPACE
    assert _lin(L, **lin, wsp=ctypes.c_void_p(0x10080), n=need) == ALIGN and _lin(L, **lin, n=need) == DEVICE
    for bad in ((-1, 8, 128), (0, 8, 128), (4, 0, 128), (4, 8, 0), (4, 8, (1 << 22) + 1), (ROWS + 1, 8, 128)):
        assert L.awq_mxfp4_linear_workspace_bytes(*bad) == 0


def _norm(L, out="", x=P, ldx=100, r=P, ldr=100, rows=4, cols=100, dtype=0, w=P, wt=0, eps=1e-6, h=P, ldh=100,
          y=P, ldy=112, sc=P, lds=4):
    head = (x, ldx, r, ldr, rows, cols, dtype, w, wt, ctypes.c_double(eps), h, ldh, y, ldy)
    if out == "":
        return L.awq_rmsnorm(*head, None)
    if out == "int8":
        return L.awq_rmsnorm_int8(*head, sc, None)
    return L.awq_rmsnorm_mxfp4(*head, sc, lds, None)


@pytest.mark.parametrize("out", ["", "int8", "mxfp4"])
def test_norm_refusals(L, out):
    def call(**k):
        return _norm(L, out, **k)
    for name in ("x", "h", "y") + (() if out == "" else ("sc",)):
        assert call(**{name: None}) == NULL, name
    assert call(r=None, h=None) == DEVICE and call(w=None) == DEVICE     # both may be absent
    assert call(dtype=2) == CONFIG and call(wt=1) == CONFIG and call(dtype=1) == CONFIG
    assert call(dtype=1, wt=1) == DEVICE and call(wt=2) == DEVICE
    for eps in (0.0, -1e-6, float("nan"), float("inf"), 1e-39):
        assert call(eps=eps) == CONFIG, eps
    for bad in (dict(rows=-1), dict(cols=0), dict(cols=-1), dict(ldx=99), dict(ldr=99), dict(ldh=99),
                dict(rows=1 << 31), dict(rows=1 << 28, ldx=1 << 20), dict(rows=1 << 28, ldh=1 << 20)):
        assert call(**bad) == SHAPE, bad
    for bad in (dict(x=P1), dict(r=P1), dict(h=P1), dict(w=P1), dict(wt=2, w=P2), dict(y=P1)):
        assert call(**bad) == ALIGN, bad
    assert call(rows=0) == OK
    if out == "":
        assert call(ldy=99) == SHAPE
    if out == "int8":
        assert call(ldy=96) == SHAPE and call(ldy=120) == SHAPE and call(y=P8) == ALIGN and call(sc=P2) == ALIGN
    if out == "mxfp4":
        assert call(ldy=48) == SHAPE and call(ldy=72) == SHAPE and call(lds=6) == SHAPE and call(rows=5) == SHAPE
        assert call(y=P8) == ALIGN and call(sc=P8) == ALIGN


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x, w = torch.zeros(3, 64), torch.ones(64)
    c, s = torch.zeros(3, 32, dtype=torch.uint8), torch.zeros(1, 4, 4, dtype=torch.uint8)
    for f, args in ((awq.awq_rmsnorm, (x, w)), (awq.awq_rmsnorm_int8, (x, w)), (awq.awq_rmsnorm_mxfp4, (x, w)),
                    (awq.awq_mxfp4_quantize, (x,)), (awq.awq_mxfp4_dequantize, (c, s, 64)),
                    (awq.awq_mxfp4_matmul, (c, s, c, s)), (awq.awq_mxfp4_linear, (x, c, s)),
                    (awq.awq_int8_dequantize, (c.view(torch.int8), w, 32))):
        with pytest.raises((ValueError, RuntimeError)):
            f(*args)
        with pytest.raises((TypeError, RuntimeError)):
            f(3.0, *args[1:])


def test_plain_rows_are_the_format():
    """The reference's rows against the definition by hand: ties to the even code, saturation, subnormal
    scales, NaN."""
    v = np.zeros((1, 96), np.float32)
    v[0, :16] = [7.9, 6.0, 5.0, 4.999, 5.001, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, 0.2501, -0.25, -5.0, -0.0, 4]
    v[0, 32:34] = [2.0 ** -126, 2.0 ** -128]
    v[0, 64:66] = [1.0, np.inf]
    codes, scales = mx_ref.quantise(v)
    got = mx_ref.values(codes, scales, 96)[0]
    assert list(got[:16]) == [6, 6, 4, 4, 6, 4, 2, 2, 1, 1, 0, 0.5, 0, -4, 0, 4]
    assert np.signbit(got[14]) and np.signbit(got[12])
    assert list(scales[0, 0]) == [127, 0, 255, 0]
    assert list(got[32:34]) == [2.0 ** -126, 2.0 ** -128] and np.isnan(got[64:]).all()
    assert codes.shape == (1, 48) and scales.shape == (1, 4, 4) and not codes[0, 32:].any()


def test_forms_are_covered(tmp_path):
    """The sizes that the GPU tests run land on the forms that they are meant for, so that a changed rule
    cannot leave a form untested."""
    src = tmp_path / "plan.cpp"
    src.write_text("""#include <stdio.h>
#include "mxfp4_plan.h"
int main() {
  long long T, M, K;
  const char* name[] = {"few", "32k", "32x64k", "64k", "64", "64x128", "128w", "128", "256"};
  while (scanf("%lld %lld %lld", &T, &M, &K) == 3)
    printf("%s\\n", name[awq::mxfp4_form(T, M, (K + 31) / 32 * 16)]);
}
""")
    exe = tmp_path / "plan"
    csrc = os.path.join(os.path.dirname(awq.LIB_PATH), "csrc")
    subprocess.run(["g++", "-std=c++17", "-I", csrc, str(src), "-o", str(exe)], check=True)
    sizes = "\n".join("%d %d %d" % s[1:] for s in SHAPES)
    out = subprocess.run([str(exe)], input=sizes, capture_output=True, text=True, check=True).stdout.split()
    assert out == [s[0] for s in SHAPES], [(s, f) for s, f in zip(SHAPES, out) if s[0] != f]
    assert set(out) == {"few", "32k", "32x64k", "64k", "64", "64x128", "128w", "128", "256"}
