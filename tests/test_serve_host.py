"""C ABI of the serving operators on the host: the library exports every entry point of
awq_serve.h, the binding declares the same set, and bad arguments are refused with the
documented status codes before anything touches the GPU (fake pointers, never dereferenced)."""
import ctypes
import os
import re

import pytest

import weight_only_quantization_act_amd as awq
from weight_only_quantization_act_amd import _serve

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "awq_serve.h")
OK, NULL, SHAPE, CONFIG, WORKSPACE, ALIGN = 0, 1, 2, 3, 5, 9
P, P_ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10001)


@pytest.fixture(scope="module")
def L():
    return _serve.lib()


def test_exports_every_declared_symbol(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|size_t)\s+(awq_\w+)\s*\(", text, flags=re.M))
    assert names == set(_serve._SIGNATURES)
    for n in names:
        assert hasattr(L, n) and hasattr(awq, n)


def _quant(L, A=P, rows=4, cols=100, lda=100, dtype=0, s=None, fold=0, codes=P, ldc=112, steps=P):
    return L.awq_int8_quantize(A, rows, cols, lda, dtype, s, fold, codes, ldc, steps, None)


def test_int8_quantize_refusals(L):
    assert _quant(L, A=None) == NULL and _quant(L, codes=None) == NULL
    assert _quant(L, steps=None) == NULL
    assert _quant(L, dtype=2) == CONFIG and _quant(L, fold=2) == CONFIG
    assert _quant(L, rows=-1) == SHAPE and _quant(L, cols=-1) == SHAPE
    assert _quant(L, lda=99) == SHAPE
    assert _quant(L, ldc=104) == SHAPE and _quant(L, ldc=96) == SHAPE
    assert _quant(L, rows=1 << 31) == SHAPE and _quant(L, rows=1 << 30, lda=1 << 20) == SHAPE
    assert _quant(L, A=P_ODD) == ALIGN and _quant(L, codes=ctypes.c_void_p(0x10008)) == ALIGN
    assert _quant(L, steps=ctypes.c_void_p(0x10002)) == ALIGN
    assert _quant(L, s=ctypes.c_void_p(0x10002)) == ALIGN
    assert _quant(L, rows=0) == OK


def _mm(L, fn="awq_int8_matmul", x=P, ldx=128, xs=P, T=4, w=P, ldw=128, ws=P, M=8, K=128, bias=None,
        dtype=0, y=P, ldy=8, wsp=P, n=1 << 40):
    f = getattr(L, fn)
    return f(x, ldx, xs, T, w, ldw, ws, M, K, bias, dtype, y, ldy, wsp, n, None)


def test_int8_matmul_refusals(L):
    for name in ("x", "xs", "w", "ws", "y"):
        assert _mm(L, **{name: None}) == NULL, name
    assert _mm(L, dtype=-1) == CONFIG
    assert _mm(L, T=-1) == SHAPE and _mm(L, M=-1) == SHAPE and _mm(L, K=-1) == SHAPE
    assert _mm(L, K=131057, ldx=1 << 18, ldw=1 << 18) == SHAPE
    assert _mm(L, ldx=112) == SHAPE and _mm(L, ldw=112) == SHAPE
    assert _mm(L, ldx=136) == SHAPE and _mm(L, ldw=136) == SHAPE
    assert _mm(L, K=120, ldx=120) == SHAPE
    assert _mm(L, ldy=7) == SHAPE
    assert _mm(L, ldw=1 << 22) == SHAPE and _mm(L, ldx=1 << 22) == SHAPE
    assert _mm(L, x=ctypes.c_void_p(0x10008)) == ALIGN and _mm(L, w=ctypes.c_void_p(0x10008)) == ALIGN
    assert _mm(L, xs=P_ODD) == ALIGN and _mm(L, ws=P_ODD) == ALIGN
    assert _mm(L, bias=P_ODD) == ALIGN and _mm(L, y=P_ODD) == ALIGN
    assert _mm(L, T=0) == OK and _mm(L, M=0) == OK


def test_int8_linear_refusals(L):
    def lin(**k):
        return _mm(L, fn="awq_int8_linear", **k)
    for name in ("x", "w", "ws", "y"):
        assert lin(**{name: None}) == NULL, name
    assert lin(dtype=2) == CONFIG
    assert lin(ldx=127) == SHAPE and lin(K=131057, ldx=1 << 18, ldw=1 << 18) == SHAPE
    assert lin(x=P_ODD) == ALIGN
    need = L.awq_int8_linear_workspace_bytes(64, 8, 128)
    assert need >= 64 * 128 + 64 * 4
    assert lin(T=64, wsp=None, n=0) == WORKSPACE and lin(T=64, n=need - 1) == WORKSPACE
    assert lin(T=64, wsp=ctypes.c_void_p(0x10080), n=need) == ALIGN
    assert lin(T=0, wsp=None, n=0) == OK
    for bad in ((-1, 8, 128), (0, 8, 128), (4, 0, 128), (4, 8, 131057)):
        assert L.awq_int8_linear_workspace_bytes(*bad) == 0
        assert L.awq_int8_matmul_workspace_bytes(*bad) == 0
