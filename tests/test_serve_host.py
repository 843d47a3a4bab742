"""C ABI of the serving operators on the host: the library exports every entry point of
awq_serve.h, the binding declares the same set, and bad arguments are refused with the
documented status codes before anything touches the GPU (fake pointers, never dereferenced)."""
import ctypes
import os
import re
import subprocess

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


def _cfg(D=128, H=2, page=32, g=64, zp=1):
    return ctypes.byref(awq.awq_kv4_config(D, H, page, g, zp))


BAD_CFGS = [dict(D=96), dict(D=256), dict(H=0), dict(H=65536), dict(page=8), dict(page=48), dict(page=512),
            dict(g=16), dict(g=256), dict(D=64, g=128), dict(zp=2)]


def _append(L, k=P, kt=256, kh=128, v=P, vt=256, vh=128, T=4, dtype=0, cache=P, pages=10, tab=P, n=2, mb=4,
            lens=P, starts=P, cfg=None):
    return L.awq_kv4_append(k, kt, kh, v, vt, vh, T, dtype, cache, pages, tab, n, mb, lens, starts,
                            _cfg() if cfg is None else cfg, None)


def _read(L, cache=P, pages=10, tab=P, n=2, mb=4, lens=P, starts=P, T=4, cfg=None, dtype=0, k=P, v=P):
    return L.awq_kv4_read(cache, pages, tab, n, mb, lens, starts, T, _cfg() if cfg is None else cfg, dtype,
                          k, v, None)


def _attend(L, q=P, qt=1024, qh=128, T=4, H=8, dtype=0, cache=P, pages=10, tab=P, n=2, mb=4, lens=P,
            starts=P, cfg=None, max_q=2, max_len=100, scale=0.1, window=0, out=P, lse=P, ws=P, nb=1 << 40):
    return L.awq_kv4_attention(q, qt, qh, T, H, dtype, cache, pages, tab, n, mb, lens, starts,
                               _cfg() if cfg is None else cfg, max_q, max_len, scale, window, out, lse, ws,
                               nb, None)


def test_kv4_record_bytes(L):
    assert L.awq_kv4_record_bytes(_cfg(128, 8, 64, 64, 1)) == 64 * 128 + 8 * 64 * 2
    for bad in BAD_CFGS:
        assert L.awq_kv4_record_bytes(_cfg(**bad)) == 0, bad
    assert L.awq_kv4_record_bytes(None) == 0


def test_kv4_common_refusals(L):
    for call in (_append, _read, _attend):
        for name in ("cache", "tab", "lens", "starts"):
            assert call(L, **{name: None}) == NULL, (call, name)
            assert call(L, **{name: P_ODD}) == ALIGN, (call, name)
        for bad in BAD_CFGS:
            assert call(L, cfg=_cfg(**bad)) == CONFIG, (call, bad)
        assert call(L, dtype=2) == CONFIG
        for bad in (dict(pages=0), dict(pages=1 << 31), dict(n=-1), dict(n=65536), dict(mb=0),
                    dict(mb=(1 << 31) // 32), dict(T=-1), dict(T=1 << 31)):
            assert call(L, **bad) == SHAPE, (call, bad)
        assert call(L, T=0) == OK


def test_kv4_append_and_read_refusals(L):
    assert _append(L, k=None) == NULL and _append(L, v=None) == NULL
    assert _append(L, k=ctypes.c_void_p(0x10008)) == ALIGN
    for name in ("kt", "kh", "vt", "vh"):
        assert _append(L, **{name: 4}) == SHAPE and _append(L, **{name: -8}) == SHAPE
    assert _append(L, n=0) == OK
    assert _read(L, k=None) == NULL and _read(L, v=None) == NULL
    assert _read(L, v=ctypes.c_void_p(0x10008)) == ALIGN


def test_kv4_attention_refusals(L):
    assert _attend(L, q=None) == NULL and _attend(L, out=None) == NULL
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert _attend(L, scale=scale) == CONFIG, scale
    for bad in (dict(H=0), dict(H=7), dict(H=65536), dict(window=-1), dict(max_q=-1), dict(max_len=-1),
                dict(max_len=(1 << 30) + 1), dict(qt=12), dict(qh=-8), dict(T=1 << 30)):
        assert _attend(L, **bad) == SHAPE, bad
    assert _attend(L, q=ctypes.c_void_p(0x10008)) == ALIGN
    assert _attend(L, out=ctypes.c_void_p(0x10008)) == ALIGN and _attend(L, lse=P_ODD) == ALIGN
    need = L.awq_kv4_attention_workspace_bytes(2, 2, 8, _cfg(), 1, 100000)
    assert need > 0
    args = dict(T=2, max_q=1, max_len=100000)
    assert _attend(L, ws=None, nb=0, **args) == WORKSPACE and _attend(L, nb=need - 1, **args) == WORKSPACE
    assert _attend(L, ws=ctypes.c_void_p(0x10080), **args) == ALIGN
    assert _attend(L, n=0) == OK and _attend(L, max_q=0) == OK
    for bad in ((-1, 2, 8, 1, 10), (2, 2, 7, 1, 10), (2, 65536, 8, 1, 10), (2, 2, 8, -1, 10)):
        T, n, H, mq, ml = bad
        assert L.awq_kv4_attention_workspace_bytes(T, n, H, _cfg(), mq, ml) == 0


def test_c_symbols_are_the_library_s_own(L):
    """Every symbol of C linkage that the library exports carries its prefix (another could stand in the
    way of a program's own)."""
    out = subprocess.run(["nm", "-D", "--defined-only", awq.LIB_PATH], capture_output=True, text=True, check=True)
    names = [line.split()[-1] for line in out.stdout.splitlines() if line]
    own = [n for n in names if not n.startswith(("_Z", "__hip", "_init", "_fini", "_edata", "_end", "__bss"))]
    assert len(own) > 30 and all(n.startswith("awq_") for n in own), [n for n in own if not n.startswith("awq_")]
