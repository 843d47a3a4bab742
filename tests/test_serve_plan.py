"""How the serving operators lay a call out, on the host: the workspace that a query names covers
what the call it is made for uses.  Nothing is launched (fake pointers, never dereferenced)."""
import ctypes
import os
import random
import subprocess

import pytest

import weight_only_quantization_act_amd as awq
from tests.int8_forms import SHAPES
from weight_only_quantization_act_amd import _serve


# a workspace smaller than required, a pointer that must be device memory and is not
WORKSPACE, DEVICE = 5, 6


@pytest.fixture(scope="module")
def L():
    return _serve.lib()


def test_int8_workspace_counts_whole_chunks(L):
    """A product reads rows of whole 16-byte chunks and is laid out by them, so its workspace is that
    of the rounded-up columns: with fewer the sums of a divided K would be written past its end."""
    rng = random.Random(1)
    sizes = [(32, 128, 2040), (16, 16384, 4095), (64, 512, 1023), (333, 5120, 13823), (5, 16385, 4081)]
    sizes += [(round(2 ** rng.uniform(0, 13)), round(2 ** rng.uniform(0, 15)),
               max(1, 1024 * rng.randint(1, 16) - rng.randint(-20, 20))) for _ in range(3000)]
    divided = 0
    for T, M, K in sizes:
        whole = (K + 15) // 16 * 16
        need = L.awq_int8_matmul_workspace_bytes(T, M, whole)
        divided += need > 0
        assert L.awq_int8_matmul_workspace_bytes(T, M, K) == need, (T, M, K)
        assert L.awq_int8_linear_workspace_bytes(T, M, K) == L.awq_int8_linear_workspace_bytes(T, M, whole), \
            (T, M, K)
    assert divided > 500


def _attend(L, cfg, n, heads, max_q, max_len, window, ws, nbytes):
    P = ctypes.c_void_p(0x10000)
    return L.awq_kv4_attention(P, cfg.head_dim * heads, cfg.head_dim, n * max_q, heads, 0, P, 10, P, n, 4, P,
                               P, ctypes.byref(cfg), max_q, max_len, 0.1, window, P, P, ws, nbytes, None)


def test_attention_workspace_covers_every_window(L):
    """A call is given what the query names, which does not know the window.  A window is a smaller
    bound on the keys, so a larger bound may never need less; and no window makes the call ask for
    more than it was given: with these pointers it gets as far as finding that they are no device
    memory."""
    rng = random.Random(2)
    P = ctypes.c_void_p(0x10000)
    sizes = [(64, 8, 8, 1, 1 << 30, 8192), (32, 8, 4, 1, 1 << 30, 8192), (64, 8, 8, 1, 1 << 29, 8192),
             (2048, 1, 4, 1, 1 << 24, 8192), (1, 8, 4, 1, 1 << 30, (1 << 63) - 1),
             (3, 8, 4, 500, 1 << 30, (1 << 63) - 1), (40, 8, 4, 1, 1 << 30, 6000), (4, 2, 1, 40, 1 << 30, 3)]
    for _ in range(3000):
        hk = rng.choice([1, 2, 8, 40])
        sizes.append((round(2 ** rng.uniform(0, 12)), hk, rng.choice([1, 3, 8]),
                      rng.choice([1, 1, 2, 5, round(2 ** rng.uniform(0, 10))]),
                      round(2 ** rng.uniform(0, 30)), round(2 ** rng.uniform(0, 31))))
    needed = 0
    for n, hk, grp, max_q, max_len, window in sizes:
        cfg = awq.awq_kv4_config(128, hk, 64, 128, 1)
        H = hk * grp

        def query(length):
            return L.awq_kv4_attention_workspace_bytes(n * max_q, n, H, ctypes.byref(cfg), max_q, length)
        need = query(max_len)
        needed += need > 0
        where = (n, hk, grp, max_q, max_len, window)
        for smaller in (window + max_q, window, max_len // 2, 5000, 6000, 100000):
            assert query(min(smaller, max_len)) <= need, (where, smaller)
        for w in (0, window, 1, 8192):
            got = _attend(L, cfg, n, H, max_q, max_len, w, P if need else None, need)
            assert got == DEVICE, (where, w, need, got)
    assert needed > 500


def test_window_beyond_every_key_is_none(L):
    """Windows up to the type's largest are laid out as no window is (window + max_q stays in 64
    bits): such a call asks for the same workspace."""
    cfg = awq.awq_kv4_config(128, 8, 64, 128, 1)
    for n, max_q, max_len in ((1, 1, 1 << 30), (3, 500, 1 << 20), (8, 1, 8192)):
        need = L.awq_kv4_attention_workspace_bytes(n * max_q, n, 32, ctypes.byref(cfg), max_q, max_len)
        assert need > 0
        P = ctypes.c_void_p(0x10000)
        for window in (0, max_len, 1 << 31, (1 << 63) - max_q, (1 << 63) - 1):
            assert _attend(L, cfg, n, 32, max_q, max_len, window, P, need) == DEVICE, window
            assert _attend(L, cfg, n, 32, max_q, max_len, window, P, need - 256) == WORKSPACE, window


def test_int8_forms_are_covered(tmp_path):
    """The sizes that the GPU tests run land on the forms that they are meant for, so that a changed rule
    cannot leave a form untested."""
    src = tmp_path / "plan.cpp"
    src.write_text("""#include <stdio.h>
#include "int8_plan.h"
int main() {
  long long T, M, K;
  const char* name[] = {"few", "32", "64", "128", "256"};
  while (scanf("%lld %lld %lld", &T, &M, &K) == 3) {
    const awq::Int8Plan p = awq::int8_plan(T, M, K);
    printf("%s %d %d\\n", name[p.form], p.splits, awq::few_rows(M));
  }
}
""")
    exe = tmp_path / "plan"
    csrc = os.path.join(os.path.dirname(awq.LIB_PATH), "csrc")
    subprocess.run(["g++", "-std=c++17", "-I", csrc, str(src), "-o", str(exe)], check=True)
    sizes = "\n".join("%d %d %d" % s[2:] for s in SHAPES)
    out = subprocess.run([str(exe)], input=sizes, capture_output=True, text=True, check=True).stdout.split("\n")
    got = [line.split() for line in out if line]
    for shape, (form, splits, rows) in zip(SHAPES, got):
        assert (form, int(splits)) == shape[:2], (shape, form, splits)
    assert len(got) == len(SHAPES)
    assert {s[0] for s in SHAPES} == {"few", "32", "64", "128", "256"}
    assert {int(rows) for (form, _, rows) in got if form == "few"} == {1, 2}
    for form in ("32", "64", "128"):
        assert {s[1] > 1 for s in SHAPES if s[0] == form} == {True, False}, form


def test_calls_of_too_many_blocks_are_refused_for_their_size(L):
    """Sizes within their own bounds that together make more blocks than a launch numbers: a status that
    says so, before anything is launched."""
    P = ctypes.c_void_p(0x10000)
    SHAPE = 2

    def append(hk, n, T):
        cfg = awq.awq_kv4_config(128, hk, 64, 128, 1)
        return L.awq_kv4_append(P, 128 * hk, 128, P, 128 * hk, 128, T, 0, P, 10, P, n, 4, P, P, ctypes.byref(cfg), None)

    def read(hk, n, T):
        cfg = awq.awq_kv4_config(128, hk, 64, 128, 1)
        return L.awq_kv4_read(P, 10, P, n, 4, P, P, T, ctypes.byref(cfg), 0, P, P, None)
    for call in (append, read):
        assert call(65535, 65535, 1) == SHAPE and call(65535, 1, 1 << 20) == SHAPE
        assert call(8000, 65535, 1) == DEVICE and call(8, 65535, 1 << 30) == DEVICE
    cfg = awq.awq_kv4_config(128, 65535, 64, 128, 1)
    assert _attend(L, cfg, 65535, 65535, 1, 8, 0, P, 1 << 60) == SHAPE
    cfg = awq.awq_kv4_config(128, 8000, 64, 128, 1)
    assert _attend(L, cfg, 30000, 8000, 1, 8, 0, P, 1 << 60) == DEVICE
