"""How the serving operators lay a call out, on the host: the workspace that a query names covers
what the call it is made for uses.  Nothing is launched (fake pointers, never dereferenced)."""
import random

import pytest

import weight_only_quantization_act_amd as awq
from weight_only_quantization_act_amd import _serve


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
