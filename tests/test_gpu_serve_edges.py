"""Edges of the serving operators on the GPU: sizes at which a call is laid out in another way than
its neighbours, values at the ends of their types, work on other streams."""
import numpy as np
import pytest
import torch

import weight_only_quantization_act_amd as awq
from tests.gpu_util import requires_gpu, say
from tests.test_gpu_kv4 import Case, _check, _compare

pytestmark = [pytest.mark.gpu, requires_gpu]

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.mark.parametrize("T,M,K", [(32, 128, 2040), (16, 16384, 4095), (333, 640, 3063), (2, 16500, 4085),
                                   (40, 300, 1023), (100, 1000, 5 * 1024 - 1)])
def test_linear_stays_in_its_workspace(T, M, K):
    """Columns that are no multiple of 16 and end just below another division of K: the result is the
    two calls' and the bytes behind the workspace stay as they were."""
    say(f"int8 linear workspace T={T} M={M} K={K}")
    g = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(T, K, generator=g, device="cuda").half()
    W = (torch.randn(M, K, generator=g, device="cuda") * 0.02).half()
    wq, ws = awq.awq_int8_quantize(W)
    need = awq.awq_int8_linear_workspace_bytes(T, M, K)
    guard = 2 * T * M * 4 * 8 + 4096               # more than any division's sums
    buf = torch.full((need + guard,), 0x5A, dtype=torch.uint8, device="cuda")
    y = awq.awq_int8_linear(x, wq, ws, workspace=buf[:need])
    assert (buf[need:] == 0x5A).all()
    xq, xs = awq.awq_int8_quantize(x)
    assert torch.equal(y, awq.awq_int8_matmul(xq, xs, wq, ws))
    acc = xq.cpu().numpy().astype(np.float64) @ wq.cpu().numpy().astype(np.float64).T  # exact
    want = (acc.astype(np.float32) * xs.cpu().numpy()[:, None] * ws.cpu().numpy()).astype(np.float16)
    assert np.array_equal(y.cpu().numpy(), want)


@pytest.mark.parametrize("n,Hk,grp", [(64, 8, 8), (2048, 1, 4), (40, 2, 1)])
def test_window_with_a_loose_bound(n, Hk, grp):
    """A bound on the lengths so loose that only the window lets the tiles be counted: the keys are
    divided, into the workspace that the query named, and the result is that of a tight bound."""
    lens = [int(x) for x in np.random.default_rng(n).integers(0, 300 if n > 100 else 2000, n)]
    c = Case(64, Hk, 16, 64, 1, lens, [1] * n, seed=n)
    c.fill()
    q = torch.randn(n, Hk * grp, 64, device="cuda").half()
    for window, max_len in ((8192, 1 << 30), (1 << 20, 1 << 30), ((1 << 63) - 1, 1 << 30), (8192, 1 << 24),
                            (50, 1 << 30)):
        say(f"kv4 window={window} max_len={max_len} n={n}")
        need = awq.awq_kv4_attention_workspace_bytes(n, n, Hk * grp, c.cfg, 1, max_len)
        buf = torch.full((need + (1 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
        out, lse = awq.awq_kv4_attention(q, c.cache, c.dtable, c.dlens, c.dstarts, c.cfg, max_q=1,
                                         max_len=max_len, window=window, workspace=buf[:need])
        assert (buf[need:] == 0x5A).all()
        _compare(c, q, out, lse, None, min(window, 1 << 20), where=(n, window, max_len))
