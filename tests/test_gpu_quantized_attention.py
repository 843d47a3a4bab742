"""The attention block of examples/quantized_attention.py: int8 projection, 4-bit cache, attention
and 4-bit output projection in one program.

Bar of the comparison with the same block on 16-bit weights and keys, derived from the steps for
unit normal data: a group of 64 keys or values spans about 4.7 sigma, so its step is 0.31 and its
rounding error 0.31 / sqrt(12) = 0.09 of a value; a sum of values with random errors keeps that
ratio (0.09); errors of the keys move a score by 0.09 and so each weight by 9% (0.09); groups of
128 weights span 5.2 sigma (0.10); the int8 projection adds about 0.01.  Together 0.16 of the
output's norm; the bar is twice that.  The replayed graph runs the same kernels with the same
bounds as the plain calls: equal bit for bit.
"""
import importlib.util
import os

import pytest
import torch

import weight_only_quantization_act_amd as awq
from tests.gpu_util import requires_gpu, say

pytestmark = [pytest.mark.gpu, requires_gpu]

PATH = os.path.join(os.path.dirname(__file__), "..", "examples", "quantized_attention.py")


def _example():
    spec = importlib.util.spec_from_file_location("quantized_attention", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_block_decodes_and_replays():
    say("attention block")
    prompts, tokens = (70, 1, 33), 6
    got, want, replayed, last = _example().run(tokens, hidden=512, heads=8, kv_heads=2, prompts=prompts,
                                               max_len=256)
    for p, o, w in zip(prompts, got, want):
        assert o.shape == w.shape == (p + tokens, 512)
        assert float((o.float() - w).norm() / w.norm()) < 0.32
    assert torch.equal(replayed, last)


def test_layers_carry_the_scales_of_the_search():
    """What the example says of its two layers: the projection's codes stand for its weights times the
    scales that the search found on the calibration tokens, the output layer is packed with its own."""
    say("attention block: scales")
    b = _example().Block(hidden=512, heads=8, kv_heads=2, max_seqs=1, max_len=64)
    found = awq.awq_search_scales(b.w_qkv, b.calib, awq.awq_act_stats(b.calib), b.alphas, b.cfg4)
    assert torch.equal(b.s, found["s"]) and int(found["best"]) > 0
    wq, wstep = awq.awq_int8_quantize(b.w_qkv, found["s"], fold="multiply")
    assert torch.equal(b.wq, wq) and torch.equal(b.wstep, wstep)
    o = b.attend_plain(b.calib).half()
    found = awq.awq_search_scales(b.w_out, o, awq.awq_act_stats(o), b.alphas, b.cfg4)
    assert torch.equal(b.s_out, found["s"])
    codes, scales, zeros = awq.awq_quantize_pack(b.w_out, found["s"], b.cfg4)
    assert torch.equal(b.codes, codes) and torch.equal(b.scales, scales) and torch.equal(b.zeros, zeros)
