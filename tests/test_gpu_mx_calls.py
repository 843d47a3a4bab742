"""The short way into the calls of the norm and of MXFP4 on the GPU: what it does with the C ABI's answers.

A child process puts functions of the C ABI's names, which count their calls and return a chosen status, before the
library's for the extension module alone; the binding's longer way calls the library itself.
"""
import os
import subprocess
import sys
import types

import pytest
import torch

import weight_only_quantization_act_amd as awq
from tests.conftest import ROOT
from tests.gpu_util import requires_gpu, say
from tests.test_mx_calls_host import CALLS

pytestmark = [pytest.mark.gpu, requires_gpu]

ENTRIES = ("rmsnorm", "rmsnorm_int8", "rmsnorm_mxfp4", "int8_dequantize", "mxfp4_quantize", "mxfp4_dequantize",
           "mxfp4_matmul", "mxfp4_linear")
FAKE = "int awq_fake_status = 0, awq_fake_calls = 0;\n" + "".join(
    f"int awq_{e}(void) {{ ++awq_fake_calls; return awq_fake_status; }}\n" for e in ENTRIES)

CHILD = """
import ctypes, sys
import torch
fake = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)     # before the extension module is loaded
status, calls = (ctypes.c_int.in_dll(fake, "awq_fake_" + n) for n in ("status", "calls"))
import weight_only_quantization_act_amd as awq
from weight_only_quantization_act_amd import _mx

x = torch.randn(5, 128, device="cuda").half()
status.value = 2
c, s = awq.awq_mxfp4_quantize(x)
q, st = awq.awq_int8_quantize(x)
run = {"rmsnorm": lambda: awq.awq_rmsnorm(x), "rmsnorm_int8": lambda: awq.awq_rmsnorm_int8(x),
       "rmsnorm_mxfp4": lambda: awq.awq_rmsnorm_mxfp4(x), "int8_dequantize": lambda: awq.awq_int8_dequantize(q, st, 128),
       "mxfp4_quantize": lambda: awq.awq_mxfp4_quantize(x), "mxfp4_dequantize": lambda: awq.awq_mxfp4_dequantize(c, s, 128),
       "mxfp4_matmul": lambda: awq.awq_mxfp4_matmul(c, s, c, s), "mxfp4_linear": lambda: awq.awq_mxfp4_linear(x, c, s)}
real = {}
library = _mx._lib()

class Counted:
    n = 0
    def __getattr__(self, name):
        fn = getattr(library, name)
        def call(*a):
            Counted.n += not name.endswith("_bytes")
            return fn(*a)
        return call

_mx._C = Counted()
for name, call in run.items():
    for code in (1, 2, 3, 4, 5, 6, 9):                           # refusals: the library's answer counts
        status.value, calls.value, Counted.n = code, 0, 0
        call()
        assert (calls.value, Counted.n) == (1, 1), (name, code, calls.value, Counted.n)
    status.value, calls.value, Counted.n = 7, 0, 0             # a launch that failed: said, not done again
    try:
        call()
    except awq.AwqError as e:
        assert e.status == 7 and "awq_" + name in str(e), (name, str(e))
    else:
        raise AssertionError(name + ": a failed launch was not reported")
    assert (calls.value, Counted.n) == (1, 0), (name, calls.value, Counted.n)
torch.cuda.synchronize()
print("done")
"""


def test_failed_launches_are_reported_once(tmp_path):
    say("statuses of the short way into the calls")
    (tmp_path / "fake.c").write_text(FAKE)
    (tmp_path / "child.py").write_text(CHILD)
    fake = tmp_path / "libfake.so"
    subprocess.run(["gcc", "-shared", "-fPIC", str(tmp_path / "fake.c"), "-o", str(fake)], check=True)
    res = subprocess.run([sys.executable, str(tmp_path / "child.py"), str(fake)], cwd=ROOT, capture_output=True,
                         text=True, timeout=100, env={**os.environ, "PYTHONPATH": ROOT})
    assert res.returncode == 0 and "done" in res.stdout, res.stderr[-3000:]


@pytest.mark.parametrize("name", CALLS)
def test_first_arguments(name):
    """What is refused without a GPU is refused with one."""
    say(f"first arguments of {name}")
    call, (first, args, more) = getattr(awq, name), CALLS[name]
    for kw in ({}, more):
        with pytest.raises(ValueError, match="device"):
            call(first, *args, **kw)
        for bad in (3.0, 0, None, [1], "x"):
            with pytest.raises(TypeError, match="torch.Tensor"):
                call(bad, *args, **kw)


def _outcome(call):
    """What a call gives, so that two can be compared: its tensors with their layout, or its error."""
    try:
        got = call()
    except Exception as e:  # noqa: BLE001  (the error is the outcome)
        return type(e), str(e)
    torch.cuda.synchronize()
    return [(t.dtype, tuple(t.shape), t.stride(), t.device, t.requires_grad, t) for t in
            (got if isinstance(got, tuple) else (got,))]


def _alike(a, b, rows):
    if not isinstance(a, list) or not isinstance(b, list):
        return a == b
    for x, y in zip(a, b):
        s, t = x[-1], y[-1]
        if s.dim() == 3:                                          # scales: rows past the last are not written
            s, t = s[:, :rows], t[:, :rows]
        bits = (lambda v: v.contiguous().flatten().view(torch.uint8))
        if x[:-1] != y[:-1] or not torch.equal(bits(s), bits(t)):
            return False
    return len(a) == len(b)


def _arguments():
    """(name, rows, call): the usual, the odd and the refused ones of every entry point."""
    g = torch.Generator(device="cuda").manual_seed(0)

    def rand(*shape, dtype=torch.float16):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)
    f32, bf16, f16 = torch.float32, torch.bfloat16, torch.float16
    wide = rand(9, 1300)
    xs = {"plain": rand(5, 200), "bf16": rand(5, 200, dtype=bf16), "one row": rand(1, 200), "one column": rand(5, 1),
          "view": wide[1:6, 3:203], "rows apart": wide[::2, 8:208], "row of many": wide[4:5, 1:201],
          "transposed": rand(200, 5).t(), "expanded": rand(1, 200).expand(5, 200), "no rows": rand(0, 200),
          "no columns": rand(5, 0), "fp32": rand(5, 200, dtype=f32), "1-D": rand(200), "3-D": rand(5, 2, 100),
          "parameter": torch.nn.Parameter(rand(5, 200)), "column step 2": rand(5, 400)[:, ::2],
          "sparse": rand(5, 200).to_sparse(), "host": rand(5, 200).cpu()}
    ws = {"none": None, "same": rand(200), "fp32": rand(200, dtype=f32), "bf16": rand(200, dtype=bf16), "short": rand(199),
          "2-D": rand(1, 200), "step 2": rand(400)[::2], "offset": rand(205)[5:], "host": rand(200).cpu(),
          "number": 1.0, "int": torch.ones(200, dtype=torch.int32, device="cuda")}
    norms = (awq.awq_rmsnorm, awq.awq_rmsnorm_int8, awq.awq_rmsnorm_mxfp4)
    for fn in norms:
        for k, x in xs.items():
            rows = x.shape[0]
            yield f"{fn.__name__} x {k}", rows, lambda fn=fn, x=x: fn(x)
            yield f"{fn.__name__} residual {k}", 5, lambda fn=fn, x=x: fn(xs["plain"], residual=x)
        for k, w in ws.items():
            yield f"{fn.__name__} weight {k}", 5, lambda fn=fn, w=w: fn(xs["plain"], w)
        for eps in (1e-6, 1, 0, 0.0, -1.0, 1e-39, float("nan"), float("inf"), True, "1", None, 2 ** 70):
            yield f"{fn.__name__} eps {eps}", 5, lambda fn=fn, eps=eps: fn(xs["plain"], None, eps)
        yield f"{fn.__name__} residual number", 5, lambda fn=fn: fn(xs["plain"], residual=1.0)
    for k, x in xs.items():
        yield f"quantize A {k}", x.shape[0], lambda x=x: awq.awq_mxfp4_quantize(x)
    for fold in ("divide", "multiply", "add"):
        for k, w in ws.items():
            yield f"quantize s {k} {fold}", 5, lambda w=w, fold=fold: awq.awq_mxfp4_quantize(xs["plain"], w, fold)
    (xc, xss), (wc, wss) = awq.awq_mxfp4_quantize(xs["plain"]), awq.awq_mxfp4_quantize(rand(33, 200))
    pad = torch.zeros(5, xc.shape[1] + 32, dtype=torch.uint8, device="cuda")
    pad[:, 16:-16] = xc
    codes = {"plain": xc, "view": pad[:, 16:-16], "unaligned": pad[:, 8:-24], "int8": xc.view(torch.int8),
             "fewer": xc[:3], "half": xc[:, :104], "none": xc[:0], "one": xc[:1], "1-D": xc[0], "host": xc.cpu()}
    scales = {"plain": xss, "int8": xss.view(torch.int8), "short": xss[:, :4], "words": xss[:1],
              "step": xss.repeat(1, 2, 1)[:, ::2], "2-D": xss[0], "host": xss.cpu(), "number": 3}
    for k, c in codes.items():
        yield f"dequantize codes {k}", 5, lambda c=c: awq.awq_mxfp4_dequantize(c, xss, 200)
        yield f"matmul xc {k}", 5, lambda c=c: awq.awq_mxfp4_matmul(c, xss, wc, wss)
        yield f"matmul wc {k}", 33, lambda c=c: awq.awq_mxfp4_matmul(wc, wss, c, xss)
        yield f"linear wc {k}", 5, lambda c=c: awq.awq_mxfp4_linear(xs["plain"], c, xss)
    for k, s in scales.items():
        yield f"dequantize scales {k}", 5, lambda s=s: awq.awq_mxfp4_dequantize(xc, s, 200)
        yield f"matmul xs {k}", 5, lambda s=s: awq.awq_mxfp4_matmul(xc, s, wc, wss)
        yield f"matmul ws {k}", 33, lambda s=s: awq.awq_mxfp4_matmul(wc, wss, xc, s)
        yield f"linear ws {k}", 5, lambda s=s: awq.awq_mxfp4_linear(xs["plain"], xc, s)
    q, st = awq.awq_int8_quantize(xs["plain"])
    for cols in (200, 193, 208, 209, 192, 0, -1, True, 200.0, None, 2 ** 70):
        yield f"int8 cols {cols}", 5, lambda cols=cols: awq.awq_int8_dequantize(q, st, cols)
        yield f"dequantize cols {cols}", 5, lambda cols=cols: awq.awq_mxfp4_dequantize(xc, xss, cols)
    for dt in (f16, bf16, f32, torch.int8, None, "fp16"):
        yield f"int8 dtype {dt}", 5, lambda dt=dt: awq.awq_int8_dequantize(q, st, 200, dt)
        yield f"dequantize dtype {dt}", 5, lambda dt=dt: awq.awq_mxfp4_dequantize(xc, xss, 200, dt)
        yield f"matmul dtype {dt}", 5, lambda dt=dt: awq.awq_mxfp4_matmul(xc, xss, wc, wss, dt)
    for k, c in {"steps none": (q, None), "steps short": (q, st[:4]), "steps half": (q, st.half()), "uint8": (
            q.view(torch.uint8), st), "rows": (q[1:3], st[1:3]), "host": (q, st.cpu())}.items():
        yield f"int8 {k}", 5, lambda c=c: awq.awq_int8_dequantize(*c, 200)
    bias = {"none": None, "same": rand(33), "bf16": rand(33, dtype=bf16), "short": rand(32), "step 2": rand(66)[::2],
            "host": rand(33).cpu(), "number": 0.0}
    for k, b in bias.items():
        yield f"matmul bias {k}", 5, lambda b=b: awq.awq_mxfp4_matmul(xc, xss, wc, wss, f16, b)
        yield f"linear bias {k}", 5, lambda b=b: awq.awq_mxfp4_linear(xs["plain"], wc, wss, bias=b)
    for k, x in xs.items():
        yield f"linear x {k}", x.shape[0], lambda x=x: awq.awq_mxfp4_linear(x, wc, wss)
    for k, w in ws.items():
        yield f"linear s {k}", 5, lambda w=w: awq.awq_mxfp4_linear(xs["plain"], wc, wss, s=w)


def test_both_ways_agree(monkeypatch):
    """The extension module's way into the calls and the binding's own give the same tensors and the same
    errors, over arguments that either takes or refuses."""
    from weight_only_quantization_act_amd import _mx
    assert isinstance(_mx._native(), types.ModuleType)
    off, n = [], 0
    for name, rows, call in _arguments():
        say(name)
        short = _outcome(call)
        with monkeypatch.context() as m:
            m.setattr(_mx, "_N", _mx._NoCalls())
            longer = _outcome(call)
        n += 1
        if not _alike(short, longer, rows):
            off.append((name, short if not isinstance(short, list) else "tensors", longer if not isinstance(longer, list)
                        else "tensors"))
    assert n > 250 and not off, off
