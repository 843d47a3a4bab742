"""The short way into the calls of the norm and of MXFP4 on the GPU: what it does with the C ABI's answers.

A child process puts functions of the C ABI's names, which count their calls and return a chosen status, before the
library's for the extension module alone; the binding's longer way calls the library itself.
"""
import os
import subprocess
import sys

import pytest

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
