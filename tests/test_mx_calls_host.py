"""The binding of the norm and of MXFP4 on the host: what it refuses and how it says so, without a GPU."""
import types

import pytest
import torch

import weight_only_quantization_act_amd as awq

X, W = torch.zeros(3, 64).half(), torch.ones(64)
C, S = torch.zeros(3, 32, dtype=torch.uint8), torch.zeros(1, 4, 4, dtype=torch.uint8)
Q = torch.zeros(3, 64, dtype=torch.int8)
# entry point, first argument, the others, an argument that leaves the short way
CALLS = {
    "awq_rmsnorm": (X, (W,), dict(out=X)),
    "awq_rmsnorm_int8": (X, (W,), dict(residual=X, h_out=X)),
    "awq_rmsnorm_mxfp4": (X, (W,), dict(residual=X, h_out=X)),
    "awq_mxfp4_quantize": (X, (), dict(s=W)),
    "awq_mxfp4_dequantize": (C, (S, 64), dict(out=X)),
    "awq_mxfp4_matmul": (C, (S, C, S), dict(out=X)),
    "awq_mxfp4_linear": (X, (C, S), dict(out=X)),
    "awq_int8_dequantize": (Q, (W[:3], 64), dict(out=X)),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("longer", [False, True])
def test_first_arguments(name, longer):
    """A tensor of the host is a ValueError, what is no tensor a TypeError, on either way into the call."""
    call, (first, args, more) = getattr(awq, name), CALLS[name]
    kw = more if longer else {}
    with pytest.raises(ValueError, match="device"):
        call(first, *args, **kw)
    for bad in (3.0, 0, None, [1], "x"):
        with pytest.raises(TypeError, match="torch.Tensor"):
            call(bad, *args, **kw)


class Elsewhere(torch.Tensor):
    """A host tensor that says it is on a GPU: for checks that come before any use of it."""
    at = 0
    is_cuda = True
    device = property(lambda self: torch.device("cuda", self.at))

    def get_device(self):
        return self.at


def _claimed(value):
    return value.as_subclass(Elsewhere) if isinstance(value, torch.Tensor) else value


@pytest.mark.parametrize("name", CALLS)
def test_stream_of_another_device_is_refused(name, monkeypatch):
    """It would run on its tensors' device, on that device's current stream."""
    from weight_only_quantization_act_amd import _mx
    call, (first, args, more) = getattr(awq, name), CALLS[name]
    for current in (0, 1):
        monkeypatch.setattr(_mx, "_current_device", lambda: current)
        for kw in ({}, more):
            with pytest.raises(ValueError, match="stream"):
                call(_claimed(first), *map(_claimed, args), **{k: _claimed(v) for k, v in kw.items()},
                     stream=types.SimpleNamespace(device=torch.device("cuda", 1)))
