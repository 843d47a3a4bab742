"""The binding of the norm and of MXFP4 on the host: what it refuses and how it says so, without a GPU."""
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
