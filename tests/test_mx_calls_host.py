"""The binding of the norm and of MXFP4 on the host: what it refuses and how it says so, without a GPU."""
import sys
import sysconfig
import types
import warnings

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


def test_calls_without_the_extension_module(monkeypatch):
    """The binding needs the library alone: without the module calls go the longer way, said once."""
    from weight_only_quantization_act_amd import _mx
    monkeypatch.delattr(awq, "_calls", raising=False)
    monkeypatch.setitem(sys.modules, awq.__name__ + "._calls", None)
    monkeypatch.setattr(_mx, "_N", None)
    with pytest.warns(RuntimeWarning, match="_calls"):
        with pytest.raises(ValueError, match="device"):
            awq.awq_rmsnorm(X)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        for name, (first, args, more) in CALLS.items():
            with pytest.raises(ValueError, match="device"):
                getattr(awq, name)(first, *args)


@pytest.fixture
def building(tmp_path, monkeypatch):
    """The build in an empty folder, its commands written down in place of being run."""
    from weight_only_quantization_act_amd import build
    ran = []

    def run(cmd):
        if build.broken and any(build.broken in c for c in cmd):
            raise RuntimeError(build.broken)
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("new")
        return ""
    monkeypatch.setattr(build, "broken", "", raising=False)
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build, "_run", run)
    (tmp_path / "_calls.so").write_text("old")
    (tmp_path / build.LIB_NAME).write_text("old")
    return build, ran, tmp_path


def test_build(building):
    build, ran, where = building
    assert build.build() == str(where / build.LIB_NAME)
    assert (where / build.LIB_NAME).read_text() == "new" and (where / "_calls.so").read_text() == "new"
    assert sum("calls.cpp" in c for cmd in ran for c in cmd) >= 1


def test_build_without_header_files(building, monkeypatch, tmp_path):
    """The library is built where Python's header files, which it does not need, are not installed; a module on top
    of the library before does not stay."""
    build, ran, where = building
    get = sysconfig.get_path
    monkeypatch.setattr(build.sysconfig, "get_path", lambda n, *a, **k: str(tmp_path / "none") if n == "include"
                        else get(n, *a, **k))
    build.broken = "calls.cpp"                                  # as the compiler would without them
    assert build.build() == str(where / build.LIB_NAME)
    assert (where / build.LIB_NAME).read_text() == "new" and not (where / "_calls.so").exists()


@pytest.mark.parametrize("step", ["calls.cpp", "-ltorch_python"])
def test_build_whose_module_fails(building, step):
    """An error in the module's own build is one, with the library in place."""
    build, ran, where = building
    build.broken = step
    with pytest.raises(RuntimeError, match=step):
        build.build()
    assert (where / build.LIB_NAME).read_text() == "new" and not (where / "_calls.so").exists()


def test_outputs_over_operands_are_refused(monkeypatch):
    """A linear layer's out over its tokens would be read by blocks that others have written to already; the norm's
    out and h_out are two results."""
    from weight_only_quantization_act_amd import _mx
    monkeypatch.setattr(_mx, "_current_device", lambda: 0)
    c, s = torch.zeros(64, 32, dtype=torch.uint8), torch.zeros(1, 64, 4, dtype=torch.uint8)
    for rows in (1, 3, 40):
        x = _claimed(torch.zeros(rows, 64).half())
        with pytest.raises(ValueError, match="out"):
            awq.awq_mxfp4_linear(x, _claimed(c), _claimed(s), out=x)
        h = _claimed(torch.zeros(rows, 64).half())
        with pytest.raises(ValueError, match="out"):
            awq.awq_rmsnorm(x, residual=_claimed(torch.zeros(rows, 64).half()), h_out=h, out=h)
