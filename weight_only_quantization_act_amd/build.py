"""Build libawq_act.so (HIP kernels for gfx950 + the C ABI) in-tree.

    python -m weight_only_quantization_act_amd.build

Compiles every .hip file under csrc/ with hipcc for gfx950 and the host-only C ABI
(api.cpp), then links one shared library next to this file, and an extension module of this
interpreter on top of it (csrc/python/, the short way from a Python call to the C ABI).  Where the
header files that the module needs are not installed only the library is built; the binding does without
the module.  Always recompiles.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB_NAME = "libawq_act.so"
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
ARCH = "gfx950"

# Numerics flags are part of the contract: no FMA contraction, IEEE division and sqrt,
# fp32 denormals kept (the gfx9 default), no fast-math.  Packed fp32 vector ops are
# disabled for all device code.
HIP_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt", "-fno-fast-math",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]
# Per-source additions.  The clip-search kernels keep their small MFMA accumulators in
# VGPRs (no accumulator-register moves in the epilogue), and so does the cache attention
# (its running rescale); the large-tile GEMMs need AGPRs.
HIP_FILE_FLAGS = {
    "kv4_attention.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
    "clip_search.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
}
HOST_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__",
              f"-I{ROCM}/include"]


# The extension module.
CALLS = os.path.join(PKG, "_calls" + sysconfig.get_config_var("EXT_SUFFIX"))


def _calls_commands(clangxx, incs):
    """The commands that compile and link the extension module, or None where the header files of Python or of
    torch on HIP are missing."""
    import torch
    at = os.path.dirname(torch.__file__)
    python = sysconfig.get_path("include")
    dirs = [os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include")]
    if not (torch.version.hip and os.path.exists(os.path.join(python, "Python.h"))
            and os.path.exists(os.path.join(dirs[0], "ATen", "hip", "EmptyTensor.h"))):
        return None
    obj = os.path.join(BUILD, "calls.cpp.o")
    return ([clangxx, *HOST_FLAGS, "-DUSE_ROCM", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
             *incs, f"-I{python}", *(f"-isystem{d}" for d in dirs), "-c", os.path.join(CSRC, "python", "calls.cpp"),
             "-o", obj],
            [clangxx, "-shared", "-fPIC", obj, "-o", CALLS + ".tmp", f"-L{os.path.join(at, 'lib')}", "-ltorch_python",
             "-ltorch_cpu", "-ltorch_hip", "-lc10", "-lc10_hip", f"-L{PKG}", f"-l:{LIB_NAME}", "-Wl,-rpath,$ORIGIN"])


def _run(cmd):
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(l for l in res.stdout.splitlines()
                    if "packed-fp32-ops' is not a recognized feature" not in l)
    if res.returncode != 0:
        raise RuntimeError(f"command failed ({res.returncode}): {' '.join(cmd)}\n{out}")
    return out


def lib_path() -> str:
    return os.path.join(PKG, LIB_NAME)


def build(verbose: bool = False, jobs: int = 8) -> str:
    hipcc = shutil.which("hipcc") or os.path.join(ROCM, "bin", "hipcc")
    clangxx = os.path.join(ROCM, "bin", "amdclang++")
    os.makedirs(BUILD, exist_ok=True)
    incs = [f"-I{INCLUDE}", f"-I{CSRC}"]
    jobs_list = []
    for f in sorted(os.listdir(CSRC)):
        src = os.path.join(CSRC, f)
        obj = os.path.join(BUILD, f + ".o")
        if f.endswith(".hip"):
            jobs_list.append([hipcc, *HIP_FLAGS, *HIP_FILE_FLAGS.get(f, []), *incs, "-c", src,
                              "-o", obj])
        elif f.endswith(".cpp"):
            jobs_list.append([clangxx, *HOST_FLAGS, *incs, "-c", src, "-o", obj])
    calls = _calls_commands(clangxx, incs)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        calls_out = ex.submit(_run, calls[0]) if calls else None
        outs = list(ex.map(_run, jobs_list))
    if os.path.exists(CALLS):
        os.remove(CALLS)  # it fits the library before
    tmp = lib_path() + ".tmp"
    _run([hipcc, f"--offload-arch={ARCH}", "-shared", "-fPIC", *(cmd[-1] for cmd in jobs_list), "-o", tmp,
          f"-L{ROCM}/lib", "-lamdhip64"])
    os.replace(tmp, lib_path())
    if calls:  # with the library in place, whatever happens here
        outs.append(calls_out.result())
        _run(calls[1])
        os.replace(CALLS + ".tmp", CALLS)
    else:
        print("header files of Python or of torch on HIP not found: built without the extension module _calls")
    if verbose:
        for o in outs:
            if o.strip():
                print(o)
    if verbose:
        print("built", lib_path())
    return lib_path()


if __name__ == "__main__":
    build(verbose="-q" not in sys.argv)
