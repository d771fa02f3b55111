"""Build the CUDA library libattn_jvp.so in-tree for sm_100a with nvcc, and then the
Python binding of the serving operators, _serving.so, with the C++ compiler.

    python -m attention_jvp_attn_b200.build [--force] [--verbose]

The library needs nvcc only. The binding also needs torch's and Python's headers and
g++; where one is missing it is left out, with a message, and the serving operators
say so when they are called from Python.
The library is a plain shared object with a C ABI (include/attn_jvp.h); the
CUDA runtime is linked statically, and the driver entry point for tensor-map
encoding is resolved at run time, so loading it needs no GPU.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libattn_jvp.so")
BINDING = os.path.join(PKG, "_serving.so")
# Opt-in variant whose bf16 kernel records per-tile event clocks of CTA 0.
TRACE_LIB = os.path.join(PKG, "libattn_jvp_trace.so")

BINDING_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden"]

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(f) <= t for f in _deps())


def _run(cmd, verbose: bool):
    if verbose:
        print(" ".join(cmd))
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    return res.stdout + res.stderr


def binding_built_for() -> str:
    """What a binding must have been built for: it reads the tensors of one torch, in
    the Python of one ABI. The binding holds this text as `built_for`."""
    import torch
    return (f"torch {torch.__version__} abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)} python "
            f"{sysconfig.get_config_var('EXT_SUFFIX')} flags {' '.join(BINDING_FLAGS)}")


def binding_lacks():
    """What is missing here to build the binding."""
    have = {"torch": importlib.util.find_spec("torch"), "g++": shutil.which("g++"),
            "Python.h": os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h"))}
    return [name for name, found in have.items() if not found]


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """_serving.so: it reads torch tensors, so it is built against this torch,
    and by the g++ that nvcc takes too: one with a C++ runtime of its own linked
    in statically crashes beside torch's as soon as a message formats a number."""
    src, header = os.path.join(CSRC, "serve_binding.cpp"), os.path.join(INCLUDE, "attn_jvp.h")
    key = binding_built_for()
    if not force and os.path.exists(BINDING) and \
            all(os.path.getmtime(f) <= os.path.getmtime(BINDING) for f in (src, header)):
        with open(BINDING, "rb") as f:
            if key.encode() + b"\0" in f.read():
                return BINDING
    import torch
    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    includes = [INCLUDE, os.path.join(at, "include"), os.path.join(at, "include/torch/csrc/api/include"),
                os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    out = _run([shutil.which("g++"), *BINDING_FLAGS,
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DAJVP_BUILT_FOR="{key}"',
                *(f for i in includes for f in ("-isystem", i)), "-o", BINDING + ".tmp", src,
                "-L" + os.path.join(at, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"], verbose)
    if verbose:
        sys.stdout.write(out)
    os.replace(BINDING + ".tmp", BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False,
          trace: bool = False) -> str:
    lib = build_library(force, verbose, ptxas_info, trace)
    if not trace:
        lacks = binding_lacks()
        if lacks:
            print(f"serving binding not built: no {' and no '.join(lacks)} here", file=sys.stderr)
        else:
            build_binding(force, verbose)
    return lib


def build_library(force: bool = False, verbose: bool = False, ptxas_info: bool = False,
                  trace: bool = False) -> str:
    lib = TRACE_LIB if trace else LIB
    if not force and up_to_date(lib):
        return lib
    cmd = [_nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
           "-Xcompiler", "-fPIC,-O2", "-shared", "-I", INCLUDE, "-I", CSRC,
           *(["-DAJVP_TRACE"] if trace else []), "-o", lib + ".tmp", *_sources()]
    if ptxas_info:
        cmd[1:1] = ["-Xptxas", "-v"]
    out = _run(cmd, verbose)
    if verbose or ptxas_info:
        sys.stdout.write(out)
    os.replace(lib + ".tmp", lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv,
                ptxas_info="--ptxas-info" in sys.argv, trace="--trace" in sys.argv))
