"""Build libmsa.so (the CUDA library behind include/msa.h) for sm_100a, and
_msa_torch.so, the compiled binding of its paged-cache calls.

Run ``python -m block_sparse_long_05_b200.build`` or call ``build()``.  The
shared objects are written next to this file (in-tree).  libmsa has the CUDA
runtime linked statically, so it loads on any machine with an NVIDIA driver;
the binding belongs to the torch and Python it was built with (recorded in
_msa_torch.json beside it), and is built anew under others.
"""
from __future__ import annotations

import contextlib
import glob
import json
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmsa.so")
BINDING = os.path.join(HERE, "_msa_torch.so")
BINDING_KEY = os.path.join(HERE, "_msa_torch.json")
BINDING_SRC = os.path.join(HERE, "csrc_torch", "binding.cpp")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
    "-I", os.path.join(ROOT, "include"),
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(CSRC, "*.h")) + [os.path.join(ROOT, "include", "msa.h"), __file__]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every .cu under csrc/ into libmsa.so (sm_100a), then the binding
    (which needs a C++ compiler and the headers of Python and torch; the library does not).
    Returns the library's path."""
    build_library(force, verbose, ptxas_info)
    build_binding(force, verbose)
    return LIB


def build_library(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every .cu under csrc/ into libmsa.so (sm_100a).  Returns its path."""
    if not force and not ptxas_info and up_to_date():
        return LIB
    objs = []
    build_dir = os.path.join(HERE, "_build")
    os.makedirs(build_dir, exist_ok=True)
    procs = []
    for src in sources():  # the translation units compile in parallel
        obj = os.path.join(build_dir, os.path.basename(src) + ".o")
        cmd = [NVCC, *FLAGS, "-c", src, "-o", obj]
        if ptxas_info:
            cmd += ["-Xptxas", "-v"]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((cmd, subprocess.Popen(cmd)))
        objs.append(obj)
    for cmd, p in procs:
        if p.wait() != 0:
            raise subprocess.CalledProcessError(p.returncode, cmd)
    tmp = LIB + ".tmp"
    cmd = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-cudart", "static",
           "-Xcompiler", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


def _binding_key() -> dict:
    """What the binding's binary interface depends on, beside its source."""
    import torch
    return {"torch": torch.__version__, "cxx11_abi": bool(torch._C._GLIBCXX_USE_CXX11_ABI),
            "python": sysconfig.get_config_var("SOABI")}


def _recorded_key():
    try:
        with open(BINDING_KEY) as f:
            return json.load(f)
    except (OSError, ValueError):
        return None


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc_torch/binding.cpp into _msa_torch.so, unless it is newer than its
    sources and was built with this torch and Python.  Returns the path."""
    header = os.path.join(ROOT, "include", "msa.h")
    key = _binding_key()
    if not force and os.path.exists(BINDING) and _recorded_key() == key and all(
            os.path.getmtime(f) <= os.path.getmtime(BINDING) for f in (BINDING_SRC, header, __file__)):
        return BINDING
    import torch
    base = os.path.dirname(torch.__file__)
    include = [os.path.join(base, "include"),
               os.path.join(base, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"],
               os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"),
               os.path.join(ROOT, "include")]
    tmp = f"{BINDING}.{os.getpid()}.tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f for i in include for f in ("-isystem", i)), BINDING_SRC, "-o", tmp,
           "-L", os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
           "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    with contextlib.suppress(FileNotFoundError):
        os.remove(BINDING_KEY)  # (it never speaks for a module that it does not belong to)
    os.replace(tmp, BINDING)
    with open(tmp, "w") as f:
        json.dump(key, f)
    os.replace(tmp, BINDING_KEY)
    return BINDING


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
