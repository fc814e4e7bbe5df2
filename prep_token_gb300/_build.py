"""Builds libdsaprep.so in-tree with nvcc for sm_103a (no torch extension
machinery: the library is plain C ABI over CUDA), and beside it _binding-*.so, the
marshalling in C++ of the calls that a decode step makes eagerly.  The library does
without the binding, which fits one torch and one Python and carries their versions
in its name."""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB_PATH = os.path.join(PKG, "libdsaprep.so")
BINDING_SOURCE = os.path.join(PKG, "csrc", "binding.cpp")
INCLUDE = os.path.join(ROOT, "include")
NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17", "--diag-suppress=177",
    "-Xcompiler", "-fPIC", "-shared",
    "-cudart", "shared", "-Xlinker", "-rpath,/usr/local/cuda/lib64",
]


def _nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(home, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(PKG, "csrc", "*.cu")))


def _older(path: str, deps: list[str]) -> bool:
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(d) > t for d in deps)


def _headers() -> list[str]:
    return glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale() -> bool:
    return _older(LIB_PATH, sources() + glob.glob(os.path.join(PKG, "csrc", "*.cuh")) + _headers())


def binding_path() -> str:
    """The binding for this torch and this Python."""
    import torch
    return os.path.join(PKG, f"_binding-torch{torch.__version__}-{sys.implementation.cache_tag}.so")


def _torch_include() -> str:
    import torch
    return os.path.join(os.path.dirname(torch.__file__), "include")


def _binding_needs() -> list[str]:
    """Headers that an installation may lack."""
    return [os.path.join(_torch_include(), "torch", "csrc", "autograd", "python_variable.h"),
            os.path.join(sysconfig.get_paths()["include"], "Python.h")]


def _binding_command(out: str) -> list[str]:
    import torch
    include = _torch_include()
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    return ["g++", "-O1", "-std=c++17", "-fPIC", "-shared", "-I", INCLUDE, "-I", include,
            "-I", os.path.join(include, "torch", "csrc", "api", "include"),
            "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-o", out, BINDING_SOURCE, "-L", os.path.join(os.path.dirname(include), "lib"),
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile every .cu under csrc/ (in parallel, one nvcc per file) and
    link them into one shared library, and the binding beside them (left out, and
    said so, where torch's or Python's headers are not installed)."""
    import torch
    tag = f"{os.getpid()}"
    path, binding = binding_path(), None
    made = path + f".tmp{tag}"
    if force or _older(path, [BINDING_SOURCE, torch.__file__] + _headers()):
        missing = [h for h in _binding_needs() if not os.path.exists(h)]
        if missing:
            print(f"{os.path.basename(path)} is not built: no {', '.join(missing)}", file=sys.stderr)
        else:
            binding = subprocess.Popen(_binding_command(made))
    try:
        if force or _stale():
            _build_cuda(tag, verbose)
        if binding:
            if binding.wait():
                raise subprocess.CalledProcessError(binding.returncode, "g++ binding.cpp")
            os.replace(made, path)
    finally:
        if binding:
            binding.wait()
            if os.path.exists(made):
                os.remove(made)
    return LIB_PATH


def _build_cuda(tag: str, verbose: bool) -> None:
    objs, procs = [], []
    compile_flags = [f for f in NVCC_FLAGS if f not in ("-shared",)]
    for src in sources():
        obj = os.path.join(PKG, "csrc", os.path.basename(src) + f".{tag}.o")
        cmd = [_nvcc(), *compile_flags, "-I", INCLUDE, "-c", "-o", obj, src]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append(subprocess.Popen(cmd))
        objs.append(obj)
    try:
        codes = [p.wait() for p in procs]
        if any(codes):
            raise subprocess.CalledProcessError(max(codes), "nvcc -c")
        tmp = LIB_PATH + f".tmp{tag}"
        subprocess.check_call([_nvcc(), *NVCC_FLAGS, "-o", tmp, *objs])
        os.replace(tmp, LIB_PATH)
    finally:
        for obj in objs:
            if os.path.exists(obj):
                os.remove(obj)
