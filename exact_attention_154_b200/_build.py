"""Build step for ``libfa_sm100.so`` (nvcc, sm_100a only, in-tree)."""
from __future__ import annotations

import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libfa_sm100.so")
BINDING_SOURCE = os.path.join(CSRC, "fa_torch.cpp")
SOURCES = ["fa_api.cu"]


def headers():
    """Every header under csrc/: a change to any of them rebuilds the library."""
    return sorted(f for f in os.listdir(CSRC) if f.endswith((".cuh", ".h")))
NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-Xptxas", "-v",
]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, f) for f in SOURCES + headers()]
    files.append(os.path.join(ROOT, "include", "fa.h"))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library next to the package, then, where torch is installed, its
    torch binding; returns the library's path.  (A program that calls the C ABI
    needs no torch, nor a binding that compiles.)"""
    if force or not up_to_date():
        build_library(verbose)
    try:
        import torch  # noqa: F401
    except ImportError:
        return LIB
    build_binding(force)
    return LIB


def build_library(verbose: bool = False) -> None:
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc_path(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"),
           "-o", tmp, *[os.path.join(CSRC, s) for s in SOURCES]]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    if verbose:
        print(res.stderr)
    check_register_split(res.stdout + res.stderr)
    os.replace(tmp, LIB)


BINDING_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-shared"]


def binding_path() -> str:
    """The torch binding's file for the running torch and Python: its classes'
    layout and its module's form are theirs, so each has a file of its own."""
    import hashlib
    import sysconfig

    import torch
    key = "\n".join([torch.__version__, str(torch.version.cuda),
                     str(int(torch._C._GLIBCXX_USE_CXX11_ABI)),
                     str(sysconfig.get_config_var("SOABI")), *BINDING_FLAGS])
    return os.path.join(PKG, f"_fa_torch-{hashlib.sha256(key.encode()).hexdigest()[:12]}.so")


def build_binding(force: bool = False) -> str:
    """Compile the torch side of the layer's calls (host code, resolved against
    the library when it is loaded); returns its path."""
    binding = binding_path()
    inputs = [BINDING_SOURCE, os.path.join(ROOT, "include", "fa.h")]
    if not force and os.path.exists(binding) and \
            all(os.path.getmtime(f) <= os.path.getmtime(binding) for f in inputs):
        return binding
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    include = [os.path.join(root, "include"),
               os.path.join(root, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = binding + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", *BINDING_FLAGS,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[x for p in include for x in ("-isystem", p)], "-o", tmp, BINDING_SOURCE,
           "-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python", "-ldl"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + res.stdout + res.stderr)
    os.replace(tmp, binding)
    return binding


# The two-Q-tile kernels run 640 threads (96 registers each at launch) and
# redistribute them with setmaxnreg: 4 * 128 * 104 + 128 * 64 = 61440.
SPLIT_THREADS = 640
SPLIT_REQUEST = 4 * 128 * 104 + 128 * 64


def check_register_split(ptxas_log: str) -> None:
    """Refuse a build whose setmaxnreg requests exceed the registers the
    640-thread kernels are launched with: such a request would never be
    granted and the kernel would wait for it forever."""
    import re
    entry, seen = None, 0
    for line in ptxas_log.splitlines():
        m = re.search(r"Compiling entry function '(\S+)'", line)
        if m:
            entry = m.group(1)
            continue
        m = re.search(r"Used (\d+) registers", line)
        if m and entry and re.search(r"fa_fwd_kernelILi\d+ELi2E", entry):
            regs = int(m.group(1))
            if regs * SPLIT_THREADS < SPLIT_REQUEST:
                raise RuntimeError(f"{entry}: {regs} registers x {SPLIT_THREADS} threads < "
                                   f"setmaxnreg requests {SPLIT_REQUEST}")
            seen += 1
    if seen == 0:
        raise RuntimeError("ptxas register report for the two-Q-tile kernels not found")


if __name__ == "__main__":
    print(build(force=True, verbose=True))
