"""Build the CUDA library in-tree: tensor_gemm_reduce_gb300/lib/libgemm_rs.so,
and the Python entry of its operators beside it (_ops_<hash>.so).

Sources compile for sm_103a (tcgen05 / TMA need the arch-specific target) side
by side, one nvcc for each, and are linked into one library.  The library links the CUDA runtime statically and resolves the one driver call
it needs (cuTensorMapEncodeTiled) at run time, so it has no link-time
dependency on libcuda.
"""
from __future__ import annotations

import contextlib
import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libgemm_rs.so")
SOURCES = [os.path.join(CSRC, f) for f in ("gemm_rs.cu", "block_norm.cu", "act8.cu", "backward.cu", "w4.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in ("kernels.cuh", "ptx.cuh", "schedule.h",
                                                  "ops_common.cuh", "act8.cuh")] + [
    os.path.join(ROOT, "include", f) for f in ("gemm_rs.h", "gemm_rs_ops.h")]

BINDING_SOURCE = os.path.join(CSRC, "ops_binding.cpp")
BINDING_HEADERS = [os.path.join(ROOT, "include", f) for f in ("gemm_rs.h", "gemm_rs_ops.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
]


def nvcc_path() -> str:
    p = shutil.which("nvcc")
    if p:
        return p
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found")


def _stale(target: str, sources) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in sources)


def build_library(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile the library if it is missing or older than its sources; return its path."""
    if not force and not _stale(LIB, DEPS):
        return LIB
    os.makedirs(LIBDIR, exist_ok=True)
    tmp = LIB + f".tmp{os.getpid()}"
    nvcc = [nvcc_path()] + NVCC_FLAGS + list(extra_flags or [])
    with tempfile.TemporaryDirectory(prefix="gemm_rs_build_") as work:
        objects = [os.path.join(work, os.path.basename(s) + ".o") for s in SOURCES]
        steps = [[nvcc + ["-c", "-o", o, s] for o, s in zip(objects, SOURCES)],
                 [nvcc + ["-shared", "-Xlinker", "-soname=libgemm_rs.so", "-o", tmp] + objects]]
        for cmds in steps:
            if verbose:
                print("\n".join(" ".join(c) for c in cmds), file=sys.stderr)
            procs = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
                     for c in cmds]
            outs = [p.communicate()[0] for p in procs]
            for p, out in zip(procs, outs):
                if p.returncode != 0:
                    raise RuntimeError(f"nvcc failed ({p.returncode}):\n{out}")
                if verbose and out:
                    print(out, file=sys.stderr)
    os.replace(tmp, LIB)
    return LIB


def binding_path() -> str:
    """Where the binding lies that was compiled from these sources for this torch and Python.  One
    of another interface or another torch has another name, so it is never loaded in its place."""
    import torch
    h = hashlib.sha256(f"{torch.__version__} {sys.version}".encode())
    for path in [BINDING_SOURCE] + BINDING_HEADERS:
        with open(path, "rb") as f:
            h.update(f.read())
    return os.path.join(LIBDIR, f"_ops_{h.hexdigest()[:12]}.so")


def build_binding(force: bool = False) -> str:
    """Compile csrc/ops_binding.cpp against torch and the library; return its path."""
    binding = binding_path()
    if not force and os.path.exists(binding):
        return binding
    lib = build_library()
    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    tmp = binding + f".tmp{os.getpid()}"
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-o", tmp, BINDING_SOURCE,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
    for inc in (sysconfig.get_paths()["include"], os.path.join(home, "include"),
                os.path.join(home, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")):
        cmd += ["-isystem", inc]
    cmd += [lib, "-Wl,-rpath,$ORIGIN", "-L", os.path.join(home, "lib"), "-Wl,-rpath," + os.path.join(home, "lib"),
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")
    for old in glob.glob(os.path.join(LIBDIR, "_ops*.so")):
        with contextlib.suppress(FileNotFoundError):  # another process built it too
            os.remove(old)
    os.replace(tmp, binding)
    return binding


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose=True))
    print(build_binding(force="--force" in sys.argv))
