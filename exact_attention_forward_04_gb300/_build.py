"""Build the CUDA library in-tree with nvcc for sm_103a.

    python -m exact_attention_forward_04_gb300._build [--force]

Output: exact_attention_forward_04_gb300/_lib/libfa_fwd.so (git-ignored) and
fa_torch.so, a Python module that takes PyTorch tensors to some of its entry
points, and the ptxas resource report (registers, spills, shared memory) beside them.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(OUT_DIR, "libfa_fwd.so")
TORCH_PATH = os.path.join(OUT_DIR, "fa_torch.so")
ARCH = "-gencode=arch=compute_103a,code=sm_103a"
UNITS = ("fa_fwd.cu", "fa_cache.cu", "fa_cache4.cu", "fa_rope.cu")


def _sources():
    files = []
    for d in (CSRC, INCLUDE):
        for name in sorted(os.listdir(d)):
            if name.endswith((".cu", ".cuh", ".cpp", ".h")):
                files.append(os.path.join(d, name))
    return files


def _nvcc():
    cand = shutil.which("nvcc")
    if cand:
        return cand
    for p in ("/usr/local/cuda/bin/nvcc",):
        if os.path.exists(p):
            return p
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def needs_build() -> bool:
    if not (os.path.exists(LIB_PATH) and os.path.exists(TORCH_PATH)):
        return True
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(TORCH_PATH))
    return any(os.path.getmtime(f) > t for f in _sources())


def _torch_command(out):
    """The compiler's for fa_torch.so, against the installed PyTorch."""
    import torch
    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    include = [INCLUDE, os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(f"-I{p}" for p in include), os.path.join(CSRC, "fa_torch.cpp"), "-o", out, "-L" + os.path.join(at, "lib"),
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libfa_fwd.so if it is missing or older than its sources."""
    if not force and not needs_build():
        return LIB_PATH
    os.makedirs(OUT_DIR, exist_ok=True)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    flags = [ARCH, "-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
    jobs = []  # one compiler per translation unit, at the same time
    torch_tmp = TORCH_PATH + f".tmp{os.getpid()}"
    cmd = _torch_command(torch_tmp)
    jobs.append((cmd, None, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    for unit in UNITS:
        obj = os.path.join(OUT_DIR, f"{unit}.{os.getpid()}.o")
        cmd = [_nvcc(), *flags, "-Xptxas", "-v", "-c", "-o", obj, os.path.join(CSRC, unit)]
        jobs.append((cmd, obj, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    report, failed = "", False
    for cmd, _, proc in jobs:
        out = proc.communicate()[0]
        report += " ".join(cmd) + "\n" + out
        failed = failed or proc.returncode != 0
    objs = [obj for _, obj, _ in jobs if obj]
    if not failed:
        cmd = [_nvcc(), ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        report += " ".join(cmd) + "\n" + res.stdout + res.stderr
        failed = res.returncode != 0
    for obj in objs:
        if os.path.exists(obj):
            os.remove(obj)
    with open(os.path.join(OUT_DIR, "ptxas_report.txt"), "w") as f:
        f.write(report)
    if failed:
        raise RuntimeError("the build failed:\n" + report)
    os.replace(torch_tmp, TORCH_PATH)
    os.replace(tmp, LIB_PATH)
    if verbose:
        print(report)
    return LIB_PATH


if __name__ == "__main__":
    path = build(force="--force" in sys.argv, verbose=True)
    print(path)
