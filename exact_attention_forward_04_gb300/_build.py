"""Build the CUDA library in-tree with nvcc for sm_103a.

    python -m exact_attention_forward_04_gb300._build [--force]

Output: exact_attention_forward_04_gb300/_lib/libfa_fwd.so (git-ignored), the ptxas
resource report (registers, spills, shared memory) beside it and, where g++, Python's
and PyTorch's headers are there, fa_torch.so, a Python module that takes PyTorch
tensors to some of its entry points with less time on the host.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(OUT_DIR, "libfa_fwd.so")
TORCH_PATH = os.path.join(OUT_DIR, "fa_torch.so")
TORCH_FLAGS = ("-O2", "-std=c++17", "-fPIC", "-shared")
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


def _older(path, sources):
    return not os.path.exists(path) or any(os.path.getmtime(f) > os.path.getmtime(path) for f in sources)


def needs_build() -> bool:
    return _older(LIB_PATH, [f for f in _sources() if not f.endswith(".cpp")]) or _torch_stale()


def torch_key() -> str:
    """What fa_torch.so depends on beside its sources: PyTorch's C++ interface and
    Python's, and the compiler's flags."""
    import torch
    return f"PyTorch {torch.__version__}, {sysconfig.get_config_var('SOABI')}, {' '.join(TORCH_FLAGS)}"


def torch_built_for() -> str:
    """The torch_key that fa_torch.so was built for, as noted beside it."""
    try:
        with open(TORCH_PATH[:-3] + ".txt") as f:
            return f.read()
    except OSError:
        return ""


def _torch_stale() -> bool:
    sources = [os.path.join(CSRC, "fa_torch.cpp"), os.path.join(INCLUDE, "fa_fwd.h")]
    try:
        return _older(TORCH_PATH, sources) or torch_built_for() != torch_key()
    except ImportError:
        return True


def _torch_command(out):
    """The compiler's for fa_torch.so, against the installed PyTorch."""
    import torch
    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    include = [INCLUDE, os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    return ["g++", *TORCH_FLAGS, f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(f"-I{p}" for p in include), os.path.join(CSRC, "fa_torch.cpp"), "-o", out, "-L" + os.path.join(at, "lib"),
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _start(cmd):
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def _start_torch():
    """The compiler of fa_torch.so at work, and where it writes; None with the
    reason where there is none."""
    tmp = TORCH_PATH + f".tmp{os.getpid()}"
    try:
        return _start(_torch_command(tmp)), tmp
    except (ImportError, OSError, RuntimeError) as e:
        return None, str(e)


def _finish_torch(proc, tmp) -> str:
    """Puts fa_torch.so in its place; the compiler's output.  Where it cannot be
    built, the calls it serves go through Python: a warning, no error."""
    out = proc.communicate()[0] if proc else tmp
    if proc and proc.returncode == 0:
        note = TORCH_PATH[:-3] + ".txt"
        if os.path.exists(note):  # never beside a module that it is not about
            os.remove(note)
        os.replace(tmp, TORCH_PATH)
        with open(tmp, "w") as f:
            f.write(torch_key())
        os.replace(tmp, note)
    else:
        warnings.warn("fa_torch.so was not built, calls from PyTorch go through Python:\n" + out, stacklevel=3)
        if proc and os.path.exists(tmp):
            os.remove(tmp)
    return out


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libfa_fwd.so and fa_torch.so, where missing or older than their
    sources; fa_torch.so also where it is another PyTorch's or Python's."""
    os.makedirs(OUT_DIR, exist_ok=True)
    module = _start_torch() if force or _torch_stale() else None
    try:
        if force or _older(LIB_PATH, [f for f in _sources() if not f.endswith(".cpp")]):
            report = _build_library()
            if verbose:
                print(report)
    finally:
        if module:
            report = _finish_torch(*module)
            if verbose:
                print(report)
    return LIB_PATH


def _build_library() -> str:
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    flags = [ARCH, "-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]
    jobs = []  # one nvcc per translation unit, at the same time
    for unit in UNITS:
        obj = os.path.join(OUT_DIR, f"{unit}.{os.getpid()}.o")
        cmd = [_nvcc(), *flags, "-Xptxas", "-v", "-c", "-o", obj, os.path.join(CSRC, unit)]
        jobs.append((cmd, obj, _start(cmd)))
    report, failed = "", False
    for cmd, _, proc in jobs:
        out = proc.communicate()[0]
        report += " ".join(cmd) + "\n" + out
        failed = failed or proc.returncode != 0
    objs = [obj for _, obj, _ in jobs]
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
        if os.path.exists(tmp):
            os.remove(tmp)
        raise RuntimeError("nvcc failed:\n" + report)
    os.replace(tmp, LIB_PATH)
    return report


if __name__ == "__main__":
    path = build(force="--force" in sys.argv, verbose=True)
    print(path)
