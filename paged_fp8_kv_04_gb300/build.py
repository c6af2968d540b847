"""Builds libpagedfp8.so for sm_103a with nvcc, and pa_torch.so (the torch side of the cache
operators' calls) with the host compiler, in-tree (paged_fp8_kv_04_gb300/_build/)."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libpagedfp8.so")
# The same library with the decode kernel's launch trace compiled in (pa_debug_trace).
TRACE_LIB_PATH = os.path.join(BUILD_DIR, "libpagedfp8_trace.so")
TORCH_SOURCE = os.path.join(CSRC, "pa_torch.cpp")
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpagedfp8")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        [os.path.join(INCLUDE, "pa.h"), os.path.abspath(__file__)]


def up_to_date(path: str = LIB_PATH, inputs: list[str] | None = None) -> bool:
    """Whether `path` is newer than its inputs (default: the library's), this file's flags among them."""
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(f) <= t for f in (inputs or _inputs()))


def torch_module_path() -> str:
    """The torch module is built against one torch and one interpreter: both are in the name."""
    import sysconfig

    import torch
    return os.path.join(BUILD_DIR, f"pa_torch.{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _torch_module_inputs() -> list[str]:
    return [TORCH_SOURCE, os.path.join(INCLUDE, "pa.h"), os.path.abspath(__file__)]


def _start_torch_module(force: bool):
    """Starts the compilation of pa_torch.cpp if it is due: (process, temporary file) or None."""
    import sysconfig

    import torch
    out = torch_module_path()
    if not force and up_to_date(out, _torch_module_inputs()):
        return None
    os.makedirs(BUILD_DIR, exist_ok=True)
    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = out + f".tmp{os.getpid()}"
    includes = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-I" + INCLUDE]
    for i in includes:
        cmd += ["-isystem", i]
    cmd += [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-o", tmp, TORCH_SOURCE,
            "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True), tmp, out


def build_all(force: bool = False) -> str:
    """libpagedfp8.so and pa_torch.so, side by side."""
    started = _start_torch_module(force)
    lib = build(force)
    if started is not None:
        proc, tmp, out = started
        text, _ = proc.communicate()
        if proc.returncode != 0:
            raise RuntimeError("pa_torch.cpp failed to compile:\n" + text)
        os.replace(tmp, out)
    return lib


def build(force: bool = False, verbose: bool = False, trace: bool = False) -> str:
    """Compile every .cu under csrc/ into one shared library (static cudart); with trace,
    the diagnostic variant whose decode kernel records its launch trace."""
    out = TRACE_LIB_PATH if trace else LIB_PATH
    if not force and up_to_date(out):
        return out
    os.makedirs(BUILD_DIR, exist_ok=True)
    tmp = out + f".tmp{os.getpid()}"
    cmd = [nvcc(), ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-shared",
           "-I" + INCLUDE, "-I" + CSRC, "-o", tmp] + (["-DPA_TRACE"] if trace else []) + sources()
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    if verbose:
        print(res.stdout + res.stderr)
    os.replace(tmp, out)
    return out
