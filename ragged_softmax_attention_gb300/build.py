"""Build libfw_attn.so in-tree with nvcc for sm_103a (GB300).

Each .cu under csrc/ is compiled to an object in parallel, then linked into
one shared library with the CUDA runtime linked statically.  Objects are
rebuilt when their source or any header changed.  Beside it, g++ compiles
csrc/fast_binding.cpp against torch's headers into a module, the Python entry
points of the operators whose calls take a few microseconds.  Its file name holds
the versions it was compiled for, so that no other torch or interpreter loads it
(their objects may be laid out otherwise).  The library
does not depend on it: where the module cannot be compiled (no g++, no headers of
Python or torch), build() links the library all the same and warns.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfw_attn.so")
FAST_SRC = os.path.join(CSRC, "fast_binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; the CUDA 13 toolkit is required to build libfw_attn.so")


def _newest_header() -> float:
    hdrs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    return max((os.path.getmtime(h) for h in hdrs), default=0.0)


def fast_path() -> str:
    """The Python module's file for the running interpreter and its torch."""
    import sysconfig

    import torch
    return os.path.join(HERE, f"_fw_fast.{sysconfig.get_config_var('SOABI')}-torch-{torch.__version__}.so")


def _fast_command(out: str) -> list:
    """g++ command of the Python module: torch's and Python's headers and torch's
    libraries, at the versions of the running interpreter."""
    import sysconfig

    import torch
    cuda_home = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    torch_dir = os.path.dirname(torch.__file__)
    incs = [os.path.join(torch_dir, "include"), os.path.join(cuda_home, "include"), sysconfig.get_paths()["include"],
            os.path.join(ROOT, "include")]
    libdir = os.path.join(torch_dir, "lib")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", FAST_SRC, "-o", out,
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(f"-isystem{i}" for i in incs), f"-L{libdir}", f"-Wl,-rpath,{libdir}", "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch_python"]


def build(verbose: bool = False, force: bool = False, extra_flags=()) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_time = _newest_header()
    procs = []
    objects = []
    fast = fast_proc = fast_error = None
    try:
        fast = fast_path()
        fast_tmp = fast + f".tmp{os.getpid()}"
        if force or not os.path.exists(fast) or os.path.getmtime(fast) < max(
                os.path.getmtime(FAST_SRC), os.path.getmtime(os.path.join(ROOT, "include", "fw_attn.h"))):
            fast_cmd = _fast_command(fast_tmp)
            if verbose:
                print(" ".join(fast_cmd), flush=True)
            fast_proc = subprocess.Popen(fast_cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    except (ImportError, OSError) as e:                    # no torch, no g++
        fast_error = str(e)
    for src in sources:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objects.append(obj)
        stale = force or not os.path.exists(obj) or \
            os.path.getmtime(obj) < max(os.path.getmtime(src), hdr_time)
        if not stale:
            continue
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj + ".tmp"]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((obj, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for obj, pr in procs:
        out, _ = pr.communicate()
        text = out.decode(errors="replace")
        if pr.returncode != 0:
            failed.append((obj, text))
        else:
            os.replace(obj + ".tmp", obj)
            if verbose and text.strip():
                print(text, flush=True)
    if fast_proc is not None:
        out, _ = fast_proc.communicate()
        if fast_proc.returncode != 0:
            fast_error = out.decode(errors="replace")
        else:
            os.replace(fast_tmp, fast)
    if failed:
        msg = "\n".join(f"--- {o}\n{t}" for o, t in failed)
        raise RuntimeError(f"nvcc failed:\n{msg}")
    if procs or not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objects):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objects, "-cudart", "static"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        os.replace(tmp, LIB)
    if fast_error is not None:
        if fast and os.path.exists(fast):                  # made from older sources
            os.remove(fast)
        warnings.warn(f"{fast or '_fw_fast'} was not built, its Python entry points will raise:\n{fast_error}",
                      RuntimeWarning)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
