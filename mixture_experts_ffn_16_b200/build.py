"""Build libmoe.so in-tree: every .cu under csrc/ compiled for sm_100a with nvcc
and linked into one shared library (CUDA runtime linked statically, so the
library loads on a machine without a GPU driver; it needs the driver only
when a kernel is launched).  And, where there is torch, the Python binding's
native part (csrc/fastcall.cpp), compiled with the host compiler against
torch's headers, whose layout of tensors it takes over: the file's name says
which torch and which Python it is for, and no other loads it."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmoe.so")
BUILD = os.path.join(HERE, "_build")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", INCLUDE]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    return sources() + sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)
                              if f.endswith((".cuh", ".h"))) + [os.path.join(INCLUDE, "moe.h")]


def _newer(out, deps):
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(p) <= t for p in deps)


def up_to_date():
    return _newer(LIB, _deps())


def fastcall_path() -> str:
    """Where the binding's native part for this torch and this Python is, or would be."""
    import torch
    abi = f"torch-{torch.__version__}-cxx11abi{int(torch.compiled_with_cxx11_abi())}"
    return os.path.join(HERE, f"_fastcall-{abi}{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_fastcall(force: bool = False, verbose: bool = False) -> str:
    import torch
    out = fastcall_path()
    src = os.path.join(CSRC, "fastcall.cpp")
    if not force and _newer(out, [src, os.path.join(INCLUDE, "moe.h")]):
        return out
    inc, libs = (os.path.join(os.path.dirname(torch.__file__), d) for d in ("include", "lib"))
    cuda = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
    tmp = out + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", INCLUDE, "-isystem", inc,
           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
           "-isystem", sysconfig.get_paths()["include"], src, "-o", tmp,
           "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, out)
    return out


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """The library, then the binding's native part.  The library needs neither torch nor that part, and the binding
    does without it: where it cannot be built there is a warning, and without torch nothing."""
    lib = build_library(force, verbose, ptxas_info)
    try:
        build_fastcall(force, verbose)
    except ImportError:
        pass
    except (OSError, subprocess.CalledProcessError) as e:
        warnings.warn(f"the binding's native part was not built, its calls will go through ctypes: {e}")
    return lib


def build_library(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    objs = []
    procs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [NVCC] + ARCH + FLAGS + (["-Xptxas", "-v"] if ptxas_info else []) + ["-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    failed = []
    for src, pr in procs:
        out, _ = pr.communicate()
        if out and (verbose or ptxas_info or pr.returncode):
            sys.stdout.write(out.decode(errors="replace"))
        if pr.returncode:
            failed.append(src)
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(failed))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv, ptxas_info="--ptxas-info" in sys.argv)
    print(LIB)
