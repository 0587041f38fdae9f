"""Build the native library ``libmoe_gb300.so`` in-tree for sm_103a.

Each CUDA translation unit is compiled to an object in parallel, then linked
into one shared library next to this file; beside it goes the extension module
that hands torch tensors to the decode-block calls, where torch, g++ and Python's
headers are there (the library needs none of them).  Objects are rebuilt only when a
source or header is newer, the extension also for another torch.  Set ``MOE_PTXAS_VERBOSE=1`` to print register and
shared-memory use per kernel.
"""

from __future__ import annotations

import concurrent.futures
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
OBJDIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_gb300.so")
BIND = os.path.join(PKG, "_block_bind.so")
SOURCES = ("api.cu", "route_dispatch.cu", "ffn.cu", "ffn_tc.cu", "balance.cu", "formp.cu",
           "block_api.cu", "norm.cu", "kv_append.cu", "attn_decode.cu", "lora_project.cu",
           "lora_gemv.cu")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("CUDA_HOME"), os.environ.get("CUDA_PATH"), "/usr/local/cuda"):
        if cand and os.path.exists(os.path.join(cand, "bin", "nvcc")):
            return os.path.join(cand, "bin", "nvcc")
    found = shutil.which("nvcc")
    if not found:
        raise RuntimeError("nvcc not found (set CUDA_HOME)")
    return found


def _headers():
    hs = [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    hs += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    return hs


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _run(cmd):
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError("command failed:\n" + " ".join(cmd) + "\n" + r.stdout)
    return r.stdout


def _bind_command():
    """(command, None) of the extension module, or (None, what it lacks on this machine)."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None, "torch"
    torch = os.path.dirname(spec.origin)
    include, lib, python = os.path.join(torch, "include"), os.path.join(torch, "lib"), sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "c10", "cuda", "CUDAStream.h")):
        return None, "a torch with CUDA"
    if shutil.which("g++") is None:
        return None, "g++"
    if not os.path.exists(os.path.join(python, "Python.h")):
        return None, "Python's headers"
    inc = [INCLUDE, include, os.path.join(include, "torch", "csrc", "api", "include"), python,
           os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")]
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", os.path.join(CSRC, "block_bind.cpp"), "-o", BIND]
            + [a for i in inc for a in ("-I", i)]
            + ["-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{lib}"]), None


def _read(path: str):
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return None


def _bind_stamp(cmd) -> str:
    """What the extension was built by and against: a torch of another version has another C++ ABI."""
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    return " ".join(cmd) + "\n" + (_read(os.path.join(torch, "version.py")) or "")


def build(force: bool = False, verbose: bool = False) -> str:
    nvcc = nvcc_path()
    os.makedirs(OBJDIR, exist_ok=True)
    headers = _headers()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-I", INCLUDE, "-I", CSRC]
    if os.environ.get("MOE_PTXAS_VERBOSE"):
        flags += ["-Xptxas", "-v"]
    jobs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(OBJDIR, src.replace(".cu", ".o"))
        if force or _stale(o, [s] + headers):
            jobs.append([nvcc, "-c", s, "-o", o] + flags)
    bind, lacks = _bind_command()
    if bind is None:
        print(f"decode-block calls not built: no {lacks}", file=sys.stderr)
    else:
        stamp_path, stamp = os.path.join(OBJDIR, "block_bind.stamp"), _bind_stamp(bind)
        if not force and _read(stamp_path) == stamp and not _stale(BIND, [os.path.join(CSRC, "block_bind.cpp")] + [
                os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]):
            bind = None
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(jobs) + 1) as ex:
        extension = ex.submit(_run, bind) if bind else None
        for out in ex.map(_run, jobs):
            if verbose or os.environ.get("MOE_PTXAS_VERBOSE"):
                sys.stdout.write(out)
    # the library needs nothing of the extension's, whose failure comes after it
    objs = [os.path.join(OBJDIR, s.replace(".cu", ".o")) for s in SOURCES]
    if force or jobs or _stale(LIB, objs):
        _run([nvcc, "-shared", "-cudart", "shared"] + ARCH + objs + ["-o", LIB])
    if extension:
        extension.result()
        with open(stamp_path, "w") as f:
            f.write(stamp)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
