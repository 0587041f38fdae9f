"""Build the native library ``libmoe_gb300.so`` in-tree for sm_103a.

Each CUDA translation unit is compiled to an object in parallel, then linked
into one shared library next to this file; beside it goes the extension module
that hands torch tensors to the decode-block calls.  Objects are rebuilt only when a
source or header is newer.  Set ``MOE_PTXAS_VERBOSE=1`` to print register and
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
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    inc = [INCLUDE, os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")]
    lib = os.path.join(torch, "lib")
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", os.path.join(CSRC, "block_bind.cpp"), "-o", BIND]
            + [a for i in inc for a in ("-I", i)]
            + ["-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{lib}"])


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
    compiled = list(jobs)
    if force or _stale(BIND, [os.path.join(CSRC, "block_bind.cpp")] + [
            os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]):
        jobs.append(_bind_command())
    if jobs:
        with concurrent.futures.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            for out in ex.map(_run, jobs):
                if verbose or os.environ.get("MOE_PTXAS_VERBOSE"):
                    sys.stdout.write(out)
    objs = [os.path.join(OBJDIR, s.replace(".cu", ".o")) for s in SOURCES]
    if force or compiled or _stale(LIB, objs):
        _run([nvcc, "-shared", "-cudart", "shared"] + ARCH + objs + ["-o", LIB])
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
