"""Build libnc.so in-tree for sm_100a with nvcc (one object per .cu, then link),
and _ncpy.so, the native part of the Python binding (csrc/nc_py.cpp), with g++.
Only the latter needs torch and Python's headers; without them it is left out.

    python -m decoder_only_transformer_fwd_b200.build [--force] [--verbose]

Objects go to decoder_only_transformer_fwd_b200/_build/, the library to
decoder_only_transformer_fwd_b200/libnc.so.  A source is recompiled when it or
any header under csrc/ or include/ is newer than its object.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libnc.so")
PYLIB = os.path.join(PKG, "_ncpy.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
                "-I", os.path.join(ROOT, "include"), "--expt-relaxed-constexpr"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h"))


def _stale(src, obj, hdr_mtime):
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return os.path.getmtime(src) > t or hdr_mtime > t


def build_py(force: bool = False, verbose: bool = False) -> str | None:
    """_ncpy.so against torch's headers and libraries (which are loaded by the time it is) and libnc.so beside it.
    None where torch or Python's headers are not installed: C users need neither."""
    torch = importlib.util.find_spec("torch")
    python_h = os.path.join(sysconfig.get_paths()["include"], "Python.h")
    if torch is None or not os.path.exists(python_h):
        sys.stderr.write(f"_ncpy.so (Python binding) is not built: no {'torch' if torch is None else python_h}\n")
        return None
    torch_dir = torch.submodule_search_locations[0]
    with open(os.path.join(torch_dir, "version.py")) as f:  # what it is built for: it loads with no other
        target = f"{sysconfig.get_config_var('EXT_SUFFIX')}\n{torch_dir}\n{f.read()}"
    src, built_for = os.path.join(CSRC, "nc_py.cpp"), os.path.join(OBJ, "_ncpy.target")
    newest = max(os.path.getmtime(f) for f in (src, os.path.join(ROOT, "include", "nc.h")))
    if not force and os.path.exists(PYLIB) and os.path.getmtime(PYLIB) > newest and os.path.exists(built_for):
        with open(built_for) as f:
            if f.read() == target:
                return PYLIB
    cuda = os.path.dirname(os.path.dirname(NVCC))
    include = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", *(f"-I{d}" for d in include), src, "-o", PYLIB,
           f"-L{torch_dir}/lib", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-L{PKG}", "-l:libnc.so",
           "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed:\n{r.stderr}")
    os.makedirs(OBJ, exist_ok=True)
    with open(built_for, "w") as f:
        f.write(target)
    if verbose:
        sys.stderr.write(f"[g++] nc_py.cpp\n{r.stderr}")
    return PYLIB


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    srcs = _sources()
    hdr_mtime = max((os.path.getmtime(h) for h in _headers()), default=0.0)
    objs = [os.path.join(OBJ, os.path.basename(s)[:-3] + ".o") for s in srcs]
    todo = [(s, o) for s, o in zip(srcs, objs) if force or _stale(s, o, hdr_mtime)]

    def compile_one(so):
        s, o = so
        cmd = [NVCC, *FLAGS, *(["-Xptxas", "-v"] if ptxas_info else []), "-c", s, "-o", o]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return s, r

    failed = []
    with cf.ThreadPoolExecutor(max_workers=min(8, max(1, len(todo)))) as ex:
        for s, r in ex.map(compile_one, todo):
            if r.returncode != 0:
                failed.append((s, r.stderr))
            elif verbose or ptxas_info:
                sys.stderr.write(f"[nvcc] {os.path.basename(s)}\n{r.stderr}")
    if failed:
        msg = "\n".join(f"--- {s}\n{err}" for s, err in failed)
        raise RuntimeError(f"nvcc failed:\n{msg}")
    if todo or not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs):
        cmd = [NVCC, *ARCH, "-shared", "-o", LIB, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
    build_py(force=force, verbose=verbose)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose, ptxas_info=a.ptxas_info))
