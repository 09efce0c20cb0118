"""Build libctr.so (the CUDA path) in-tree for sm_103a.

Each .cu file under csrc/ is compiled by nvcc in parallel, then linked with the
static CUDA runtime into sparse_embeddings_feature_gb300/_build/libctr.so.
csrc/calls.cpp, which reads the arguments of small calls from tensors, is compiled
against the installed Python and PyTorch into _build/ctr_calls.so.  libctr needs
neither: where that fails (no Python headers, say) there is a warning, and the
binding in ctr.py serves every call.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libctr.so")
CALLS = os.path.join(OUT_DIR, "ctr_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-Wall", "-I", INCLUDE]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libctr")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _calls_command(out: str):
    import torch
    home = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    dirs = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
            os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
            *[a for d in dirs for a in ("-isystem", d)], os.path.join(CSRC, "calls.cpp"), "-o", out,
            "-L" + os.path.join(home, "lib"), "-L" + OUT_DIR,
            "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-lctr", "-Wl,-rpath,$ORIGIN"]


def _hash_files(h, paths) -> None:
    for p in paths:
        with open(p, "rb") as f:
            h.update(p.encode())
            h.update(f.read())


def _fingerprint(extra=()) -> str:
    h = hashlib.sha256()
    _hash_files(h, _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [os.path.join(INCLUDE, "ctr.h"), __file__])
    h.update(" ".join(ARCH + NVCC_FLAGS + list(extra)).encode())
    return h.hexdigest()


def _calls_fingerprint() -> str:
    """Of the extension's source, its compile command, and the Python and PyTorch it is for."""
    import torch
    try:
        command = _calls_command("")
    except RuntimeError:      # no CUDA toolkit: nothing can be compiled, but what is there may be used
        command = []
    h = hashlib.sha256(repr((sys.version, sysconfig.get_config_var("SOABI"), torch.__version__, command[:6])).encode())
    _hash_files(h, [os.path.join(CSRC, "calls.cpp"), os.path.join(INCLUDE, "ctr.h")])
    return h.hexdigest()


def build_calls(force: bool = False):
    """The extension's path, compiled if need be, or None where it cannot be (said once, by a warning)."""
    stamp = os.path.join(OUT_DIR, "calls_fingerprint")
    fp = _calls_fingerprint()
    seen = open(stamp).read() if os.path.exists(stamp) else ""
    if not force and seen == fp and os.path.exists(CALLS):
        return CALLS
    if not force and seen == fp + " failed":
        return None
    tmp = CALLS + ".tmp%d" % os.getpid()
    try:
        r = subprocess.run(_calls_command(tmp), capture_output=True, text=True)
        failed = f"{r.stdout}\n{r.stderr}" if r.returncode != 0 else ""
    except (OSError, RuntimeError) as e:
        failed = str(e)
    if failed:
        warnings.warn(f"calls.cpp was not compiled, the expert layer's calls read their arguments in Python:\n{failed}",
                      RuntimeWarning)
    else:
        os.replace(tmp, CALLS)
    with open(stamp, "w") as f:
        f.write(fp + (" failed" if failed else ""))
    return None if failed else CALLS


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    stamp = os.path.join(OUT_DIR, "fingerprint")
    extra_flags = list(extra_flags or []) + os.environ.get("CTR_NVCC_EXTRA", "").split()
    fp = _fingerprint(extra_flags)
    if not force and os.path.exists(LIB) and os.path.exists(stamp) and open(stamp).read() == fp:
        build_calls()
        return LIB
    cc = nvcc()
    flags = ARCH + NVCC_FLAGS + extra_flags

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src) + ".o")
        cmd = [cc, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 4))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs, "-lpthread", "-ldl", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    with open(stamp, "w") as f:
        f.write(fp)
    build_calls(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else None))
