"""Build libctr.so (the CUDA path) in-tree for sm_103a.

Each .cu file under csrc/ is compiled by nvcc in parallel, then linked with the
static CUDA runtime into sparse_embeddings_feature_gb300/_build/libctr.so.
csrc/calls.cpp, which reads the arguments of small calls from tensors, is compiled
against the installed PyTorch into _build/ctr_calls.so.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import os
import shutil
import subprocess
import sys

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


def _calls_command(src: str, out: str):
    import sysconfig

    import torch
    home = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    dirs = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
            os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
            *[a for d in dirs for a in ("-isystem", d)], src, "-o", out, "-L" + os.path.join(home, "lib"), "-L" + OUT_DIR,
            "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-lctr", "-Wl,-rpath,$ORIGIN"]


def _fingerprint(extra=()) -> str:
    import torch
    h = hashlib.sha256(torch.__version__.encode())
    for p in sorted(glob.glob(os.path.join(CSRC, "*")) + [os.path.join(INCLUDE, "ctr.h"), __file__]):
        with open(p, "rb") as f:
            h.update(p.encode())
            h.update(f.read())
    h.update(" ".join(ARCH + NVCC_FLAGS + list(extra)).encode())
    return h.hexdigest()


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    stamp = os.path.join(OUT_DIR, "fingerprint")
    extra_flags = list(extra_flags or []) + os.environ.get("CTR_NVCC_EXTRA", "").split()
    fp = _fingerprint(extra_flags)
    if not force and os.path.exists(LIB) and os.path.exists(CALLS) and os.path.exists(stamp) and open(stamp).read() == fp:
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
    tmp = CALLS + ".tmp%d" % os.getpid()
    r = subprocess.run(_calls_command(os.path.join(CSRC, "calls.cpp"), tmp), capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"calls.cpp failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)
    with open(stamp, "w") as f:
        f.write(fp)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else None))
