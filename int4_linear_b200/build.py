"""Build libfq.so in-tree with nvcc for sm_100a.

Usage: python -m int4_linear_b200.build   (or call build()).
"""
from __future__ import annotations

import fcntl
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libfq.so")
SOURCES = ["abi.cu", "quant.cu", "quant_int.cu", "gemm.cu", "linear.cu", "ternary.cu", "kv_cache.cu", "kv_attn.cu",
           "mx.cu", "mx_gemm.cu"]
HEADERS = ["fq_device.cuh", "fq_host.h", "kv_cache.cuh", "mx.cuh", os.path.join("..", "..", "include", "fq.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
]


def _nvcc() -> str:
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    p = os.path.join(cuda, "bin", "nvcc")
    return p if os.path.exists(p) else "nvcc"


def _stamp() -> str:
    """The file that names the compiler and flags of the objects beside it."""
    return os.path.join(HERE, "_build", "flags")


def _flags() -> str:
    return "\n".join([_nvcc(), *NVCC_FLAGS])


def _other_flags() -> bool:
    try:
        with open(_stamp()) as f:
            return f.read() != _flags()
    except OSError:
        return True


def _stale() -> bool:
    if not os.path.exists(LIB) or _other_flags():
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, s) for s in SOURCES] + [os.path.join(CSRC, h) for h in HEADERS]
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    # one process builds at a time; the others find its library (the lock goes with the file object)
    with open(os.path.join(objdir, "lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)
        if force or _stale():
            _build(objdir, force, verbose)
    return LIB


def _build(objdir: str, force: bool, verbose: bool) -> None:
    newest = max(os.path.getmtime(os.path.join(CSRC, h)) for h in HEADERS)
    force = force or _other_flags()
    if os.path.exists(_stamp()):
        os.remove(_stamp())  # until all objects are of one set of flags
    objs = [os.path.join(objdir, s.replace(".cu", ".o")) for s in SOURCES]

    def compile_one(job):
        src, obj = os.path.join(CSRC, job[0]), job[1]
        if not force and os.path.exists(obj) and os.path.getmtime(obj) > max(newest, os.path.getmtime(src)):
            return
        cmd = [_nvcc(), *NVCC_FLAGS, "-c", src, "-o", obj + ".tmp.o"]
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
        os.replace(obj + ".tmp.o", obj)  # an object that is there is whole

    with ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 1)) as pool:
        list(pool.map(compile_one, zip(SOURCES, objs)))
    with open(_stamp(), "w") as f:
        f.write(_flags())
    tmp = LIB + ".tmp"
    cmd = [_nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-cudart", "static", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
