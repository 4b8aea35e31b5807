"""Compile the CUDA sources under csrc/ into the in-tree libkda.so (sm_100a).

nvcc cross-compiles for sm_100a without a GPU.  The library links the CUDA
runtime statically and reaches the driver API through the runtime's
entry-point query, so it loads on a host without a GPU as well.
"""
import glob
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libkda.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin",
                        "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def build(force=False, verbose=False, extra=()):
    """Compiles the sources side by side (nvcc takes one core a source) and
    links them."""
    if not force and not _stale():
        return LIB
    tmp = LIB + ".tmp"

    def run(cmd):
        if verbose:
            print(" ".join(cmd))
        subprocess.check_call(cmd)

    with tempfile.TemporaryDirectory() as objs:
        def compile_one(src):
            obj = os.path.join(objs, os.path.basename(src) + ".o")
            run([nvcc(), *NVCC_FLAGS, *extra, "-I",
                 os.path.join(ROOT, "include"), "-c", "-o", obj, src])
            return obj
        with ThreadPoolExecutor(os.cpu_count() or 1) as pool:
            done = list(pool.map(compile_one, sources()))
        run([nvcc(), *NVCC_FLAGS[:2], "-shared", "-o", tmp, *done])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra=[a for a in sys.argv[1:] if a != "--force"]))
