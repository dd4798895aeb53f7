"""Build the sm_100a shared library ``libnq.so`` in-tree (nvcc, no JIT cache).

    python rank_binary_factorization_b200/build.py [--force]
"""
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libnq.so")
SOURCES = ["api.cu", "gemm_tc.cu", "kernels.cu", "chol.cu", "binary.cu", "calib_noalloc.cu",
           "selftest.cu", "w4.cu", "w4_tc.cu", "moe.cu"]
HEADERS = ["common.cuh", "gemm_tc.cuh", "kernels.cuh", "layout.h", "tc_ptx.cuh", "w4.cuh",
           os.path.join("..", "..", "include", "nq.h")]
NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC,-O2", "-Xptxas", "-v"]


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def stale():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def build(force=False, verbose=False):
    """Compile every CUDA source for sm_100a into libnq.so beside this file."""
    if not force and not stale():
        return LIB
    with tempfile.TemporaryDirectory() as tmp:
        objects = [os.path.join(tmp, f + ".o") for f in SOURCES]
        cmds = [[_nvcc()] + NVCC_FLAGS + ["-c", "-o", o, os.path.join(CSRC, f)]
                for f, o in zip(SOURCES, objects)]
        with ThreadPoolExecutor(os.cpu_count() or 1) as pool:
            runs = list(pool.map(lambda c: subprocess.run(c, capture_output=True, text=True), cmds))
        if all(r.returncode == 0 for r in runs):
            runs.append(subprocess.run([_nvcc()] + NVCC_FLAGS + ["-shared", "-o", LIB + ".tmp"] + objects,
                                       capture_output=True, text=True))
    for r in runs:
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("nvcc failed building libnq.so")
        if verbose:
            sys.stderr.write(r.stderr)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
    print(LIB)
