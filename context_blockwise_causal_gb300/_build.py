"""Build step for libcpattn.so (the C-ABI library), in-tree, for sm_103a,
and for libcpattn_checked.so, the same library with the kernels' bounds
tests compiled in (-DCPATTN_CHECKS; see include/cpattn.h). The sources of both
compile in parallel.

Run ``python -m context_blockwise_causal_gb300._build`` or call ``build()``.
"""
import os
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG_DIR, "csrc")
LIB_PATH = os.path.join(PKG_DIR, "libcpattn.so")
CHECKED_LIB_PATH = os.path.join(PKG_DIR, "libcpattn_checked.so")
SOURCES = ["cpattn_api.cu", "window_api.cu", "qk_api.cu", "decode_api.cu"]
NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-O2"]


def _nvcc():
    for cand in (os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc"), "nvcc"):
        if os.path.sep not in cand or os.path.exists(cand):
            return cand
    return "nvcc"


def is_stale():
    """True when a library is missing or older than a source or header."""
    if not (os.path.exists(LIB_PATH) and os.path.exists(CHECKED_LIB_PATH)):
        return True
    built = min(os.path.getmtime(LIB_PATH), os.path.getmtime(CHECKED_LIB_PATH))
    inc = os.path.join(os.path.dirname(PKG_DIR), "include")
    for d in (CSRC, inc):
        for f in os.listdir(d):
            if os.path.getmtime(os.path.join(d, f)) > built:
                return True
    return False


def _run(cmds, verbose):
    """Runs the commands in parallel; raises for the first that fails."""
    if verbose:
        for cmd in cmds:
            print(" ".join(cmd), flush=True)
    procs = [(cmd, subprocess.Popen(cmd)) for cmd in cmds]
    failed = [cmd for cmd, proc in procs if proc.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])


def build(verbose=False):
    """Compile every CUDA source of the library into one shared object, and
    the checked build beside it."""
    objdir = os.path.join(PKG_DIR, "build")
    os.makedirs(objdir, exist_ok=True)
    compiles, links = [], []
    for out, extra, tag in ((LIB_PATH, [], ""), (CHECKED_LIB_PATH, ["-DCPATTN_CHECKS"], ".checked")):
        objs = []
        for src in SOURCES:
            obj = os.path.join(objdir, f"{os.path.splitext(src)[0]}{tag}.o")
            flags = [*NVCC_FLAGS, *extra] + (["-Xptxas=-v"] if verbose else [])
            compiles.append([_nvcc(), *flags, "-c", "-o", obj, os.path.join(CSRC, src)])
            objs.append(obj)
        links.append([_nvcc(), *NVCC_FLAGS, "-shared", "-o", out + ".tmp", *objs])
    _run(compiles, verbose)
    _run(links, verbose)
    for out in (LIB_PATH, CHECKED_LIB_PATH):
        os.replace(out + ".tmp", out)
    return LIB_PATH


if __name__ == "__main__":
    build(verbose="-v" in sys.argv)
    print(LIB_PATH)
