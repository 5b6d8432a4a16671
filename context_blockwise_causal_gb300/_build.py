"""Build step for libcpattn.so (the C-ABI library), in-tree, for sm_103a,
for libcpattn_checked.so, the same library with the kernels' bounds tests
compiled in (-DCPATTN_CHECKS; see include/cpattn.h), and for _binding.so, the
native half of the Python binding. All sources compile in parallel.

Run ``python -m context_blockwise_causal_gb300._build`` or call ``build()``.
"""
import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG_DIR, "csrc")
LIB_PATH = os.path.join(PKG_DIR, "libcpattn.so")
CHECKED_LIB_PATH = os.path.join(PKG_DIR, "libcpattn_checked.so")
BINDING_PATH = os.path.join(PKG_DIR, "_binding.so")
SOURCES = ["cpattn_api.cu", "window_api.cu", "qk_api.cu", "decode_api.cu"]
NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-O2"]


def _nvcc():
    for cand in (os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc"), "nvcc"):
        if os.path.sep not in cand or os.path.exists(cand):
            return cand
    return "nvcc"


def is_stale():
    """True when a built file is missing or older than a source or header."""
    outs = (LIB_PATH, CHECKED_LIB_PATH, BINDING_PATH)
    if not all(os.path.exists(p) for p in outs):
        return True
    built = min(os.path.getmtime(p) for p in outs)
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


def _binding_command(out):
    """Compiles csrc/binding.cpp against the installed PyTorch's C++ headers."""
    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(_nvcc()))))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            *(x for p in inc for x in ("-isystem", p)), os.path.join(CSRC, "binding.cpp"), "-o", out,
            "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]


def build(verbose=False):
    """Compile every CUDA source of the library into one shared object, the
    checked build beside it, and the native half of the Python binding."""
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
    compiles.append(_binding_command(BINDING_PATH + ".tmp"))
    _run(compiles, verbose)
    _run(links, verbose)
    for out in (LIB_PATH, CHECKED_LIB_PATH, BINDING_PATH):
        os.replace(out + ".tmp", out)
    return LIB_PATH


if __name__ == "__main__":
    build(verbose="-v" in sys.argv)
    print(LIB_PATH)
