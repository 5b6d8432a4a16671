"""Build step for libcpattn.so (the C-ABI library), in-tree, for sm_103a,
for libcpattn_checked.so, the same library with the kernels' bounds tests
compiled in (-DCPATTN_CHECKS; see include/cpattn.h), and for _binding.so, the
native half of the Python binding. All sources compile in parallel. The two
libraries need nvcc alone and are put in place whatever becomes of the
binding, which needs the C++ headers of Python and PyTorch besides.

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
    """True when a built file is missing or older than a source or header (the
    binding only where it can be built)."""
    outs = (LIB_PATH, CHECKED_LIB_PATH) + (() if _binding_lacks() else (BINDING_PATH,))
    if not all(os.path.exists(p) for p in outs):
        return True
    if BINDING_PATH in outs and binding_made_for() != _made_for():
        return True
    built = min(os.path.getmtime(p) for p in outs)
    inc = os.path.join(os.path.dirname(PKG_DIR), "include")
    for d in (CSRC, inc):
        for f in os.listdir(d):
            if os.path.getmtime(os.path.join(d, f)) > built:
                return True
    return False


def _made_for():
    """What the binding's machine code depends on: it uses PyTorch's and Python's
    own C++ interfaces, which change with every version."""
    import torch

    return f"torch {torch.__version__} {sysconfig.get_config_var('SOABI')}"


def binding_made_for():
    """The versions that the binding was built for ("" when not recorded)."""
    try:
        with open(BINDING_PATH + ".txt") as f:
            return f.read()
    except OSError:
        return ""


def check_binding():
    """Raises where the binding is missing or made for another PyTorch or
    Python than the ones that run."""
    if not os.path.exists(BINDING_PATH):
        raise RuntimeError(f"{BINDING_PATH} is missing: build it with context_blockwise_causal_gb300.build() (it needs "
                           "g++ and the C++ headers of Python and PyTorch)")
    if binding_made_for() != _made_for():
        raise RuntimeError(f"{BINDING_PATH} was built for '{binding_made_for()}' and this is '{_made_for()}': build it "
                           "again with context_blockwise_causal_gb300.build()")


def _start(cmds, verbose):
    """Starts the commands in parallel."""
    if verbose:
        for cmd in cmds:
            print(" ".join(cmd), flush=True)
    return [(cmd, subprocess.Popen(cmd)) for cmd in cmds]


def _wait(procs):
    """Waits for all of them; raises for the first that fails."""
    failed = [cmd for cmd, proc in procs if proc.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])


def _binding_includes():
    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(_nvcc()) or _nvcc())))
    return [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
            os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]


def _binding_lacks():
    """What the machine lacks for compiling the binding, or None."""
    if shutil.which("g++") is None:
        return "g++"
    inc = _binding_includes()
    for header in ("Python.h", "cuda_runtime_api.h", os.path.join("torch", "csrc", "autograd", "python_variable.h")):
        if not any(os.path.exists(os.path.join(d, header)) for d in inc):
            return header
    return None


def _binding_command(out):
    """Compiles csrc/binding.cpp against the installed PyTorch's C++ headers."""
    import torch

    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            *(x for p in _binding_includes() for x in ("-isystem", p)), os.path.join(CSRC, "binding.cpp"), "-o", out,
            "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
            "-ltorch_python"]


def build(verbose=False):
    """Compile every CUDA source of the library into one shared object, the
    checked build beside it, and the native half of the Python binding.

    The libraries are in place before anything about the binding is reported.
    Where its compiler or headers are missing it is left out, with a line on
    stderr (the Python calls that need it raise); where its compilation fails,
    this raises. Either way no older binding stays beside the new library."""
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
    lacks = _binding_lacks()
    binding = [] if lacks else _start([_binding_command(BINDING_PATH + ".tmp")], verbose)
    try:
        _wait(_start(compiles, verbose))
        _wait(_start(links, verbose))
        for out in (LIB_PATH, CHECKED_LIB_PATH):
            os.replace(out + ".tmp", out)
        if os.path.exists(BINDING_PATH):
            os.remove(BINDING_PATH)
    finally:
        for _, proc in binding:
            proc.wait()
    if lacks:
        print(f"{BINDING_PATH} is not built ({lacks} is missing): the C library is complete, the Python calls for "
              "rotations, norms, windows and decoding need it", file=sys.stderr)
        return LIB_PATH
    _wait(binding)
    with open(BINDING_PATH + ".txt", "w") as f:
        f.write(_made_for())
    os.replace(BINDING_PATH + ".tmp", BINDING_PATH)
    return LIB_PATH


if __name__ == "__main__":
    build(verbose="-v" in sys.argv)
    print(LIB_PATH)
