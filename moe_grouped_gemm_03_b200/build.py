"""Build libdg.so (the C-ABI library, CUDA for sm_100a) and _rowwise.so (the binding of the row-wise operators) in-tree."""
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libdg.so")
BINDING = os.path.join(HERE, "_rowwise.so")
SOURCES = [os.path.join(CSRC, "libdg.cu")]
BINDING_SOURCE = os.path.join(CSRC, "rowwise_binding.cpp")
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))] + \
    [os.path.join(INCLUDE, "dg.h")]
BINDING_DEPS = [BINDING_SOURCE, os.path.join(INCLUDE, "dg.h")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def flags(verbose: bool = False):
    f = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17", "--shared",
         "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "-I" + INCLUDE, "-I" + CSRC,
         "--expt-relaxed-constexpr"]
    if verbose:
        f += ["-Xptxas", "-v"]
    return f


def _newer(target, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(d) <= os.path.getmtime(target) for d in deps)


def up_to_date() -> bool:
    return _newer(LIB, DEPS) and _newer(BINDING, BINDING_DEPS)


def build_binding() -> None:
    """_rowwise.so: a CPython module against torch's headers, linked to libdg.so beside it."""
    import torch

    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    includes = [INCLUDE, os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] + ["-I" + i for i in includes] + \
        [BINDING_SOURCE, "-o", tmp, "-L" + HERE, "-l:libdg.so", "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(base, "lib"),
         "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose: bool = False) -> str:
    if force or not _newer(LIB, DEPS):
        tmp = LIB + ".tmp"
        cmd = [nvcc()] + flags(verbose) + SOURCES + ["-o", tmp]
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    if force or not _newer(BINDING, BINDING_DEPS):
        try:
            import torch  # noqa: F401
        except ImportError:  # the C library needs none of it
            print(f"no torch: {BINDING}, the Python binding of the row-wise operators, is not built", file=sys.stderr)
        else:
            build_binding()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
