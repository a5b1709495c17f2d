"""Build libulysses.so in-tree with nvcc for sm_103a (no cmake, no torch), and
the C++ marshalling of the binding's small calls (_fastcall-*.so, g++).

Each .cu file compiles to an object in parallel; one nvcc link makes the
shared library.  The CUDA runtime is linked statically, and the driver's
tensor-map encoder is fetched at run time, so the library needs only the
driver at load time.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libulysses.so")
# The bounds-checked variant (-DULYSSES_CHECKS): every kernel checks its
# global-memory indexes against the buffers' sizes, records a failed check in
# the device error word (ulysses_check returns ULYSSES_ERR_BOUNDS) and skips
# the access.  Same ABI; loaded instead of LIB when ULYSSES_CHECKED=1.
BUILD_CHECKED = os.path.join(PKG, "_build_checked")
LIB_CHECKED = os.path.join(PKG, "libulysses_checked.so")

# Marshalling of the strided calls; the binding works without it, slower.
FAST_SRC = os.path.join(PKG, "csrc_py", "fastcall.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _stale(lib: str, deps) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra=None, checked: bool = False) -> str:
    srcs = sources()
    lib_path = LIB_CHECKED if checked else LIB
    build_dir = BUILD_CHECKED if checked else BUILD
    deps = srcs + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    deps.append(os.path.join(INCLUDE, "ulysses.h"))
    deps.append(os.path.abspath(__file__))
    if not force and not _stale(lib_path, deps):
        return lib_path
    os.makedirs(build_dir, exist_ok=True)
    cc = nvcc()
    extra = list(extra or []) + (["-DULYSSES_CHECKS"] if checked else [])

    def compile_one(src):
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = lib_path + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-ldl", "-lpthread", "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib_path)
    return lib_path


def fastcall_path() -> str:
    """Where the marshalling for this interpreter and this torch is: it uses the
    layouts of both, so another's, left in the tree, must not be taken for it."""
    import torch
    return os.path.join(PKG, f"_fastcall-{sys.implementation.cache_tag}-torch{torch.__version__}.so")


def build_fastcall(force: bool = False) -> str:
    """Compile the marshalling with the host compiler, against the headers and
    libraries of the installed torch; raises with the compiler's words if that
    fails, and leaves none behind then."""
    path = fastcall_path()
    if not force and not _stale(path, [FAST_SRC, os.path.join(INCLUDE, "ulysses.h"), os.path.abspath(__file__)]):
        return path
    if os.path.exists(path):
        os.remove(path)
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = path + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + INCLUDE,
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(root, "include"),
           "-I" + os.path.join(root, "include", "torch", "csrc", "api", "include"), "-I" + os.path.join(cuda, "include"),
           FAST_SRC, "-o", tmp, "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
           "-ltorch_python"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"compiling {FAST_SRC} failed: {e}") from e
    if r.returncode != 0:
        raise RuntimeError(f"compiling {FAST_SRC} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)
    return path


def try_build_fastcall(force: bool = False) -> str | None:
    """build_fastcall; where it fails, its words on stderr and None: the calls
    are then marshalled in Python."""
    try:
        return build_fastcall(force)
    except RuntimeError as e:
        print(f"warning: no C++ marshalling of the strided calls (Python's serves): {e}", file=sys.stderr)
        return None


if __name__ == "__main__":
    try_build_fastcall(force="--force" in sys.argv)
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else None, checked="--checked" in sys.argv))
