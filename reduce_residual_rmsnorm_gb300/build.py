"""Build the CUDA library ``libts_fused_norm.so`` in-tree with nvcc (sm_103a only).

Each ``csrc/*.cu`` translation unit is compiled in parallel, then linked into
one shared object with the CUDA runtime linked statically, so the library
loads on any machine with a CUDA driver.  No fast-math: IEEE division and
square root, denormals kept (the quantisers depend on them).  Beside it
``_python_calls.so`` (g++ against the installed PyTorch) marshals the calls of
``_nvfp4_moe``.  The library needs none of PyTorch: it is linked first, and
alone where no PyTorch with CUDA is installed.
"""
from __future__ import annotations

import concurrent.futures as cf
import fcntl
import glob
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libts_fused_norm.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
CALLS_SRC = os.path.join(CSRC, "python_calls.cpp")
CALLS_PATH = os.path.join(PKG, "_python_calls.so")
BUILD_DIR = os.path.join(PKG, "_build")
CALLS_STAMP = "python_calls.built_for"  # in BUILD_DIR

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "-Xcompiler", "-fvisibility=hidden",
              "-ftz=false", "-prec-div=true", "-prec-sqrt=true", "--expt-relaxed-constexpr",
              "-Xptxas", "-warn-spills", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return path


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(path: str, deps: list[str]) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(d) <= t for d in deps)


def _common_deps() -> list[str]:
    return glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def library_up_to_date() -> bool:
    return _newer(LIB_PATH, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  _common_deps())


def _calls_for() -> str:
    """What the compiled calls are bound to: the layout of PyTorch's tensors and Python's objects."""
    import torch

    return "PyTorch %s, CXX11 ABI %d, %s" % (torch.__version__, int(torch._C._GLIBCXX_USE_CXX11_ABI),
                                             sysconfig.get_config_var("SOABI"))


def calls_match() -> bool:
    """Whether the compiled calls were built for the installed PyTorch and this Python."""
    try:
        with open(os.path.join(BUILD_DIR, CALLS_STAMP), encoding="utf-8") as f:
            return f.read() == _calls_for()
    except OSError:
        return False


def calls_up_to_date() -> bool:
    return _newer(CALLS_PATH, [CALLS_SRC] + _common_deps()) and calls_match()


def calls_wanted() -> bool:
    """Whether there is a PyTorch whose CUDA tensors the compiled calls could take."""
    try:
        import torch
    except ImportError:
        return False
    return torch.version.cuda is not None


def up_to_date() -> bool:
    return library_up_to_date() and (not calls_wanted() or calls_up_to_date())


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    # one build at a time: processes started together (torchrun ranks, test
    # workers) share the object files; the later ones find the library built
    with open(os.path.join(BUILD_DIR, ".lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)
        if not force and up_to_date():
            return LIB_PATH
        calls = calls_wanted() and (force or not calls_up_to_date())
        with cf.ThreadPoolExecutor(max_workers=1) as ex:
            # compiled beside the library, whose link waits for none of it
            calls_obj = ex.submit(_compile_calls) if calls else None
            if force or not library_up_to_date():
                _build_library(verbose, extra_flags)
            if calls_obj is not None:
                _link_calls(calls_obj.result())
        return LIB_PATH


def _compile_calls() -> str:
    """The object file of python_calls.cpp."""
    import torch

    top = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    obj = os.path.join(BUILD_DIR, "python_calls.cpp.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), "-I", INCLUDE,
           "-isystem", os.path.join(top, "include"),
           "-isystem", os.path.join(top, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"],
           "-c", CALLS_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {CALLS_SRC}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_calls(obj: str) -> None:
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = CALLS_PATH + ".tmp%d" % os.getpid()
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:" + LIB_NAME, "-Wl,-rpath,$ORIGIN", "-L", lib,
           "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of {CALLS_PATH} failed:\n{r.stdout}\n{r.stderr}")
    stamp = os.path.join(BUILD_DIR, CALLS_STAMP)
    if os.path.exists(stamp):
        os.remove(stamp)  # (it never stands beside calls built for another PyTorch)
    os.replace(tmp, CALLS_PATH)
    with open(stamp, "w", encoding="utf-8") as f:
        f.write(_calls_for())


def _build_library(verbose: bool, extra_flags: list[str] | None) -> None:
    cc = nvcc()
    flags = NVCC_FLAGS + (extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB_PATH + ".tmp%d" % os.getpid()
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "-v" in sys.argv else None))
