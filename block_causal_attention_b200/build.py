"""Build libbca.so (the C-ABI library) in-tree with nvcc for sm_100a, and, where there is a PyTorch
to build it for, the Python module that calls the library's paged cache."""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libbca.so")
BINDING = os.path.join(PKG, "_paged_binding.so")
BINDING_FOR = os.path.join(BUILD, "paged_binding.for")   # what BINDING was compiled against
SOURCES = ["api.cpp", "plan.cpp", "fwd.cu", "fwd_static.cu", "bwd.cu", "cp_passes.cu", "paged_api.cpp", "paged.cu",
           "paged_rows.cu", "paged_tiles.cu"]
HEADERS = ["plan.hpp", "kernels.hpp", "sm100.cuh", "prologue.cuh", "paged.hpp", "paged_device.cuh", "paged_mma.cuh"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
                     "-Xcompiler", "-fPIC,-O2,-Wall", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _read(path: str) -> str:
    if not os.path.exists(path):
        return ""
    with open(path) as f:
        return f.read()


def _torch_version() -> str:
    try:
        return importlib.metadata.version("torch")   # without the seconds that importing it takes
    except importlib.metadata.PackageNotFoundError:  # a source tree on the path
        import torch
        return torch.__version__


def _binding_lacks() -> str:
    """What the module's build needs and is not there, or nothing.  The library needs none of it."""
    if importlib.util.find_spec("torch") is None:
        return "PyTorch"
    if not os.path.exists(os.path.join(sysconfig.get_path("include"), "Python.h")):
        return "Python's headers"
    return ""


def _binding_command(target: str) -> list:
    """The Python module over torch tensors (csrc/paged_binding.cpp), against libbca.so."""
    import torch
    from torch.utils import cpp_extension as ext
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [f"-I{p}" for p in [*ext.include_paths(), sysconfig.get_path("include"), os.path.join(cuda, "include")]]
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w", *inc,
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            os.path.join(CSRC, "paged_binding.cpp"), "-o", target, f"-L{PKG}", "-l:libbca.so", f"-L{lib}",
            "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"]


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "bca.h")]
    jobs = []
    objs = []
    for s in SOURCES:
        src = os.path.join(CSRC, s)
        obj = os.path.join(BUILD, s + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + hdrs):
            cmd = [nvcc, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
            if verbose and s.endswith(".cu"):
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        return r.stdout + r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(jobs) or 1) as ex:
        for out in ex.map(run, jobs):
            if verbose and out:
                print(out)
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lpthread"])
        os.replace(tmp, LIB)
    header = os.path.join(ROOT, "include", "bca.h")
    lacks = _binding_lacks()
    versions = "" if lacks else f"torch {_torch_version()}, Python {sys.version}\n"
    if lacks:
        warnings.warn(f"libbca.so is built; the module of the paged cache is not: {lacks} not found. "
                      "PagedCache needs it, plans and the C ABI do not.")
    elif force or _stale(BINDING, [os.path.join(CSRC, "paged_binding.cpp"), header]) or _read(BINDING_FOR) != versions:
        tmp = BINDING + f".tmp{os.getpid()}"
        run(_binding_command(tmp))
        os.replace(tmp, BINDING)
        with open(BINDING_FOR, "w") as f:
            f.write(versions)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
