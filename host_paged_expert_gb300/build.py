"""Build libpe.so in-tree with nvcc for GB300 (sm_103a).

Every .cu file under csrc/ is compiled in parallel to an object file, then
linked into ``host_paged_expert_gb300/libpe.so``; the Python binding of the
dense operators (csrc/py_dense.cpp) becomes ``_dense.so`` next to it.  Run as
``python -m host_paged_expert_gb300.build`` or call ``build()``.
"""

from __future__ import annotations

import concurrent.futures
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpe.so")
PYEXT = os.path.join(PKG, "_dense.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if "-v" in extra and r.stderr:
        print(r.stderr, file=sys.stderr)
    return obj


def build(verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile and link libpe.so, then the Python binding; returns the
    library's path.  The library needs nvcc alone and is in place before the
    binding is asked for; a host without torch gets no binding."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    extra = list(extra or [])
    if verbose:
        extra += ["-Xptxas", "-v"]
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(12, len(srcs) + 1)) as ex:
        # the longest one first
        binding = ex.submit(_compile_binding) if importlib.util.find_spec("torch") else None
        objs = list(ex.map(lambda s: _compile(s, extra), srcs))
        _link(objs)
    if binding is None:
        print("torch is not installed: libpe.so is built, the Python binding of the dense operators is not", file=sys.stderr)
    else:
        _link_binding(binding.result())
    return LIB


def _link(objs: list[str]) -> None:
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def _compile_binding() -> str:
    """Compile the CPython binding of the dense operators."""
    import torch

    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        raise RuntimeError("no C++ compiler found")
    tinc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    obj = os.path.join(BUILD, "py_dense.o")
    cmd = [cxx, "-O1", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-Wno-sign-compare",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{sysconfig.get_paths()['include']}",
           f"-I{os.path.join(ROOT, 'include')}", f"-isystem{tinc}", f"-isystem{os.path.join(tinc, 'torch', 'csrc', 'api', 'include')}",
           f"-isystem{cuda}", "-c", os.path.join(CSRC, "py_dense.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling the binding failed:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    """Link it against libpe.so beside it and torch's libraries."""
    import torch

    tlib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = PYEXT + ".tmp"
    cmd = [shutil.which("g++") or "c++", "-shared", obj, f"-L{PKG}", "-l:libpe.so", f"-L{tlib}", "-ltorch_python", "-ltorch_cuda",
           "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking the binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, PYEXT)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
