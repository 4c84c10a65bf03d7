"""Build libmuon.so in-tree for sm_103a (nvcc, no cmake), and the compiled half
of layers.py against the installed PyTorch (host compiler), as a file that is
named for that PyTorch: another installation builds and loads another file.
Where PyTorch's parts for it are missing, libmuon.so is built alone.

Translation units are compiled in parallel into newton_schulz_05_gb300/_build
and linked into newton_schulz_05_gb300/libmuon.so.  The CUDA runtime is
linked statically; driver entry points are resolved at run time, so the
library loads on a machine without a GPU (symbols can be inspected there).
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
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmuon.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["plan.cpp", "step.cu", "dense.cu", "skinny.cu", "tc_gemm.cu", "noalloc.cu", "adamw.cu",
           "host.cu", "norm.cu", "norm_grad.cu", "dropout.cu", "route.cu"]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmuon")


def _flags(verbose_ptxas: bool):
    f = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC] + ARCH
    if verbose_ptxas:
        f += ["-Xptxas", "-v"]
    return f


def _deps_mtime() -> float:
    t = 0.0
    for d in (CSRC, os.path.join(ROOT, "include")):
        for fn in os.listdir(d):
            t = max(t, os.path.getmtime(os.path.join(d, fn)))
    return t


class Unavailable(Exception):
    """A part that the binding is built from is not installed."""


def binding_path() -> str:
    """Where the binding for this interpreter and the installed PyTorch is: both
    fix the ABI it is compiled against."""
    import torch
    return os.path.join(PKG, "_binding.%s-torch-%s-abi%d.so"
                        % (sys.implementation.cache_tag, torch.__version__,
                           int(torch._C._GLIBCXX_USE_CXX11_ABI)))


def _binding_current() -> bool:
    try:
        path = binding_path()
    except ImportError:
        return False
    return os.path.exists(path) and os.path.getmtime(path) >= _deps_mtime()


def _compile_binding() -> str:
    """The binding from binding.cpp; it is handed libmuon's entry points when
    it is loaded, so it links only with PyTorch."""
    import sysconfig

    try:
        import torch
    except ImportError as e:
        raise Unavailable("PyTorch cannot be imported (%s)" % e) from None
    home = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    compiler = shutil.which("g++")
    if compiler is None:
        raise Unavailable("g++ not found")
    python_include = sysconfig.get_paths()["include"]
    for part in (os.path.join(home, "include", "ATen", "core", "Tensor.h"),
                 os.path.join(home, "lib", "libc10_cuda.so"), os.path.join(python_include, "Python.h")):
        if not os.path.exists(part):
            raise Unavailable("%s not found" % part)
    path = binding_path()
    tmp = path + ".tmp%d" % os.getpid()
    cmd = [compiler, "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-w",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(home, "include"),
           "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-isystem", python_include,
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L", os.path.join(home, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("compiling the binding failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose_ptxas: bool = False, quiet: bool = True) -> str:
    lib_current = not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps_mtime()
    binding_current = not force and _binding_current()
    if lib_current and binding_current:
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    flags = _flags(verbose_ptxas)

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src + ".o")
        cmd = [nvcc] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        if src.endswith(".cpp"):
            cmd = [nvcc] + flags + ["-x", "cu", "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr))
        if not quiet or verbose_ptxas:
            sys.stderr.write(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = None if binding_current else ex.submit(_compile_binding)
        if not lib_current:
            objs = list(ex.map(compile_one, SOURCES))
            tmp = LIB + ".tmp%d" % os.getpid()
            cmd = [nvcc, "-shared", "-o", tmp] + objs + ARCH
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
            os.replace(tmp, LIB)
        try:
            if binding:
                binding.result()
        except Unavailable as e:
            sys.stderr.write("libmuon.so built; not the binding that layers.py needs: %s\n" % e)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv, quiet=False))
