"""Build step of the CUDA library: ``csrc/*.cu`` -> ``liblosa.so`` (in-tree), and
of the binding's native argument checks: ``csrc/torch_binding.cpp`` ->
``_binding.<torch and Python it is built for>.so``.

nvcc cross-compiles for sm_100a; no GPU is needed to build.  The library needs no
torch; without one the native argument checks are left out.
``python -m sparse_long_context_mse_b200.build`` rebuilds when a source or
header is newer than the library.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "liblosa.so")
BINDING_SRC = os.path.join(CSRC, "torch_binding.cpp")
OBJDIR = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def up_to_date() -> bool:
    if not os.path.exists(LIB) or _binding_stale():
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def binding_name():
    """File name of the native argument checks for this Python and torch: they are
    compiled against torch's C++ classes, so another version's are another file.
    None without torch."""
    try:
        import torch
    except ImportError:
        return None
    return "_binding.torch-%s.cxx11abi-%d%s" % (
        torch.__version__.replace("+", "-"), torch._C._GLIBCXX_USE_CXX11_ABI,
        sysconfig.get_config_var("EXT_SUFFIX"))


def _binding_deps():
    return [BINDING_SRC, os.path.join(INCLUDE, "losa.h"), os.path.abspath(__file__)]


def _binding_stale() -> bool:
    name = binding_name()
    if name is None:
        return False
    path = os.path.join(PKG, name)
    return not os.path.exists(path) or any(
        os.path.getmtime(p) > os.path.getmtime(path) for p in _binding_deps())


def build_binding(force: bool = False):
    """The native argument checks, against the installed torch's headers: their path,
    or None without torch."""
    name = binding_name()
    if name is None:
        sys.stderr.write("no torch: the native argument checks are not built\n")
        return None
    path = os.path.join(PKG, name)
    if not force and not _binding_stale():
        return path
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    tmp = path + ".tmp.%d" % os.getpid()
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-isystem", inc, "-isystem", cuda,
           "-I", sysconfig.get_paths()["include"], "-I", INCLUDE,
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, BINDING_SRC, "-o", tmp,
           "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-lc10_cuda"]  # (loaded already: the package imports torch first)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{res.stderr}")
    os.replace(tmp, path)
    return path


TRACE_LIB = os.path.join(PKG, "liblosa_trace.so")


def build(force: bool = False, verbose: bool = False, ptxas_v: bool = False,
          trace: bool = False) -> str:
    """The library; with ``trace`` a separate copy, ``liblosa_trace.so``,
    whose step kernel records per-phase timestamps (``phase_trace.py``)."""
    lib = TRACE_LIB if trace else LIB
    if not force and os.path.exists(lib) and all(
            os.path.getmtime(p) <= os.path.getmtime(lib) for p in _deps()):
        build_binding(force)
        return lib
    objdir = os.path.join(OBJDIR, "trace") if trace else OBJDIR
    os.makedirs(objdir, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_v else []
    if trace:
        extra.append("-DLOSA_PHASE_TRACE")

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [cc, *NVCC_FLAGS, *ARCH, *extra, "-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stderr}")
        if verbose or ptxas_v:
            sys.stderr.write(res.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = lib + ".tmp.%d" % os.getpid()
    subprocess.check_call([cc, *ARCH, "-shared", "-o", tmp, *objs])
    os.replace(tmp, lib)
    build_binding(force)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_v="-v" in sys.argv,
                trace="--trace" in sys.argv))
