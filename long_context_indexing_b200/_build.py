"""Builds liblsa.so in-tree: nvcc for sm_100a, static CUDA runtime.

Each .cu under csrc/ is compiled to an object in parallel, then linked into
long_context_indexing_b200/liblsa.so.  The library depends only on the CUDA
driver at run time (the runtime is linked statically), so loading it on a
host without a GPU succeeds; the first CUDA call then fails cleanly.

csrc/py/paged_binding.cpp, the binding of the paged cache's per-token calls, is
compiled against the installed torch and Python into _paged_binding with Python's own
suffix beside it.  It is optional: without torch or a C++ compiler that takes it, the
library is built all the same and those calls go through ctypes.
"""
import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "liblsa.so")
BINDING_SRC = os.path.join(CSRC, "py", "paged_binding.cpp")
BINDING = os.path.join(PKG, "_paged_binding" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
CXX = os.environ.get("CXX", "g++")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
         "--expt-relaxed-constexpr"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src, verbose_ptxas=False):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    if not _stale(obj, [src, *_headers()]):
        return obj, ""
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
    return obj, r.stderr


def _build_binding(force=False):
    torch = importlib.util.find_spec("torch")
    if torch is None:
        raise RuntimeError("no torch")
    torch_dir = torch.submodule_search_locations[0]
    version_py = os.path.join(torch_dir, "version.py")
    if not force and not _stale(BINDING, [BINDING_SRC, version_py, *_headers()]):
        return
    with open(version_py) as f:
        version = re.search(r"__version__ = ['\"]([^'\"]+)['\"]", f.read()).group(1)
    tmp = BINDING + ".tmp.%d" % os.getpid()
    inc = os.path.join(torch_dir, "include")
    cmd = [CXX, "-O2", "-fPIC", "-shared", "-std=c++17", '-DLSA_TORCH_VERSION="%s"' % version,
           "-I", INCLUDE, "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"), BINDING_SRC,
           "-o", tmp, "-L", os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s%s" % (CXX, r.stdout, r.stderr))
    os.replace(tmp, BINDING)


def _finish_binding(result):
    """Takes the outcome of _build_binding: where it failed there is no binding, not an old one."""
    any_python = os.path.join(os.path.dirname(BINDING), "_paged_binding.so")
    gone = [any_python] if any_python != BINDING else []
    try:
        result()
    except Exception as e:
        sys.stderr.write("warning: no compiled binding of the paged cache's calls (they go through "
                         "ctypes): %s\n" % e)
        gone.append(BINDING)
    for path in gone:
        if os.path.exists(path):
            os.remove(path)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compiles every CUDA source for sm_100a and links liblsa.so."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    if force:
        for s in srcs:
            o = os.path.join(BUILD, os.path.basename(s) + ".o")
            if os.path.exists(o):
                os.remove(o)
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        binding = ex.submit(_build_binding, force)
        results = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    objs = [o for o, _ in results]
    if verbose_ptxas:
        for (_, log), s in zip(results, srcs):
            if log:
                sys.stderr.write("== %s\n%s" % (os.path.basename(s), log))
    if _stale(LIB, objs):
        tmp = LIB + ".tmp.%d" % os.getpid()
        cmd = [NVCC, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
        os.replace(tmp, LIB)
    _finish_binding(binding.result)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
