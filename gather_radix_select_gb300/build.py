"""Builds libsel.so (the CUDA kernels + C ABI) in-tree for sm_103a, and the Python module that calls its serving part.

    python -m gather_radix_select_gb300.build [--force] [--debug] [-v]

Each .cu under csrc/ is compiled by its own nvcc process (in parallel), then
the objects are linked into gather_radix_select_gb300/_lib/libsel.so with the
CUDA runtime linked statically, so the library needs only the driver.

--debug builds libsel_debug.so instead: the same sources with SEL_DEBUG
defined, whose kernels check selected accesses (staged-list and region
offsets, workspace slots, output positions, gathered key rows), skip the ones
that would leave their buffer and report SEL_EBOUNDS in err_flag.  It is
loaded instead of libsel.so when SEL_LIBRARY=debug is set.

csrc/binding.cpp, the module _binding, is compiled by g++ against the installed PyTorch and the running Python, whose
versions its folder's name has (its ABI goes with both).
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_lib")
SO = os.path.join(OUT_DIR, "libsel.so")
DEBUG_SO = os.path.join(OUT_DIR, "libsel_debug.so")
ROOT = os.path.dirname(HERE)
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if not f.startswith(".")]
    for where, _, names in os.walk(os.path.join(ROOT, "include")):
        files += [os.path.join(where, f) for f in names if f.endswith(".h")]
    return files


def up_to_date(so: str = SO) -> bool:
    if not os.path.exists(so):
        return False
    t = os.path.getmtime(so)
    return all(os.path.getmtime(f) <= t for f in _deps())


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None,
          debug: bool = False) -> str:
    so = DEBUG_SO if debug else SO
    if not force and up_to_date(so):
        return so
    obj_dir = os.path.join(OUT_DIR, "debug" if debug else "release")
    os.makedirs(obj_dir, exist_ok=True)
    cc = nvcc()
    flags = NVCC_FLAGS + (["-DSEL_DEBUG"] if debug else []) + list(extra_flags or [])
    objs = []
    cmds = []
    for src in sources():
        obj = os.path.join(obj_dir, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmds.append([cc, *ARCH, *flags, "-c", src, "-o", obj])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for " + cmd[-3])
        return r

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(cmds)) as ex:
        list(ex.map(run, cmds))
    tmp = so + ".tmp%d" % os.getpid()
    run([cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs])
    os.replace(tmp, so)
    return so


def binding_path() -> str:
    import torch
    return os.path.join(OUT_DIR, "binding-%s-%s" % (torch.__version__, sysconfig.get_config_var("SOABI")), "_binding.so")


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """The Python module of csrc/binding.cpp."""
    import torch
    so = binding_path()
    if not force and up_to_date(so):
        return so
    os.makedirs(os.path.dirname(so), exist_ok=True)
    home, cuda = os.path.dirname(torch.__file__), os.path.dirname(os.path.dirname(nvcc()))
    libs = os.path.join(home, "lib")
    tmp = so + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "c++", "-O2", "-std=c++17", "-shared", "-fPIC",
           "-fvisibility=hidden", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-isystem", os.path.join(home, "include"), "-isystem",
           os.path.join(home, "include", "torch", "csrc", "api", "include"), "-isystem", os.path.join(cuda, "include"),
           "-isystem", sysconfig.get_paths()["include"], "-L" + libs, "-Wl,-rpath," + libs, "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        if os.path.exists(so):
            os.remove(so)  # (an earlier build's would call a library that it does not know)
        raise RuntimeError("g++ failed for binding.cpp")
    os.replace(tmp, so)
    return so


def _binding_or_warning(force: bool = False, verbose: bool = False) -> list[str]:
    """The binding, or a warning of what is missing without it: the library's other calls go by ctypes."""
    try:
        return [build_binding(force=force, verbose=verbose)]
    except (RuntimeError, OSError) as e:
        warnings.warn("cache_append, and cache_attention with a window or a shared prefix, are not available: %s" % e,
                      RuntimeWarning, stacklevel=3)
        return []


def build_all(force: bool = False) -> list[str]:
    """libsel.so, libsel_debug.so and, where it can be built, the binding, compiled side by side."""
    with concurrent.futures.ThreadPoolExecutor(max_workers=2) as ex:
        jobs = [ex.submit(build, force=force), ex.submit(build, force=force, debug=True)]
        binding = _binding_or_warning(force)
        return [j.result() for j in jobs] + binding


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv))
    for so in _binding_or_warning(force="--force" in sys.argv, verbose="-v" in sys.argv):
        print(so)
