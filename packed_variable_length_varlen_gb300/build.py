"""Builds libvarlen_attn.so in-tree for sm_103a with nvcc.

``--bounds`` (``build(bounds=True)``) builds the bounds-checking variant into
``_build/bounds/libvarlen_attn.so``: the same sources compiled with
-DVARLEN_DEBUG_BOUNDS, whose kernels check every plain global access against
its operand's extent (load it by setting VARLEN_ATTN_LIB to that path).

Each .cu translation unit compiles in parallel to an object file, then nvcc
links them into one shared library with the CUDA runtime linked statically
(the library depends on no CUDA shared object at load time; the driver API
entry points it needs are fetched at run time).

binding() builds _varlen_binding, the native way from torch tensors into the
entry points around a step (csrc/varlen_binding.cpp, g++ against torch's
headers); a process that cannot load one for its torch, header and library goes
by ctypes alone.

    python -m packed_variable_length_varlen_gb300.build
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import platform
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libvarlen_attn.so")
BOUNDS_LIB = os.path.join(BUILD, "bounds", "libvarlen_attn.so")
HEADER = os.path.join(INCLUDE, "varlen_attn.h")
BINDING = os.path.join(BUILD, "_varlen_binding.so")
BINDING_SOURCE = os.path.join(CSRC, "varlen_binding.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
              "--expt-relaxed-constexpr", "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libvarlen_attn")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    return sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + [
        HEADER, os.path.abspath(__file__)]


def _digest(*paths) -> str | None:
    """Of the files' contents; None where one cannot be read."""
    h = hashlib.sha256()
    try:
        for path in paths:
            with open(path, "rb") as f:
                h.update(f.read() + b"\0")
    except OSError:
        return None
    return h.hexdigest()


def _stamp(path: str) -> str | None:
    try:
        with open(path) as f:
            return f.read().strip()
    except OSError:
        return None


def _put(tmp: str, path: str, stamps: dict) -> None:
    """A finished build in its place, with what says where it comes from: never beside what spoke for the one before."""
    for name in stamps:
        if os.path.exists(path + name):
            os.remove(path + name)
    os.replace(tmp, path)
    for name, text in stamps.items():
        with open(path + name, "w") as f:
            f.write(text)


def of_this_header(lib: str) -> bool:
    """Whether a library was compiled with the header that is here now."""
    digest = _digest(HEADER)
    return digest is not None and _stamp(lib + ".header") == digest


def up_to_date(lib: str | None = None) -> bool:
    lib = lib or LIB
    if not os.path.exists(lib) or _stamp(lib + ".arch") != platform.machine() or not of_this_header(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(d) <= t for d in _deps())


def _compile(src: str, verbose: bool, out_dir: str, defines=()) -> str:
    obj = os.path.join(out_dir, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *defines, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
    log = os.path.join(out_dir, os.path.basename(src)[:-3] + ".ptxas.txt")
    with open(log, "w") as f:
        f.write(r.stdout + r.stderr)
    if verbose:
        sys.stderr.write(r.stderr)
    return obj


def binding_tag() -> str:
    """What a built binding belongs to: machine type, Python, torch, and the header and source that it was compiled from
    (it calls the library by the header's struct layouts and argument lists)."""
    import torch
    return " ".join((platform.machine(), sys.implementation.cache_tag, torch.__version__,
                     _digest(HEADER, BINDING_SOURCE) or "no source"))


def _binding_current() -> bool:
    return (os.path.exists(BINDING) and _digest(HEADER, BINDING_SOURCE) is not None
            and _stamp(BINDING + ".tag") == binding_tag())


def binding_built(lib: str | None = None) -> bool:
    """Whether there is a binding for this Python, torch, header and library."""
    return _binding_current() and of_this_header(lib or LIB)


def binding(force: bool = False) -> str:
    """Compiles the native binding unless it is up to date; returns its path."""
    if not force and _binding_current() and os.path.getmtime(BINDING) >= os.path.getmtime(os.path.abspath(__file__)):
        return BINDING
    import torch
    os.makedirs(BUILD, exist_ok=True)
    if os.path.exists(BINDING + ".tag"):  # should this fail, the one before is not taken for it
        os.remove(BINDING + ".tag")
    tag = binding_tag()
    home = os.path.dirname(os.path.abspath(torch.__file__))
    dirs = (INCLUDE, os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"))
    tmp = BINDING + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), *["-I" + d for d in dirs], BINDING_SOURCE,
           "-o", tmp, "-L" + os.path.join(home, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed for %s:\n%s\n%s" % (cmd[0], BINDING_SOURCE, r.stdout, r.stderr))
    _put(tmp, BINDING, {".tag": tag})
    return BINDING


def build(force: bool = False, verbose: bool = False, bounds: bool = False) -> str:
    """Compile and link; returns the library path.  Skips work when the
    library is newer than every source and was built on this machine type with this header.
    ``bounds`` builds the bounds-checking variant (BOUNDS_LIB) instead."""
    lib = BOUNDS_LIB if bounds else LIB
    if not force and up_to_date(lib):
        return lib
    out_dir = os.path.dirname(lib)
    os.makedirs(out_dir, exist_ok=True)
    header = _digest(HEADER)
    defines = ["-DVARLEN_DEBUG_BOUNDS"] if bounds else []
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose, out_dir, defines), sources()))
    tmp = lib + ".tmp%d" % os.getpid()
    cmd = [nvcc(), *ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    _put(tmp, lib, {".arch": platform.machine(), ".header": header})
    return lib


if __name__ == "__main__":
    if "--bounds" not in sys.argv:
        print(binding(force="--force" in sys.argv))
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, bounds="--bounds" in sys.argv))
