"""Build libhm.so in-tree with nvcc for sm_100a.

Every .cu under csrc/ is compiled separately (in parallel) and linked into one
shared object with the CUDA runtime linked statically, so the library loads
without a GPU (its symbols can be inspected on a build host) and needs only
the driver on a GPU host.

csrc/marshal.cpp becomes the extension module _marshal.so beside it, with the
host compiler, against torch's headers and libraries.  It only saves the helpers
time, so where it cannot be built the library stands without it.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libhm.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
OBJDIR = os.path.join(HERE, "_build")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
                     "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
                     "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def marshal_tag() -> str:
    """What a build of csrc/marshal.cpp is good for: it reads torch's and Python's objects at the
    places that this torch and this Python have them."""
    import sys
    import torch
    return "torch %s abi %d %s" % (torch.__version__, torch._C._GLIBCXX_USE_CXX11_ABI, sys.implementation.cache_tag)


def build_marshal(force: bool = False) -> str:
    """Compile csrc/marshal.cpp into _marshal.so; returns its path."""
    src, stamp, tag = os.path.join(CSRC, "marshal.cpp"), os.path.join(OBJDIR, "marshal.tag"), marshal_tag()
    built = open(stamp).read() if os.path.exists(stamp) else ""
    if not force and built == tag and not _stale(MARSHAL, [src, os.path.join(INCLUDE, "hm.h")]):
        return MARSHAL
    import sysconfig
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = MARSHAL + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-w",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, '-DHM_MARSHAL_TAG="%s"' % tag, "-I", INCLUDE,
           "-I", os.path.join(base, "include"), "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-I", cuda, "-I", sysconfig.get_paths()["include"], src, "-o", tmp, "-L", os.path.join(base, "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s\n%s%s" % (" ".join(cmd), r.stdout, r.stderr))
    os.replace(tmp, MARSHAL)
    os.makedirs(OBJDIR, exist_ok=True)
    with open(stamp, "w") as f:
        f.write(tag)
    return MARSHAL


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile csrc/*.cu and link libhm.so, then build _marshal.so; returns the library's path."""
    os.makedirs(OBJDIR, exist_ok=True)
    srcs = _sources()
    hdrs = _headers()
    cc = nvcc()
    objs = []
    jobs = []
    for s in srcs:
        o = os.path.join(OBJDIR, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            cmd = [cc, *NVCC_FLAGS, *extra_flags, "-c", s, "-o", o]
            jobs.append(cmd)
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(8, len(jobs))) as ex:
            results = list(ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs))
        for cmd, r in zip(jobs, results):
            if verbose and (r.stdout or r.stderr):
                print(r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError("nvcc failed:\n%s\n%s%s" % (" ".join(cmd), r.stdout, r.stderr))
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n%s\n%s%s" % (" ".join(cmd), r.stdout, r.stderr))
        os.replace(tmp, LIB)
    try:
        build_marshal(force)
    except Exception as e:      # no torch, its headers or Python's, or no host compiler
        warnings.warn("_marshal.so was not built; the helpers fill their structs in Python: %s" % e, RuntimeWarning)
    return LIB


if __name__ == "__main__":  # pragma: no cover
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
