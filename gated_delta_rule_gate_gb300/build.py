"""Builds libgdn.so (the CUDA library) in-tree for sm_103a, and _layer.so (the
native Python binding of the recurrent-layer operators).

Each .cu translation unit is compiled by nvcc in parallel, then linked into
one shared library next to this file.  Only sm_103a is targeted.  The binding is
one C++ file, compiled by g++ against the headers of Python and torch, whose
libraries are loaded already when it is; the library needs neither it nor them, and is
built whether or not it can be.
"""
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libgdn.so")
BINDING = os.path.join(HERE, "_layer.so")
OBJDIR = os.path.join(HERE, "_build")
STAMP = os.path.join(OBJDIR, "_layer.stamp")  # the Python and torch that the binding was built for

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgdn")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _newer(made, deps):
    return os.path.exists(made) and all(os.path.getmtime(d) <= os.path.getmtime(made) for d in deps)


def up_to_date():
    return _newer(LIB, _deps())


def _host():
    import torch
    return "python %s, torch %s in %s" % (sys.version, torch.__version__, os.path.dirname(torch.__file__))


def _binding_deps():
    return [os.path.join(CSRC, "layer_binding.cpp"), os.path.join(INCLUDE, "gdn.h"), os.path.abspath(__file__)]


def binding_up_to_date():
    if not _newer(BINDING, _binding_deps()) or not os.path.exists(STAMP):
        return False
    with open(STAMP) as f:
        return f.read() == _host()


def build_binding(force=False):
    if not force and binding_up_to_date():
        return BINDING
    import torch
    gxx = shutil.which("g++")
    if not gxx:
        raise RuntimeError("g++ not found: it is required to build the binding of the recurrent-layer operators")
    home = os.path.dirname(torch.__file__)
    inc = os.path.join(home, "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    tmp = BINDING + ".tmp%d" % os.getpid()
    cmd = [gxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch.compiled_with_cxx11_abi(), "-I", INCLUDE, "-isystem", inc, "-isystem",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", sysconfig.get_paths()["include"],
           "-isystem", cuda, os.path.join(CSRC, "layer_binding.cpp"), "-o", tmp, "-L", os.path.join(home, "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on layer_binding.cpp:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, BINDING)
    os.makedirs(OBJDIR, exist_ok=True)
    with open(STAMP, "w") as f:
        f.write(_host())
    return BINDING


def build_all(**kw):
    """Library and binding side by side; the library is there even where the binding fails."""
    with ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(build_binding, force=kw.get("force", False))
        lib = build(**kw)
        binding.result()
    return lib


def build(force=False, verbose=False, extra=()):
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(OBJDIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVFLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    srcs = _sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 4))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    args = sys.argv[1:]
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in args else []
    print(build_all(force="--force" in args or bool(extra), verbose=bool(extra), extra=extra))
