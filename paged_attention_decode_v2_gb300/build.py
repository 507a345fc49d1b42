"""Build ``libpa.so`` (the C-ABI library) in-tree with nvcc for sm_103a, and
``_marshal.so`` (its torch argument marshalling, host code) with g++.

Each ``csrc/*.cu`` file is compiled in parallel into ``_build/``, then the
objects are linked into ``paged_attention_decode_v2_gb300/libpa.so``.  A file
is recompiled only when it or a header under ``csrc/`` or ``include/`` is
newer than its object.  ``_marshal.so`` serves Python callers only: where torch,
its headers or the host compiler are missing, ``libpa.so`` alone is built and the
reason goes to stderr.

Usage: ``python -m paged_attention_decode_v2_gb300.build [--force] [--verbose]
[--no-binding]``
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
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
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpa.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpa.so")


def _headers():
    return (glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
            glob.glob(os.path.join(INCLUDE, "*.h")))


def _flags(verbose: bool):
    f = ["-std=c++17", "-O3", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I", INCLUDE,
         "-I", CSRC, "--expt-relaxed-constexpr"]
    if verbose:
        f += ["-Xptxas", "-v"]
    return f


def binding_stamp() -> str:
    """What ``_marshal.so`` is compiled against: it reads tensors by the C++
    layout of one torch and one Python, and fits no other."""
    import torch

    return (f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}, "
            f"cxx11abi {int(torch.compiled_with_cxx11_abi())}")


def _cxx() -> str:
    return os.environ.get("CXX", "g++")


def _build_marshal(force: bool) -> None:
    """Compile and link ``csrc/marshal.cpp`` against torch's headers and libpa,
    where it is out of date or was compiled against something else."""
    import torch

    src, header = os.path.join(CSRC, "marshal.cpp"), os.path.join(INCLUDE, "pa.h")
    newest = max(os.path.getmtime(src), os.path.getmtime(header))
    version = subprocess.run([_cxx(), "-dumpfullversion"], capture_output=True, text=True).stdout
    stamp = f"{binding_stamp()}; {_cxx()} {version.strip()}"  # kept in the binary
    if not force and os.path.exists(MARSHAL) and os.path.getmtime(MARSHAL) >= newest:
        with open(MARSHAL, "rb") as f:
            if stamp.encode() + b"\0" in f.read():
                return
    troot = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = [_cxx(), "-std=c++17", "-O2", "-fPIC", "-shared",
           "-fvisibility=hidden", src, "-o", tmp, "-I", INCLUDE,
           "-isystem", os.path.join(troot, "include"),
           "-isystem", os.path.join(troot, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(cuda, "include"),
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           f'-DPA_MARSHAL_STAMP="{stamp}"',
           "-L", os.path.join(troot, "lib"), f"-Wl,-rpath,{os.path.join(troot, 'lib')}",
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
           "-L", PKG, "-l:libpa.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"build of _marshal.so failed:\n{r.stderr[-4000:]}")
    os.replace(tmp, MARSHAL)


def _no_binding() -> str | None:
    """Why ``_marshal.so`` cannot be built here, if so."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return "torch is not installed"
    if not os.path.exists(os.path.join(os.path.dirname(spec.origin), "include", "ATen", "core",
                                       "Tensor.h")):
        return "torch's headers are not installed"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers are not installed"
    if shutil.which(_cxx()) is None:
        return f"{_cxx()} is not installed"
    return None


def build(force: bool = False, verbose: bool = False, jobs: int | None = None,
          binding: bool = True) -> str:
    """Build what is out of date and return the path of ``libpa.so``."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    newest_header = max((os.path.getmtime(h) for h in _headers()), default=0.0)
    exe = nvcc()
    flags = _flags(verbose)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        if (not force and os.path.exists(obj) and
                os.path.getmtime(obj) >= max(os.path.getmtime(src), newest_header)):
            return obj, ""
        tmp = obj + f".tmp{os.getpid()}"
        r = subprocess.run([exe, *flags, "-c", src, "-o", tmp], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        os.replace(tmp, obj)
        return obj, r.stderr

    jobs = jobs or min(len(srcs), os.cpu_count() or 4)
    with cf.ThreadPoolExecutor(jobs) as ex:
        results = list(ex.map(compile_one, srcs))
    if verbose:
        for _, log in results:
            if log:
                sys.stderr.write(log)
    objs = [o for o, _ in results]
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < max(map(os.path.getmtime, objs)):
        tmp = LIB + f".tmp{os.getpid()}"
        r = subprocess.run([exe, "-shared", *ARCH, *objs, "-o", tmp, "-cudart", "static",
                            "-Xlinker", "-soname=libpa.so",
                            "-Xlinker", "-Bsymbolic", "-Xlinker", "--exclude-libs,ALL"],
                           capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link of libpa.so failed:\n{r.stderr}")
        os.replace(tmp, LIB)
    if binding:
        why = _no_binding()
        if why:
            sys.stderr.write(f"_marshal.so is not built: {why}\n")
        else:
            _build_marshal(force)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true", help="print ptxas register/spill reports")
    ap.add_argument("--no-binding", action="store_true", help="libpa.so only (nvcc alone)")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose, binding=not args.no_binding))
