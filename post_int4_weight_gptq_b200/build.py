"""Build the in-tree shared libraries with nvcc and g++: ``lib/libpiq.so`` (the
kernels and the C ABI, sm_100a) and ``lib/piq_serve.so`` (the Python entry of the
8-bit serving calls, ``csrc/serve_binding.cpp``, against torch's headers).

Usage: ``python -m post_int4_weight_gptq_b200.build [--force] [--verbose]``.
Sources are ``csrc/*.cu``; the C ABI is ``include/piq.h`` at the repository
root.  Objects are rebuilt when a source or header is newer than the library, the
binding also when Python or torch has changed.
"""
from __future__ import annotations

import argparse
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
LIBDIR = os.path.join(PKG, "lib")
OBJDIR = os.path.join(PKG, "_build")
LIB = os.path.join(LIBDIR, "libpiq.so")
SERVE = os.path.join(LIBDIR, "piq_serve.so")
SERVE_SRC = os.path.join(CSRC, "serve_binding.cpp")
SERVE_FOR = os.path.join(OBJDIR, "piq_serve.for")  # what piq_serve.so was built for
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-warn-spills"] + ARCH


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libpiq")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(CSRC, "*.h")) + [os.path.join(INCLUDE, "piq.h")]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _serve_for() -> str:
    """The Python and torch whose headers and libraries the binding is built against."""
    import torch
    return (f"python {sys.version}\ntorch {torch.__version__} {torch.version.git_version} "
            f"cxx11abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)}\n")


def serve_up_to_date() -> bool:
    if not os.path.exists(SERVE) or any(
            os.path.getmtime(p) > os.path.getmtime(SERVE)
            for p in (SERVE_SRC, os.path.join(INCLUDE, "piq.h"))):
        return False
    try:
        with open(SERVE_FOR) as f:
            return f.read() == _serve_for()
    except OSError:
        return False


def build_serve(force: bool = False) -> str:
    """The serving binding; needs libpiq.so to link to."""
    if not force and serve_up_to_date():
        return SERVE
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = SERVE + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", SERVE_SRC, "-o", tmp,
           "-I" + os.path.join(base, "include"),
           "-I" + os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-I" + os.path.join(cuda, "include"), "-I" + sysconfig.get_paths()["include"],
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
           "-lc10_cuda", "-lc10", "-L" + LIBDIR, "-lpiq", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {os.path.basename(SERVE_SRC)}:\n{r.stderr}")
    os.replace(tmp, SERVE)
    os.makedirs(OBJDIR, exist_ok=True)
    with open(SERVE_FOR, "w") as f:
        f.write(_serve_for())
    return SERVE


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    if not force and up_to_date():
        build_serve()
        return LIB
    os.makedirs(LIBDIR, exist_ok=True)
    os.makedirs(OBJDIR, exist_ok=True)
    flags = NVCC_FLAGS + list(extra_flags or [])
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
        cmd = [cc, "-c", src, "-o", obj, "-I", INCLUDE] + flags
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        if verbose and r.stderr.strip():
            print(r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + ".tmp"
    cmd = [cc, "-shared", "-o", tmp] + objs + ARCH + ["-lcudart_static", "-ldl", "-lpthread",
                                                      "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    build_serve(force)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-v", action="store_true", help="print register/smem usage")
    a = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if a.ptxas_v else []
    print(build(force=a.force or a.ptxas_v, verbose=a.verbose or a.ptxas_v, extra_flags=extra))


if __name__ == "__main__":
    main()
