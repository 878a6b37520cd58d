"""Build libfp8q.so in-tree with nvcc for sm_100a (B200), and the binding's native part.

    python -m dequantisation_fp8q_token_b200.build [--force] [--verbose]

Each csrc/*.cu compiles to an object in _build/ (in parallel), then nvcc links
them into dequantisation_fp8q_token_b200/libfp8q.so with the CUDA runtime
linked statically, so the library needs only the driver at run time.
csrc/torch_ops.cpp (marshalling and autograd functions over the C ABI, no
device code) compiles with g++ against the installed torch into _fp8q_torch.so
beside it.
Flags keep IEEE semantics: no fast-math, precise division, denormals kept.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build", "libfp8q")
LIB = os.path.join(PKG, "libfp8q.so")
TORCH_SRC = os.path.join(CSRC, "torch_ops.cpp")
TORCH_EXT = os.path.join(PKG, "_fp8q_torch.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                     "-prec-div=true", "-ftz=false", "-prec-sqrt=true", "-fmad=false",
                     "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libfp8q needs the CUDA toolkit to build")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    hdrs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hdrs.append(os.path.join(INCLUDE, "fp8q.h"))
    return hdrs


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in sources() + _deps() + [__file__])


def torch_ext_tag() -> str:
    """What _fp8q_torch.so is built for; the module holds it as `built_for`."""
    import torch
    return f"fp8q for torch {torch.__version__}, cxx11 abi {int(torch.compiled_with_cxx11_abi())}, {sys.implementation.cache_tag}"


def torch_ext_up_to_date() -> bool:
    if not os.path.exists(TORCH_EXT):
        return False
    with open(TORCH_EXT, "rb") as f:
        if torch_ext_tag().encode() + b"\0" not in f.read():
            return False
    t = os.path.getmtime(TORCH_EXT)
    return all(os.path.getmtime(p) <= t for p in (TORCH_SRC, os.path.join(INCLUDE, "fp8q.h"), __file__))


def build_torch_ext(force: bool = False, verbose: bool = False) -> str:
    """_fp8q_torch.so, against libfp8q.so (found beside it at run time) and the installed torch."""
    if not force and torch_ext_up_to_date():
        return TORCH_EXT
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    cxx = shutil.which("g++") or "g++"
    tmp = TORCH_EXT + ".tmp.%d" % os.getpid()
    cuda_include = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-DTORCH_EXTENSION_NAME=_fp8q_torch",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch.compiled_with_cxx11_abi(), f'-DFP8Q_BUILT_FOR="{torch_ext_tag()}"',
           "-I", INCLUDE]
    for d in [*cpp_extension.include_paths(), cuda_include, sysconfig.get_paths()["include"]]:
        cmd += ["-isystem", d]
    cmd += [TORCH_SRC, "-o", tmp]
    for d in cpp_extension.library_paths():
        cmd += ["-L", d]
    cmd += ["-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-ltorch_python", "-L", PKG, "-l:libfp8q.so",
            "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed on {TORCH_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TORCH_EXT)
    return TORCH_EXT


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """libfp8q.so and _fp8q_torch.so, whichever is stale; the path of the former."""
    lib = build_lib(force, verbose, extra_flags)
    build_torch_ext(force, verbose)
    return lib


def build_lib(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    srcs = sources()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers / spills per kernel")
    a = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if a.ptxas_info else []
    print(build(force=a.force or a.ptxas_info, verbose=a.verbose or a.ptxas_info, extra_flags=extra))


if __name__ == "__main__":
    sys.exit(main())
