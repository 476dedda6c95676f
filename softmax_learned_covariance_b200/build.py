"""Build the Parallax CUDA library (libparallax.so) in-tree with nvcc for sm_100a.

    python -m softmax_learned_covariance_b200.build [--force] [--verbose]

Each csrc/*.cu is compiled to an object under _build/ (recompiled when it or a
header changed) and the objects are linked into a shared library next to this
file.  The CUDA runtime is linked statically so the library loads wherever the
NVIDIA driver is present; the driver API entry point for TMA descriptors is
resolved at run time.  csrc/binding.cpp, the native part of the Python binding,
becomes the extension module _binding.so next to it (g++ against torch's headers; the
library itself does not need torch and is built without it as well).
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libparallax.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(HERE, "_binding.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(src, obj, newest_header):
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return os.path.getmtime(src) > t or newest_header > t


def _built_against():
    """What _binding.so fits, as text: this torch and this Python; None without torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "?"
    return f"torch {version} {spec.origin} python {sysconfig.get_config_var('EXT_SUFFIX')}\n"


def build_binding(force: bool = False, verbose: bool = False) -> str | None:
    fits = _built_against()
    if fits is None:
        print("torch is not installed: the library is built, its Python binding is not", file=sys.stderr)
        return None
    header = os.path.join(INCLUDE, "parallax.h")
    stamp = os.path.join(BUILD, "binding.txt")
    fresh = os.path.exists(stamp) and open(stamp).read() == fits
    if not force and fresh and not _stale(BINDING_SRC, BINDING, os.path.getmtime(header)):
        return BINDING
    import torch
    from torch.utils import cpp_extension

    inc = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"], INCLUDE,
           os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-isystem{i}" for i in inc),
           BINDING_SRC, "-o", tmp, f"-L{libs}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python",
           f"-Wl,-rpath,{libs}"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        print(r.stdout + r.stderr, file=sys.stderr)
        raise RuntimeError("g++ failed for: " + BINDING_SRC)
    os.replace(tmp, BINDING)
    os.makedirs(BUILD, exist_ok=True)
    with open(stamp, "w") as f:
        f.write(fits)
    return BINDING


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    newest_header = max((os.path.getmtime(h) for h in _headers()), default=0.0)
    cc = nvcc()
    jobs = []
    for src in srcs:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        if force or ptxas_info or _stale(src, obj, newest_header):
            cmd = [cc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
            if ptxas_info:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append((src, cmd))
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def run(job):
        src, cmd = job
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, r

    failed = []
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        for src, r in ex.map(run, jobs):
            out = (r.stdout or "") + (r.stderr or "")
            if out.strip() and (verbose or ptxas_info or r.returncode):
                print(out, file=sys.stderr)
            if r.returncode:
                failed.append(src)
    if failed:
        raise RuntimeError(f"nvcc failed for: {failed}")
    if jobs or force or not os.path.exists(LIB):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs, "-lpthread", "-ldl", "-lrt"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        os.replace(tmp, LIB)
    build_binding(force, verbose)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers/spills/smem per kernel")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose, ptxas_info=a.ptxas_info))
