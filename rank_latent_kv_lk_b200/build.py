"""Builds liblk.so (the C-ABI library) in-tree with nvcc for sm_100a.

Usage: python rank_latent_kv_lk_b200/build.py [--force] [--verbose] [--ptxas-info]
(run as a script: importing the package would load the library it builds).

Each .cu file compiles to an object under ``_build/`` (in parallel), then the
objects link into ``rank_latent_kv_lk_b200/liblk.so``; the torch binding of the
serving operators (``csrc/lk_serving_py.cpp``) compiles with g++ into
``_serving_ext.so`` beside it.  Objects are rebuilt when their source or any
header is newer, the binding also for another Python or torch than it was built
for (kept in ``_build/``); without torch it is left out.  IEEE fp32 semantics are kept
(no fast-math, no flush-to-zero): the latent quantiser is bit-exact.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "liblk.so")
EXT_SRC = os.path.join(CSRC, "lk_serving_py.cpp")
EXT = os.path.join(PKG, "_serving_ext.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
    "-ftz=false", "-prec-div=true", "-prec-sqrt=true",
    "-I", INCLUDE, "-I", CSRC,
]


def _nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build liblk.so")
    return cand


def _newest_header():
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _compile(src, obj, verbose, extra):
    cmd = [_nvcc(), *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{p.stdout}\n{p.stderr}")
    return p.stderr


def _build_ext(force, verbose):
    """The torch binding; links against liblk.so beside it."""
    import importlib.metadata
    import importlib.util
    import sysconfig
    spec = importlib.util.find_spec("torch")
    if spec is None:
        print("torch is not installed: liblk.so stands alone, without the binding of the serving operators", flush=True)
        return
    deps = [EXT_SRC, os.path.join(INCLUDE, "lk.h"), os.path.join(INCLUDE, "lk_serving.h")]
    built_for = f"python {sys.version_info[:2]} torch {importlib.metadata.version('torch')} {spec.origin}\n"
    stamp = os.path.join(BUILD, "serving_ext.txt")

    def stamped():
        if not os.path.exists(stamp):
            return ""
        with open(stamp) as f:
            return f.read()

    if not force and os.path.exists(EXT) and stamped() == built_for and \
            os.path.getmtime(EXT) >= max(os.path.getmtime(d) for d in deps):
        return
    import torch
    from torch.utils import cpp_extension
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [INCLUDE, sysconfig.get_paths()["include"], os.path.join(cuda, "include"), *cpp_extension.include_paths()]
    libs = cpp_extension.library_paths()
    tmp = EXT + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-DTORCH_EXTENSION_NAME=_serving_ext",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{d}" for d in inc], EXT_SRC,
           "-o", tmp, f"-L{PKG}", "-l:liblk.so", "-Wl,-rpath,$ORIGIN", *[f"-L{d}" for d in libs],
           "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"g++ failed on {os.path.basename(EXT_SRC)}:\n{p.stdout}\n{p.stderr}")
    os.replace(tmp, EXT)
    with open(stamp, "w") as f:
        f.write(built_for)


def build(force=False, verbose=False, extra_flags=()):
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_time = _newest_header()
    jobs = []
    objs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or not os.path.exists(o) or os.path.getmtime(o) < max(os.path.getmtime(s), hdr_time):
            jobs.append((s, o))
    logs = []
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            futs = [ex.submit(_compile, s, o, verbose, list(extra_flags)) for s, o in jobs]
            for f in futs:
                logs.append(f.result())
    if jobs or not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + ".tmp"
        cmd = [_nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
        p = subprocess.run(cmd, capture_output=True, text=True)
        if p.returncode != 0:
            raise RuntimeError(f"link failed:\n{p.stdout}\n{p.stderr}")
        os.replace(tmp, LIB)
    _build_ext(force, verbose)
    for log in logs:
        if log.strip() and verbose:
            print(log)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers / spills per kernel")
    args = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if args.ptxas_info else []
    if args.ptxas_info:
        os.makedirs(BUILD, exist_ok=True)
        for s in sorted(glob.glob(os.path.join(CSRC, "*.cu"))):
            o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
            print(_compile(s, o, args.verbose, extra))
    print(build(force=args.force, verbose=args.verbose))
    return 0


if __name__ == "__main__":
    sys.exit(main())
