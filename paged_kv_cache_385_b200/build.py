"""Build libpagedattn.so in-tree with nvcc for sm_100a (no GPU needed: nvcc cross-compiles), and the
binding's ``_views`` extension module with gcc.

    python paged_kv_cache_385_b200/build.py [--force] [--verbose] [--ptxas-v]

Run it as a file, not as ``-m paged_kv_cache_385_b200.build``: importing the package loads the
library, which is what this script produces.

Objects go to ``<package>/_build``; the shared library to ``<package>/libpagedattn.so``.
A rebuild happens when any source or header is newer than the library. The binding works without the
``_views`` extension: where it cannot be built (no gcc, no Python headers) the build warns and goes on.
"""
from __future__ import annotations

import argparse
import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpagedattn.so")
VIEWS_SOURCE = os.path.join(CSRC, "views.c")  # the binding's tensor marshalling, a CPython extension module
VIEWS = os.path.join(PKG, "_views" + sysconfig.get_config_var("EXT_SUFFIX"))

SOURCES = ["api.cu", "decode.cu", "decode_units.cu", "multiquery.cu", "prefill_tc.cu", "tree.cu", "tree_few.cu", "tree_commit.cu",
           "rope.cu", "cache.cu", "no_alloc.cu", "selftest.cu", "allocator.cpp"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-I" + INCLUDE, "-I" + CSRC,
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpagedattn.so")


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES]
    for d in (CSRC, INCLUDE):
        files += [os.path.join(d, f) for f in os.listdir(d) if f.endswith((".h", ".cuh"))]
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _views_up_to_date() -> bool:
    return os.path.exists(VIEWS) and all(os.path.getmtime(f) <= os.path.getmtime(VIEWS)
                                         for f in (VIEWS_SOURCE, os.path.join(INCLUDE, "pa.h")))


def _compile(src: str, verbose: bool, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc()] + ARCH + NVCC_FLAGS + list(extra) + ["-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, flush=True)
    return obj


def _build_views(verbose: bool) -> None:
    """The binding works without the extension, which saves a call about 6 us: no compiler or no Python headers
    is a warning."""
    tmp = VIEWS + ".tmp"
    cmd = ["gcc", "-O2", "-Wall", "-shared", "-fPIC", "-I" + sysconfig.get_paths()["include"], "-I" + INCLUDE, VIEWS_SOURCE,
           "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        said = None if r.returncode == 0 else r.stdout + r.stderr
    except OSError as e:
        said = str(e)
    if said is not None:
        warnings.warn(f"the _views extension was not built (the binding does without it): {said}", stacklevel=3)
        return
    os.replace(tmp, VIEWS)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile every source for sm_100a and link libpagedattn.so; returns its path."""
    if force or not up_to_date():
        _build_library(verbose, extra_flags)
    if force or not _views_up_to_date():
        _build_views(verbose)
    return LIB


def _build_library(verbose: bool, extra_flags) -> None:
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose, extra_flags), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-v", action="store_true", help="print registers / spills / shared memory per kernel")
    a = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if a.ptxas_v else []
    print(build(force=a.force or a.ptxas_v, verbose=a.verbose or a.ptxas_v, extra_flags=extra))
    return 0


if __name__ == "__main__":
    sys.exit(main())
