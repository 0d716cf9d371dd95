"""Build libdspark.so in-tree with nvcc for sm_103a (GB300).

Each .cu file compiles in its own nvcc process (in parallel), then one link step makes
speculative_decoding_draft_markov_gb300/lib/libdspark.so.  No cmake, no torch extension:
the library exports a plain C ABI (include/dspark.h).  Beside it lib/_calls.so (csrc/calls.cpp, the
CPython C API): the Python calls that are made per layer and per token."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libdspark.so")
CALLS = os.path.join(LIBDIR, "_calls.so")
SOURCES = ["api.cu", "draft.cu", "draft_tc.cu", "decide_tc.cu", "sched_pack.cu", "verify.cu", "draft_noalloc.cu", "rnn.cu",
           "observe.cu", "serve_api.cu", "kv_append.cu", "window_attention.cu", "attention_windows.cu", "attention_prompts.cu",
           "logit_rules.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    for c in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(d) <= t for d in deps)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(ROOT, "include", "dspark.h"))
    objs, jobs = [], []
    for s in SOURCES:
        src = os.path.join(CSRC, s)
        obj = os.path.join(BUILD, s.replace(".cu", ".o"))
        objs.append(obj)
        if force or not _newer(obj, [src, *headers]):
            jobs.append([nvcc(), *ARCH, *FLAGS, *extra, "-c", src, "-o", obj])
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        for cmd, res in zip(jobs, ex.map(lambda c: subprocess.run(c, capture_output=True, text=True), jobs)):
            if verbose or res.returncode != 0:
                sys.stderr.write(" ".join(cmd) + "\n" + res.stdout + res.stderr)
            if res.returncode != 0:
                raise RuntimeError(f"nvcc failed on {cmd[-3]}")
    if force or jobs or not _newer(LIB, objs):
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", LIB, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            sys.stderr.write(res.stdout + res.stderr)
            raise RuntimeError("link of libdspark.so failed")
    _build_calls(force)
    return LIB


def _build_calls(force: bool) -> None:
    """lib/_calls.so.  Without Python's headers the library alone is built: its other calls need no extension module, and
    the calls that do need one say that it is missing."""
    src, include = os.path.join(CSRC, "calls.cpp"), sysconfig.get_paths()["include"]
    if not force and _newer(CALLS, [src, os.path.join(ROOT, "include", "dspark.h")]):
        return
    if not os.path.exists(os.path.join(include, "Python.h")):
        if os.path.exists(CALLS):
            os.remove(CALLS)  # of older sources
        sys.stderr.write(f"_calls.so is not built: no Python.h in {include}\n")
        return
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-I" + os.path.join(ROOT, "include"),
           "-I" + include, src, "-o", CALLS, "-L" + LIBDIR, "-ldspark", "-Wl,-rpath,$ORIGIN"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("build of _calls.so failed")


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
