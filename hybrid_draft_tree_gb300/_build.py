"""Build libgraft.so in-tree with nvcc for sm_103a (one translation unit per
kernel file, compiled in parallel, then linked)."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libgraft.so")
# the binding's per-layer calls, a CPython extension: its name holds the interpreter's ABI, so that one over the same tree
# with another ABI builds its own and loads no other's
FASTCALL = os.path.join(PKG, "_fastcall" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
OBJDIR = os.path.join(PKG, "_build")
SOURCES = ("api.cu", "assemble.cu", "scan.cu", "umax.cu", "select.cu", "coverage.cu", "sample.cu", "scan_tma.cu", "noalloc.cu",
           "cluster_select.cu", "logit_rules.cu", "kv.cu", "kv_append.cu", "kv_read.cu", "kv_attend.cu",
           "kv_attend_windowed.cu", "kv_attend_capped.cu", "kv_attend_biased.cu", "kv_attend_any.cu", "kv_attend_eight.cu",
           "kv_attend_eight_windowed.cu", "kv_attend_eight_capped.cu", "kv_attend_eight_biased.cu", "kv_attend_eight_any.cu")
NVCC_FLAGS = ["-O3", "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-lineinfo",
              "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]


def _newest_input() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "graft.h")]
    return max(os.path.getmtime(f) for f in files)


def build_fastcall(force: bool = False) -> str | None:
    """The extension, or None where Python's headers or a C compiler are missing (the binding then makes those calls
    itself)."""
    include = sysconfig.get_paths()["include"]
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None or not os.path.exists(os.path.join(include, "Python.h")):
        return None
    src = os.path.join(CSRC, "fastcall.c")
    newest = max(os.path.getmtime(src), os.path.getmtime(os.path.join(INCLUDE, "graft.h")))
    if not force and os.path.exists(FASTCALL) and os.path.getmtime(FASTCALL) >= newest:
        return FASTCALL
    tmp = FASTCALL + f".tmp{os.getpid()}"
    subprocess.check_call([cc, "-O2", "-fPIC", "-shared", "-I" + include, "-I" + INCLUDE, src, "-o", tmp])
    os.replace(tmp, FASTCALL)
    return FASTCALL


def build(force: bool = False, verbose: bool = False) -> str:
    build_fastcall(force)
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest_input():
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(OBJDIR, src.replace(".cu", ".o"))
        cmd = ["nvcc", *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call(["nvcc", "-shared", "-o", tmp, *[o for o, _ in results], "-lcudart", "-ldl"])
    os.replace(tmp, LIB)
    if verbose:
        for _, log in results:
            print(log)
    return LIB
