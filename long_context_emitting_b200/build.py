"""Build libkascade.so in-tree with nvcc for sm_100a.

Usage: python -m long_context_emitting_b200.build [--force]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libkascade.so")
# CPython module: calls of the decode step's small entry points.  Its name carries the interpreter's
# tag, so that another Python of the same checkout neither imports it nor takes it for its own.
HOSTCALL = os.path.join(HERE, "_hostcall" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ["api.cu", "decode.cu", "topk.cu", "prefill.cu", "noalloc.cu", "calib.cu", "selftest.cu",
           "norm_rope.cu", "cache_q4.cu", "decode_q4.cu"]
HEADERS = ["common.cuh", "internal.h", "tcgen05.cuh", "exp2_poly.cuh", "f32x2.cuh", "q4.cuh"]

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills", f"-I{os.path.join(ROOT, 'include')}"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES]
    files += [os.path.join(CSRC, h) for h in HEADERS if os.path.exists(os.path.join(CSRC, h))]
    files.append(os.path.join(CSRC, "hostcall.c"))
    files.append(os.path.join(ROOT, "include", "kascade.h"))
    return files


def python_headers() -> str | None:
    """Where Python.h is, or None: without it the library goes without its CPython module."""
    inc = sysconfig.get_paths()["include"]
    return inc if os.path.exists(os.path.join(inc, "Python.h")) else None


def up_to_date() -> bool:
    made = [LIB, HOSTCALL] if python_headers() else [LIB]
    if not all(os.path.exists(f) for f in made):
        return False
    t = min(os.path.getmtime(f) for f in made)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def hostcall_command(out: str) -> list:
    """nvcc, which hands C files to the host compiler that it uses anyway."""
    return [nvcc(), *ARCH, "-O2", "-shared", "-cudart", "none", "-Xcompiler", "-fPIC,-Wall", f"-I{python_headers()}",
            os.path.join(CSRC, "hostcall.c"), "-o", out]


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    objs = []
    procs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc(), *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0 or verbose:
            sys.stderr.write(out.decode(errors="replace"))
        if p.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError(f"nvcc failed for {failed}")
    tmp = LIB + ".tmp"
    subprocess.check_call([nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static"])
    os.replace(tmp, LIB)
    untagged = os.path.join(HERE, "_hostcall.so")  # of earlier builds: any interpreter would import it
    if os.path.exists(untagged):
        os.remove(untagged)
    if python_headers():
        tmp = HOSTCALL + ".tmp"
        subprocess.check_call(hostcall_command(tmp))
        os.replace(tmp, HOSTCALL)
    else:
        sys.stderr.write("no Python.h: built without _hostcall, its calls go through ctypes (2 us each)\n")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
