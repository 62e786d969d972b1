"""Build libmhc.so in-tree with nvcc for sm_103a.

Each translation unit under csrc/ is compiled in parallel to an object file,
then linked (CUDA runtime linked statically) into
layers_proj_rms_gb300/_build/libmhc.so; gcc builds the binding's C part, which
belongs to one Python ABI and says so in its name (_build/_marshal.cpython-...).
Rebuilds only what changed.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.machinery
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libmhc.so")
# the binding's C part (csrc/marshal.c)
MARSHAL = os.path.join(OUT, "_marshal" + importlib.machinery.EXTENSION_SUFFIXES[0])
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", f"-I{INCLUDE}"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmhc")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers_mtime():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(INCLUDE, "mhc.h"))
    return max(os.path.getmtime(h) for h in hs)


def _compile(src: str, obj: str, extra) -> None:
    cmd = [_nvcc()] + NVCC_FLAGS + list(extra) + ["-c", src, "-o", obj + ".tmp"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    os.replace(obj + ".tmp", obj)


def _build_marshal(force: bool) -> None:
    src = os.path.join(CSRC, "marshal.c")
    newest = max(os.path.getmtime(src), os.path.getmtime(os.path.join(INCLUDE, "mhc.h")))
    if not force and os.path.exists(MARSHAL) and os.path.getmtime(MARSHAL) >= newest:
        return
    headers = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(headers, "Python.h")):
        warnings.warn(f"no Python.h in {headers}: mhc_qk_norm_rope_* and mhc_moe_* cannot be "
                      "called from Python (their binding, csrc/marshal.c, is not built)")
        return
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = [shutil.which("gcc") or "cc", "-O2", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-I{headers}", f"-I{INCLUDE}", src, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"gcc failed for marshal.c:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(OUT, exist_ok=True)
    hdr = _headers_mtime()
    jobs = []
    objs = []
    for src in sources():
        obj = os.path.join(OUT, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or not os.path.exists(obj) or os.path.getmtime(obj) < max(
                os.path.getmtime(src), hdr):
            jobs.append((src, obj))
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            futs = [ex.submit(_compile, s, o, extra_flags) for s, o in jobs]
            for f in futs:
                f.result()
    if jobs or not os.path.exists(LIB):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [_nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    _build_marshal(force)
    if verbose:
        print(f"libmhc: {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
