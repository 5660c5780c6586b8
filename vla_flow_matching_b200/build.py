"""Build libpi0x.so in-tree from csrc/*.cu with nvcc for sm_100a, and the Python
binding of its small calls, _binding.so, from csrc/binding.c.

``python -m vla_flow_matching_b200.build`` (or ``build()``) compiles each CUDA
source to an object under ``_build/`` in parallel and links the shared library
next to this file.  Nothing is rebuilt when no source or header is newer than
the library.
"""
from __future__ import annotations

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
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpi0x.so")
BINDING = os.path.join(PKG, "_binding.so")
NO_BINDING = os.path.join(BUILD, "binding.failed")  # why the last build made no binding

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.c")) +
            glob.glob(os.path.join(ROOT, "include", "*.h")))


def up_to_date() -> bool:
    made = [LIB]
    if importlib.util.find_spec("torch"):
        made.append(NO_BINDING if os.path.exists(NO_BINDING) else BINDING)
    if not all(os.path.exists(p) for p in made):
        return False
    t = min(os.path.getmtime(p) for p in made)
    return all(os.path.getmtime(p) <= t for p in _deps())


def build(force: bool = False, verbose: bool = False, extra: list | None = None) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = list(extra or [])

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    why = _build_binding(verbose)
    if os.path.exists(NO_BINDING):
        os.remove(NO_BINDING)
    if why:  # the sampler does without, and the paged-cache calls say so
        if os.path.exists(BINDING):
            os.remove(BINDING)
        with open(NO_BINDING, "w") as f:
            f.write(why)
        print(f"_binding.so, which the paged-cache calls need, was not built: {why}", file=sys.stderr)
    return LIB


def _build_binding(verbose: bool) -> str:
    """Compile csrc/binding.c where there is a torch; returns why it could not be, or ""."""
    torch = importlib.util.find_spec("torch")
    if torch is None:  # the paged-cache calls take torch tensors
        return ""
    # finds libpi0x.so beside itself; Python's own symbols are the interpreter's; of torch only the
    # DLPack header is used
    cmd = ["gcc", "-O2", "-Wall", "-Wextra", "-shared", "-fPIC", "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(torch.submodule_search_locations[0], "include"),
           os.path.join(CSRC, "binding.c"), "-o", BINDING + ".tmp", "-L", PKG, "-l:libpi0x.so", "-Wl,-rpath,$ORIGIN"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        return str(e)
    if r.returncode != 0:
        return f"gcc failed on binding.c:\n{r.stdout}\n{r.stderr}"
    if verbose and r.stderr:
        print(r.stderr, file=sys.stderr)
    os.replace(BINDING + ".tmp", BINDING)
    return ""


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else None))
