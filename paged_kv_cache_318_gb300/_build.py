"""Build libpkv.so in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` translation unit compiles in parallel to an object under
``_build/``; the objects link into ``paged_kv_cache_318_gb300/lib/libpkv.so``
with the CUDA runtime linked statically.  A rebuild happens only when a
source or header is newer than the library.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import re
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_DIR = os.path.join(PKG, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libpkv.so")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH_FLAGS + [
    "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
    "-Xcompiler", "-fvisibility=hidden",
    "-I" + INCLUDE, "-I" + CSRC,
]


def nvcc_path() -> str:
    for cand in (os.environ.get("CUDA_HOME"), "/usr/local/cuda"):
        if cand and os.path.exists(os.path.join(cand, "bin", "nvcc")):
            return os.path.join(cand, "bin", "nvcc")
    found = shutil.which("nvcc")
    if not found:
        raise RuntimeError("nvcc not found: set CUDA_HOME")
    return found


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__])


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(f) <= t for f in _inputs())


# Kernels whose warps trade registers (setmaxnreg) and have no stand-in: the
# registers a thread that their split adds up to (LAUNCH_REGS in tree_attn.cuh).
# With fewer the warps that ask for more would wait for ever.
LAUNCH_REGS = ((re.compile(r"tree_attn_kernelI\w+?Li(64|128)ELi[12]E"), 96),
               (re.compile(r"tree_attn_kernelI\w+?Li256ELi[12]E"), 128))


def check_registers(log):
    """Raises if ptxas (-v) gave one of those kernels another count; returns
    how many of them it saw."""
    want, name, seen = None, "", 0
    for line in log.splitlines():
        if "Compiling entry function" in line:
            name = line.split("'")[1]
            want = next((n for pat, n in LAUNCH_REGS if pat.search(name)),
                        None)
        used = re.search(r"Used (\d+) registers", line)
        if used and want is not None:
            if int(used.group(1)) != want:
                raise RuntimeError(
                    "%s: compiled for %s registers, its register split needs "
                    "%d" % (name, used.group(1), want))
            seen, want = seen + 1, None
    return seen


def _compile(nvcc, src, extra):
    obj = os.path.join(BUILD_DIR,
                       os.path.basename(src).replace(".cu", ".o"))
    split = os.path.basename(src) == "tree_codes.cu"
    cmd = [nvcc] + NVCC_FLAGS + extra + (["-Xptxas", "-v"] if split else []) \
        + ["-c", src, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" %
                           (src, " ".join(cmd), res.stderr))
    if split and check_registers(res.stderr) == 0:
        raise RuntimeError("no register counts from ptxas for %s" % src)
    return obj, res.stderr


def build(force: bool = False, verbose: bool = False,
          extra_flags=()) -> str:
    """Compile and link libpkv.so; returns its path."""
    if not force and up_to_date():
        return LIB_PATH
    nvcc = nvcc_path()
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    srcs = sources()
    workers = max(1, min(len(srcs), os.cpu_count() or 1))
    with cf.ThreadPoolExecutor(workers) as ex:
        results = list(ex.map(lambda s: _compile(nvcc, s, list(extra_flags)),
                              srcs))
    if verbose:
        for _, log in results:
            if log:
                print(log)
    objs = [o for o, _ in results]
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc] + ARCH_FLAGS + ["-shared", "-cudart", "static", "-o", tmp] \
        + objs
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd),
                                                     res.stderr))
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
