"""Builds libmea.so in-tree with nvcc for sm_100a (no JIT cache, so the library ships with the tree)."""
from __future__ import annotations

import glob
import hashlib
import os
import shutil
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmea.so")
STAMP = LIB + ".sha256"  # hash of the sources and flags libmea.so was built from
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: cannot build libmea.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(CSRC, "*.h"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def source_hash() -> str:
    """SHA-256 over the kernel sources, the public header and the compiler flags."""
    h = hashlib.sha256(" ".join(NVCC_FLAGS).encode())
    for path in sources():
        h.update(os.path.relpath(path, os.path.dirname(HERE)).encode())
        with open(path, "rb") as f:
            h.update(f.read())
    return h.hexdigest()


def up_to_date() -> bool:
    """True when libmea.so exists and was built from exactly the current sources (a stamp file
    beside the library holds their hash; modification times are not trusted, since a copied
    tree can carry a newer library built from other sources)."""
    if not (os.path.exists(LIB) and os.path.exists(STAMP)):
        return False
    with open(STAMP) as f:
        return f.read().strip() == source_hash()


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd))
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    if verbose:
        print(res.stderr)


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compiles every csrc/*.cu (side by side) and links them into libmea.so; returns its path."""
    if not force and up_to_date():
        return LIB
    units = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as work:
        objs = [os.path.join(work, os.path.basename(u) + ".o") for u in units]
        flags = [*NVCC_FLAGS, "-Xptxas=-v"] if verbose else NVCC_FLAGS
        with ThreadPoolExecutor(len(units)) as pool:
            list(pool.map(lambda uo: _run([_nvcc(), *flags, "-c", "-o", uo[1], uo[0]], verbose),
                          zip(units, objs)))
        _run([_nvcc(), *NVCC_FLAGS, "-shared", "-o", tmp, *objs], verbose)
    os.replace(tmp, LIB)
    with open(STAMP, "w") as f:
        f.write(source_hash() + "\n")
    return LIB


if __name__ == "__main__":
    import sys
    print(build_library(force="--force" in sys.argv, verbose="-v" in sys.argv))
