"""Compile the CUDA library (sm_103a only) into persistent_megakernel_sm_gb300/_build."""
from __future__ import annotations

import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
REPO = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "_build", "libmoe.so")
SOURCES = ["moe.cu", "router.cu", "w4.cu"]
DEPS = SOURCES + ["tasks.cuh", "layer.cuh", "ptx.cuh", "error.h", "tmap.h", "w4_tiles.cuh"]
HEADER = os.path.join(REPO, "include", "moe.h")

NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-cudart", "shared"]


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, d) for d in DEPS] + [HEADER]
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Build libmoe.so if missing or older than its sources; return its path."""
    if not force and not _stale():
        return LIB
    os.makedirs(os.path.dirname(LIB), exist_ok=True)
    nvcc = os.environ.get("NVCC", "nvcc")
    flags = [*NVCC_FLAGS, *(["-Xptxas=-v"] if verbose else []), "-I", os.path.join(REPO, "include")]
    # beside the library, so that it can be moved into place; gone whatever fails
    with tempfile.TemporaryDirectory(prefix="tmp", dir=os.path.dirname(LIB)) as tmp:
        def compile_one(src: str) -> str:
            obj = os.path.join(tmp, f"{src}.o")
            subprocess.run([nvcc, *flags, "-c", "-o", obj, os.path.join(CSRC, src)], check=True)
            return obj

        with ThreadPoolExecutor(len(SOURCES)) as ex:  # one compiler process per source
            objs = list(ex.map(compile_one, SOURCES))
        lib = os.path.join(tmp, "libmoe.so")
        subprocess.run([nvcc, *NVCC_FLAGS, "-shared", "-o", lib, *objs], check=True)
        os.replace(lib, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
