"""Build libspecverify.so in-tree for sm_103a with nvcc (no CMake, no torch extension machinery)."""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "spec_verify.cu")
SRC_CTRL = os.path.join(PKG, "csrc", "spec_control.cpp")
SRC_DECODE = [os.path.join(PKG, "csrc", f) for f in ("spec_kv.cu", "spec_attention.cu", "spec_pages.cu", "spec_weigh.cu", "spec_select.cu", "spec_logits.cu")]
HDR = os.path.join(ROOT, "include", "spec_verify.h")
HDR_CTRL = os.path.join(ROOT, "include", "spec_control.h")
HDR_DECODE = [os.path.join(ROOT, "include", "spec_decode.h"), os.path.join(PKG, "csrc", "decode_common.cuh"),
              os.path.join(PKG, "csrc", "tile_stream.cuh")]
LIB = os.path.join(PKG, "libspecverify.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
]


def nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(home, "bin", "nvcc")
    return path if os.path.exists(path) else "nvcc"


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in (SRC, SRC_CTRL, HDR, HDR_CTRL, *SRC_DECODE, *HDR_DECODE, __file__))


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library if it is missing or older than its sources; returns its path."""
    if not force and not stale():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    flags = [*(["-Xptxas=-v"] if verbose else []), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include")]
    sources = [SRC, *SRC_DECODE, SRC_CTRL]
    with tempfile.TemporaryDirectory() as objects, ThreadPoolExecutor(len(sources)) as ex:  # compiled side by side
        objs = [os.path.join(objects, os.path.basename(s) + ".o") for s in sources]
        list(ex.map(lambda so: subprocess.run([nvcc(), *flags, "-c", so[0], "-o", so[1]], check=True),
                    zip(sources, objs)))
        subprocess.run([nvcc(), *NVCC_FLAGS, "-shared", *objs, "-o", tmp], check=True)
    os.replace(tmp, LIB)  # atomic: a process that already mapped the old file keeps it intact
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
