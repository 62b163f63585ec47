"""Builds the in-tree shared library libbgtq.so for sm_100a with nvcc."""
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libbgtq.so")
SOURCES = ["csrc/encode.cu", "csrc/decode.cu", "csrc/diag.cu", "csrc/api.cu", "csrc/host_tables.cpp",
           "csrc/byte_append.cu", "csrc/byte_decode.cu", "csrc/api_byte.cu", "csrc/pages.cu", "csrc/api_pages.cu",
           "csrc/rope.cu", "csrc/api_rope.cu"]
NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC,-O2",
    "-I", os.path.join(ROOT, "include"),
]


def sources():
    return [os.path.join(PKG, s) for s in SOURCES] + [
        os.path.join(PKG, "csrc", h) for h in ("device_tables.h", "host_tables.h", "common.cuh",
                                                      "byte_cache.h", "pages.h", "rope.h", "state.h")] + [
        os.path.join(ROOT, "include", "bgtq.h")]


def up_to_date():
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in sources())


def build(force=False, verbose=False):
    if not force and up_to_date():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    cmd = [nvcc] + NVCC_FLAGS + ["-o", LIB] + [os.path.join(PKG, s) for s in SOURCES]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
