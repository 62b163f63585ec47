"""Builds the in-tree shared library libbgtq.so for sm_100a with nvcc, and _marshal.so (the Python binding's checks and
calls of the serving operators), which links to it."""
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libbgtq.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
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


def build_marshal(force=False, verbose=False):
    """Builds _marshal.so; None, with a word on stderr, where Python's headers or a C compiler are missing (the packed
    cache does without it; the serving operators then say what to build)."""
    src, header = os.path.join(PKG, "csrc", "marshal.c"), os.path.join(ROOT, "include", "bgtq.h")
    if not force and os.path.exists(MARSHAL) and os.path.getmtime(MARSHAL) >= max(map(os.path.getmtime, (src, header))):
        return MARSHAL
    cc, include = os.environ.get("CC", "gcc"), sysconfig.get_paths()["include"]
    missing = ([] if os.path.exists(os.path.join(include, "Python.h")) else [os.path.join(include, "Python.h")]) + (
        [] if shutil.which(cc.split()[0]) else [cc])
    if missing:
        print(f"_marshal.so not built: {', '.join(missing)} not found", file=sys.stderr)
        return None
    cmd = cc.split() + ["-shared", "-fPIC", "-O2", "-std=c11", "-Wall", "-I", include, "-o", MARSHAL, src, "-L", PKG,
                        "-lbgtq", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    return MARSHAL


def build(force=False, verbose=False):
    if force or not up_to_date():
        nvcc = os.environ.get("NVCC", "nvcc")
        cmd = [nvcc] + NVCC_FLAGS + ["-o", LIB] + [os.path.join(PKG, s) for s in SOURCES]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
    build_marshal(force, verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
