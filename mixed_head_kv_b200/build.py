"""Build libduo.so (the C-ABI library of include/duo.h) in-tree with nvcc for sm_100a."""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libduo.so")
SOURCES = ["duo_abi.cu", "append.cu", "decode.cu", "decode_tc.cu", "prefill.cu", "prefill_stream.cu", "decode_static.cu",
           "paged_abi.cu", "paged_pages.cu", "paged_append.cu", "paged_decode.cu", "prefill_packed.cu"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "-I" + os.path.join(ROOT, "include")]


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "duo.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    # One nvcc per source, side by side, then one link.
    with tempfile.TemporaryDirectory() as objects:
        def compile_one(src: str) -> str:
            obj = os.path.join(objects, src[:-3] + ".o")
            cmd = [NVCC, *FLAGS, *(["-Xptxas=-v"] if verbose else []), "-c", os.path.join(CSRC, src), "-o", obj]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            subprocess.check_call(cmd)
            return obj

        with concurrent.futures.ThreadPoolExecutor(os.cpu_count() or 1) as pool:
            objs = list(pool.map(compile_one, SOURCES))
        subprocess.check_call([NVCC, *FLAGS, "-shared", *objs, "-o", tmp])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="-v" in sys.argv)
