"""Build libopq.so (two translation units, compiled side by side) for sm_100a, in-tree."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
SO = os.path.join(HERE, "libopq.so")
SOURCES = ["opq_capi.cu", "opq_fp8.cu"]
HEADERS = ["opq_bits.h", "opq_device.cuh", "opq_quantize.cuh", "opq_quantize_stream.cuh", "opq_dequantize.cuh",
           "opq_linear.cuh", "opq_linear_wide.cuh", "opq_grouped.cuh", "opq_host.h", "opq_fp8_format.cuh",
           "opq_fp8_quantize.cuh", "opq_fp8_cache.cuh", "opq_fp8_linear.cuh"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _stale() -> bool:
    if not os.path.exists(SO):
        return True
    t = os.path.getmtime(SO)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(INCLUDE, "opq.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return SO
    tmp = SO + f".tmp{os.getpid()}"
    flags = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
             "-I", INCLUDE, "-I", CSRC]
    if verbose:
        flags.append("-Xptxas=-v")
    objs = [f"{tmp}.{i}.o" for i in range(len(SOURCES))]
    try:
        jobs = [subprocess.Popen([_nvcc(), *flags, "-c", os.path.join(CSRC, src), "-o", obj])
                for src, obj in zip(SOURCES, objs)]
        codes = [j.wait() for j in jobs]
        if any(codes):
            raise subprocess.CalledProcessError(max(codes), "nvcc")
        subprocess.check_call([_nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs])
    finally:
        for obj in objs:
            if os.path.exists(obj):
                os.remove(obj)
    os.replace(tmp, SO)
    return SO


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
