"""Build libopq.so (two translation units, compiled side by side) for sm_100a, and _fp8.so, the torch
binding of its 8-bit calls, in-tree."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
SO = os.path.join(HERE, "libopq.so")
EXT = os.path.join(HERE, "_fp8.so")
EXT_SOURCE = "opq_fp8_torch.cpp"
SOURCES = ["opq_capi.cu", "opq_fp8.cu"]
HEADERS = ["opq_bits.h", "opq_device.cuh", "opq_quantize.cuh", "opq_quantize_stream.cuh", "opq_dequantize.cuh",
           "opq_linear.cuh", "opq_linear_wide.cuh", "opq_grouped.cuh", "opq_host.h", "opq_fp8_format.cuh",
           "opq_fp8_quantize.cuh", "opq_fp8_cache.cuh", "opq_fp8_linear.cuh"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _cuda_include() -> str:
    """The CUDA headers beside the nvcc in use (which may be a name on PATH, or a link into the toolkit)."""
    nvcc = shutil.which(_nvcc()) or _nvcc()
    for path in (nvcc, os.path.realpath(nvcc)):
        include = os.path.join(os.path.dirname(os.path.dirname(path)), "include")
        if os.path.exists(os.path.join(include, "cuda_runtime_api.h")):
            return include
    raise FileNotFoundError(f"no CUDA headers beside {nvcc}")


def _older(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _stale() -> bool:
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(INCLUDE, "opq.h")]
    return _older(SO, deps)


def _torch_version() -> str:
    import torch
    return torch.__version__


def _ext_stale() -> bool:
    """Older than its sources, or built for another torch (whose C++ interface need not be the same)."""
    try:
        with open(EXT + ".torch") as f:
            if f.read() != _torch_version():
                return True
    except (OSError, ImportError):      # (no torch: building the binding says so)
        return True
    return _older(EXT, [os.path.join(CSRC, EXT_SOURCE), os.path.join(INCLUDE, "opq.h")])


def _start_ext(obj: str) -> subprocess.Popen:
    """Compile the torch binding (host code only)."""
    import torch
    tinc = os.path.join(os.path.dirname(torch.__file__), "include")
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return subprocess.Popen(["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={abi}", "-I", INCLUDE,
                             "-isystem", tinc, "-isystem", os.path.join(tinc, "torch", "csrc", "api", "include"),
                             "-isystem", sysconfig.get_paths()["include"], "-isystem", _cuda_include(),
                             "-c", os.path.join(CSRC, EXT_SOURCE), "-o", obj])


def _link_ext(obj: str, out: str):
    import torch
    tlib = os.path.join(os.path.dirname(torch.__file__), "lib")
    subprocess.check_call(["g++", "-shared", "-o", out, obj, "-L", HERE, "-lopq", "-Wl,-rpath,$ORIGIN", "-L", tlib,
                           "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"])


def build(force: bool = False, verbose: bool = False) -> str:
    lib, ext = force or _stale(), force or _ext_stale()
    if not lib and not ext:
        return SO
    tmp = SO + f".tmp{os.getpid()}"
    flags = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
             "-I", INCLUDE, "-I", CSRC]
    if verbose:
        flags.append("-Xptxas=-v")
    objs = [f"{tmp}.{i}.o" for i in range(len(SOURCES))] if lib else []
    ext_obj = f"{tmp}.ext.o"
    try:
        jobs = [subprocess.Popen([_nvcc(), *flags, "-c", os.path.join(CSRC, src), "-o", obj])
                for src, obj in zip(SOURCES, objs)]
        ext_job = ext_error = None
        if ext:
            try:
                ext_job = _start_ext(ext_obj)
            except (ImportError, OSError) as e:
                ext_error = e
        codes = [j.wait() for j in jobs]
        ext_code = ext_job.wait() if ext_job else 0
        # the library first: it does not need the binding
        if any(codes):
            raise subprocess.CalledProcessError(next(c for c in codes if c), "nvcc")
        if lib:
            subprocess.check_call([_nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs])
            os.replace(tmp, SO)
        if ext_error:
            raise ext_error
        if ext_code:
            raise subprocess.CalledProcessError(ext_code, f"g++ {EXT_SOURCE}")
        if ext:
            _link_ext(ext_obj, tmp)
            os.replace(tmp, EXT)
            with open(EXT + ".torch", "w") as f:
                f.write(_torch_version())
    finally:
        for f in objs + [ext_obj, tmp]:
            if os.path.exists(f):
                os.remove(f)
    return SO


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
