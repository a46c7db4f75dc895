"""Python binding of the 8-bit block format (opq_fp8_* in include/opq.h): e4m3 codes with one
float32 scale per block of 128 values along the row.

    m     = max(largest finite |x| of the block, 2^-64)
    scale = m / 448
    code  = the e4m3 number nearest 448 x / m (ties to even; infinities -> +-448, NaN -> NaN)

Codes are torch.float8_e4m3fn tensors of the input's shape; the scales of a matrix [R, K] are
float32 [ceil(K / 128), ceil(R / block_rows)] (a block's scales of neighbouring rows side by
side). 16-bit tensors are bfloat16 or float16.

Like the rest of the binding, these calls only marshal arguments to the library's kernels on the
current stream of the tensors' device (through the extension _fp8.so, built with the library);
wrong arguments raise ValueError or OPQError before anything is launched. They take no workspace,
so calls on several streams and captured graphs are independent of one another.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

import bit_diffusion_transformer_b200 as _opq

FP8_BLOCK = 128
EXT_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_fp8.so")

_ext = None


def _load():
    """The extension (raises if it, or the library behind it, has not been built)."""
    global _ext
    if _ext is None:
        _opq.load()
        if not os.path.exists(EXT_PATH):
            raise ImportError(f"_fp8.so not found at {EXT_PATH}; build it with "
                              f"`python -m bit_diffusion_transformer_b200.build`")
        from . import _fp8
        if not re.match(re.escape(_fp8.TORCH_VERSION) + r"(?!\d)", torch.__version__):    # (2.9.0a0+git..: 2.9.0)
            raise ImportError(f"_fp8.so was built for torch {_fp8.TORCH_VERSION}, this is {torch.__version__}; build it "
                              f"again with `python -m bit_diffusion_transformer_b200.build`")
        _fp8.set_error(_opq.OPQError)
        _ext = _fp8
    return _ext


def fp8_quantize(x: torch.Tensor, block_rows: int = 1, out=None):
    """Quantize a 16-bit matrix [R, K] (K % 32 == 0) -> (codes [R, K], scales).

    ``block_rows`` 1 gives each row its own scale per 128 columns (activations), 128 gives one
    scale per 128 x 128 block (weights). Rows may be strided (a multiple of 8 elements); R is 1 or more.
    ``out`` = (codes, scales) to write into."""
    return (_ext or _load()).quantize(x, block_rows, out)


def fp8_linear(x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
               bias: torch.Tensor | None = None, act: str = "none", dtype: torch.dtype = torch.bfloat16, out=None):
    """y = act(x @ W^T + bias) -> [M, N] of ``dtype`` (bfloat16 or float16).

    ``x``, ``x_scales`` from fp8_quantize(., 1); ``w``, ``w_scales`` from fp8_quantize(., 128);
    ``bias`` [N] of the output's type; ``act`` one of ACTIVATIONS, evaluated to fp32's accuracy. Rows
    may be strided (codes: multiples of 16), so slices of a batch's codes and scales serve; M is 1 or
    more. ``out`` (its type stands for ``dtype``) to write into, inside a wider buffer too."""
    code = _opq.ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"opq: act must be one of {', '.join(_opq.ACTIVATIONS)}")
    return (_ext or _load()).linear(x, x_scales, w, w_scales, bias, code, dtype, out)


def fp8_linear_plan(M: int, N: int, K: int):
    """The tiles fp8_linear uses for x [M, K] and W [N, K] -> (rows of x, rows of W, CTAs that share a tile)."""
    out = [ctypes.c_int() for _ in range(3)]
    _opq._check(_opq.load().opq_fp8_linear_plan(M, N, K, *[ctypes.byref(v) for v in out]), "opq_fp8_linear_plan")
    return tuple(v.value for v in out)


class Fp8Cache(ctypes.Structure):
    """Keys or values of a cache (the C struct opq_fp8_cache)."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("head_dim", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("scale_page_stride", ctypes.c_int64), ("scale_token_stride", ctypes.c_int64),
                ("scale_head_stride", ctypes.c_int64)]


class Fp8Rows(ctypes.Structure):
    """Rows [tokens, heads, head_dim] (the C struct opq_rows)."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


def fp8_cache_write(k: torch.Tensor, v: torch.Tensor | None, cache, slots: torch.Tensor):
    """Quantize keys and values [T, heads, head_dim] into their slots of a paged cache.

    ``cache`` = (k_codes, k_scales, v_codes, v_scales), or (codes, scales) with ``v`` None: codes
    float8_e4m3fn [pages, page_size, heads, head_dim] and scales float32 [pages, page_size, heads,
    ceil(head_dim / 128)]; views of other layouts (heads before tokens in a page) and slices of a
    fused projection's output serve, as long as no two elements share memory. head_dim % 16 == 0; values may have their own head_dim.
    ``slots`` int64 [T]: page * page_size + offset; negative entries are skipped, entries past the
    cache are skipped and reported by device_error() (DEVERR_INDEX). Slots >= 0 must differ."""
    (_ext or _load()).cache_write(k, v, cache, slots)


def fp8_cache_read(cache, page_table: torch.Tensor, cu_rows: torch.Tensor, rows: int | None = None,
                   starts: torch.Tensor | None = None, dtype: torch.dtype = torch.bfloat16, out=None):
    """Decode a batch of sequences from a paged cache -> (k [rows, heads, head_dim], v).

    ``page_table`` int32 [B, W]: the pages of each sequence in order. ``cu_rows`` int32 [B + 1]:
    sequence b's tokens go to rows cu_rows[b] .. cu_rows[b + 1] - 1, from position ``starts``[b]
    (int32 [B]; None: 0) on. ``rows`` is the number of output rows (cu_rows[B] or more, on the
    host); rows that no sequence holds stay as they were (unset in a new output). ``out`` = (k, v)
    to write into, any strides with contiguous channels. A cache of keys alone, (codes, scales),
    gives (k,). Pages out of range leave their rows unwritten and are reported by device_error()
    (DEVERR_INDEX)."""
    return (_ext or _load()).cache_read(cache, page_table, cu_rows, rows, starts, dtype, out)
