"""Python binding of the 8-bit block format (opq_fp8_* in include/opq.h): e4m3 codes with one
float32 scale per block of 128 values along the row.

    m     = max(largest finite |x| of the block, 2^-64)
    scale = m / 448
    code  = the e4m3 number nearest 448 x / m (ties to even; infinities -> +-448, NaN -> NaN)

Codes are torch.float8_e4m3fn tensors of the input's shape; the scales of a matrix [R, K] are
float32 [ceil(K / 128), ceil(R / block_rows)] (a block's scales of neighbouring rows side by
side). 16-bit tensors are bfloat16 or float16.

Like the rest of the binding, these calls only marshal arguments to the library's kernels on the
current stream of the tensors' device; wrong arguments raise ValueError or OPQError before
anything is launched. They take no workspace, so calls on several streams and captured graphs
are independent of one another.
"""
from __future__ import annotations

import ctypes

import torch

import bit_diffusion_transformer_b200 as _opq

FP8_BLOCK = 128
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
_F8 = torch.float8_e4m3fn


def _fail(msg: str):
    raise ValueError(f"opq: {msg}")


def _dtype(t, what: str) -> int:
    d = _DTYPES.get(t.dtype if isinstance(t, torch.Tensor) else t)
    if d is None:
        _fail(f"{what} must be bfloat16 or float16")
    return d


def _check(dtype, what: str, t, dim: int, device=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        _fail(f"{what} must be a tensor on a CUDA device")
    if device is not None and t.device != device:
        _fail(f"{what} is on {t.device}, not {device}")
    if dtype is not None and t.dtype != dtype:
        _fail(f"{what} must be {dtype}")
    if t.dim() != dim:
        _fail(f"{what} must have {dim} dimensions")


def _rows(what: str, t, written: bool = False) -> int:
    """Row stride of a matrix whose rows are contiguous."""
    if t.shape[1] > 1 and t.stride(1) != 1:
        _fail(f"{what}: the last dimension must be contiguous")
    if t.shape[0] <= 1:
        return t.shape[1]
    if written and t.stride(0) < t.shape[1]:
        _fail(f"{what}: rows overlap")
    return t.stride(0)


def _call(fn: str, device, *args):
    """The library call on `device`'s current stream, with that device current."""
    f = getattr(_opq.load(), fn)
    if torch.cuda.current_device() == device.index:
        _opq._check(f(*args, torch._C._cuda_getCurrentRawStream(device.index)), fn)
    else:
        with torch.cuda.device(device):
            _opq._check(f(*args, torch._C._cuda_getCurrentRawStream(device.index)), fn)


def fp8_quantize(x: torch.Tensor, block_rows: int = 1, out=None):
    """Quantize a 16-bit matrix [R, K] (K % 32 == 0) -> (codes [R, K], scales).

    ``block_rows`` 1 gives each row its own scale per 128 columns (activations), 128 gives one
    scale per 128 x 128 block (weights). Rows may be strided (a multiple of 8 elements).
    ``out`` = (codes, scales) to write into."""
    _check(None, "x", x, 2)
    dt = _dtype(x, "x")
    if block_rows not in (1, 128):
        _fail("block_rows must be 1 or 128")
    R, K = x.shape
    shape = (-(-K // FP8_BLOCK), -(-R // block_rows))
    if out is None:
        codes = torch.empty((R, K), dtype=_F8, device=x.device)
        scales = torch.empty(shape, dtype=torch.float32, device=x.device)
        ldc, lds = K, shape[1]
    else:
        codes, scales = out
        _check(_F8, "codes", codes, 2, x.device)
        _check(torch.float32, "scales", scales, 2, x.device)
        if codes.shape != x.shape or tuple(scales.shape) != shape:
            _fail(f"out must be codes {tuple(x.shape)} and scales {shape}")
        ldc, lds = _rows("codes", codes, True), _rows("scales", scales, True)
    _call("opq_fp8_quantize", x.device, x.data_ptr(), dt, R, K, _rows("x", x), block_rows, codes.data_ptr(), ldc,
          scales.data_ptr(), lds)
    return codes, scales


def fp8_linear(x: torch.Tensor, x_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
               bias: torch.Tensor | None = None, act: str = "none", dtype: torch.dtype = torch.bfloat16, out=None):
    """y = act(x @ W^T + bias) -> [M, N] of ``dtype`` (bfloat16 or float16).

    ``x``, ``x_scales`` from fp8_quantize(., 1); ``w``, ``w_scales`` from fp8_quantize(., 128);
    ``bias`` [N] of ``dtype``; ``act`` one of ACTIVATIONS. Rows may be strided (codes: multiples of
    16), so slices of a batch's codes and scales serve."""
    if out is not None:
        dtype = out.dtype
    dt = _dtype(dtype, "dtype")
    _check(_F8, "x", x, 2)
    dev = x.device
    _check(_F8, "w", w, 2, dev)
    _check(torch.float32, "x_scales", x_scales, 2, dev)
    _check(torch.float32, "w_scales", w_scales, 2, dev)
    if act not in _opq.ACTIVATIONS:
        _fail(f"act must be one of {', '.join(_opq.ACTIVATIONS)}")
    M, K = x.shape
    N = w.shape[0]
    kb = -(-K // FP8_BLOCK)
    if w.shape[1] != K:
        _fail(f"x has {K} columns, w {w.shape[1]}")
    if tuple(x_scales.shape) != (kb, M):
        _fail(f"x_scales must be {(kb, M)} (fp8_quantize with block_rows = 1)")
    if tuple(w_scales.shape) != (kb, -(-N // FP8_BLOCK)):
        _fail(f"w_scales must be {(kb, -(-N // FP8_BLOCK))} (fp8_quantize with block_rows = 128)")
    if bias is not None:
        _check(dtype, "bias", bias, 1, dev)
        if bias.shape[0] != N or (N > 1 and bias.stride(0) != 1):
            _fail(f"bias must be a contiguous [{N}]")
    if out is None:
        out = torch.empty((M, N), dtype=dtype, device=dev)
    else:
        _check(dtype, "out", out, 2, dev)
        if tuple(out.shape) != (M, N):
            _fail(f"out must be {(M, N)}")
    _call("opq_fp8_linear", dev, x.data_ptr(), _rows("x", x), x_scales.data_ptr(), _rows("x_scales", x_scales), M, K,
          w.data_ptr(), _rows("w", w), w_scales.data_ptr(), _rows("w_scales", w_scales), N,
          None if bias is None else bias.data_ptr(), _opq.ACTIVATIONS[act], out.data_ptr(), dt,
          _rows("out", out, True))
    return out


class Fp8Cache(ctypes.Structure):
    """Keys or values of a cache (the C struct opq_fp8_cache)."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("head_dim", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("scale_page_stride", ctypes.c_int64), ("scale_token_stride", ctypes.c_int64),
                ("scale_head_stride", ctypes.c_int64)]


class Fp8Rows(ctypes.Structure):
    """Rows [tokens, heads, head_dim] (the C struct opq_rows)."""
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


def _overlaps(t) -> bool:
    return any(n > 1 and s == 0 for n, s in zip(t.shape, t.stride()))


def _cache(cache):
    """(C structs, pages, page size, heads, head dims, device) of (k_codes, k_scales[, v_codes, v_scales])."""
    if len(cache) not in (2, 4):
        _fail("cache must be (codes, scales) or (k_codes, k_scales, v_codes, v_scales)")
    n = len(cache) // 2
    arr = (Fp8Cache * n)()
    dims = []
    for i in range(n):
        codes, scales = cache[2 * i], cache[2 * i + 1]
        _check(_F8, "cache codes", codes, 4, None if i == 0 else cache[0].device)
        _check(torch.float32, "cache scales", scales, 4, codes.device)
        D = codes.shape[3]
        if codes.shape[:3] != cache[0].shape[:3]:
            _fail("keys and values must have the same pages, page size and heads")
        if scales.shape[:3] != codes.shape[:3] or scales.shape[3] != -(-D // FP8_BLOCK):
            _fail(f"scales must be {tuple(codes.shape[:3]) + (-(-D // FP8_BLOCK),)}")
        if (D > 1 and codes.stride(3) != 1) or (scales.shape[3] > 1 and scales.stride(3) != 1):
            _fail("cache: the last dimension must be contiguous")
        if _overlaps(codes) or _overlaps(scales):
            _fail("cache: elements overlap")
        arr[i] = Fp8Cache(codes.data_ptr(), scales.data_ptr(), D, *_strides(codes), *_strides(scales))
        dims.append(D)
    return arr, *cache[0].shape[:3], dims, cache[0].device


def _strides(t):
    """Strides of all dimensions but the last; 0 where there is one entry (its stride is never used)."""
    return [s if n > 1 else 0 for n, s in zip(t.shape[:-1], t.stride()[:-1])]


def _row_array(what, tensors, heads, dims, device, dtype, written):
    arr = (Fp8Rows * len(tensors))()
    for i, (t, D) in enumerate(zip(tensors, dims)):
        _check(dtype, what, t, 3, device)
        if t.shape[0] != tensors[0].shape[0] or t.shape[1] != heads or t.shape[2] != D:
            _fail(f"{what} must be [{tensors[0].shape[0]}, {heads}, {D}]")
        if D > 1 and t.stride(2) != 1:
            _fail(f"{what}: the last dimension must be contiguous")
        if written and _overlaps(t):
            _fail(f"{what}: elements overlap")
        arr[i] = Fp8Rows(t.data_ptr(), *_strides(t))
    return arr


def fp8_cache_write(k: torch.Tensor, v: torch.Tensor | None, cache, slots: torch.Tensor):
    """Quantize keys and values [T, heads, head_dim] into their slots of a paged cache.

    ``cache`` = (k_codes, k_scales, v_codes, v_scales), or (codes, scales) with ``v`` None: codes
    float8_e4m3fn [pages, page_size, heads, head_dim] and scales float32 [pages, page_size, heads,
    ceil(head_dim / 128)]; views of other layouts (heads before tokens in a page) and slices of a
    fused projection's output serve. head_dim % 16 == 0; values may have their own head_dim.
    ``slots`` int64 [T]: page * page_size + offset; negative entries are skipped, entries past the
    cache are skipped and reported by device_error() (DEVERR_INDEX). Slots >= 0 must differ."""
    arr, pages, page_size, heads, dims, dev = _cache(cache)
    tensors = [k] if v is None else [k, v]
    if len(tensors) != len(dims):
        _fail("values go with a cache of keys and values")
    _check(None, "k", k, 3, dev)
    dt = _dtype(k, "k")
    rows = _row_array("k and v", tensors, heads, dims, dev, k.dtype, False)
    _check(torch.int64, "slots", slots, 1, dev)
    T = k.shape[0]
    if slots.shape[0] != T or (T > 1 and slots.stride(0) != 1):
        _fail(f"slots must be a contiguous [{T}]")
    _call("opq_fp8_cache_write", dev, arr, rows, len(dims), pages, page_size, heads, dt, T, slots.data_ptr())


def fp8_cache_read(cache, page_table: torch.Tensor, cu_rows: torch.Tensor, rows: int | None = None,
                   starts: torch.Tensor | None = None, dtype: torch.dtype = torch.bfloat16, out=None):
    """Decode a batch of sequences from a paged cache -> (k [rows, heads, head_dim], v).

    ``page_table`` int32 [B, W]: the pages of each sequence in order. ``cu_rows`` int32 [B + 1]:
    sequence b's tokens go to rows cu_rows[b] .. cu_rows[b + 1] - 1, from position ``starts``[b]
    (int32 [B]; None: 0) on. ``rows`` is the number of output rows (cu_rows[B] or more, on the
    host); rows that no sequence holds stay as they were (unset in a new output). ``out`` = (k, v) to write into,
    any strides with contiguous channels. A cache of keys alone, (codes, scales), gives (k,).
    Pages out of range leave their rows unwritten and are reported by device_error()."""
    arr, pages, page_size, heads, dims, dev = _cache(cache)
    _check(torch.int32, "page_table", page_table, 2, dev)
    _check(torch.int32, "cu_rows", cu_rows, 1, dev)
    B, W = page_table.shape
    ld = _rows("page_table", page_table)
    if cu_rows.shape[0] != B + 1 or (B > 0 and cu_rows.stride(0) != 1):
        _fail(f"cu_rows must be a contiguous [{B + 1}]")
    if starts is not None:
        _check(torch.int32, "starts", starts, 1, dev)
        if starts.shape[0] != B or (B > 1 and starts.stride(0) != 1):
            _fail(f"starts must be a contiguous [{B}]")
    if out is None:
        if rows is None:
            _fail("rows (the number of output rows) or out is needed")
        _dtype(dtype, "dtype")
        out = tuple(torch.empty((rows, heads, D), dtype=dtype, device=dev) for D in dims)
    else:
        if len(out) != len(dims):
            _fail(f"out must hold {len(dims)} tensors")
        _check(None, "out", out[0], 3, dev)
        if rows is not None and rows != out[0].shape[0]:
            _fail(f"out has {out[0].shape[0]} rows, not {rows}")
    dt = _dtype(out[0], "out")
    oarr = _row_array("out", out, heads, dims, dev, out[0].dtype, True)
    _call("opq_fp8_cache_read", dev, arr, oarr, len(dims), pages, page_size, heads, dt, out[0].shape[0],
          cu_rows.data_ptr(), B, page_table.data_ptr(), max(ld, W), W, None if starts is None else starts.data_ptr())
    return tuple(out)
