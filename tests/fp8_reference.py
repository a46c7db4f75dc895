"""The 8-bit block format in plain float64 torch on the CPU: the definition, element by element,
for the tests of fp8_quantize, fp8_linear, fp8_cache_write and fp8_cache_read."""
import math

import torch

BLOCK = 128
F8 = torch.float8_e4m3fn


def e4m3_values():
    """All non-negative finite e4m3 numbers in order, from the bit fields (exponent bias 7)."""
    out = []
    for code in range(0x7F):
        e, m = code >> 3, code & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return torch.tensor(out, dtype=torch.float64)


def nearest_e4m3(v):
    """Nearest e4m3 number of float64 v, ties to the even code, magnitudes above 448 to 448; NaN stays."""
    grid = e4m3_values()
    a = v.abs().clamp(max=448.0)
    a = torch.where(torch.isnan(a), torch.zeros_like(a), a)
    hi = torch.searchsorted(grid, a).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - grid[lo], grid[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    r = torch.copysign(torch.where(up, grid[hi], grid[lo]), v)
    return torch.where(torch.isnan(v), v, r)


def block_codes(x):
    """x [..., n] float64, one block along the last axis -> (numbers the codes hold, scales)."""
    fin = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    m = fin.amax(-1, keepdim=True).clamp(min=2.0 ** -64)
    q = torch.where(torch.isinf(x), torch.copysign(torch.full_like(x, 448.0), x), 448.0 * x / m)
    return nearest_e4m3(q), (m / 448.0).squeeze(-1)


def quantize(x, block_rows):
    """x [R, K] -> (codes' numbers float64 [R, K], scales float64 [ceil(K / 128), ceil(R / block_rows)])."""
    x = x.double()
    R, K = x.shape
    codes = torch.empty_like(x)
    scales = torch.empty((-(-K // BLOCK), -(-R // block_rows)), dtype=torch.float64)
    for b in range(scales.shape[0]):
        for r in range(scales.shape[1]):
            part = x[r * block_rows:(r + 1) * block_rows, b * BLOCK:(b + 1) * BLOCK]
            c, s = block_codes(part.reshape(-1))
            codes[r * block_rows:(r + 1) * block_rows, b * BLOCK:(b + 1) * BLOCK] = c.view(part.shape)
            scales[b, r] = s
    return codes, scales


def decode(codes, scales, block_rows):
    """Float64 values of a quantized matrix (codes as numbers or e4m3)."""
    R, K = codes.shape
    s = scales.double().t().repeat_interleave(block_rows, 0)[:R].repeat_interleave(BLOCK, 1)[:, :K]
    return codes.double() * s


def linear(xc, xs, wc, ws, bias=None, act="none"):
    """(y float64, B = |x| |W|^T, v = the value before the activation)."""
    x, w = decode(xc, xs, 1), decode(wc, ws, BLOCK)
    v = x @ w.t()
    if bias is not None:
        v = v + bias.double()
    y = v
    if act == "silu":
        y = v / (1.0 + torch.exp(-v))
    elif act == "gelu_tanh":
        y = 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    return y, x.abs() @ w.abs().t(), v


def linear_tolerance(y, B, v, bias, act, dtype, K):
    """How far fp8_linear may be from the float64 result.

    Products of two e4m3 numbers are exact in fp32. A 128-term sum is off by at most 128 truncations
    of 2^-23 of the terms' magnitudes; the scale product rounds once (2^-24), its product with the sum
    and the running sum once each per block (fused: once), so kblocks + 2 roundings of 2^-24 of B.
    The bias adds one. The activations' slopes are below 1.15, and tanh.approx (largest relative error
    2^-11) moves v (1 + tanh) / 2 by at most 2^-12 |v|, plus a few fp32 roundings (4 x 2^-24 |v|).
    The result is rounded once to the output type: eps / 2 of its size, or half of the smallest
    subnormal step."""
    kb = -(-K // BLOCK)
    err = (128 * 2.0 ** -23 + (kb + 2) * 2.0 ** -24) * B
    if bias is not None:
        err = err + 2.0 ** -24 * (v.abs() + bias.double().abs())
    if act != "none":
        err = 1.15 * err + (2.0 ** -12 + 4 * 2.0 ** -24) * v.abs()
    fi = torch.finfo(dtype)
    return err + (y.abs() + err) * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def to_codes(numbers):
    """float64 e4m3 numbers -> float8_e4m3fn (exact)."""
    return numbers.float().to(F8)
