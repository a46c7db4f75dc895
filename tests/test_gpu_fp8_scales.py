"""The 8-bit linear over scales whose products leave fp32's normal range although the outputs do not:
y = sum_b sx sw P_b for any fp32 scales, P_b a block's sum of code products.

How far an output may be off: each block's sum by 128 truncations of 2^-23 of its terms' magnitudes;
the scale product's rounding (or the sum's with its first scale), the fused multiply-add and the running
sum of blocks make at most blocks + 3 roundings of 2^-24 of B = sum |x| |w|; a block's contribution below
fp32's normal range adds half of 2^-149 per block. The result is rounded once."""
import pytest
import torch

import bit_diffusion_transformer_b200 as opq
import fp8_reference as ref
from test_gpu_fp8_activations import exact, tolerance

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn
# narrow tiles of 16 rows (one range of blocks, several), of 32 and 64; 128 x 128, 128 x 256, pairs
SHAPES = [(1, 130, 96), (5, 300, 2048), (20, 300, 640), (40, 3840, 10240), (300, 300, 384), (1100, 3845, 640),
          (2001, 4001, 640)]


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    torch.cuda.synchronize()
    assert opq.device_error() == 0


def codes(rows, K, seed, low=0x30, high=0x70):
    """Positive e4m3 codes between two bit patterns."""
    g = torch.Generator(DEV).manual_seed(seed)
    return torch.randint(low, high, (rows, K), generator=g, device=DEV, dtype=torch.uint8)


def powers(shape, lo, hi, seed):
    """fp32 numbers of random mantissas with exponents lo .. hi."""
    g = torch.Generator(DEV).manual_seed(seed)
    e = torch.randint(lo, hi + 1, shape, generator=g, device=DEV)
    return torch.ldexp(1.0 + torch.rand(shape, generator=g, device=DEV, dtype=torch.float64), e).float()


def check(xc, xs, wc, ws, dtype=torch.bfloat16):
    K = xc.shape[1]
    xc, wc = xc.view(F8), wc.view(F8)
    y = opq.fp8_linear(xc, xs, wc, ws, dtype=dtype).double()
    want, B, _ = ref.linear(xc, xs, wc, ws)
    assert float(want.abs().max()) < torch.finfo(dtype).max
    kb, fi = -(-K // 128), torch.finfo(dtype)
    err = (128 * 2.0 ** -23 + (kb + 3) * 2.0 ** -24) * B + kb * 2.0 ** -150
    tol = err + (want.abs() + err) * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2
    off = (y - want).abs()
    bad = ~(off <= tol)
    at = int(torch.where(bad, off / tol, torch.zeros_like(off)).nan_to_num(nan=1e300).argmax())
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} out; {float(y.flatten()[at])} for {float(want.flatten()[at])}"
    return want


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_products_below_the_normal_range(M, N, K):
    """Scale products of 2^-148 .. 2^-128 under sums of 2^8 .. 2^24: outputs in bf16's normal range."""
    kb = -(-K // 128)
    want = check(codes(M, K, 1), powers((kb, M), -75, -66, 2), codes(N, K, 3), powers((kb, -(-N // 128)), -73, -62, 4))
    assert float((want >= torch.finfo(torch.bfloat16).smallest_normal).double().mean()) > 0.3
    # one scale far below the other's reciprocal
    check(codes(M, K, 1), powers((kb, M), -149, -130, 5), codes(N, K, 3), powers((kb, -(-N // 128)), 0, 12, 6))


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_products_above_the_range(M, N, K):
    """Scale products past fp32's largest: under sums of zero the output is zero, under small ones finite."""
    kb = -(-K // 128)
    xc, wc = codes(M, K, 1, 1, 3), codes(N, K, 2, 1, 3)        # codes of 2^-9 and 2^-8: terms 2^-18 .. 2^-16
    xc[:, 8:] = 0
    xs, ws = powers((kb, M), 62, 64, 3), powers((kb, -(-N // 128)), 65, 66, 4)
    odd = torch.arange(M, device=DEV) % 3 == 1
    xc[odd, 0:8:2] = 0
    wc[:, 1:8:2] = 0                                           # these rows meet no column of W
    want = check(xc, xs, wc, ws)
    assert bool((want[odd] == 0).all()) and bool((want[~odd] > 2.0 ** 100).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_rows_and_blocks_apart(M, N, K, dtype):
    """Ordinary, tiny, huge and zero scales in neighbouring rows and blocks of one tile."""
    kb, nb = -(-K // 128), -(-N // 128)
    xc, wc = codes(M, K, 1), codes(N, K, 2)
    xs, ws = powers((kb, M), -22, -21, 3), powers((kb, nb), -9, -8, 4)
    m, b = torch.arange(M, device=DEV), torch.arange(kb, device=DEV)
    xs[:, m % 5 == 1] = powers((kb, M), -149, -120, 5)[:, m % 5 == 1]
    xs[:, m % 5 == 2] = 0.0
    ws[b % 3 == 1] = powers((kb, nb), -126, -110, 6)[b % 3 == 1]
    if kb > 1:                                                 # a block of huge scales over zero codes
        last = slice((kb - 1) * 128, K)
        xc[:, last] = 0
        xs[kb - 1] = 3e38
        ws[kb - 1] = 2e38
    else:
        xs[:, m % 5 == 2] = 0.0
        ws[:] = 1e-3
    want = check(xc, xs, wc, ws, dtype)
    assert bool((want[m % 5 == 2] == 0).all())


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_zero_scales_beside_huge_ones(M, N, K):
    kb, nb = -(-K // 128), -(-N // 128)
    xs, ws = torch.zeros((kb, M), device=DEV), torch.full((kb, nb), 3e38, device=DEV)
    assert bool((check(codes(M, K, 1), xs, codes(N, K, 2), ws) == 0).all())
    assert bool((check(codes(M, K, 1), xs + 3e38, codes(N, K, 2), ws * 0) == 0).all())


@pytest.mark.parametrize("act", ["none", "silu", "gelu_tanh"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_second_pass_strides_bias_and_activation(M, N, K, act):
    """Operands and output inside wider buffers; what lies around the output stays."""
    kb, nb = -(-K // 128), -(-N // 128)
    wide = torch.full((M + 2, K + 48), 0x7F, dtype=torch.uint8, device=DEV)        # NaN codes around the rows
    wpad = torch.full((N, K + 16), 0x7F, dtype=torch.uint8, device=DEV)
    xc, wc = wide[1:M + 1, 16:16 + K], wpad[:, :K]
    xc.copy_(codes(M, K, 1))
    wc.copy_(codes(N, K, 2))
    xs, ws = powers((kb, M + 5), -22, -21, 3)[:, 2:M + 2], powers((kb, nb), -9, -8, 4)
    xs[:, ::3] = powers((kb, M + 5), -149, -120, 5)[:, 2:M + 2][:, ::3]
    ws[-1] *= 2.0 ** -20
    bias = (torch.randn(N, generator=torch.Generator(DEV).manual_seed(6), device=DEV) * 4).to(torch.bfloat16)
    buf = torch.full((M + 9, N + 19), 99.0, dtype=torch.bfloat16, device=DEV)
    out = buf[8:M + 8, 8:8 + N]          # (8 rows and 8 columns in: 16-byte aligned)
    opq.fp8_linear(xc.view(F8), xs, wc.view(F8), ws, bias=bias, act=act, out=out)
    _, B, v = ref.linear(xc.view(F8), xs, wc.view(F8), ws, bias)
    dv = (128 * 2.0 ** -23 + (kb + 3) * 2.0 ** -24) * B + 2.0 ** -24 * (v.abs() + bias.double().abs()) + kb * 2.0 ** -150
    if act == "none":
        want, tol = v, dv + (v.abs() + dv) * 2.0 ** -8 + 2.0 ** -134
    else:
        want, z, slope = exact(v, act)
        tol = tolerance(want, z, slope, v, dv, torch.bfloat16)
    assert bool(((out.double() - want).abs() <= tol).all())
    out.fill_(99.0)
    assert bool((buf == 99.0).all())


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_zero_rows_against_zero_blocks(M, N, K):
    """Padded tokens against padded weights: both operands' smallest scales meet (2^-146), over zeros."""
    x = torch.randn((M, K), device=DEV, generator=torch.Generator(DEV).manual_seed(1)).to(torch.bfloat16)
    w = torch.randn((N, K), device=DEV, generator=torch.Generator(DEV).manual_seed(2)).to(torch.bfloat16)
    x[M // 2:] = 0
    w[(N - 1) // 128 * 128:] = 0
    xc, xs = opq.fp8_quantize(x)
    wc, ws = opq.fp8_quantize(w, 128)
    want = check(xc, xs, wc, ws)
    assert bool((want[M // 2:] == 0).all())
    y = opq.fp8_linear(xc, xs, wc, ws)
    assert bool((y[M // 2:] == 0).all()) and bool((y[:, (N - 1) // 128 * 128:] == 0).all())
