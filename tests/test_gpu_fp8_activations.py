"""The 8-bit linear's SiLU and GELU, to fp32's accuracy over the whole line, negative tail included.

How far an output may be off (u = 2^-24, fp32's half step; f the activation, v its argument, z the
exponent: y = v / (1 + e^-z), z = v for SiLU, 2 sqrt(2 / pi) (v + 0.044715 v^3) for GELU):
  v       off by dv <= (128 2^-23 + (blocks + 2) u) B + u (|v| + |bias|), B = sum |x| |w|, as for the
          product without an activation: moves y by |f'(v)| dv + dv^2 / 2 (|f''| < 1)
  e^-|z|  the exponent by 3.5 u relative (a rounded constant, up to three operations), which is 3.5 u |z|
          of the exponential; ex2.approx at 2^-22 = 4 u twice (half the exponent, squared) and a rounding
  y       1 + e^-|z| (its exponential's error counts half), a shared reciprocal (2 u) of up to four such
          sums, the products that undo the sharing, the two last products: at most 20 roundings,
          (32 + 6 |z|) u |y| with the above
  result  rounded once: eps / 2 of its size, or half of the smallest subnormal step; intermediate
          subnormals add at most (|v| + 1) 2^-149
"""
import math

import pytest
import torch

import bit_diffusion_transformer_b200 as opq
import fp8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
# tile kinds by shape: narrow tiles of 16 rows (one range of blocks, two), of 32, of 64; 128 x 128,
# 128 x 256 and pairs of 256 x 256 with whole rows and with rows that TMA cannot store
SHAPES = [(1, 1500, 32), (1, 1500, 512), (20, 1500, 512), (40, 3840, 10240), (300, 1500, 128), (1089, 3840, 640),
          (1100, 3845, 640), (2000, 4000, 640), (2001, 4001, 640)]


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    torch.cuda.synchronize()
    assert opq.device_error() == 0


def exact(v, act):
    """(y, |z|, |f'|) of float64 v, without cancellation."""
    if act == "silu":
        z, dz = v, torch.ones_like(v)
    else:
        c = 2.0 * math.sqrt(2.0 / math.pi)
        z, dz = c * (v + 0.044715 * v ** 3), c * (1.0 + 3 * 0.044715 * v ** 2)
    s = torch.sigmoid(z)
    y = v * s
    return y, z.abs(), (s + y * torch.sigmoid(-z) * dz).abs()


def tolerance(y, z, slope, v, dv, dtype):
    fi = torch.finfo(dtype)
    err = slope * dv + dv * dv / 2 + (32 + 6 * z) * 2.0 ** -24 * y.abs() + (v.abs() + 1) * 2.0 ** -149
    return err + (y.abs() + err) * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


def grid(n, dtype):
    a = torch.cat([torch.linspace(-24, 0, n // 2, dtype=torch.float64), torch.linspace(-110, -24, n // 8, dtype=torch.float64),
                   torch.logspace(-30, 1.5, n // 8, base=2, dtype=torch.float64) * -1])
    b = torch.cat([torch.linspace(0, 30, n // 8, dtype=torch.float64), torch.logspace(-8, 4, n, dtype=torch.float64)])
    return torch.cat([a, b])[:n].to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_activation_over_the_line(M, N, K, act, dtype):
    """A zero product: the activation's argument is the bias, exactly."""
    dt = DTYPES[dtype]
    bias = grid(N, dt)
    x = opq.fp8_quantize(torch.zeros((M, K), dtype=torch.bfloat16, device=DEV))
    w = opq.fp8_quantize(torch.randn((N, K), device=DEV, generator=torch.Generator(DEV).manual_seed(1)).to(torch.bfloat16), 128)
    y = opq.fp8_linear(*x, *w, bias=bias, act=act, dtype=dt)
    v = bias.double()
    want, z, slope = exact(v, act)
    tol = tolerance(want, z, slope, v, torch.zeros_like(v), dt)
    err = (y.double() - want).abs()
    bad = ~(err <= tol)
    at = int((err / tol).amax(0).argmax())
    assert not bool(bad.any()), f"{int(bad.sum())} out; worst at v = {float(v[at])}: {float(y[0, at])} for {float(want[at])}"


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_activation_of_products(M, N, K, act, dtype):
    dt = DTYPES[dtype]
    g = torch.Generator(DEV).manual_seed(M + N)
    x = opq.fp8_quantize(torch.randn((M, K), device=DEV, generator=g).to(torch.bfloat16))
    w = opq.fp8_quantize((torch.randn((N, K), device=DEV, generator=g) * (6 / math.sqrt(K))).to(torch.bfloat16), 128)
    bias = torch.randn(N, device=DEV, generator=g).to(dt)
    y = opq.fp8_linear(*x, *w, bias=bias, act=act, dtype=dt)
    _, B, v = ref.linear(*x, *w, bias)
    dv = (128 * 2.0 ** -23 + (-(-K // 128) + 2) * 2.0 ** -24) * B + 2.0 ** -24 * (v.abs() + bias.double().abs())
    want, z, slope = exact(v, act)
    err = (y.double() - want).abs()
    tol = tolerance(want, z, slope, v, dv, dt)
    assert bool((err <= tol).all()), f"{int((err > tol).sum())} out, worst {float((err / tol).max()):.3g}"


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_activation_of_special_values(M, N, K, act, dtype):
    """Infinities, NaN and zeros of the argument, each beside ordinary values: as y = v / (1 + e^-z) gives them."""
    dt = DTYPES[dtype]
    bias = grid(N, dt)
    special = torch.tensor([math.inf, -math.inf, math.nan, 0.0, -0.0, torch.finfo(dt).max, -torch.finfo(dt).max], dtype=dt)
    for i, s in enumerate(special):
        bias[3 + 5 * i] = s
        bias[N - 1 - 5 * i] = s
    x = opq.fp8_quantize(torch.zeros((M, K), dtype=torch.bfloat16, device=DEV))
    w = opq.fp8_quantize(torch.ones((N, K), dtype=torch.bfloat16, device=DEV), 128)
    y = opq.fp8_linear(*x, *w, bias=bias, act=act, dtype=dt)
    fin = torch.isfinite(bias)
    v = bias.double()
    want, z, slope = exact(torch.where(fin, v, torch.zeros_like(v)), act)
    tol = tolerance(want, z, slope, v, torch.zeros_like(v), dt)
    assert bool(((y.double() - want).abs() <= tol)[:, fin & (bias.double().abs() < 1e4)].all())
    big, low = bias == torch.finfo(dt).max, bias == -torch.finfo(dt).max
    assert bool((y[:, big] == torch.finfo(dt).max).all()) and bool((y[:, low] == 0).all())
    assert bool((y[:, bias == math.inf] == math.inf).all())
    assert bool(torch.isnan(y[:, torch.isnan(bias) | (bias == -math.inf)]).all())


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_nan_and_infinite_sums_stay_where_they_are(M, N, K, act):
    """Values that share a reciprocal are neighbours along the features or along the rows of x."""
    g = torch.Generator(DEV).manual_seed(M)
    xc, xs = opq.fp8_quantize(torch.randn((M, K), device=DEV, generator=g).to(torch.bfloat16))
    wc, ws = opq.fp8_quantize(torch.randn((N, K), device=DEV, generator=g).to(torch.bfloat16), 128)
    clean = opq.fp8_linear(xc, xs, wc, ws, act=act)
    xn, wn, xi = xc.view(torch.uint8).clone(), wc.view(torch.uint8).clone(), xs.clone()
    xn[M // 2, 5] = 0x7F
    wn[N // 3, 7] = 0xFF
    xi[0, M - 1] = math.inf                                   # sums of +-inf: inf, NaN below
    y = opq.fp8_linear(xn.view(F8), xi, wn.view(F8), ws, act=act)
    hit = torch.zeros((M, N), dtype=torch.bool, device=DEV)
    hit[M // 2], hit[:, N // 3], hit[M - 1] = True, True, True
    assert bool(torch.isnan(y[M // 2]).all()) and bool(torch.isnan(y[:, N // 3]).all())
    assert not bool(torch.isfinite(y[M - 1]).any())
    assert torch.equal(y[~hit], clean[~hit])
