"""The 8-bit linear's tile kinds and epilogues on operands quantized on the GPU (whose codes
test_gpu_fp8.py holds to the definition), against float64 products on the GPU within the derived
tolerance of fp8_reference.linear_tolerance."""
import pytest
import torch

import bit_diffusion_transformer_b200 as opq
import fp8_reference as ref
from fp8_schedules import SCHEDULES
from test_gpu_fp8_activations import exact, tolerance

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    torch.cuda.synchronize()
    assert opq.device_error() == 0


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def normal(*shape, seed=0, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen(seed), device=DEV) * scale).to(dtype)


def operands(M, N, K, seed=0):
    return (*opq.fp8_quantize(normal(M, K, seed=seed)), *opq.fp8_quantize(normal(N, K, seed=seed + 1, scale=0.02), 128))


def check(ops, bias=None, act="none", dtype=torch.bfloat16):
    y = opq.fp8_linear(*ops, bias=bias, act=act, dtype=dtype)
    want, B, v = ref.linear(*ops, bias, act)
    tol = ref.linear_tolerance(want, B, v, bias, act, dtype, ops[0].shape[1])
    err = (y.double() - want).abs()
    assert y.dtype == dtype and bool(torch.isfinite(y).all())
    assert bool((err <= tol).all()), f"{int((err > tol).sum())} of {err.numel()} out, worst {float((err / tol).max()):.3g}"


@pytest.mark.parametrize("M,N", [(1000, 4104), (2600, 5001)])
def test_bias_of_each_tile_over_one_block(M, N):
    """One block per tile: nothing but the epilogue's own barriers stands between a tile's bias, stored
    by all lanes of a warp, and its readers. Several tiles per CTA, each with a bias of its own."""
    bias = torch.arange(N, device=DEV).remainder(509).sub(254).to(torch.bfloat16)
    for K in (96, 128):
        check(operands(M, N, K, seed=K), bias)


@pytest.mark.parametrize("M,K", [(5, 96), (20, 640), (300, 384), (1100, 640), (2001, 640)])
@pytest.mark.parametrize("N", [3840, 3841, 3845, 3847, 3876])
@pytest.mark.parametrize("pad", [0, 1, 8, 24])
def test_nothing_beside_the_output_is_written(M, N, K, pad):
    """The output inside a wider buffer, its rows aligned to 16 bytes or not, its last column anywhere."""
    ops = operands(M, N, K, seed=M)
    bias = normal(N, seed=7)
    buf = torch.full((M + 16, -(-N // 8) * 8 + pad), 99.0, dtype=torch.bfloat16, device=DEV)
    out = buf[8:M + 8, :N]
    opq.fp8_linear(*ops, bias=bias, out=out)
    assert torch.equal(out, opq.fp8_linear(*ops, bias=bias))
    out.fill_(99.0)
    assert bool((buf == 99.0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ["none", "silu", "gelu_tanh"])
@pytest.mark.parametrize("M,N,K", list(SCHEDULES))
def test_every_schedule(M, N, K, act, dtype):
    """With a bias that differs from column to column, an activation and both types."""
    ops = operands(M, N, K, seed=N)
    bias = normal(N, seed=3, dtype=dtype)
    y = opq.fp8_linear(*ops, bias=bias, act=act, dtype=dtype)
    _, B, v = ref.linear(*ops, bias)
    dv = (128 * 2.0 ** -23 + (-(-K // 128) + 2) * 2.0 ** -24) * B + 2.0 ** -24 * (v.abs() + bias.double().abs())
    if act == "none":
        fi = torch.finfo(dtype)
        want, tol = v, dv + (v.abs() + dv) * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2
    else:
        want, z, slope = exact(v, act)
        tol = tolerance(want, z, slope, v, dv, dtype)
    err = (y.double() - want).abs()
    assert y.dtype == dtype and bool((err <= tol).all()), f"{int((~(err <= tol)).sum())} of {err.numel()} out"


def test_the_wait_limit_is_where_the_8_bit_kernels_read_it():
    assert opq.wait_limit_ns() == (4_000_000_000, 4_000_000_000)
    try:
        opq.set_wait_limit_ns(70_000_000)
        assert opq.wait_limit_ns() == (70_000_000, 70_000_000)
        check(operands(300, 700, 1024, seed=2))
    finally:
        opq.set_wait_limit_ns(0)
    assert opq.wait_limit_ns() == (4_000_000_000, 4_000_000_000)
