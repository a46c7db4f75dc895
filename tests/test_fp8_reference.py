"""The float64 reference of the 8-bit format against torch's own e4m3 type and hand-worked blocks,
and mistakes planted in it that these checks catch."""
import math

import torch

import fp8_reference as ref


def test_grid_is_the_e4m3_type():
    bits = torch.arange(0x7F, dtype=torch.uint8)
    assert torch.equal(bits.view(ref.F8).double(), ref.e4m3_values())


def test_nearest_ties_to_even_against_exact_midpoints():
    grid = ref.e4m3_values()
    mid = (grid[:-1] + grid[1:]) / 2
    got = ref.nearest_e4m3(mid)
    even = torch.where(torch.arange(mid.numel()) % 2 == 0, grid[:-1], grid[1:])
    assert torch.equal(got, even)
    assert torch.equal(ref.nearest_e4m3(mid * (1 - 2.0 ** -40)), grid[:-1])
    assert torch.equal(ref.nearest_e4m3(mid * (1 + 2.0 ** -40)), grid[1:])
    assert torch.equal(ref.nearest_e4m3(-mid), -even)
    assert torch.equal(ref.nearest_e4m3(mid), mid.float().to(ref.F8).double())


def test_hand_worked_block():
    # m = 7: scale 1/64, codes 64 x: 7 -> 448, 3.5 -> 224, 0.25 -> 16, 3.3125 -> 212 (between 208 and
    # 224, nearer 208), 1.0625 -> 68 (a tie of 64 and 72: 64 has the even code)
    x = torch.tensor([7.0, -3.5, 0.25, 3.3125, 1.0625, 0.0, math.inf, -math.inf], dtype=torch.float64)
    c, s = ref.block_codes(x)
    assert float(s) == 1.0 / 64
    assert c.tolist() == [448.0, -224.0, 16.0, 208.0, 64.0, 0.0, 448.0, -448.0]
    c, s = ref.block_codes(torch.tensor([math.nan, 2.0 ** -70, 0.0], dtype=torch.float64))
    assert float(s) == 2.0 ** -64 / 448 and math.isnan(c[0]) and float(c[1]) == 7.0


def test_blocks_and_decode():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(130, 160, generator=g).to(torch.bfloat16)
    for rows in (1, 128):
        c, s = ref.quantize(x, rows)
        assert s.shape == (2, -(-130 // rows))
        d = ref.decode(c, s, rows)
        # half a step of a 3-bit mantissa, or half of the smallest step at the block's scale
        sc = ref.decode(torch.ones(130, 160), s, rows)
        assert ((d - x.double()).abs() <= torch.maximum(x.double().abs() * 2.0 ** -4, sc * 2.0 ** -10) * (1 + 1e-12)).all()
    assert float(ref.quantize(x, 128)[1][1, 1]) == float(x[128:, 128:].double().abs().max()) / 448


def test_linear_reference_against_loops():
    g = torch.Generator().manual_seed(2)
    x, w = torch.randn(3, 160, generator=g), torch.randn(130, 160, generator=g)
    xc, xs = ref.quantize(x, 1)
    wc, ws = ref.quantize(w, 128)
    y, B, _ = ref.linear(xc, xs, wc, ws)
    for m, n in ((0, 0), (2, 129), (1, 127), (2, 128)):
        t = [float(xc[m, k] * wc[n, k] * xs[k // 128, m] * ws[k // 128, n // 128]) for k in range(160)]
        assert abs(float(y[m, n]) - math.fsum(t)) < 1e-12 * float(B[m, n])
    # a scale taken from the neighbouring row, block or column block is seen
    tol = ref.linear_tolerance(y, B, y, None, "none", torch.bfloat16, 160)
    for bad in (ref.linear(xc, xs.roll(1, 1), wc, ws)[0], ref.linear(xc, xs.roll(1, 0), wc, ws)[0],
                ref.linear(xc, xs, wc, ws.roll(1, 1))[0], ref.linear(xc, xs, wc, ws.roll(1, 0))[0]):
        assert ((bad - y).abs() > tol).any()
