"""GPU parity of the 8-bit format's operators against the float64 reference (fp8_reference.py):
codes and decoded values exactly, scales to one fp32 rounding, the product within a derived
tolerance (linear_tolerance)."""
import math

import pytest
import torch

import bit_diffusion_transformer_b200 as opq
import fp8_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    torch.cuda.synchronize()
    assert opq.device_error() == 0


def randn(*shape, seed=0, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def same_codes(got, want):
    """got e4m3 (GPU) holds exactly the numbers `want` (float64), NaN for NaN."""
    got = got.cpu().double()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])


def same_scales(got, want):
    # m / 448 rounded once to fp32
    assert torch.equal(got.cpu(), want.float())


def check_quantize(x, block_rows, xd=None):
    codes, scales = opq.fp8_quantize(x.to(DEV) if xd is None else xd, block_rows)
    wc, ws = ref.quantize(x, block_rows)
    assert codes.dtype == F8 and codes.shape == x.shape
    same_codes(codes, wc)
    same_scales(scales, ws)


# ---------------------------------------------------------------- quantize --
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("R,K", [(1, 32), (1, 3840), (2, 96), (31, 160), (33, 128), (128, 512), (129, 544), (300, 672)])
def test_quantize(R, K, block_rows, dtype):
    x = randn(R, K, seed=R + K, dtype=DTYPES[dtype])
    x[:, ::37] *= 30.0
    check_quantize(x, block_rows)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_special_values(block_rows, dtype):
    dt = DTYPES[dtype]
    fi = torch.finfo(dt)
    rows = [torch.zeros(128), torch.full((128,), -0.0), torch.full((128,), fi.max),
            torch.full((128,), fi.smallest_normal * fi.eps),               # the smallest subnormal
            torch.linspace(-1, 1, 128) * fi.smallest_normal * 8,           # subnormals and their neighbours
            torch.linspace(-fi.max, fi.max, 128), torch.arange(128) / 127.0]
    inf = torch.arange(128) / 16.0
    inf[5], inf[77] = math.inf, -math.inf
    nan = torch.arange(128) / 16.0
    nan[9] = math.nan
    both = torch.full((128,), math.nan)
    both[3], both[4] = -math.inf, 2.0
    only = torch.full((128,), math.inf)
    rows += [inf, nan, both, only, torch.full((128,), math.nan)]
    # exact ties: m a power of two times 7, values on every midpoint of the code grid
    grid = ref.e4m3_values()
    mid = (grid[:-1] + grid[1:]) / 2              # 126 of them
    rows += [torch.cat([torch.tensor([448.0, 0.0]), mid]).float() * s for s in (1.0, 2.0 ** -5, -2.0 ** 6)]
    x = torch.stack([r.double() for r in rows]).to(dt)
    check_quantize(x, block_rows)
    # and each alone, two blocks wide, next to an ordinary block
    for i in range(x.shape[0]):
        check_quantize(torch.cat([x[i:i + 1], randn(1, 128, seed=i, dtype=dt)], dim=1), block_rows)


def test_quantize_every_bf16_magnitude_in_a_block():
    """All finite bf16 values below several block maxima (ties, subnormal codes, tiny maxima)."""
    bits = torch.arange(0, 0x7F80, dtype=torch.int32)
    vals = (bits << 16).view(torch.float32)
    for m in (1.0, 7.0, 1.9921875, 3.0e38, 2.0 ** -63, 2.0 ** -66):
        v = vals[vals <= m]
        v = v[-127 * 200:]
        v = torch.cat([v, torch.zeros((-v.numel()) % 127)]).view(-1, 127)
        x = torch.cat([torch.full((v.shape[0], 1), m), v], dim=1).to(torch.bfloat16)
        check_quantize(x, 1)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_strides_and_guards(block_rows):
    R, K = 70, 288
    big = randn(R, 1024, seed=3)
    x = big[:, 64:64 + K]
    codes = torch.zeros((R + 2, K + 64), dtype=torch.uint8, device=DEV)
    codes.fill_(0x5A)
    sc = torch.full((3 + 2, 200), -7.0, device=DEV)
    n = R if block_rows == 1 else 1
    out = (codes.view(F8)[1:R + 1, 16:16 + K], sc[1:4, 3:3 + n])
    opq.fp8_quantize(big.to(DEV)[:, 64:64 + K], block_rows, out=out)
    wc, ws = ref.quantize(x, block_rows)
    same_codes(out[0], wc)
    same_scales(out[1], ws)
    codes[1:R + 1, 16:16 + K] = 0x5A
    sc[1:4, 3:3 + n] = -7.0
    assert bool((codes == 0x5A).all()) and bool((sc == -7.0).all())


# ------------------------------------------------------------------ linear --
def operands(M, N, K, seed=0):
    xc, xs = ref.quantize(randn(M, K, seed=seed) * (1 + 20 * (torch.arange(K) % 61 == 3)), 1)
    wc, ws = ref.quantize(randn(N, K, seed=seed + 1, scale=0.02), 128)
    return ref.to_codes(xc), xs.float(), ref.to_codes(wc), ws.float()


def check_linear(ops, bias=None, act="none", dtype=torch.bfloat16, out=None, dev_ops=None):
    xc, xs, wc, ws = ops
    y = opq.fp8_linear(*(dev_ops or [t.to(DEV) for t in ops]), bias=None if bias is None else bias.to(DEV), act=act,
                       dtype=dtype, out=out)
    want, B, v = ref.linear(xc, xs, wc, ws, bias, act)
    tol = ref.linear_tolerance(want, B, v, bias, act, dtype, xc.shape[1])
    err = (y.cpu().double() - want).abs()
    assert y.dtype == dtype and bool(torch.isfinite(y).all())
    assert bool((err <= tol).all()), f"{int((err > tol).sum())} of {err.numel()} out, worst {float((err / tol).max()):.3g} of the tolerance"
    return y


@pytest.mark.parametrize("M", [1, 2, 16, 17, 32, 33, 64, 65, 127, 129, 256, 300])
@pytest.mark.parametrize("N,K", [(1, 32), (130, 96), (128, 128), (300, 672), (513, 1280)])
def test_linear_shapes(M, N, K):
    check_linear(operands(M, N, K, seed=M))


@pytest.mark.parametrize("M,N,K", [(1, 11520, 3840), (37, 3840, 10240), (333, 2560, 3840), (1089, 3840, 640),
                                   (2048, 2304, 512), (3, 40, 32768)])
def test_linear_larger(M, N, K):
    check_linear(operands(M, N, K, seed=5))


@pytest.mark.parametrize("M,N,K,act", [
    # narrow tiles: one to eight ranges of blocks, with blocks left over, several row tiles
    (7, 40000, 384, "none"), (20, 18000, 1152, "silu"), (60, 6500, 2720, "none"), (16, 4600, 3104, "gelu_tanh"),
    (90, 2100, 2912, "none"), (130, 500, 4000, "silu"), (9, 129, 2048, "none"),
    # whole tiles on single CTAs and on pairs: one round and several, rows that TMA cannot store
    (700, 2001, 1024, "gelu_tanh"), (1000, 4104, 416, "none"), (2300, 4100, 288, "silu"), (2600, 5001, 416, "gelu_tanh"),
    (4400, 2568, 160, "none")])
def test_linear_schedules(M, N, K, act):
    check_linear(operands(M, N, K, seed=M), randn(N, seed=3), act)


def test_linear_outputs_past_31_bits():
    """2.2 G outputs: the last rows are at offsets past 2^31 elements."""
    M, N, K = 70016, 32000, 32
    x = torch.empty((M, K), dtype=torch.bfloat16, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(1))
    w = torch.empty((N, K), dtype=torch.bfloat16, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(2))
    ops = (*opq.fp8_quantize(x), *opq.fp8_quantize(w, 128))
    y = opq.fp8_linear(*ops)
    assert y.numel() > 1 << 31
    xc, xs, wc, ws = [t.cpu() for t in ops]
    for rows in (slice(0, 40), slice(M // 2, M // 2 + 40), slice(M - 40, M)):
        want, B, v = ref.linear(xc[rows], xs[:, rows], wc, ws)
        tol = ref.linear_tolerance(want, B, v, None, "none", torch.bfloat16, K)
        assert bool(((y[rows].cpu().double() - want).abs() <= tol).all())


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_past_31_bits(block_rows):
    R, K = 66000, 32768
    x = torch.empty((R, K), dtype=torch.bfloat16, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(1))
    assert x.numel() > 1 << 31
    codes, scales = opq.fp8_quantize(x, block_rows)
    for r0 in (0, 65920):                      # the last one starts a 128-row block and ends the matrix
        c, s = ref.quantize(x[r0:r0 + 128, -256:].cpu(), block_rows)
        same_codes(codes[r0:r0 + 128, -256:], c)
        same_scales(scales[-2:, r0 // block_rows:r0 // block_rows + s.shape[1]], s)


def test_linear_after_a_changed_wait_limit():
    """The bounded waits' limit reaches these kernels too, and no wait of a healthy call comes near it."""
    ops = operands(300, 700, 1024, seed=2)
    try:
        opq.set_wait_limit_ns(50_000_000)
        check_linear(ops)
        assert opq.device_error() == 0
    finally:
        opq.set_wait_limit_ns(0)
    check_linear(ops)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("act", ["none", "silu", "gelu_tanh"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 300, 512), (45, 257, 1152), (100, 130, 256), (520, 770, 640)])
def test_linear_epilogue(M, N, K, with_bias, act, dtype):
    dt = DTYPES[dtype]
    bias = randn(N, seed=9, scale=2.0, dtype=dt) if with_bias else None
    check_linear(operands(M, N, K, seed=N), bias, act, dt)


@pytest.mark.parametrize("M", [1, 40, 200, 700])
def test_linear_strides_and_guards(M):
    """Slices of a larger batch's codes and scales, padded rows, a guarded output."""
    N, K = 200, 288
    xc, xs, wc, ws = operands(M + 9, N, K, seed=M)
    wide = torch.zeros((M + 9, K + 96), dtype=torch.uint8)
    wide[:, 32:32 + K] = xc.view(torch.uint8)
    wpad = torch.full((N, K + 16), 0x7F, dtype=torch.uint8)      # NaN codes right behind each row
    wpad[:, :K] = wc.view(torch.uint8)
    y = torch.full((M + 2, N + 24), 99.0, dtype=torch.bfloat16, device=DEV)
    out = y[1:M + 1, 8:8 + N]
    dev = [wide.to(DEV).view(F8)[4:4 + M, 32:32 + K], xs.to(DEV)[:, 4:4 + M], wpad.to(DEV).view(F8)[:, :K], ws.to(DEV)]
    check_linear((xc[4:4 + M], xs[:, 4:4 + M], wc, ws), out=out, dev_ops=dev)
    out.fill_(99.0)
    assert bool((y == 99.0).all())


@pytest.mark.parametrize("M,N", [(5, 140), (300, 300)])
def test_linear_nan_stays_in_its_row(M, N):
    xc, xs, wc, ws = operands(M, N, 256, seed=1)
    clean = opq.fp8_linear(*[t.to(DEV) for t in (xc, xs, wc, ws)])
    xn = xc.view(torch.uint8).clone()
    xn[M // 2, 200] = 0x7F
    wn = wc.view(torch.uint8).clone()
    wn[N - 2, 3] = 0xFF
    y = opq.fp8_linear(xn.to(DEV).view(F8), xs.to(DEV), wn.to(DEV).view(F8), ws.to(DEV))
    bad = torch.zeros((M, N), dtype=torch.bool)
    bad[M // 2], bad[:, N - 2] = True, True
    assert torch.equal(torch.isnan(y).cpu(), bad)
    assert torch.equal(y.cpu()[~bad], clean.cpu()[~bad])


def test_linear_zero_and_extreme_scales():
    M, N, K = 20, 130, 384
    xc, xs, wc, ws = operands(M, N, K, seed=4)
    xs[:, 3] = 0.0
    xs[1] *= 2.0 ** -90
    ws[2] *= 2.0 ** 30
    y = check_linear((xc, xs, wc, ws))
    assert bool((y[3] == 0).all())


@pytest.mark.parametrize("M", [1, 50, 400])
def test_linear_repeats_bitwise(M):
    ops = [t.to(DEV) for t in operands(M, 1000, 2048, seed=M)]
    a = opq.fp8_linear(*ops)
    for _ in range(3):
        assert torch.equal(opq.fp8_linear(*ops), a)


# ------------------------------------------------------------------- cache --
def make_cache(pages, page, heads, dims, layout="token", seed=0):
    """[(codes, scales)] per tensor, CPU copies filled with recognizable content, GPU views."""
    g = torch.Generator().manual_seed(seed)
    cpu, dev = [], []
    for D in dims:
        nb = -(-D // 128)
        shape = (pages, page, heads) if layout == "token" else (pages, heads, page)
        c = torch.randint(0, 0x7F, shape + (D,), generator=g, dtype=torch.uint8)
        s = torch.rand(shape + (nb,), generator=g) + 0.5
        cd, sd = c.to(DEV), s.to(DEV)
        if layout == "head":
            c, s, cd, sd = [t.transpose(1, 2) for t in (c, s, cd, sd)]
        cpu += [c.view(F8), s]
        dev += [cd.view(F8), sd]
    return cpu, dev


def ref_write(cpu, tensors, slots, page):
    want = []
    for i, x in enumerate(tensors):
        c, s = cpu[2 * i].double(), cpu[2 * i + 1].double()
        for t, slot in enumerate(slots.tolist()):
            if 0 <= slot < c.shape[0] * page:
                for b in range(s.shape[-1]):
                    part = x[t, :, b * 128:(b + 1) * 128].double()
                    codes, sc = ref.block_codes(part)
                    c[slot // page, slot % page, :, b * 128:(b + 1) * 128] = codes
                    s[slot // page, slot % page, :, b] = sc
        want += [c, s]
    return want


def check_cache(dev, want):
    for got, w in zip(dev, want):
        (same_codes if got.dtype == F8 else same_scales)(got, w)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("T,heads,dims,page,pages", [
    (1, 1, (16, 16), 1, 3), (5, 2, (64, 64), 16, 2), (33, 3, (128, 80), 7, 9), (100, 8, (128, 128), 16, 8),
    (40, 1, (576, 512), 24, 3), (17, 5, (192, 128), 5, 6), (64, 4, (48, 256), 64, 2)])
def test_cache_write(T, heads, dims, page, pages, layout, dtype):
    dt = DTYPES[dtype]
    cpu, dev = make_cache(pages, page, heads, dims, layout, seed=T)
    kv = [randn(T, heads, D, seed=D + i, dtype=dt) for i, D in enumerate(dims)]
    kv[0][0, 0, 3] = math.inf
    kv[1][T - 1, heads - 1, 7] = math.nan
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(T))[:T].long()
    if T > 4:
        slots[2], slots[T - 1] = -1, -100
    opq.fp8_cache_write(*[t.to(DEV) for t in kv], dev, slots.to(DEV))
    check_cache(dev, ref_write(cpu, kv, slots, page))


def test_cache_write_sliced_inputs_and_one_tensor():
    """Keys as a slice of a fused projection's output; a cache of one tensor; an expanded head."""
    T, heads, D, page, pages = 21, 4, 96, 8, 4
    qkv = randn(T, 3 * heads * D, seed=2)
    k = qkv[:, heads * D:2 * heads * D].view(T, heads, D)
    cpu, dev = make_cache(pages, page, heads, (D,), seed=1)
    slots = torch.arange(T).flip(0) + 5
    opq.fp8_cache_write(qkv.to(DEV)[:, heads * D:2 * heads * D].view(T, heads, D), None, dev, slots.to(DEV))
    check_cache(dev, ref_write(cpu, [k], slots, page))
    one = randn(T, 1, D, seed=3)
    cpu, dev = make_cache(pages, page, heads, (D,), seed=1)
    opq.fp8_cache_write(one.to(DEV).expand(T, heads, D), None, dev, slots.to(DEV))
    check_cache(dev, ref_write(cpu, [one.expand(T, heads, D)], slots, page))


def test_cache_write_long():
    """Enough tokens for the several-items-per-lane variant, a partial last CTA."""
    T, heads, page, pages = 1501, 8, 16, 100
    cpu, dev = make_cache(pages, page, heads, (64, 128), seed=8)
    kv = [randn(T, heads, D, seed=D) for D in (64, 128)]
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(1))[:T].long()
    opq.fp8_cache_write(*[t.to(DEV) for t in kv], dev, slots.to(DEV))
    for i, x in enumerate(kv):
        D = x.shape[2]
        c, s = ref.quantize(x.reshape(T * heads, D), 1)
        same_codes(dev[2 * i].view(torch.uint8).view(-1, heads, D)[slots.to(DEV)].view(F8), c.view(T, heads, D))
        same_scales(dev[2 * i + 1].view(-1, heads)[slots.to(DEV)], s.view(T, heads))
    # narrow heads: eight lanes per block
    cpu, dev = make_cache(pages, page, heads, (64, 32), seed=9)
    kv = [randn(T, heads, D, seed=D) for D in (64, 32)]
    opq.fp8_cache_write(*[t.to(DEV) for t in kv], dev, slots.to(DEV))
    for i, x in enumerate(kv):
        D = x.shape[2]
        c, s = ref.quantize(x.reshape(T * heads, D), 1)
        same_codes(dev[2 * i].view(torch.uint8).view(-1, heads, D)[slots.to(DEV)].view(F8), c.view(T, heads, D))
        same_scales(dev[2 * i + 1].view(-1, heads)[slots.to(DEV)], s.view(T, heads))


def test_cache_write_nothing():
    cpu, dev = make_cache(2, 4, 2, (64, 64))
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    opq.fp8_cache_write(e, e, dev, torch.empty((0,), dtype=torch.int64, device=DEV))
    x = randn(3, 2, 64).to(DEV)
    opq.fp8_cache_write(x, x, dev, torch.full((3,), -1, dtype=torch.int64, device=DEV))
    check_cache(dev, [t.double() for t in cpu])


def test_cache_slots_out_of_range_are_skipped_and_reported():
    cpu, dev = make_cache(3, 4, 2, (64, 64))
    kv = [randn(4, 2, 64, seed=i) for i in (1, 2)]
    slots = torch.tensor([12, 3, 1 << 40, 11])
    opq.fp8_cache_write(*[t.to(DEV) for t in kv], dev, slots.to(DEV))
    check_cache(dev, ref_write(cpu, kv, slots, 4))
    assert opq.device_error() == opq.DEVERR_INDEX
    assert opq.device_error() == 0


def ref_read(cpu, table, cu, starts, page, dt, outs):
    for i, out in enumerate(outs):
        c, s = cpu[2 * i], cpu[2 * i + 1]
        for b in range(table.shape[0]):
            for r in range(int(cu[b]), int(cu[b + 1])):
                pos = r - int(cu[b]) + (int(starts[b]) if starts is not None else 0)
                if not 0 <= pos // page < table.shape[1] or not 0 <= int(table[b, pos // page]) < c.shape[0]:
                    continue
                p, o = int(table[b, pos // page]), pos % page
                # code * scale rounded to fp32, then to the output type
                v = c[p, o].double() * s[p, o].double().repeat_interleave(128, 1)[:, :c.shape[3]]
                out[r] = v.float().to(dt)
    return outs


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("lens,heads,dims,page", [
    ([1], 1, (16, 16), 1), ([0, 5, 0, 17, 1, 0], 2, (64, 64), 16), ([33, 64], 3, (128, 80), 7),
    ([100, 1, 30], 8, (128, 128), 16), ([9, 50], 1, (576, 512), 24), ([40] * 9, 5, (192, 48), 5)])
def test_cache_read(lens, heads, dims, page, layout, dtype):
    dt = DTYPES[dtype]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    cpu, dev = make_cache(pages, page, heads, dims, layout, seed=len(lens))
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(3))
    table = torch.full((len(lens), max(max(need), 1)), -5, dtype=torch.int32)   # unused entries are never read
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)
    rows = sum(lens) + 3                      # rows behind the last sequence stay as they are
    want = ref_read(cpu, table, cu, None, page, dt, [torch.full((rows, heads, D), 7.0, dtype=dt) for D in dims])
    out = [torch.full((rows, heads, D), 7.0, dtype=dt, device=DEV) for D in dims]
    got = opq.fp8_cache_read(dev, table.to(DEV), cu.to(DEV), out=out)
    for g, w in zip(got, want):
        assert torch.equal(g.cpu(), w)
    fresh = opq.fp8_cache_read(dev, table.to(DEV), cu.to(DEV), sum(lens), dtype=dt)
    for g, w in zip(fresh, want):
        assert torch.equal(g.cpu(), w[:sum(lens)])


def test_cache_read_starts_strides_and_bad_pages():
    page, pages, heads, D = 6, 8, 3, 96
    cpu, dev = make_cache(pages, page, heads, (D,), seed=4)
    table = torch.tensor([[3, 1, 7, 0], [2, 9, 5, -1], [4, 6, 0, 0]], dtype=torch.int32)
    wide = torch.zeros((3, 9), dtype=torch.int32)
    wide[:, 2:6] = table
    cu = torch.tensor([2, 12, 20, 24], dtype=torch.int32)       # rows 0 and 1 belong to no sequence
    starts = torch.tensor([5, 3, 23], dtype=torch.int32)        # the last sequence runs past its table
    want = ref_read(cpu, table, cu, starts, page, torch.bfloat16, [torch.full((26, heads, D), 7.0, dtype=torch.bfloat16)])
    buf = torch.full((heads, 26, 2 * D), 7.0, dtype=torch.bfloat16, device=DEV)
    opq.fp8_cache_read(dev, wide.to(DEV)[:, 2:6], cu.to(DEV), starts=starts.to(DEV), out=[buf[:, :, 32:32 + D].transpose(0, 1)])
    assert torch.equal(buf[:, :, 32:32 + D].transpose(0, 1).cpu(), want[0])
    buf[:, :, 32:32 + D] = 7.0
    assert bool((buf == 7.0).all())
    assert opq.device_error() == opq.DEVERR_INDEX


def test_cache_offsets_past_31_bits():
    """A cache of 2.3 GB: the last pages are written and read at byte offsets past 2^31."""
    pages, page, heads, D = 9000, 64, 16, 256
    codes = torch.zeros((pages, page, heads, D), dtype=torch.uint8, device=DEV)
    assert codes.numel() > 1 << 31
    scales = torch.zeros((pages, page, heads, 2), device=DEV)
    x = randn(65, heads, D, seed=6)
    slots = torch.arange(65) + (pages * page - 70)
    opq.fp8_cache_write(x.to(DEV), None, (codes.view(F8), scales), slots.to(DEV))
    c, s = ref.quantize(x.reshape(65 * heads, D), 1)
    flat = codes.view(-1, heads, D)
    same_codes(flat[-70:-5].view(F8), c.view(65, heads, D))
    assert int(flat[:-70].max()) == 0 and int(flat[-5:].max()) == 0
    table = torch.tensor([[pages - 2, pages - 1]], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 65], dtype=torch.int32, device=DEV)
    got, = opq.fp8_cache_read((codes.view(F8), scales), table, cu, 65, starts=torch.tensor([58], dtype=torch.int32, device=DEV))
    v = (c.view(65, heads, 2, 128) * s.float().double().view(2, 65, heads).permute(1, 2, 0)[..., None]).view(65, heads, D)
    assert torch.equal(got.cpu(), v.float().to(torch.bfloat16))


# --------------------------------------------------- refusals of the binding --
def test_binding_refusals():
    x = randn(4, 64).to(DEV)
    c, s = opq.fp8_quantize(x)
    w, sw = opq.fp8_quantize(x, 128)
    cache = [torch.zeros(2, 8, 2, 64, device=DEV).to(F8), torch.ones(2, 8, 2, 1, device=DEV)]
    kv = randn(3, 2, 64).to(DEV)
    slots = torch.arange(3, device=DEV)
    table = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    bad = [lambda: opq.fp8_quantize(x.float()), lambda: opq.fp8_quantize(x[0]), lambda: opq.fp8_quantize(x, 64),
           lambda: opq.fp8_quantize(x.t().contiguous().t()), lambda: opq.fp8_quantize(x, out=(c, s[:, :3])),
           lambda: opq.fp8_quantize(x, out=(c.view(torch.uint8), s)),
           lambda: opq.fp8_linear(c, s, w, sw, act="relu"), lambda: opq.fp8_linear(c, s, w, s),
           lambda: opq.fp8_linear(c, s.t(), w, sw), lambda: opq.fp8_linear(c, s, w[:, :32], sw),
           lambda: opq.fp8_linear(c, s, w, sw, dtype=torch.float32),
           lambda: opq.fp8_linear(c, s, w, sw, bias=torch.zeros(4, device=DEV)),
           lambda: opq.fp8_linear(c, s, w, sw, bias=torch.zeros(3, dtype=torch.bfloat16, device=DEV)),
           lambda: opq.fp8_linear(c.view(torch.uint8), s, w, sw), lambda: opq.fp8_linear(c, s.cpu(), w, sw),
           lambda: opq.fp8_linear(c, s, w, sw, out=torch.empty(4, 5, dtype=torch.bfloat16, device=DEV)),
           lambda: opq.fp8_linear(c, s, w, sw, out=torch.empty(1, 4, dtype=torch.bfloat16, device=DEV).expand(4, 4)),
           lambda: opq.fp8_cache_write(kv, kv, cache, slots), lambda: opq.fp8_cache_write(kv, None, cache[:1], slots),
           lambda: opq.fp8_cache_write(kv[:, :1], None, cache, slots), lambda: opq.fp8_cache_write(kv, None, cache, slots[:2]),
           lambda: opq.fp8_cache_write(kv, None, cache, slots.int()),
           lambda: opq.fp8_cache_write(kv, None, [cache[0][:1].expand(2, 8, 2, 64), cache[1]], slots),
           lambda: opq.fp8_cache_write(kv, None, [cache[0], cache[1][..., :0]], slots),
           lambda: opq.fp8_cache_read(cache, table, cu), lambda: opq.fp8_cache_read(cache, table, cu[:1], 1),
           lambda: opq.fp8_cache_read(cache, table.long(), cu, 1), lambda: opq.fp8_cache_read(cache, table, cu.long(), 1),
           lambda: opq.fp8_cache_read(cache, table, cu, 1, dtype=torch.float32),
           lambda: opq.fp8_cache_read(cache, table, cu, 1, starts=cu),
           lambda: opq.fp8_cache_read(cache, table, cu, 2, out=[kv[:1]])]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    for f in (lambda: opq.fp8_quantize(randn(4, 48).to(DEV)), lambda: opq.fp8_quantize(x[:0]),
              lambda: opq.fp8_linear(c[:0], s[:, :0], w, sw), lambda: opq.fp8_quantize(randn(4, 65).to(DEV)[:, 1:])):
        with pytest.raises(opq.OPQError):
            f()


# ------------------------------------------------------------ used together --
def layer(x, w, bias, ws, cache, slots, table, cu, heads, D):
    """A layer's keys and values: quantize the tokens, project, write to the cache, read back."""
    xq = opq.fp8_quantize(x)
    kv = opq.fp8_linear(*xq, *w, bias=bias)
    k, v = kv[:, :heads * D].view(-1, heads, D), kv[:, heads * D:].view(-1, heads, D)
    opq.fp8_cache_write(k, v, cache, slots)
    return kv, opq.fp8_cache_read(cache, table, cu, x.shape[0])


def layer_inputs(T, seed=0, heads=4, D=64, K=512, page=16):
    x, wt = randn(T, K, seed=seed), randn(2 * heads * D, K, seed=seed + 1, scale=0.05)
    bias = randn(2 * heads * D, seed=seed + 2)
    pages = -(-T // page) + 3
    _, cache = make_cache(pages, page, heads, (D, D), seed=seed)
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    table = perm[:-(-T // page)].int().view(1, -1)
    t = torch.arange(T)
    slots = table[0].long()[t // page] * page + t % page
    cu = torch.tensor([0, T], dtype=torch.int32)
    return x, wt, bias, cache, slots.to(DEV), table.to(DEV), cu.to(DEV), heads, D


@pytest.mark.parametrize("T", [1, 50, 300])
def test_layer_together(T):
    x, wt, bias, cache, slots, table, cu, heads, D = layer_inputs(T)
    w = opq.fp8_quantize(wt.to(DEV), 128)
    kv, (k, v) = layer(x.to(DEV), w, bias.to(DEV), None, cache, slots, table, cu, heads, D)
    xc, xs = ref.quantize(x, 1)
    wc, ws = ref.quantize(wt, 128)
    same_codes(w[0], wc)
    want, B, pre = ref.linear(xc, xs.float(), wc, ws.float(), bias)
    err = (kv.cpu().double() - want).abs()
    assert bool((err <= ref.linear_tolerance(want, B, pre, bias, "none", torch.bfloat16, x.shape[1])).all())
    # the cache step from the GPU's own projection: exact
    for got, part in ((k, kv[:, :heads * D]), (v, kv[:, heads * D:])):
        c, s = ref.quantize(part.cpu().reshape(T * heads, D), 1)
        assert torch.equal(got.cpu().view(T * heads, D), (c * s.float().double().t()).float().to(torch.bfloat16))


def test_layer_captured_and_replayed_with_new_inputs():
    x, wt, bias, cache, slots, table, cu, heads, D = layer_inputs(50)
    w = opq.fp8_quantize(wt.to(DEV), 128)
    xd, b = x.to(DEV), bias.to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(xd, w, b, None, cache, slots, table, cu, heads, D)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):                       # two graphs of the same call: nothing is shared between them
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = layer(xd, w, b, None, cache, slots, table, cu, heads, D)
        graphs.append((g, res))
    for seed in (11, 12):
        xd.copy_(randn(*x.shape, seed=seed))
        for g, (kv, (k, v)) in graphs:
            g.replay()
        torch.cuda.synchronize()
        ekv, (ek, ev) = layer(xd, w, b, None, cache, slots, table, cu, heads, D)
        for _, (kv, (k, v)) in graphs:
            assert torch.equal(kv, ekv) and torch.equal(k, ek) and torch.equal(v, ev)


def test_layers_on_two_streams_at_once():
    jobs = [layer_inputs(T, seed=T) for T in (64, 200)]
    ready = [([t.to(DEV) for t in j[:3]], j[3:]) for j in jobs]
    ws = [opq.fp8_quantize(r[0][1], 128) for r in ready]
    alone = [layer(r[0][0], w, r[0][2], None, *r[1]) for r, w in zip(ready, ws)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    outs = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(layer(ready[i][0][0], ws[i], ready[i][0][2], None, *ready[i][1]))
    torch.cuda.synchronize()
    for i in range(2):
        for kv, (k, v) in outs[i]:
            assert torch.equal(kv, alone[i][0]) and torch.equal(k, alone[i][1][0]) and torch.equal(v, alone[i][1][1])
