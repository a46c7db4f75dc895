"""opq_fp8_*: arguments refused before any launch (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import bit_diffusion_transformer_b200 as opq
from bit_diffusion_transformer_b200 import build as opq_build
from bit_diffusion_transformer_b200 import fp8

INVALID, SHAPE, MISALIGNED, HOST = 1, 2, 3, 6


@pytest.fixture(scope="module")
def lib():
    opq_build.build()
    return opq.load()


@pytest.fixture
def buf():
    keep = []

    def make(off=0):
        a = np.zeros(4096 + 64, np.uint8)
        keep.append(a)
        return ctypes.c_void_p(a.ctypes.data + (-a.ctypes.data) % 16 + off)
    return make


def test_quantize_refusals(lib, buf):
    def q(x="x", dtype=0, R=4, K=64, ldx=64, rows=1, codes="c", ldc=64, scales="s", lds=4):
        x, codes, scales = [buf() if isinstance(p, str) else p for p in (x, codes, scales)]
        return lib.opq_fp8_quantize(x, dtype, R, K, ldx, rows, codes, ldc, scales, lds, None)
    for kw in (dict(x=None), dict(codes=None), dict(scales=None), dict(dtype=2), dict(dtype=-1), dict(R=0), dict(K=0),
               dict(R=-1), dict(rows=0), dict(rows=64), dict(rows=2), dict(ldx=56), dict(ldx=68), dict(ldc=48),
               dict(ldc=72), dict(lds=3)):
        assert q(**kw) == INVALID, kw
    assert q(K=48, ldx=48, ldc=48) == SHAPE
    assert q(K=1 << 32, ldx=1 << 32, ldc=1 << 32) == SHAPE
    assert q(x=buf(2)) == MISALIGNED and q(codes=buf(8)) == MISALIGNED and q(scales=buf(2)) == MISALIGNED
    assert q() == HOST and q(rows=128, lds=1) == HOST and q(scales=buf(4)) == HOST


def test_linear_refusals(lib, buf):
    def lin(x="x", ldx=64, xs="xs", ldxs=4, M=4, K=64, w="w", ldw=64, ws="ws", ldws=1, N=8, bias=None, act=0, y="y",
            dtype=0, ldy=8):
        x, xs, w, ws, y = [buf() if isinstance(p, str) else p for p in (x, xs, w, ws, y)]
        return lib.opq_fp8_linear(x, ldx, xs, ldxs, M, K, w, ldw, ws, ldws, N, bias, act, y, dtype, ldy, None)
    for kw in (dict(x=None), dict(w=None), dict(xs=None), dict(ws=None), dict(y=None), dict(M=0), dict(N=0), dict(K=0),
               dict(M=-5), dict(act=3), dict(act=-1), dict(dtype=7), dict(ldx=48), dict(ldx=72), dict(ldw=48),
               dict(ldw=72), dict(ldy=7), dict(ldxs=3), dict(ldws=0), dict(N=129, ldy=129, ldws=1)):
        assert lin(**kw) == INVALID, kw
    for kw in (dict(K=48, ldx=48, ldw=48), dict(M=1 << 31, ldxs=1 << 31), dict(N=1 << 31, ldy=1 << 31, ldws=1 << 30)):
        assert lin(**kw) == SHAPE, kw
    for kw in (dict(x=buf(8)), dict(w=buf(4)), dict(y=buf(2)), dict(xs=buf(2)), dict(ws=buf(1))):
        assert lin(**kw) == MISALIGNED, kw
    assert lin() == HOST


def _side(buf, **kw):
    f = dict(codes=buf(), scales=buf(), head_dim=64, page_stride=1024, token_stride=128, head_stride=64,
             scale_page_stride=16, scale_token_stride=2, scale_head_stride=1)
    f.update(kw)
    return fp8.Fp8Cache(**f)


def _write(lib, buf, side=None, row=None, tensors=1, pages=2, page=8, heads=2, dtype=0, tokens=3, slots="s"):
    c = (fp8.Fp8Cache * 2)(side or _side(buf), side or _side(buf))
    r = (fp8.Fp8Rows * 2)(*[row or fp8.Fp8Rows(buf(), 128, 64)] * 2)
    return lib.opq_fp8_cache_write(c, r, tensors, pages, page, heads, dtype, tokens, buf() if slots == "s" else slots, None)


SIDE_ERRORS = [(dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(head_dim=0), INVALID),
               (dict(head_dim=24), SHAPE), (dict(head_dim=131072), SHAPE), (dict(page_stride=-16), INVALID),
               (dict(token_stride=8), MISALIGNED), (dict(head_stride=40), MISALIGNED),
               (dict(scale_token_stride=-1), INVALID)]


def test_cache_write_refusals(lib, buf):
    for kw, want in SIDE_ERRORS:
        assert _write(lib, buf, side=_side(buf, **kw)) == want, kw
    assert _write(lib, buf, side=_side(buf, codes=buf(8))) == MISALIGNED
    assert _write(lib, buf, side=_side(buf, scales=buf(2))) == MISALIGNED
    for kw in (dict(tensors=0), dict(tensors=3), dict(pages=0), dict(page=0), dict(heads=0), dict(dtype=2),
               dict(tokens=-1), dict(slots=None), dict(row=fp8.Fp8Rows(None, 128, 64)),
               dict(row=fp8.Fp8Rows(buf(), -128, 64))):
        assert _write(lib, buf, **kw) == INVALID, kw
    for kw in (dict(pages=1 << 32), dict(page=1 << 32), dict(heads=1 << 31), dict(tokens=1 << 31), dict(tokens=1 << 40)):
        assert _write(lib, buf, **kw) in (SHAPE, HOST), kw
    for kw in (dict(slots=buf(4)), dict(row=fp8.Fp8Rows(buf(), 132, 64)), dict(row=fp8.Fp8Rows(buf(8), 128, 64))):
        assert _write(lib, buf, **kw) == MISALIGNED, kw
    assert _write(lib, buf, tokens=0, slots=None) == 0        # nothing to do
    assert _write(lib, buf) == HOST and _write(lib, buf, tensors=2) == HOST


def test_cache_read_refusals(lib, buf):
    def read(side=None, row=None, tensors=1, pages=2, page=8, heads=2, dtype=0, rows=3, cu="c", seqs=1, table="t", ld=2,
             width=2, starts=None):
        c = (fp8.Fp8Cache * 2)(side or _side(buf), side or _side(buf))
        r = (fp8.Fp8Rows * 2)(*[row or fp8.Fp8Rows(buf(), 128, 64)] * 2)
        return lib.opq_fp8_cache_read(c, r, tensors, pages, page, heads, dtype, rows, buf() if cu == "c" else cu, seqs,
                                      buf() if table == "t" else table, ld, width, starts, None)
    for kw, want in SIDE_ERRORS:
        assert read(side=_side(buf, **kw)) == want, kw
    for kw in (dict(tensors=0), dict(tensors=3), dict(pages=0), dict(page=0), dict(heads=0), dict(dtype=-1),
               dict(rows=-1), dict(seqs=-1), dict(cu=None), dict(table=None), dict(width=0), dict(ld=1),
               dict(row=fp8.Fp8Rows(None, 128, 64))):
        assert read(**kw) == INVALID, kw
    for kw in (dict(cu=buf(2)), dict(table=buf(1)), dict(starts=buf(2)), dict(row=fp8.Fp8Rows(buf(), 128, 12))):
        assert read(**kw) == MISALIGNED, kw
    assert read(rows=1 << 31) == SHAPE and read(seqs=1 << 31) == SHAPE
    assert read(rows=0) == 0 and read(seqs=0) == 0
    assert read() == HOST and read(tensors=2) == HOST


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(4, 64).to(torch.float8_e4m3fn), torch.ones(1, 4)
    with pytest.raises(ValueError):
        opq.fp8_quantize(x)
    with pytest.raises(ValueError):
        opq.fp8_linear(c, s, c, torch.ones(1, 1))
    cache = (torch.zeros(2, 8, 2, 64).to(torch.float8_e4m3fn), torch.ones(2, 8, 2, 1))
    with pytest.raises(ValueError):
        opq.fp8_cache_write(torch.zeros(3, 2, 64, dtype=torch.bfloat16), None, cache, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        opq.fp8_cache_read(cache, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 1)


def test_division_by_multiplication():
    """The kernels' n / d for n < 2^31 (a multiplication and a shift), as computed on the host side:
    shift 31 + s with 2^s >= d, multiplier ceil(2^(31 + s) / d)."""
    rng = np.random.default_rng(0)
    ds = list(range(1, 300)) + [2 ** k + e for k in range(9, 31) for e in (-1, 0, 1)] + [2 ** 31 - 1]
    for d in ds:
        s = 0
        while (1 << s) < d:
            s += 1
        mul = -(-(1 << (31 + s)) // d)
        assert mul < 1 << 32
        ns = np.concatenate([rng.integers(0, 2 ** 31, 50), [0, 1, d - 1, d, 2 ** 31 - 1],
                             (rng.integers(1, max(2, 2 ** 31 // d), 20) * d - 1)])
        for n in ns.tolist():
            if 0 <= n < 2 ** 31:
                assert (n * mul) >> (31 + s) == n // d
