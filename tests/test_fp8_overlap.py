"""Caches and outputs whose elements share memory are refused where they are written: two CTAs would
write one place in any order (no GPU needed)."""
import pytest

from bit_diffusion_transformer_b200 import fp8
from test_fp8_abi import HOST, INVALID, _side, _write, buf, lib  # noqa: F401 (fixtures)

# pages 2, page 8, heads 2, head_dim 64 in _write; every stride that makes elements meet
OVERLAPPING = [dict(page_stride=1008), dict(page_stride=16), dict(token_stride=112), dict(token_stride=64),
               dict(head_stride=48), dict(head_stride=0), dict(token_stride=0), dict(page_stride=0),
               dict(scale_page_stride=15), dict(scale_token_stride=1), dict(scale_head_stride=0),
               dict(head_stride=512, token_stride=48)]
# other orders and gaps
APART = [dict(), dict(head_stride=512, token_stride=64), dict(page_stride=128, token_stride=256),
         dict(page_stride=4096, token_stride=256, head_stride=128), dict(scale_head_stride=8, scale_token_stride=1),
         dict(scale_page_stride=100, scale_token_stride=7, scale_head_stride=3)]


@pytest.mark.parametrize("kw", OVERLAPPING)
def test_overlapping_cache_is_not_written(lib, buf, kw):  # noqa: F811
    assert _write(lib, buf, side=_side(buf, **kw)) == INVALID


@pytest.mark.parametrize("kw", APART)
def test_other_layouts_are(lib, buf, kw):  # noqa: F811
    assert _write(lib, buf, side=_side(buf, **kw)) == HOST       # (past the checks: the memory is the host's)


def test_strides_of_single_entries_do_not_count(lib, buf):  # noqa: F811
    one = _side(buf, page_stride=0, token_stride=0, head_stride=0, scale_page_stride=0, scale_token_stride=0,
                scale_head_stride=0)
    assert _write(lib, buf, side=one, pages=1, page=1, heads=1) == HOST
    assert _write(lib, buf, side=one, pages=2, page=1, heads=1) == INVALID


def test_inputs_may_overlap_and_outputs_may_not(lib, buf):  # noqa: F811
    def read(row, side=None):
        c, r = (fp8.Fp8Cache * 1)(side or _side(buf)), (fp8.Fp8Rows * 1)(row)
        return lib.opq_fp8_cache_read(c, r, 1, 2, 8, 2, 0, 3, buf(), 1, buf(), 2, 2, None, None)
    for strides in ((0, 64), (128, 0), (120, 64), (64, 32), (32, 96)):
        row = fp8.Fp8Rows(buf(), *strides)
        assert _write(lib, buf, row=row) == HOST, strides        # a head shared by all: read only
        assert read(row) == INVALID, strides
    assert read(fp8.Fp8Rows(buf(), 64, 192)) == HOST and read(fp8.Fp8Rows(buf(), 128, 64)) == HOST
    assert read(fp8.Fp8Rows(buf(), 128, 64), _side(buf, token_stride=64)) == HOST      # the cache is only read
