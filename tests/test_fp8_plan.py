"""The 8-bit linear's schedules by shape (no GPU needed)."""
import pytest

import bit_diffusion_transformer_b200 as opq
from bit_diffusion_transformer_b200 import build as opq_build
from fp8_schedules import SCHEDULES


@pytest.fixture(scope="module", autouse=True)
def built():
    opq_build.build()


@pytest.mark.parametrize("shape", list(SCHEDULES))
def test_schedule_of_each_tested_shape(shape):
    assert opq.fp8_linear_plan(*shape) == SCHEDULES[shape]


def test_every_tile_kind_is_among_them():
    kinds = {plan[:2] for plan in SCHEDULES.values()}
    assert kinds == {(16, 128), (32, 128), (64, 128), (128, 128), (128, 256), (256, 256)}


def test_refusals():
    for shape in ((0, 8, 64), (8, 0, 64), (8, 8, 0)):
        with pytest.raises(opq.OPQError, match="INVALID_ARG"):
            opq.fp8_linear_plan(*shape)
    for shape in ((8, 8, 48), (1 << 31, 8, 64), (8, 1 << 31, 64), (8, 8, 1 << 31)):
        with pytest.raises(opq.OPQError, match="UNSUPPORTED_SHAPE"):
            opq.fp8_linear_plan(*shape)
