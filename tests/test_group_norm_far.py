"""Group norm of values far from zero where sequences are cut into strips and tiles: mean and variance of a
group are put together from pieces, and neither the pieces' nor their sums may lose the variance to the
size of the mean. Against the float64 oracle element by element."""

import pytest

from test_block import name_of
from test_recurrent import run_group_norm

pytestmark = pytest.mark.gpu


# a strip or two, many, sequences of a few rows and of none in one, groups across tiles; the narrow groups of
# few rows have nothing to average a rounding over
@pytest.mark.parametrize("lay", [dict(batch=25, L=2), dict(batch=3, L=130), dict(batch=2, L=2100),
                                 dict(lens=[3, 0, 1, 2, 40, 300, 7], spare=20)], ids=name_of)
@pytest.mark.parametrize("io,C,G,shift", [
    ("f32", 96, 48, 100.0), ("f32", 96, 48, 1000.0), ("f32", 24, 2, 1000.0), ("f32", 1064, 7, -1000.0),
    ("bf16", 40, 10, 30.0)])
def test_values_far_from_zero_in_strips(lay, io, C, G, shift):
    run_group_norm(lay, io, C, G, 8, False, "both", shift=shift)
