"""The recurrence's longer chains against the float64 oracle element by element: the forward's chunks of
sixteen waves that wait for one another, and the backward's chains of more chunks than one round takes."""

import pytest

from test_block import name_of
from test_recurrent import run_recurrence

pytestmark = pytest.mark.gpu


# Chunks of eight waves (128 rows) of all channel tiles (128 bf16 channels, 64 fp32) are more than 256
# blocks here, those of sixteen not: 272 or 288 against 144 or 160.
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("decay,gated", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("lay", [dict(batch=2, L=1100), dict(lens=[255, 1, 0, 1000, 17, 790], spare=37)],
                         ids=name_of)
def test_chunks_of_sixteen_waves(io, decay, gated, lay):
    run_recurrence(lay, io, 2048 if io == "bf16" else 1024, 8, decay, gated, True)


# The backward's chunks are 28 bf16 or 48 fp32 rows, a round of the chain is 256 chunks: a round to its
# end, one chunk more, a part of a second, a third, and sequences that begin around the rounds' borders.
@pytest.mark.parametrize("io,decay,lay", [
    ("bf16", True, dict(batch=1, L=7168)), ("bf16", True, dict(batch=2, L=7169)),
    ("bf16", False, dict(batch=2, L=7400)), ("f32", True, dict(batch=1, L=12400)),
    ("bf16", True, dict(batch=1, L=14400)),
    ("bf16", True, dict(lens=[7100, 67, 1, 1, 0, 7000], spare=900)),
    ("f32", False, dict(lens=[3, 12285, 12, 700], spare=5))],
    ids=lambda v: name_of(v) if isinstance(v, dict) else str(v))
def test_backward_chains_of_several_rounds(io, decay, lay):
    run_recurrence(lay, io, 24, 8, decay, True, True)
