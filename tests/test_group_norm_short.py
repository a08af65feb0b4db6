"""Group norm over short sequences in groups of any width, so many that blocks of the backward pass take
several of them in turn, against the float64 oracle element by element."""

import pytest

from test_recurrent import run_group_norm

pytestmark = pytest.mark.gpu


# strips shared by many sequences, by few, a last strip that is not full, one sequence a strip
@pytest.mark.parametrize("io,batch,L,C,G", [
    ("bf16", 9001, 1, 600, 50), ("f32", 5003, 1, 24, 2), ("bf16", 4099, 3, 40, 8), ("f32", 2100, 7, 1064, 7),
    ("bf16", 6007, 9, 64, 1), ("f32", 4200, 12, 600, 5), ("bf16", 2057, 31, 520, 5), ("bf16", 5000, 2, 8200, 1),
    ("f32", 4100, 33, 24, 1), ("f32", 1500, 1, 2600, 4)])
@pytest.mark.parametrize("affine", ["both", None])
def test_many_short_sequences(io, batch, L, C, G, affine):
    run_group_norm(dict(batch=batch, L=L), io, C, G, 8, affine == "both", affine)
