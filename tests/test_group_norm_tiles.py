"""Groups of the group norm that cross a border of the kernels' channel tiles (512 channels): every block
that needs such a group's statistics forms the same ones, bit for bit, whatever other groups it has."""

import numpy as np
import pytest
import torch

import mamba_ssd_chunked_cumsum_amd as ssd

from gpu_util import DEV, note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("C,G", [(600, 5), (768, 16), (768, 32), (1064, 7), (1536, 1)])
@pytest.mark.parametrize("L", [704, 2112])
def test_one_pair_of_statistics_a_group(C, G, L):
    """Every row holds one value in all channels, so without weights a group's outputs of a row are one
    value, too, as long as its mean and its root are one. The values cancel in pairs and span twelve powers
    of ten: what is left of their sum is decided by the order of its terms, and the outputs of the rows of
    zeros show it whole."""
    note(f"group_norm across tiles C{C} G{G} L{L}")
    rng = np.random.default_rng(101)
    n = L // 16  # runs of 16 rows: one or several make a strip
    half = rng.uniform(1, 9, n // 2 - 4) * 10.0 ** rng.integers(0, 12, n // 2 - 4)
    v = rng.permutation(np.concatenate([half, -half, np.zeros(n - 2 * len(half))]))
    x = torch.from_numpy(np.repeat(v, 16).astype(np.float32)).to(DEV)[None, :, None]
    x = torch.cat([x, x.flip(1)]).expand(2, L, C).contiguous()
    y, stats = ssd.group_norm(x, ngroups=G, activation=None)
    y = y.view(2, L, G, C // G)
    assert torch.equal(y, y[..., :1].expand_as(y))
    # the means of the backward pass, too
    unit = torch.stack([torch.zeros(2, G), torch.ones(2, G)], -1).to(DEV)
    dx = ssd.group_norm_backward(torch.zeros_like(x), None, None, unit, x, ngroups=G,
                                 activation=None)["dx"].view(2, L, G, C // G)
    assert torch.equal(dx, dx[..., :1].expand_as(dx))
