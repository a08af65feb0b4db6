"""The group norm's workspace, without a GPU."""

import ctypes

import pytest

from mamba_ssd_chunked_cumsum_amd import block

from test_block_abi import OK, tokens


@pytest.mark.parametrize("seqlen", [1, 2, 5, 9, 16, 33, 64, 100])
@pytest.mark.parametrize("channels,groups", [(1000, 50), (600, 25), (2600, 4), (20480, 2), (96, 8)])
def test_workspace_of_many_sequences_is_smaller_than_x(seqlen, channels, groups):
    n = ctypes.c_int64()
    t = tokens(batch=2 ** 18 // seqlen, seqlen=seqlen, nseq=2 ** 18 // seqlen, channels=channels,
               io_dtype=1)
    x = t.batch * seqlen * channels * 2
    for name in ("ssd_group_norm_workspace", "ssd_group_norm_backward_workspace"):
        assert block._function(name)(ctypes.byref(t), groups, ctypes.byref(n)) == OK
        assert n.value < x, (name, n.value / x)
