"""More packed sequences than 2^30 on the GPU: all but the last few are empty, so the results are those
of the last few alone. Indexes of sequences, and sums of two of them, pass 31 bits here."""

import pytest
import torch

import mamba_ssd_chunked_cumsum_amd as ssd

from gpu_util import DEV, note

pytestmark = pytest.mark.gpu


def offsets(S, ends):
    cu = torch.zeros(S + 1, dtype=torch.int32, device=DEV)
    cu[S + 1 - len(ends):] = torch.tensor(ends, dtype=torch.int32, device=DEV)
    return cu, torch.tensor([0, *ends], dtype=torch.int32, device=DEV)


def inputs(rows, C, W):
    g = torch.Generator(device=DEV).manual_seed(51)
    return [torch.randn(*s, device=DEV, generator=g) for s in ((1, rows, C), (C, W), (1, rows, C))]


def test_search_among_many_sequences():
    """The middle of two indexes whose sum passes 31 bits."""
    S = 1_600_000_000
    note(f"conv over {S} sequences")
    cu, few = offsets(S, [3, 5, 8])
    x, w, dy = inputs(8, 8, 4)
    y, _ = ssd.conv(x, w, cu_seqlens=cu, want_final=False)
    g = ssd.conv_backward(x, w, None, dy, cu_seqlens=cu, want_initial_grad=False)
    torch.cuda.synchronize()
    y2, _ = ssd.conv(x, w, cu_seqlens=few, want_final=False)
    g2 = ssd.conv_backward(x, w, None, dy, cu_seqlens=few, want_initial_grad=False)
    assert torch.equal(y, y2)
    assert torch.equal(g["dx"], g2["dx"]) and torch.equal(g["dweight"], g2["dweight"])


def test_rows_and_final_states_of_many_sequences():
    """Strips of rows and the sequences' final states in one launch: together more than 2^31."""
    S, rows = (1 << 31) - 4097, 40000
    note(f"conv over {S} sequences with final states")
    cu, few = offsets(S, [3, 5, rows])
    x, w, _ = inputs(rows, 8, 2)
    x = x.to(torch.bfloat16)
    y, f = ssd.conv(x, w, cu_seqlens=cu)
    torch.cuda.synchronize()
    y2, f2 = ssd.conv(x, w, cu_seqlens=few)
    assert torch.equal(y, y2) and torch.equal(f[-3:], f2)
    step = 1 << 28
    for i in range(0, S - 3, step):  # the others begin and stay at zero
        assert not f[i:min(i + step, S - 3)].flatten().view(torch.int32).any()
    del f, cu
    torch.cuda.empty_cache()
