"""Overlapping calls of the recurrence that share one workspace, which the header leaves without defined
results: every call still ends, no access leaves its tensors, and calls with workspaces of their own are not
touched."""

import ctypes

import pytest
import torch

import mamba_ssd_chunked_cumsum_amd as ssd
from mamba_ssd_chunked_cumsum_amd import block, recurrent

from gpu_util import DEV, note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("packed", [False, True])
def test_overlapping_calls_that_share_a_workspace_end(packed):
    note(f"recurrence: a shared workspace, packed {packed}")
    g = torch.Generator(DEV).manual_seed(111)
    Bt, L, C = (1, 5000, 64) if packed else (3, 1700, 64)
    cu = torch.tensor([0, 700, 4000, 5000], dtype=torch.int32, device=DEV) if packed else None
    x = [torch.randn(Bt, L, C, device=DEV, generator=g) for _ in range(2)]
    gate = torch.randn(Bt, L, C, device=DEV, generator=g)
    want = [ssd.recurrence(v, gate, cu_seqlens=cu)[0] for v in x]
    # outputs between guards of their own kind
    room = [torch.full((3, Bt * L * C), -7.5, device=DEV) for _ in x]
    S = 3
    tok = block.SSDTokens(Bt, L, C, S, None if cu is None else cu.data_ptr(), 0, 0)
    ins = [recurrent.SSDRecurrent(v.data_ptr(), gate.data_ptr(), None, 0, 0, 0, None, None, 8.0, 0)
           for v in x]
    n = ctypes.c_int64()
    assert block._function("ssd_recurrence_workspace")(ctypes.byref(tok), ctypes.byref(ins[0]),
                                                       ctypes.byref(n)) == 0 and n.value
    guard = 1 << 16
    ws = torch.zeros(n.value + 2 * guard, dtype=torch.uint8, device=DEV)
    streams = [torch.cuda.Stream() for _ in x]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, q, y in zip(streams, ins, room):
            assert block._function("ssd_recurrence")(
                ctypes.byref(tok), ctypes.byref(q), y[1].data_ptr(), None, ws.data_ptr() + guard, n.value,
                s.cuda_stream) == 0
        torch.cuda.synchronize()
    for y in room:
        assert torch.all(y[0] == -7.5) and torch.all(y[2] == -7.5)
    assert not ws[:guard].any() and not ws[-guard:].any()
    for v, w in zip(x, want):
        assert torch.equal(ssd.recurrence(v, gate, cu_seqlens=cu)[0], w)
