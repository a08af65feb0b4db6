"""Limits of the recurrence as the header states them: rows (dense: of sequences rounded up to 28) times
channel tiles below 2^28, for short sequences too, however many states they have."""

import pytest
import torch

import mamba_ssd_chunked_cumsum_amd as ssd

from gpu_util import DEV, note
from test_block_abi import NO_DEVICE, UNSUPPORTED, no_gpu, tokens
from test_recurrent_abi import BARE, Recurrence, far


@no_gpu
@pytest.mark.parametrize("seqlen,channels,io,taken,refused", [
    (1, 1024, 1, 2 ** 20, 2 ** 26), (1, 976, 1, 849592, 2 ** 26), (12, 50648, 1, 21179, 2 ** 24),
    (11, 4952, 0, 108595, 2 ** 23), (100, 8192, 1, 37449, 2 ** 21)])
def test_many_short_sequences_are_taken(seqlen, channels, io, taken, refused):
    for n, status in ((taken, NO_DEVICE), (refused, UNSUPPORTED)):
        t = tokens(batch=n, seqlen=seqlen, nseq=n, channels=channels, io_dtype=io)
        r = Recurrence(t=t, x=far(0), gate=far(1), y=far(2), fin=far(3), ws=far(4), n=1 << 43,
                       dy=far(5), df=None, dx=far(6), dg=far(7), di=None, dd=None, dh=far(8), **BARE)
        assert r.forward() == r.backward() == status
        if seqlen == 1:
            r.q["initial_state"] = far(9)
            assert r.step() == status


@pytest.mark.gpu
def test_states_past_two_to_the_29():
    """The last sequences of a call with more than 2^29 states are what they are alone, bit for bit."""
    note("recurrence of 2^29 states")
    S, C, tail = 560001, 976, 33
    assert S * C > 2 ** 29
    g = torch.Generator(device=DEV).manual_seed(103)
    x, gate, dy = (torch.empty(S, 1, C, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
                   for _ in range(3))
    h0 = torch.empty(S, C, device=DEV).normal_(generator=g)
    decay = torch.randn(C, device=DEV, generator=g)
    end = [v[-tail:].contiguous() for v in (x, gate, dy, h0)]
    y, f = ssd.recurrence(x, gate, decay, None, h0)
    y2, f2 = ssd.recurrence(end[0], end[1], decay, None, end[3])
    assert torch.equal(y[-tail:], y2) and torch.equal(f[-tail:], f2)
    d = ssd.recurrence_backward(x, gate, decay, None, dy, h0)
    d2 = ssd.recurrence_backward(end[0], end[1], decay, None, end[2], end[3])
    for k in ("dx", "dgate", "dinitial_state"):
        assert torch.equal(d[k][-tail:], d2[k]), k
    y, f = ssd.recurrence_step(h0, x[:, 0], gate[:, 0], decay)
    y2, f2 = ssd.recurrence_step(end[3], end[0][:, 0], end[1][:, 0], decay)
    assert torch.equal(y[-tail:], y2) and torch.equal(f[-tail:], f2)
