"""Limits of the group norm as the header states them, and a call near them."""

import ctypes

import pytest
import torch

import mamba_ssd_chunked_cumsum_amd as ssd
from mamba_ssd_chunked_cumsum_amd import block

from gpu_util import DEV, note
from test_block_abi import NO_DEVICE, UNSUPPORTED, no_gpu, tokens
from test_recurrent_abi import far


def norm(batch, seqlen, channels, groups):
    """Forward and backward of dense sequences, their two statuses."""
    t = tokens(batch=batch, seqlen=seqlen, nseq=batch, channels=channels, io_dtype=1)
    forward = block._function("ssd_group_norm")(
        ctypes.byref(t), far(1), 0, None, None, groups, 1e-5, 1, far(2), None, far(3), 1 << 43, None)
    backward = block._function("ssd_group_norm_backward")(
        ctypes.byref(t), far(1), 0, None, None, groups, 1, far(4), far(2), far(5), None, None, far(3),
        1 << 43, None)
    return forward, backward


@no_gpu
@pytest.mark.parametrize("call,taken,refused", [
    # a strip each: sequences of more than 8 tokens, groups of other widths, wide groups
    (lambda n: norm(n, 9, 8, 1), 2 ** 24 - 2, 2 ** 24 - 1),
    (lambda n: norm(n, 1, 24, 2), 2 ** 24 - 3, 2 ** 24 - 1),
    (lambda n: norm(n, 1, 8200, 1), (2 ** 24 - 258) // 17, 2 ** 24 // 17 + 1),
    # several strips each
    (lambda n: norm(n, 100, 8, 1), 2 ** 23 - 1, 2 ** 23),
    # more groups of short sequences than of long ones, whose totals take a launch of their own
    (lambda n: norm(n, 192, 64, 64), 5 * 2 ** 20, 2 ** 24),
    (lambda n: norm(n, 1000, 512, 512), 2 ** 17 - 1, 2 ** 17),
    # lanes of their own
    (lambda n: norm(n, 8, 24, 3), 2 ** 28 - 4097, 2 ** 29),
    (lambda n: norm(n, 1, 2560, 32), 2 ** 23 - 1, 2 ** 23)])
def test_stated_limits_of_dense_sequences(call, taken, refused):
    assert call(taken) == (NO_DEVICE, NO_DEVICE)
    assert call(refused) == (UNSUPPORTED, UNSUPPORTED)


@pytest.mark.gpu
def test_nearly_as_many_sequences_as_there_may_be():
    """The last sequences of a call with a strip each for nearly 2^24 of them are what they are in a call of
    70001, which takes strips too: bit for bit."""
    note("group_norm of 2^24 - 9 sequences")
    S, L, C, tail = 2 ** 24 - 9, 9, 8, 70001
    g = torch.Generator(device=DEV).manual_seed(102)
    x = torch.empty(S, L, C, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    w, b = (torch.randn(C, device=DEV, generator=g) for _ in range(2))
    y, st = ssd.group_norm(x, w, b, ngroups=1)
    y2, st2 = ssd.group_norm(x[-tail:].contiguous(), w, b, ngroups=1)
    assert torch.equal(y[-tail:], y2) and torch.equal(st[-tail:], st2)
    d = ssd.group_norm_backward(x, w, b, st, y, ngroups=1)
    d2 = ssd.group_norm_backward(x[-tail:].contiguous(), w, b, st2, y2, ngroups=1)
    assert torch.equal(d["dx"][-tail:], d2["dx"])
    # dweight and dbias against those of two halves: a block adds 7 sequences, 63 rows, in fp32, the rest is in
    # 64 bits and rounded once, so either is off by at most 64 roundings of the sum of absolute values. The
    # slope is at most 1.1, a value of 72 normalised ones at most sqrt(72)
    h = [ssd.group_norm_backward(v.contiguous(), w, b, s.contiguous(), u.contiguous(), ngroups=1)
         for v, s, u in zip(x.split(2 ** 23), st.split(2 ** 23), y.split(2 ** 23))]
    size = sum(u.abs().sum((0, 1), dtype=torch.float64) for u in y.split(2 ** 21)) * 1.1
    for k, most in (("dweight", 72 ** 0.5), ("dbias", 1.0)):
        both = sum(i[k].double() for i in h)
        assert torch.all((d[k].double() - both).abs() <= 2 * 64 * 2.0 ** -24 * most * size), k
