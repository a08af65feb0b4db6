"""The limits that include/ssd.h states for the operators around the scan, on the host: the largest size is
taken and one more refused (placeholder addresses, never dereferenced)."""

import ctypes

import pytest

from mamba_ssd_chunked_cumsum_amd import block

from test_block_abi import NO_DEVICE, UNSUPPORTED, len3, no_gpu, ptr3, tokens

MOST_ROWS = 2 ** 31 - 4097


def addr(i):
    return (1 << 50) + (i << 44)


def packed(rows, nseq, channels=8):
    return tokens(batch=1, seqlen=rows, channels=channels, nseq=nseq, seq_starts=addr(9))


def conv(t, stride=0):
    return block._function("ssd_conv")(ctypes.byref(t), addr(0), stride, addr(1), None, 2, 1, None,
                                       ptr3(addr(2), None, None), len3(t.channels, 0, 0), None, None)


def gated(rows, channels, groups):
    t = tokens(batch=1, seqlen=rows, channels=channels, nseq=1)
    return block._function("ssd_gated_norm")(ctypes.byref(t), addr(0), 0, None, 0, addr(1), groups,
                                             1e-5, 0, addr(2), None)


@no_gpu
@pytest.mark.parametrize("call,most", [
    (lambda n: conv(packed(n, 1)), MOST_ROWS), (lambda n: conv(packed(1, n)), MOST_ROWS),
    (lambda n: conv(packed(1, 1, 8 * n)), 2 ** 17),
    (lambda n: conv(packed(2 ** 20, 1), 8 * n), 2 ** 17),  # rows times row stride
    (lambda n: gated(n, 8, 1), 2 ** 26 - 1), (lambda n: gated(n, 1024, 1), 2 ** 26 - 1),
    (lambda n: gated(n, 128, 16), 2 ** 22 - 1), (lambda n: gated(n, 1032, 1), 2 ** 23 - 1),
    (lambda n: gated(n, 8192, 1), 2 ** 23 - 1)])
def test_stated_limits(call, most):
    assert call(most) == NO_DEVICE
    assert call(most + 1) == UNSUPPORTED
