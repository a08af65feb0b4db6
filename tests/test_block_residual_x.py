"""The residual norm's backward reads x only where there is a scale; without one nothing about x but
its shape and type matters, neither its address nor its rows."""

import ctypes

import pytest
import torch

import mamba_ssd_chunked_cumsum_amd as ssd
from mamba_ssd_chunked_cumsum_amd import block

from test_block_abi import INVALID, NO_DEVICE, addr, no_gpu, tokens


@no_gpu
@pytest.mark.parametrize("kw", [dict(x=None), dict(x=addr(0, 4)), dict(xs=36), dict(xs=68),
                                dict(x=addr(6)), dict(x=addr(5)), dict(x=addr(9))])
def test_x_is_not_checked_without_a_scale(kw):
    """Null, misaligned, with strides that are refused elsewhere, and at the outputs' addresses."""
    def call(scale, x=addr(0), xs=0):
        t = tokens(seqlen=7)
        return block._function("ssd_residual_norm_backward")(
            ctypes.byref(t), addr(1), 0, x, xs, scale, addr(3), 1e-5, addr(4), None, addr(5),
            addr(6), addr(7), addr(8) if scale else None, addr(9), 1 << 30, None)

    assert call(None, **kw) == call(addr(2)) == NO_DEVICE
    assert call(addr(2), **kw) == INVALID


@pytest.mark.gpu
def test_any_x_will_do_without_a_scale():
    rng = torch.Generator(device="cuda:0").manual_seed(61)
    r, dy = (torch.randn(2, 7, 64, device="cuda:0", generator=rng) for _ in range(2))
    w = torch.randn(64, device="cuda:0", generator=rng)
    want = ssd.residual_norm_backward(r, r, w, dy)
    wide = torch.zeros(2, 7, 101, device="cuda:0")
    for x in (wide[..., 3:67], wide[:, :, :64], w.expand(2, 7, 64)):
        got = ssd.residual_norm_backward(x, r, w, dy)
        for k in ("dx", "dresidual", "dweight"):
            assert torch.equal(got[k], want[k])
