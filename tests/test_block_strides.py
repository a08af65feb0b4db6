"""Row strides that the binding of the operators around the scan takes, without a GPU: the device
checks are stubbed and a call that reaches the library is caught. A row stride of 0 means dense to the
library, so a broadcast tensor (rows 0 apart) or one of overlapping rows has to be refused before it."""

import pytest
import torch

import mamba_ssd_chunked_cumsum_amd as ssd
from mamba_ssd_chunked_cumsum_amd import block

Bt, L, C, G, N = 3, 9, 64, 2, 16


class Reached(Exception):
    pass


@pytest.fixture
def no_device(monkeypatch):
    def reached(name, dev, *args):
        raise Reached(name)

    def tensor(t, name, shape, dtype, dev):
        return None if t is None else t.data_ptr()

    monkeypatch.setattr(block, "_place", lambda *a: None)
    monkeypatch.setattr(block, "_tensor", tensor)
    monkeypatch.setattr(block, "_run", reached)
    monkeypatch.setattr(block, "_workspace", reached)


def z(*shape):
    return torch.zeros(*shape)


def operators(lead):
    """name -> (call of its activations by name, the activations); lead: their token dimensions."""
    act, bc = z(*lead, C), z(*lead, G, N)
    A, w, nw, h = z(C, N), z(C, 4), z(C), z(lead[0], C, N)
    five = dict(x=act, dt=act, B=bc, C=bc, z=act)
    if len(lead) == 1:
        return {
            "conv_step": (lambda x: ssd.conv_step(z(lead[0], 3, C), x, w), dict(x=act)),
            "selective_step": (lambda x, dt, B, C, z: ssd.selective_step(h, x, dt, A, B, C, nw, z),
                               five),
        }
    return {
        "conv": (lambda x: ssd.conv(x, w), dict(x=act)),
        "conv_backward": (lambda x: ssd.conv_backward(x, w, None, act), dict(x=act)),
        "selective_scan": (lambda x, dt, B, C, z: ssd.selective_scan(x, dt, A, B, C, nw, z), five),
        "selective_backward": (lambda x, dt, B, C, z: ssd.selective_backward(x, dt, A, B, C, nw, z,
                                                                             act), five),
        "gated_norm": (lambda x, z: ssd.gated_norm(x, z, nw), dict(x=act, z=act)),
        "gated_norm_backward": (lambda x, z: ssd.gated_norm_backward(x, z, nw, act),
                                dict(x=act, z=act)),
        "residual_norm": (lambda x: ssd.residual_norm(x, act, nw), dict(x=act)),
        "residual_norm_backward": (lambda x: ssd.residual_norm_backward(x, act, nw, act, scale=nw),
                                   dict(x=act)),
    }


def broadcasts(t, lead):
    """t's shape with the rows of one or every token dimension at the same place, or overlapping."""
    tail = t.shape[len(lead):]
    width = tail.numel()
    if len(lead) == 1:
        yield z(1, *tail).expand(t.shape)
    else:
        yield z(1, 1, *tail).expand(t.shape)                # over both
        yield z(1, *t.shape[1:]).expand(t.shape)            # over the batch
        yield z(lead[0], 1, *tail).expand(t.shape)          # over the tokens
    rows = t.shape[:len(lead)].numel()
    flat = z(rows * width)
    yield flat.as_strided((rows, width), (width // 2, 1)).unflatten(0, lead).unflatten(-1, tail)


@pytest.mark.parametrize("lead", [(Bt, L), (Bt, 1), (1, L), (Bt,), (2,)])
def test_broadcast_and_overlapping_rows_are_refused(no_device, lead):
    for name, (call, given) in operators(lead).items():
        for arg, t in given.items():
            with pytest.raises(Reached):
                call(**given)
            for bad in broadcasts(t, lead):
                if bad.is_contiguous():  # (a dimension of one row)
                    continue
                with pytest.raises(ValueError, match=f"^{arg}: the rows of tokens must be"):
                    call(**{**given, arg: bad})


@pytest.mark.parametrize("lead", [(Bt, L), (Bt, 1), (1, L), (1, 1), (Bt,), (1,)])
def test_rows_that_are_taken(lead):
    """Slices of wider rows with their stride; dense tensors, and a single row however it is strided,
    as dense."""
    n = len(lead)

    def rows(t):
        return block._rows(t, "x", t.shape, t.dtype, t.device, n)

    with pytest.MonkeyPatch.context() as m:
        m.setattr(block, "_place", lambda *a: None)
        m.setattr(block, "_tensor", lambda t, *a: t.data_ptr())
        wide = z(*lead, 2 * C + 8)
        single = lead == (1,) * n
        for part in (wide[..., 8:8 + C], wide[..., C:C + G * N].unflatten(-1, (G, N))):
            assert rows(part) == (part.data_ptr(), 0 if single else 2 * C + 8)
        dense = z(*lead, C)
        assert rows(dense) == (dense.data_ptr(), 0)
        one = z(*lead, C).as_strided((1,) * n + (C,), (0,) * n + (1,))
        assert rows(one) == (one.data_ptr(), 0)


@pytest.mark.gpu
def test_broadcast_inputs_write_nothing_on_the_gpu():
    """The same refusals with device tensors, and the contiguous copies of what was refused."""
    dev = "cuda:0"
    x = torch.ones(Bt, L, C, device=dev)
    step = torch.full((1, 1, C), 0.25, device=dev).expand(Bt, L, C)
    A = -torch.ones(C, N, device=dev)
    B = torch.ones(1, 1, 1, N, device=dev).expand(Bt, L, 1, N)
    out = torch.full_like(x, 7.0)
    for bad in (lambda: ssd.selective_scan(x, step, A, B.contiguous(), B.contiguous(), out=out),
                lambda: ssd.selective_scan(x, step.contiguous(), A, B, B.contiguous(), out=out),
                lambda: ssd.gated_norm(x, step, A[:, 0].contiguous(), out=out),
                lambda: ssd.conv(step, torch.ones(C, 4, device=dev), out=out)):
        with pytest.raises(ValueError, match="the rows of tokens must be"):
            bad()
    torch.cuda.synchronize()
    assert torch.all(out == 7.0)
    y, h = ssd.selective_scan(x, step.contiguous(), A, B.contiguous(), B.contiguous())
    decay = torch.exp(torch.tensor(-0.25, dtype=torch.float64))
    want = 0.25 * (1 - decay ** torch.arange(1, L + 1, dtype=torch.float64)) / (1 - decay)
    # every state entry is the same sum: L steps of two roundings and the exponential's two
    bound = 2.0 ** -24 * 8 * (L + 16) * want
    assert torch.all((h.double().cpu() - want[-1]).abs() <= bound[-1])
    assert torch.all((y.double().cpu() - N * want[None, :, None]).abs()
                     <= N * bound[None, :, None] + 2.0 ** -24 * N * N * want[None, :, None])
