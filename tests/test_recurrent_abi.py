"""The operators of layers of linear recurrence without a GPU: invalid requests are rejected on the host
before any HIP call, by the C ABI (placeholder addresses, never dereferenced) and by the binding;
the stated limits; row strides; and no kernel spills registers."""

import ctypes
import os

import pytest
import torch

import mamba_ssd_chunked_cumsum_amd as ssd
from mamba_ssd_chunked_cumsum_amd import block, libssd, recurrent

from test_block_abi import INVALID, NO_DEVICE, OK, PACKED, UNSUPPORTED, addr, no_gpu, one, tokens
from test_block_strides import Reached, broadcasts, no_device  # noqa: F401
from test_build import BUILD, _kernel_descriptors


def test_exports_and_struct_layouts():
    assert set(recurrent.EXPORTS) <= set(libssd.EXPORTS)
    assert ctypes.sizeof(recurrent.SSDRecurrent) == 72
    assert ctypes.sizeof(recurrent.SSDRotation) == 136


class Recurrence:
    """A valid call of ssd_recurrence, its step or its backward, with fields to spoil."""

    def __init__(self, **kw):
        self.t = tokens()
        self.q = dict(x=addr(0), gate=addr(1), input_gate=addr(2), x_stride=0, gate_stride=0,
                      input_gate_stride=0, decay=addr(3), initial_state=addr(4), sharpness=8.0,
                      reserved=0)
        self.y, self.fin, self.dy, self.df = addr(5), addr(6), addr(7), addr(8)
        self.dx, self.dg, self.di, self.dd, self.dh = (addr(i) for i in range(9, 14))
        self.ws, self.n = addr(15), 1 << 33
        for k, v in kw.items():
            if k in self.q:
                self.q[k] = v
            else:
                setattr(self, k, v)

    def _args(self):
        names = [n for n, _ in recurrent.SSDRecurrent._fields_]
        return ctypes.byref(self.t), ctypes.byref(recurrent.SSDRecurrent(*(self.q[n] for n in names)))

    def forward(self):
        return block._function("ssd_recurrence")(*self._args(), self.y, self.fin, self.ws, self.n,
                                                 None)

    def step(self):
        return block._function("ssd_recurrence_step")(*self._args(), self.fin, self.y, None)

    def backward(self):
        return block._function("ssd_recurrence_backward")(
            *self._args(), self.dy, self.df, self.dx, self.dg, self.di, self.dd, self.dh, self.ws,
            self.n, None)


BARE = dict(input_gate=None, decay=None, initial_state=None)


@no_gpu
def test_recurrence_valid_requests_report_no_device():
    assert Recurrence().forward() == Recurrence().backward() == NO_DEVICE
    assert Recurrence(t=tokens(**PACKED)).forward() == NO_DEVICE
    assert Recurrence(t=tokens(**PACKED)).backward() == NO_DEVICE
    assert Recurrence(t=one()).step() == Recurrence(t=one(), fin=addr(4)).step() == NO_DEVICE
    assert Recurrence(fin=None, ws=None, n=0, gate_stride=72, sharpness=0.0, **BARE).forward() == \
        NO_DEVICE
    assert Recurrence(t=tokens(seqlen=28), di=None, dd=None, df=None, dh=None, ws=None, n=0,
                      **BARE).backward() == NO_DEVICE


@no_gpu
@pytest.mark.parametrize("kw,status", [
    (dict(t=tokens(batch=0)), INVALID), (dict(t=tokens(seqlen=0)), INVALID),
    (dict(t=tokens(nseq=3)), INVALID), (dict(t=tokens(io_dtype=2)), INVALID),
    (dict(t=tokens(channels=60)), UNSUPPORTED), (dict(reserved=1), INVALID),
    (dict(t=tokens(batch=1, nseq=3, seq_starts=addr(60, 2))), INVALID),
    (dict(x=None), INVALID), (dict(gate=None), INVALID), (dict(y=None), INVALID),
    (dict(x=addr(0, 8)), INVALID), (dict(gate=addr(1, 8)), INVALID),
    (dict(input_gate=addr(2, 8)), INVALID), (dict(decay=addr(3, 4)), INVALID),
    (dict(initial_state=addr(4, 4)), INVALID), (dict(y=addr(5, 8)), INVALID),
    (dict(x_stride=56), INVALID), (dict(gate_stride=68), INVALID),
    (dict(input_gate_stride=-64), INVALID),
    (dict(sharpness=0.0), INVALID), (dict(sharpness=-1.0), INVALID),
    (dict(sharpness=float("nan")), INVALID), (dict(sharpness=float("inf")), INVALID),
    (dict(y=addr(0)), INVALID), (dict(y=addr(1)), INVALID), (dict(y=addr(2)), INVALID),
    (dict(fin=addr(4)), INVALID), (dict(fin=addr(5)), INVALID), (dict(fin=addr(3)), INVALID),
    (dict(t=tokens(seqlen=5000), ws=None), INVALID), (dict(t=tokens(seqlen=5000), n=64), INVALID),
    (dict(t=tokens(seqlen=5000), ws=addr(15, 8)), INVALID),
    (dict(t=tokens(seqlen=5000), ws=addr(5)), INVALID),
])
def test_recurrence_rejects(kw, status):
    assert Recurrence(**kw).forward() == status


@no_gpu
@pytest.mark.parametrize("kw", [
    dict(t=tokens()), dict(t=one(), initial_state=None), dict(t=one(), fin=None),
    dict(t=one(), y=None), dict(t=one(), fin=addr(4, 64)), dict(t=one(), y=addr(4)),
    dict(t=tokens(**{**PACKED, "seqlen": 1}))])
def test_recurrence_step_rejects(kw):
    assert Recurrence(**kw).step() == INVALID


@no_gpu
@pytest.mark.parametrize("kw", [
    dict(dy=None), dict(dx=None), dict(dg=None), dict(di=None), dict(dd=None),
    dict(input_gate=None), dict(decay=None), dict(dx=addr(0)), dict(dg=addr(9)), dict(dd=addr(3)),
    dict(dh=addr(8)), dict(df=addr(8, 4)), dict(dy=addr(7, 8)), dict(sharpness=0.0),
    # (rows of several chunks need a workspace)
    dict(t=tokens(seqlen=5000), ws=None), dict(t=tokens(seqlen=5000), n=16),
    dict(t=tokens(seqlen=5000), ws=addr(10))])
def test_recurrence_backward_rejects(kw):
    assert Recurrence(**kw).backward() == INVALID


class Rotation:
    def __init__(self, **kw):
        self.q = dict(rows=50, ngroups=2, dstate=32, nfreq=12, sections=(4, 8, 0, 0),
                      positions=addr(0), frequencies=addr(1), B=addr(2), C=addr(3), b_stride=0,
                      c_stride=0, naxes=2, interleaved=0, inverse=0, io_dtype=1, reserved=0)
        self.bo, self.co = addr(4), addr(5)
        for k, v in kw.items():
            if k in self.q:
                self.q[k] = v
            else:
                setattr(self, k, v)

    def call(self):
        q = dict(self.q, sections=(ctypes.c_int64 * 4)(*self.q["sections"]))
        names = [n for n, _ in recurrent.SSDRotation._fields_]
        return block._function("ssd_rotate")(
            ctypes.byref(recurrent.SSDRotation(*(q[n] for n in names))), self.bo, self.co, None)


@no_gpu
@pytest.mark.parametrize("kw,status", [
    (dict(), NO_DEVICE), (dict(C=None, co=None), NO_DEVICE), (dict(b_stride=72), NO_DEVICE),
    (dict(positions=addr(0, 4)), NO_DEVICE), (dict(sections=(0, 12, 0, 0)), NO_DEVICE),
    (dict(naxes=4, sections=(3, 3, 3, 3), nfreq=12), NO_DEVICE),
    (dict(rows=0), INVALID), (dict(ngroups=0), INVALID), (dict(dstate=0), INVALID),
    (dict(nfreq=0), INVALID), (dict(naxes=0), INVALID), (dict(reserved=1), INVALID),
    (dict(io_dtype=2), INVALID), (dict(positions=None), INVALID), (dict(frequencies=None), INVALID),
    (dict(B=None), INVALID), (dict(bo=None), INVALID), (dict(C=None), INVALID),
    (dict(co=None), INVALID), (dict(nfreq=20, sections=(4, 16, 0, 0)), INVALID),
    (dict(sections=(4, 4, 4, 0)), INVALID), (dict(sections=(4, 4, 0, 0)), INVALID),
    (dict(sections=(16, -4, 0, 0)), INVALID), (dict(sections=(13, 0, 0, 0)), INVALID),
    (dict(positions=addr(0, 2)), INVALID), (dict(frequencies=addr(1, 4)), INVALID),
    (dict(B=addr(2, 8)), INVALID), (dict(b_stride=60), INVALID), (dict(c_stride=68), INVALID),
    (dict(bo=addr(2)), INVALID), (dict(co=addr(2)), INVALID), (dict(co=addr(4)), INVALID),
    (dict(bo=addr(0)), INVALID), (dict(co=addr(5, 8)), INVALID),
    (dict(naxes=5), UNSUPPORTED), (dict(dstate=28), UNSUPPORTED),
    (dict(nfreq=10, sections=(4, 6, 0, 0)), UNSUPPORTED), (dict(ngroups=1 << 16), UNSUPPORTED),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(rows=1 << 40), UNSUPPORTED),
    (dict(dstate=1 << 62, ngroups=1 << 62, nfreq=1 << 61), UNSUPPORTED),
])
def test_rotation_checks(kw, status):
    assert Rotation(**kw).call() == status


@no_gpu
def test_group_norm_valid_and_rejected():
    F, B = block._function("ssd_group_norm"), block._function("ssd_group_norm_backward")

    long = tokens(seqlen=50000)

    def forward(t=long, x=addr(0), xs=0, w=addr(1), b=addr(2), g=4, eps=1e-5, y=addr(3),
                st=addr(4), ws=addr(5), n=1 << 33):
        return F(ctypes.byref(t), x, xs, w, b, g, eps, 1, y, st, ws, n, None)

    def backward(t=long, w=addr(1), b=addr(2), g=4, st=addr(4), dy=addr(6), dx=addr(7),
                 dw=addr(8), db=addr(9), ws=addr(5), n=1 << 33):
        return B(ctypes.byref(t), addr(0), 0, w, b, g, 1, st, dy, dx, dw, db, ws, n, None)

    few = tokens(seqlen=3)
    assert forward(t=tokens(), ws=None, n=0) == backward(t=tokens()) == NO_DEVICE
    assert forward() == forward(w=None, b=None, st=None, xs=72, g=64) == NO_DEVICE
    assert forward(t=few, ws=None, n=0) == forward(t=tokens(**PACKED), eps=0.0) == NO_DEVICE
    assert backward() == backward(w=None, dw=None) == backward(b=None, db=None) == NO_DEVICE
    assert backward(t=few) == backward(t=tokens(**PACKED)) == NO_DEVICE
    for kw in (dict(x=None), dict(y=None), dict(g=0), dict(g=-1), dict(g=5), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(xs=32), dict(xs=68),
               dict(y=addr(0)), dict(st=addr(1)), dict(st=addr(3)), dict(y=addr(3, 8)),
               dict(w=addr(1, 4)), dict(ws=None), dict(n=64), dict(ws=addr(5, 4)),
               dict(ws=addr(4)), dict(t=tokens(nseq=3))):
        assert forward(**kw) == INVALID, kw
    assert forward(t=tokens(channels=60)) == UNSUPPORTED
    for kw in (dict(st=None), dict(dy=None), dict(dx=None), dict(dw=None), dict(db=None),
               dict(w=None), dict(b=None), dict(dx=addr(0)), dict(dw=addr(9)), dict(ws=None),
               dict(n=64), dict(dx=addr(4)), dict(g=3), dict(ws=addr(7))):
        assert backward(**kw) == INVALID, kw


def test_workspace_queries():
    n = ctypes.c_int64()
    long, short = tokens(batch=1, nseq=1, seqlen=1000), tokens(batch=2, nseq=2, seqlen=28)
    for name in ("ssd_recurrence_workspace", "ssd_recurrence_backward_workspace"):
        f = block._function(name)
        q = Recurrence()._args()[1]
        assert f(ctypes.byref(long), q, ctypes.byref(n)) == OK and n.value > 0
        assert f(ctypes.byref(long), q, None) == INVALID
        assert f(None, q, ctypes.byref(n)) == f(ctypes.byref(long), None, ctypes.byref(n)) == INVALID
    q = Recurrence(**BARE)._args()[1]
    for name in ("ssd_recurrence_workspace", "ssd_recurrence_backward_workspace"):
        assert block._function(name)(ctypes.byref(short), q, ctypes.byref(n)) == OK and n.value == 0
    for name in ("ssd_group_norm_workspace", "ssd_group_norm_backward_workspace"):
        f = block._function(name)
        long.seqlen = 50000
        assert f(ctypes.byref(long), 4, ctypes.byref(n)) == OK and n.value > 0
        assert f(ctypes.byref(long), 4, None) == f(ctypes.byref(long), 0, ctypes.byref(n)) == INVALID


def far(i):  # apart by more than the largest tensors
    return (1 << 50) + (i << 44)


def rows_of_recurrence(n, channels=8):
    t = tokens(batch=1, seqlen=n, channels=channels, nseq=1, seq_starts=addr(60))
    return Recurrence(t=t, x=far(0), gate=far(1), y=far(2), fin=far(3), ws=far(4), n=1 << 40,
                      **BARE).forward()


def rows_of_rotation(n, groups=1):
    return Rotation(rows=n, ngroups=groups, dstate=8, nfreq=4, sections=(4, 0, 0, 0), naxes=1,
                    positions=far(0), B=far(1), C=None, bo=far(2), co=None).call()


def groups_of_norm(n):
    t = tokens(batch=1, seqlen=100, channels=64, nseq=n, seq_starts=far(0))
    return block._function("ssd_group_norm")(ctypes.byref(t), far(1), 0, None, None, 64, 1e-5, 1,
                                             far(2), None, far(3), 1 << 43, None)


@no_gpu
@pytest.mark.parametrize("call,taken,refused", [
    (lambda n: Recurrence(t=tokens(seqlen=1, channels=8 * n)).forward(), 2 ** 17, 2 ** 17 + 1),
    (rows_of_recurrence, 2 ** 28, 2 ** 29),
    (lambda n: rows_of_recurrence(n, 1024), 2 ** 25, 2 ** 26),
    (rows_of_rotation, 2 ** 31 - 4097, 2 ** 31 - 4096),
    (lambda n: rows_of_rotation(n, 16), 2 ** 30 - 65, 2 ** 30),
    (groups_of_norm, 2 ** 20 - 1, 2 ** 20)])
def test_stated_limits(call, taken, refused):
    assert call(taken) == NO_DEVICE
    assert call(refused) == UNSUPPORTED


@pytest.mark.parametrize("source", ["ssd_recurrence", "ssd_rotate", "ssd_group_norm"])
def test_kernels_use_no_scratch(source):
    kernels = _kernel_descriptors(os.path.join(BUILD, source + ".o"))
    assert kernels, source
    bad = {k: v for k, v in kernels.items()
           if v.get("private_segment_fixed_size", 0) or v.get("vgpr_spill_count", 0)}
    assert not bad, f"{source} kernels spilling to scratch: {bad}"


# ---- the binding -----------------------------------------------------------------------------------

Bt, L, C = 2, 6, 16


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


def test_binding_rejects_shapes_and_types():
    x, bc = z(Bt, L, C), z(Bt, L, 2, 8)
    pos, f = z(1, Bt, L, dtype=torch.int32), z(4)
    two = z(2, Bt, L, dtype=torch.int32)
    cu = z(3, dtype=torch.int32)
    for match, call in (
            ("x must be", lambda: ssd.recurrence(x[0], x)),
            ("unsupported io dtype", lambda: ssd.recurrence(x.half(), x)),
            ("x must be a device", lambda: ssd.recurrence(x, x)),
            ("batch 1", lambda: ssd.recurrence(x, x, cu_seqlens=cu)),
            ("state must be", lambda: ssd.recurrence_step(None, x[:, 0], x[:, 0])),
            ("x must be", lambda: ssd.recurrence_step(z(Bt, C), x, x)),
            ("x must be a device", lambda: ssd.recurrence_backward(x, x, None, None, x)),
            ("B must be", lambda: ssd.rotate(bc[0, 0], None, pos, f)),
            ("dB must be", lambda: ssd.rotate_backward(bc[0, 0], None, pos, f)),
            ("unsupported io dtype", lambda: ssd.rotate(bc.double(), None, pos, f)),
            ("positions must be", lambda: ssd.rotate(bc, bc, pos[0], f)),
            ("positions must be", lambda: ssd.rotate(bc[:, 0], None, pos, f)),
            ("positions must be", lambda: ssd.rotate(bc, bc, z(5, Bt, L, dtype=torch.int32), f)),
            ("frequencies must be", lambda: ssd.rotate(bc, bc, pos, f[None])),
            ("sections must say", lambda: ssd.rotate(bc, bc, two, f)),
            ("sections must be", lambda: ssd.rotate(bc, bc, two, f, sections=(4,))),
            ("sections must be", lambda: ssd.rotate(bc, bc, two, f, sections=(2, 3))),
            ("sections must be", lambda: ssd.rotate(bc, bc, two, f, sections=(6, -2))),
            ("B must be a device", lambda: ssd.rotate(bc, bc, pos, f)),
            ("x must be a device", lambda: ssd.group_norm(x, ngroups=2)),
            ("unknown activation", lambda: ssd.group_norm(x, ngroups=2, activation="gelu")),
            ("x must be a device", lambda: ssd.group_norm_backward(x, None, None, None, x, ngroups=2))):
        with pytest.raises(ValueError, match=match):
            call()


def operators(lead):
    """name -> (call of its activations by name, the activations); lead: their token dimensions."""
    act, bc = z(*lead, 64), z(*lead, 2, 16)
    pos, f, h = z(1, *lead, dtype=torch.int32), z(8), z(lead[0], 64)
    gates = dict(x=act, gate=act, input_gate=act)
    ops = {"rotate": (lambda B, C: ssd.rotate(B, C, pos, f), dict(B=bc, C=bc)),
           "rotate_backward": (lambda dB, dC: ssd.rotate_backward(dB, dC, pos, f),
                               dict(dB=bc, dC=bc))}
    if len(lead) == 1:
        ops["recurrence_step"] = (
            lambda x, gate, input_gate: ssd.recurrence_step(h, x, gate, None, input_gate), gates)
        return ops
    ops.update({
        "recurrence": (lambda x, gate, input_gate: ssd.recurrence(x, gate, None, input_gate), gates),
        "recurrence_backward": (lambda x, gate, input_gate: ssd.recurrence_backward(
            x, gate, None, input_gate, act), gates),
        "group_norm": (lambda x: ssd.group_norm(x, ngroups=4), dict(x=act)),
        "group_norm_backward": (lambda x: ssd.group_norm_backward(x, None, None, z(lead[0], 4, 2),
                                                                  act, ngroups=4), dict(x=act))})
    return ops


@pytest.fixture
def caught(no_device, monkeypatch):  # noqa: F811
    for name in ("_run", "_workspace", "_tensor"):
        monkeypatch.setattr(recurrent, name, getattr(block, name))


@pytest.mark.parametrize("lead", [(3, 9), (3, 1), (1, 9), (3,), (2,)])
def test_broadcast_and_overlapping_rows_are_refused(caught, lead):
    for name, (call, given) in operators(lead).items():
        for arg, t in given.items():
            with pytest.raises(Reached):
                call(**given)
            for bad in broadcasts(t, lead):
                if bad.is_contiguous():  # (a dimension of one row)
                    continue
                with pytest.raises(ValueError, match=f"^{arg}: the rows of tokens must be"):
                    call(**{**given, arg: bad})
