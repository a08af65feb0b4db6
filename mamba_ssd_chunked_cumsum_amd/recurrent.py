"""Python binding of the operators of layers of linear recurrence: the gated linear recurrence with
one state entry a channel (forward, one token at a time, backward), the rotation of the scan's B and
C by positions of several axes (and its backward), and the group norm with its activation (forward
and backward). Argument marshalling only; activations, packed prompts (cu_seqlens), streams, outputs
and errors as in block.py.
"""

from __future__ import annotations

import ctypes

import torch

from .block import (_SIGNATURES, _T, SSDTokens, _f32, _i32, _i64, _io, _output, _PI, _rows, _run,
                    _silu, _tensor, _tokens, _vp, _workspace)
from .libssd import DTYPES


class SSDRecurrent(ctypes.Structure):
    _fields_ = [("x", _vp), ("gate", _vp), ("input_gate", _vp), ("x_stride", _i64),
                ("gate_stride", _i64), ("input_gate_stride", _i64), ("decay", _vp),
                ("initial_state", _vp), ("sharpness", _f32), ("reserved", _i32)]


class SSDRotation(ctypes.Structure):
    _fields_ = [("rows", _i64), ("ngroups", _i64), ("dstate", _i64), ("nfreq", _i64),
                ("sections", _i64 * 4), ("positions", _vp), ("frequencies", _vp), ("B", _vp),
                ("C", _vp), ("b_stride", _i64), ("c_stride", _i64), ("naxes", _i32),
                ("interleaved", _i32), ("inverse", _i32), ("io_dtype", _i32), ("reserved", _i64)]


_R, _Sections = ctypes.POINTER(SSDRecurrent), _i64 * 4
_MORE = {
    "ssd_recurrence_workspace": [_T, _R, _PI],
    "ssd_recurrence": [_T, _R, _vp, _vp, _vp, _i64, _vp],
    "ssd_recurrence_step": [_T, _R, _vp, _vp, _vp],
    "ssd_recurrence_backward_workspace": [_T, _R, _PI],
    "ssd_recurrence_backward": [_T, _R, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp],
    "ssd_rotate": [ctypes.POINTER(SSDRotation), _vp, _vp, _vp],
    "ssd_group_norm_workspace": [_T, _i64, _PI],
    "ssd_group_norm": [_T, _vp, _i64, _vp, _vp, _i64, _f32, _i32, _vp, _vp, _vp, _i64, _vp],
    "ssd_group_norm_backward_workspace": [_T, _i64, _PI],
    "ssd_group_norm_backward": [_T, _vp, _i64, _vp, _vp, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                                _i64, _vp],
}
_SIGNATURES.update(_MORE)
EXPORTS = tuple(_MORE)


def _address(t):
    return None if t is None else t.data_ptr()


def _like(given, name, like):
    """(tensor, address) of the given output, checked, or of a new dense one of `like`'s shape and
    type (empty_like is the cheapest call there is for that, where `like` is dense)."""
    if given is None:
        given = torch.empty_like(like) if like.is_contiguous() else like.new_empty(like.shape)
        return given, given.data_ptr()
    return given, _tensor(given, name, like.shape, like.dtype, like.device)


# ---- gated linear recurrence ---------------------------------------------------------------------

def _recurrent(x, gate, decay, input_gate, state, sharpness, S, lead):
    """ssd_recurrent of the inputs; `lead`: the token dimensions of x."""
    n, dev, C = len(lead), x.device, x.shape[-1]
    xp, xs = _rows(x, "x", (*lead, C), x.dtype, dev, n)
    gp, gs = _rows(gate, "gate", (*lead, C), x.dtype, dev, n)
    ip, is_ = _rows(input_gate, "input_gate", (*lead, C), x.dtype, dev, n)
    return SSDRecurrent(
        xp, gp, ip, xs, gs, is_, _tensor(decay, "decay", (C,), torch.float32, dev),
        _tensor(state, "state" if n == 1 else "initial_state", (S, C), torch.float32, dev),
        sharpness, 0)


def recurrence(x, gate, decay=None, input_gate=None, initial_state=None, *, sharpness=8.0,
               cu_seqlens=None, want_final=True, out=None, final_out=None):
    """Gated linear recurrence h_t = a_t h_{t-1} + m_t v_t over each sequence, one state entry a
    channel, v = sigmoid(input_gate) x (x without an input gate). With a decay parameter a =
    exp(-sharpness softplus(decay) sigmoid(gate)) and m = sqrt(1 - a^2); without, a =
    sigmoid(gate) and m = 1 - a.

    x, gate, input_gate [Bt, L, C] of one dtype; decay [C], initial_state [nseq, C] f32 (None:
    zeros). Returns (y = h [Bt, L, C], final_state [nseq, C] or None if not wanted)."""
    _io(x)
    dev = x.device
    tok, S = _tokens(x, cu_seqlens)
    q = _recurrent(x, gate, decay, input_gate, initial_state, sharpness, S, x.shape[:2])
    y, yp = _like(out, "out", x)
    fin = fp = None
    if want_final:
        fin, fp = _output(final_out, "final_out", x, (S, x.shape[2]), torch.float32)
    t, qr = ctypes.byref(tok), ctypes.byref(q)
    ws, wp, n = _workspace("ssd_recurrence_workspace", dev, t, qr)
    _run("ssd_recurrence", dev, t, qr, yp, fp, wp, n)
    return y, fin


def recurrence_step(state, x, gate, decay=None, input_gate=None, *, sharpness=8.0, out_state=None,
                    out=None):
    """One token of recurrence for each sequence: state [Bt, C] f32; x, gate, input_gate [Bt, C].
    Returns (y [Bt, C], new_state); out_state may be `state` itself."""
    io, dev = _io(x, dim=2), x.device
    Bt, C = x.shape
    if state is None:
        raise ValueError("state must be [batch, channels]")
    tok = SSDTokens(Bt, 1, C, Bt, None, io, 0)
    q = _recurrent(x, gate, decay, input_gate, state, sharpness, Bt, (Bt,))
    y, yp = _like(out, "out", x)
    so, sop = _like(out_state, "out_state", state)
    _run("ssd_recurrence_step", dev, ctypes.byref(tok), ctypes.byref(q), sop, yp)
    return y, so


def recurrence_backward(x, gate, decay, input_gate, dy, initial_state=None, dfinal=None, *,
                        sharpness=8.0, cu_seqlens=None, want_initial_grad=True):
    """Gradients of recurrence for dy (x's dtype and shape) and dfinal ([nseq, C] f32, None: zero).
    Returns a dict: dx, dgate, dinput_gate (x's dtype; None without an input gate), ddecay (float32;
    None without a decay) and dinitial_state (float32; None unless want_initial_grad)."""
    _io(x)
    dev = x.device
    tok, S = _tokens(x, cu_seqlens)
    C = x.shape[2]
    q = _recurrent(x, gate, decay, input_gate, initial_state, sharpness, S, x.shape[:2])
    dyp = _tensor(dy, "dy", x.shape, x.dtype, dev)
    dfp = _tensor(dfinal, "dfinal", (S, C), torch.float32, dev)
    f32 = dict(dtype=torch.float32, device=dev)
    # (dy is dense, of x's shape and type)
    g = dict(dx=torch.empty_like(dy), dgate=torch.empty_like(dy),
             dinput_gate=None if input_gate is None else torch.empty_like(dy),
             ddecay=None if decay is None else torch.empty_like(decay),
             dinitial_state=torch.empty((S, C), **f32) if want_initial_grad else None)
    t, qr = ctypes.byref(tok), ctypes.byref(q)
    ws, wp, n = _workspace("ssd_recurrence_backward_workspace", dev, t, qr)
    _run("ssd_recurrence_backward", dev, t, qr, dyp, dfp, *map(_address, g.values()), wp, n)
    return g


# ---- rotation of B and C ---------------------------------------------------------------------------

def _rotate(B, C, names, positions, frequencies, sections, interleaved, inverse, out):
    if B.dim() not in (3, 4):
        raise ValueError(f"{names[0]} must be [batch, seqlen, ngroups, dstate] or, for one token, "
                         "[batch, ngroups, dstate]")
    if B.dtype not in DTYPES:
        raise ValueError(f"unsupported io dtype {B.dtype}")
    dev, n = B.device, B.dim() - 2
    lead, G, N = B.shape[:n], B.shape[-2], B.shape[-1]
    if positions.dim() != n + 1 or not 1 <= positions.shape[0] <= 4:
        raise ValueError(f"positions must be [axes, {'batch, seqlen' if n == 2 else 'batch'}] with "
                         "up to four axes")
    if frequencies.dim() != 1:
        raise ValueError("frequencies must be [nfreq]")
    axes, nf = positions.shape[0], frequencies.shape[0]
    if sections is None:
        if axes != 1:
            raise ValueError(f"sections must say how many of the {nf} frequencies go by each of the "
                             f"{axes} axes")
        sections = (nf,)
    sections = tuple(map(int, sections))
    if len(sections) != axes or sum(sections) != nf or min(sections) < 0:
        raise ValueError(f"sections must be {axes} sizes that sum to {nf}")
    bp, bs = _rows(B, names[0], B.shape, B.dtype, dev, n)
    cp, cs = _rows(C, names[1], B.shape, B.dtype, dev, n)
    given = (None, None) if out is None else out
    Bo, bo = _like(given[0], "out", B)
    Co, co = (None, None) if C is None else _like(given[1], "out", C)
    q = SSDRotation(
        lead.numel(), G, N, nf, _Sections(*sections),
        _tensor(positions, "positions", (axes, *lead), torch.int32, dev),
        _tensor(frequencies, "frequencies", (nf,), torch.float32, dev), bp, cp, bs, cs, axes,
        1 if interleaved else 0, inverse, DTYPES[B.dtype], 0)
    _run("ssd_rotate", dev, ctypes.byref(q), bo, co)
    return Bo, Co


def rotate(B, C, positions, frequencies, *, sections=None, interleaved=False, out=None):
    """B and C turned by the positions of their tokens, before ``forward`` or ``step``: C_t . B_s then
    depends on positions by their difference alone, which gives the scan's decays a phase.

    B, C (or None) [Bt, L, G, N], or [Bt, G, N] for one token, of one dtype; positions int32 [axes,
    Bt, L] (or [axes, Bt]), up to four axes; frequencies [nfreq] f32 in radians a position, nfreq a
    multiple of 4 up to N / 2, N a multiple of 8. sections: how many of the frequencies go by each
    axis, in order (None with one axis). Frequency j turns entries j and j + nfreq, or 2j and 2j + 1
    if interleaved; entries from 2 nfreq on stay. out: two tensors. Returns (B', C')."""
    return _rotate(B, C, ("B", "C"), positions, frequencies, sections, interleaved, 0, out)


def rotate_backward(dB, dC, positions, frequencies, *, sections=None, interleaved=False, out=None):
    """Gradients of rotate's B and C from those of what it returned (float32 as ``backward`` gives
    them, or bfloat16): the same turned the other way. Returns (dB, dC) in the dtype given."""
    return _rotate(dB, dC, ("dB", "dC"), positions, frequencies, sections, interleaved, 1, out)


# ---- group norm ------------------------------------------------------------------------------------

def group_norm(x, weight=None, bias=None, *, ngroups, eps=1e-5, activation="silu", cu_seqlens=None,
               want_stats=True, out=None):
    """Group norm over each sequence's tokens and each of ngroups equal runs of the channels, with
    its SiLU: silu(weight (x - mean) / sqrt(variance + eps) + bias). x [Bt, L, C]; weight, bias [C]
    f32 (each may be None). A norm of every token by itself is that of [Bt L, 1, C]. Returns (y,
    stats [nseq, ngroups, 2] f32: mean and 1 / sqrt(variance + eps); None if not wanted)."""
    _io(x)
    act, dev = _silu(activation), x.device
    tok, S = _tokens(x, cu_seqlens)
    xp, xs = _rows(x, "x", x.shape, x.dtype, dev)
    w = _tensor(weight, "weight", x.shape[2:], torch.float32, dev)
    b = _tensor(bias, "bias", x.shape[2:], torch.float32, dev)
    y, yp = _like(out, "out", x)
    stats = sp = None
    if want_stats and ngroups > 0:
        stats, sp = _output(None, "stats", x, (S, ngroups, 2), torch.float32)
    t = ctypes.byref(tok)
    ws, wp, n = _workspace("ssd_group_norm_workspace", dev, t, ngroups)
    _run("ssd_group_norm", dev, t, xp, xs, w, b, ngroups, eps, act, yp, sp, wp, n)
    return y, stats


def group_norm_backward(x, weight, bias, stats, dy, *, ngroups, activation="silu",
                        cu_seqlens=None):
    """Gradients of group_norm for dy (x's dtype and shape), with the stats that it returned. Returns
    a dict: dx (x's dtype), dweight, dbias (float32; None where the input is)."""
    _io(x)
    act, dev = _silu(activation), x.device
    tok, S = _tokens(x, cu_seqlens)
    xp, xs = _rows(x, "x", x.shape, x.dtype, dev)
    w = _tensor(weight, "weight", x.shape[2:], torch.float32, dev)
    b = _tensor(bias, "bias", x.shape[2:], torch.float32, dev)
    st = _tensor(stats, "stats", (S, ngroups, 2), torch.float32, dev)
    dyp = _tensor(dy, "dy", x.shape, x.dtype, dev)
    g = dict(dx=torch.empty_like(dy), dweight=None if weight is None else torch.empty_like(weight),
             dbias=None if bias is None else torch.empty_like(bias))
    t = ctypes.byref(tok)
    ws, wp, n = _workspace("ssd_group_norm_backward_workspace", dev, t, ngroups)
    _run("ssd_group_norm_backward", dev, t, xp, xs, w, b, ngroups, act, st, dyp,
         *map(_address, g.values()), wp, n)
    return g
