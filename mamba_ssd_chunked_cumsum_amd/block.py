"""Python binding of the operators around the scan in a state space block: the short causal
convolution, the selective scan (a decay of its own for every channel and state entry), the gated
norm and the norm with residual; each forward, backward and, for the first two, one token at a
time. Argument marshalling only, as in libssd.py.

Activations are [batch, seqlen, channels] of float32 or bfloat16, weights and scan states
float32. An activation may be a slice of wider rows (one projection's output) as long as its
channels are adjacent, its rows evenly spaced and apart (a broadcast tensor is refused), the offset
16-byte aligned and the row stride a multiple of 8 elements (the selective scan's B and C: of 4
elements each). Packed prompts: batch 1 and cu_seqlens, int32 offsets [nseq + 1] on the
device, sequence s being the tokens [cu_seqlens[s], cu_seqlens[s + 1]) (it may be empty); states
then have nseq entries. Tokens outside every sequence (behind the last, as a rule) have no part in
any result, whatever lies there; forward outputs there are left as they are (undefined in fresh
tensors) and their gradients are zero. cu_seqlens is not read on the host: offsets that decrease or
leave [0, seqlen] give undefined results.

The calls run on the current stream of the inputs' device and allocate their outputs and workspace
with torch, so they can be captured into a graph. Given outputs (out, final_out, out_state) may not
overlap inputs, but out_state may be the state itself (updated in place).
"""

from __future__ import annotations

import ctypes

import torch

from .libssd import DTYPES, _check, load

_vp, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class SSDTokens(ctypes.Structure):
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("nseq", _i64),
                ("seq_starts", _vp), ("io_dtype", _i32), ("reserved", _i32)]


class SSDSelective(ctypes.Structure):
    _fields_ = [("dstate", _i64), ("ngroups", _i64),
                ("x", _vp), ("dt", _vp), ("B", _vp), ("C", _vp), ("z", _vp),
                ("x_stride", _i64), ("dt_stride", _i64), ("b_stride", _i64), ("c_stride", _i64),
                ("z_stride", _i64),
                ("A", _vp), ("D", _vp), ("dt_bias", _vp), ("initial_state", _vp),
                ("dt_softplus", _i32), ("reserved", _i32)]


class SSDSelectiveGrads(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("dx", "ddt", "dz", "dB", "dC", "dA", "dD", "ddt_bias",
                                   "dinitial_state")]


_Ptr3, _Split3 = _vp * 3, _i64 * 3
_T, _S = ctypes.POINTER(SSDTokens), ctypes.POINTER(SSDSelective)
_P3, _L3, _PI = ctypes.POINTER(_vp), ctypes.POINTER(_i64), ctypes.POINTER(_i64)
_SIGNATURES = {
    "ssd_conv": [_T, _vp, _i64, _vp, _vp, _i32, _i32, _vp, _P3, _L3, _vp, _vp],
    "ssd_conv_step": [_T, _vp, _i64, _vp, _vp, _i32, _i32, _vp, _vp, _P3, _L3, _vp],
    "ssd_conv_backward_workspace": [_T, _i32, _PI],
    "ssd_conv_backward": [_T, _vp, _i64, _vp, _vp, _i32, _i32, _vp, _P3, _L3, _i32, _vp, _vp, _vp,
                          _vp, _vp, _vp, _i64, _vp],
    "ssd_selective_scan_workspace": [_T, _S, _PI],
    "ssd_selective_scan": [_T, _S, _vp, _vp, _vp, _i64, _vp],
    "ssd_selective_step": [_T, _S, _vp, _vp, _vp],
    "ssd_selective_backward_workspace": [_T, _S, _PI],
    "ssd_selective_backward": [_T, _S, _vp, _vp, ctypes.POINTER(SSDSelectiveGrads), _vp, _i64,
                               _vp],
    "ssd_gated_norm": [_T, _vp, _i64, _vp, _i64, _vp, _i64, _f32, _i32, _vp, _vp],
    "ssd_gated_norm_backward_workspace": [_T, _i64, _PI],
    "ssd_gated_norm_backward": [_T, _vp, _i64, _vp, _i64, _vp, _i64, _f32, _i32, _vp, _vp, _vp,
                                _vp, _vp, _i64, _vp],
    "ssd_residual_norm": [_T, _vp, _i64, _vp, _i32, _vp, _vp, _f32, _vp, _vp, _vp],
    "ssd_residual_norm_backward_workspace": [_T, _PI],
    "ssd_residual_norm_backward": [_T, _vp, _i32, _vp, _i64, _vp, _vp, _f32, _vp, _vp, _vp, _vp,
                                   _vp, _vp, _vp, _i64, _vp],
}
EXPORTS = tuple(_SIGNATURES)

_functions = {}


def _function(name):
    f = _functions.get(name)
    if f is None:
        f = getattr(load(), name)
        f.argtypes, f.restype = _SIGNATURES[name], ctypes.c_int
        _functions[name] = f
    return f


# ---- checks ------------------------------------------------------------------------------------

def _place(t, name, dtype, dev):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")


def _tensor(t, name, shape, dtype, dev):
    """Address of a dense input or output (None for None) after checks of shape, dtype, device."""
    if t is None:
        return None
    if t.shape == shape and t.dtype == dtype and t.is_cuda and t.device == dev \
            and t.is_contiguous():
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    _place(t, name, dtype, dev)
    raise ValueError(f"{name} must be contiguous")


def _rows(t, name, shape, dtype, dev, lead=2):
    """An activation whose first `lead` dimensions are token rows: (address, row stride); the
    others are dense."""
    if t is None:
        return None, 0
    if t.is_contiguous():
        return _tensor(t, name, shape, dtype, dev), 0
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    size, stride = t.shape, t.stride()
    # the common slice of wider rows, checked at once: rows of a batch, their values side by side
    if len(size) == lead + 1 and stride[lead] == 1 and size[lead - 1] > 1:
        row = stride[lead - 1]
        if row >= size[lead] and (lead == 1 or size[0] == 1 or stride[0] == row * size[1]) \
                and lead <= 2 and t.dtype == dtype and t.is_cuda and t.device == dev:
            return t.data_ptr(), row
    width = 1
    for i in range(len(size) - 1, lead - 1, -1):
        if size[i] != 1 and stride[i] != width:
            raise ValueError(f"{name}: the values of a token must be adjacent")
        width *= size[i]
    row = None  # every leading dimension of more than one entry agrees on it
    step = 1
    for i in range(lead - 1, -1, -1):
        if size[i] != 1:
            if stride[i] % step or (row is not None and stride[i] != row * step):
                raise ValueError(f"{name}: the rows of tokens must be evenly spaced")
            row = stride[i] // step if row is None else row
        step *= size[i]
    if row is not None and row < width:  # 0, a broadcast, would mean dense to the library
        raise ValueError(f"{name}: the rows of tokens must be at least {width} elements apart, they "
                         f"are {row} (a broadcast tensor needs contiguous())")
    _place(t, name, dtype, dev)
    return t.data_ptr(), 0 if row is None else row


def _io(x, name="x", dim=3):
    if x.dim() != dim:
        raise ValueError(f"{name} must be [batch, {'seqlen, ' if dim == 3 else ''}channels]")
    if x.dtype not in DTYPES:
        raise ValueError(f"unsupported io dtype {x.dtype}")
    return DTYPES[x.dtype]


def _tokens(x, cu_seqlens=None):
    """(ssd_tokens, number of sequences) of x [batch, seqlen, channels]."""
    Bt, L, C = x.shape
    if cu_seqlens is None:
        return SSDTokens(Bt, L, C, Bt, None, _io(x), 0), Bt
    if Bt != 1:
        raise ValueError("packed sequences (cu_seqlens) need batch 1")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must be [nseq + 1] with nseq >= 1")
    S = cu_seqlens.shape[0] - 1
    p = _tensor(cu_seqlens, "cu_seqlens", (S + 1,), torch.int32, x.device)
    return SSDTokens(1, L, C, S, p, _io(x), 0), S


def _stream(dev):
    """The current stream's handle (torch.cuda.current_stream builds an object for it, which costs
    more than the rest of a small call)."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _run(name, dev, *args):
    """Calls an entry point on the current stream of `dev`, as that device's own call."""
    f = _functions.get(name) or _function(name)
    if torch.cuda.current_device() == dev.index:
        status = f(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            status = f(*args, _stream(dev))
    if status:
        _check(status, name)


def _workspace(name, dev, *args):
    n = _i64()
    f = _function(name)
    if torch.cuda.current_device() == dev.index:
        status = f(*args, ctypes.byref(n))
    else:
        with torch.cuda.device(dev):
            status = f(*args, ctypes.byref(n))
    _check(status, name)
    ws = torch.empty(n.value, dtype=torch.uint8, device=dev) if n.value else None
    return ws, (None if ws is None else ws.data_ptr()), n.value


def _output(given, name, like, shape, dtype):
    """(tensor, address) of the given output, checked, or of a new one on `like`'s device."""
    if given is None:
        given = like.new_empty(shape, dtype=dtype)
        return given, given.data_ptr()
    return given, _tensor(given, name, shape, dtype, like.device)


# ---- short causal convolution ------------------------------------------------------------------

def _split_sizes(split, C):
    if split is None:
        return (C,)
    sizes = tuple(map(int, split))
    if not 1 <= len(sizes) <= 3 or sum(sizes) != C or min(sizes) <= 0:
        raise ValueError(f"split must be up to three positive sizes that sum to {C}")
    return sizes


def _parts(ts, name, sizes, lead, dtype, dev):
    """(void*[3], int64[3]) of the tensors the channels are split over."""
    return _Ptr3(*[_tensor(t, name, (*lead, n), dtype, dev) for t, n in zip(ts, sizes)]), \
        _Split3(*sizes)


def _outputs(out, split, sizes, lead, x):
    """The tensors that the channels come in, given or new, and as _parts."""
    if out is None:
        out = tuple([x.new_empty((*lead, n)) for n in sizes])
        return out, _Ptr3(*[t.data_ptr() for t in out]), _Split3(*sizes)
    out = (out,) if split is None else tuple(out)
    if len(out) != len(sizes):
        raise ValueError(f"out must hold {len(sizes)} tensors")
    return out, *_parts(out, "out", sizes, lead, x.dtype, x.device)


def _silu(activation):
    if activation == "silu":
        return 1
    if activation is not None:
        raise ValueError(f"unknown activation {activation!r}")
    return 0


def _conv_params(weight, bias, C, dev):
    if weight.dim() != 2 or weight.shape[0] != C:
        raise ValueError(f"weight has shape {tuple(weight.shape)}, expected ({C}, width)")
    W = weight.shape[1]
    return (W, _tensor(weight, "weight", (C, W), torch.float32, dev),
            _tensor(bias, "bias", (C,), torch.float32, dev))


def conv(x, weight, bias=None, initial_state=None, *, activation="silu", split=None,
         cu_seqlens=None, want_final=True, out=None, final_out=None):
    """Depthwise causal convolution of width 2 to 4 over each sequence, with its SiLU.

    x [Bt, L, C]; weight [C, W], bias [C] f32; initial_state [nseq, W - 1, C] (x's dtype): the W - 1
    inputs before each sequence, oldest first (None: zeros). split: up to three sizes that sum to
    C; the channels then come in that many dense tensors (the scan's x, B and C) instead of one.
    Returns (y or the tuple of its parts, final_state [nseq, W - 1, C] or None if not wanted)."""
    io, dev = _io(x), x.device
    Bt, L, C = x.shape
    tok, S = _tokens(x, cu_seqlens)
    xp, xs = _rows(x, "x", (Bt, L, C), x.dtype, dev)
    W, w, b = _conv_params(weight, bias, C, dev)
    h0 = _tensor(initial_state, "initial_state", (S, W - 1, C), x.dtype, dev)
    sizes = _split_sizes(split, C)
    ys, yp, sp = _outputs(out, split, sizes, (Bt, L), x)
    fin = fp = None
    if want_final:
        fin, fp = _output(final_out, "final_out", x, (S, W - 1, C), x.dtype)
    _run("ssd_conv", dev, ctypes.byref(tok), xp, xs, w, b, W, _silu(activation), h0, yp, sp, fp)
    return (ys[0] if split is None else ys), fin


def conv_step(state, x, weight, bias=None, *, activation="silu", split=None, out_state=None,
              out=None):
    """One token of conv for each sequence: state [Bt, W - 1, C], x [Bt, C]. Returns (y [Bt, C] or
    the tuple of its parts, new_state); out_state may be `state` itself (updated in place)."""
    io, dev = _io(x, dim=2), x.device
    Bt, C = x.shape
    tok = SSDTokens(Bt, 1, C, Bt, None, io, 0)
    xp, xs = _rows(x, "x", (Bt, C), x.dtype, dev, lead=1)
    W, w, b = _conv_params(weight, bias, C, dev)
    sp_in = _tensor(state, "state", (Bt, W - 1, C), x.dtype, dev)
    sizes = _split_sizes(split, C)
    ys, yp, sp = _outputs(out, split, sizes, (Bt,), x)
    so, sop = _output(out_state, "out_state", x, (Bt, W - 1, C), x.dtype)
    _run("ssd_conv_step", dev, ctypes.byref(tok), xp, xs, w, b, W, _silu(activation), sp_in, sop,
         yp, sp)
    return (ys[0] if split is None else ys), so


def conv_backward(x, weight, bias, dy, initial_state=None, dfinal=None, *, activation="silu",
                  cu_seqlens=None, want_initial_grad=True):
    """Gradients of conv. dy: the gradient of y, or the tuple of its parts' gradients as they were
    split; x's dtype, or float32 (as ``backward`` returns dx, dB and dC). dfinal [nseq, W - 1, C]
    f32 or None (zero). Returns a dict: dx (x's dtype), dweight, dbias (None without a bias) and
    dinitial_state (None unless want_initial_grad) in float32."""
    io, dev = _io(x), x.device
    Bt, L, C = x.shape
    tok, S = _tokens(x, cu_seqlens)
    xp, xs = _rows(x, "x", (Bt, L, C), x.dtype, dev)
    W, w, b = _conv_params(weight, bias, C, dev)
    h0 = _tensor(initial_state, "initial_state", (S, W - 1, C), x.dtype, dev)
    parts = tuple(dy) if isinstance(dy, (tuple, list)) else (dy,)
    sizes = _split_sizes([d.shape[-1] for d in parts], C)
    if parts[0].dtype not in (x.dtype, torch.float32):
        raise ValueError(f"dy must be {x.dtype} or float32, got {parts[0].dtype}")
    dyp, sp = _parts(parts, "dy", sizes, (Bt, L), parts[0].dtype, dev)
    df = _tensor(dfinal, "dfinal", (S, W - 1, C), torch.float32, dev)
    f32 = dict(dtype=torch.float32, device=dev)
    g = dict(dx=torch.empty((Bt, L, C), dtype=x.dtype, device=dev),
             dweight=torch.empty((C, W), **f32),
             dbias=None if bias is None else torch.empty((C,), **f32),
             dinitial_state=torch.empty((S, W - 1, C), **f32) if want_initial_grad else None)
    ws, wp, n = _workspace("ssd_conv_backward_workspace", dev, ctypes.byref(tok), W)
    _run("ssd_conv_backward", dev, ctypes.byref(tok), xp, xs, w, b, W, _silu(activation), h0, dyp,
         sp, DTYPES[parts[0].dtype], df, *(None if t is None else t.data_ptr() for t in g.values()),
         wp, n)
    return g


# ---- selective scan ------------------------------------------------------------------------------

def _selective(x, dt, A, B, C, D, z, state, dt_bias, dt_softplus, S, lead, dev):
    """ssd_selective of the inputs; `lead`: the token dimensions of x."""
    n = len(lead)
    Dm = x.shape[-1]
    if B.dim() != n + 2:
        raise ValueError(f"B must be [{'batch, seqlen' if n == 2 else 'batch'}, ngroups, dstate]")
    G, N = B.shape[-2], B.shape[-1]
    xp, xs = _rows(x, "x", (*lead, Dm), x.dtype, dev, n)
    tp, ts = _rows(dt, "dt", (*lead, Dm), x.dtype, dev, n)
    bp, bs = _rows(B, "B", (*lead, G, N), x.dtype, dev, n)
    cp, cs = _rows(C, "C", (*lead, G, N), x.dtype, dev, n)
    zp, zs = _rows(z, "z", (*lead, Dm), x.dtype, dev, n)
    return SSDSelective(
        N, G, xp, tp, bp, cp, zp, xs, ts, bs, cs, zs,
        _tensor(A, "A", (Dm, N), torch.float32, dev), _tensor(D, "D", (Dm,), torch.float32, dev),
        _tensor(dt_bias, "dt_bias", (Dm,), torch.float32, dev),
        _tensor(state, "state" if n == 1 else "initial_state", (S, Dm, N), torch.float32, dev),
        1 if dt_softplus else 0, 0)


def selective_scan(x, dt, A, B, C, D=None, z=None, initial_state=None, *, dt_bias=None,
                   dt_softplus=False, cu_seqlens=None, want_final=True, out=None, final_out=None):
    """Selective scan: h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t, y_t = (C_t . h_t + D x_t)
    silu(z_t) for every channel, with delta = dt + dt_bias, then softplus if dt_softplus.

    x, dt, z [Bt, L, Dm] and B, C [Bt, L, G, N] of one dtype (G divides Dm; each group's B and C
    serve Dm / G neighbouring channels); A [Dm, N], D, dt_bias [Dm], initial_state [nseq, Dm, N]
    f32; D, z, dt_bias and initial_state may be None (no skip, no gate, no bias, zeros). N a
    multiple of 4 up to 64. Returns (y, final_state [nseq, Dm, N] or None if not wanted)."""
    _io(x)
    dev = x.device
    tok, S = _tokens(x, cu_seqlens)
    q = _selective(x, dt, A, B, C, D, z, initial_state, dt_bias, dt_softplus, S, x.shape[:2], dev)
    y, yp = _output(out, "out", x, x.shape, x.dtype)
    fin = fp = None
    if want_final:
        fin, fp = _output(final_out, "final_out", x, (S, x.shape[2], q.dstate), torch.float32)
    t, qr = ctypes.byref(tok), ctypes.byref(q)
    ws, wp, n = _workspace("ssd_selective_scan_workspace", dev, t, qr)
    _run("ssd_selective_scan", dev, t, qr, yp, fp, wp, n)
    return y, fin


def selective_step(state, x, dt, A, B, C, D=None, z=None, *, dt_bias=None, dt_softplus=False,
                   out_state=None, out=None):
    """One token of selective_scan for each sequence: state [Bt, Dm, N] f32; x, dt, z [Bt, Dm]; B, C
    [Bt, G, N]. Returns (y [Bt, Dm], new_state); out_state may be `state` itself."""
    io, dev = _io(x, dim=2), x.device
    Bt, Dm = x.shape
    if state is None:
        raise ValueError("state must be [batch, channels, dstate]")
    tok = SSDTokens(Bt, 1, Dm, Bt, None, io, 0)
    q = _selective(x, dt, A, B, C, D, z, state, dt_bias, dt_softplus, Bt, (Bt,), dev)
    y, yp = _output(out, "out", x, (Bt, Dm), x.dtype)
    so, sop = _output(out_state, "out_state", x, (Bt, Dm, q.dstate), torch.float32)
    _run("ssd_selective_step", dev, ctypes.byref(tok), ctypes.byref(q), sop, yp)
    return y, so


def selective_backward(x, dt, A, B, C, D, z, dy, initial_state=None, dfinal=None, *, dt_bias=None,
                       dt_softplus=False, cu_seqlens=None, want_initial_grad=True):
    """Gradients of selective_scan for dy (x's dtype and shape) and dfinal ([nseq, Dm, N] f32, None:
    zero). Returns a dict: dx, ddt, dB, dC, dz (x's dtype; dz None without z), dA, dD, ddt_bias
    (float32; None where the input is) and dinitial_state (None unless want_initial_grad)."""
    _io(x)
    dev = x.device
    tok, S = _tokens(x, cu_seqlens)
    Bt, L, Dm = x.shape
    q = _selective(x, dt, A, B, C, D, z, initial_state, dt_bias, dt_softplus, S, (Bt, L), dev)
    N = q.dstate
    dyp = _tensor(dy, "dy", (Bt, L, Dm), x.dtype, dev)
    dfp = _tensor(dfinal, "dfinal", (S, Dm, N), torch.float32, dev)
    io = dict(dtype=x.dtype, device=dev)
    f32 = dict(dtype=torch.float32, device=dev)
    g = dict(dx=torch.empty((Bt, L, Dm), **io), ddt=torch.empty((Bt, L, Dm), **io),
             dz=None if z is None else torch.empty((Bt, L, Dm), **io),
             dB=torch.empty(B.shape, **io), dC=torch.empty(B.shape, **io),
             dA=torch.empty((Dm, N), **f32),
             dD=None if D is None else torch.empty((Dm,), **f32),
             ddt_bias=None if dt_bias is None else torch.empty((Dm,), **f32),
             dinitial_state=torch.empty((S, Dm, N), **f32) if want_initial_grad else None)
    t, qr = ctypes.byref(tok), ctypes.byref(q)
    ws, wp, n = _workspace("ssd_selective_backward_workspace", dev, t, qr)
    out = SSDSelectiveGrads(*(None if v is None else v.data_ptr() for v in g.values()))
    _run("ssd_selective_backward", dev, t, qr, dyp, dfp, ctypes.byref(out), wp, n)
    return g


# ---- norms -----------------------------------------------------------------------------------------

def gated_norm(x, z, weight, *, eps=1e-5, ngroups=1, norm_before_gate=False, out=None):
    """RMS norm over each of ngroups equal runs of the channels, with the gate silu(z):
    norm(x silu(z)) weight, or norm(x) weight silu(z) with norm_before_gate; z None: no gate.
    x, z [Bt, L, C]; weight [C] f32; C / ngroups a multiple of 8 up to 8192. Returns y."""
    _io(x)
    dev = x.device
    tok, _ = _tokens(x)
    xp, xs = _rows(x, "x", x.shape, x.dtype, dev)
    zp, zs = _rows(z, "z", x.shape, x.dtype, dev)
    w = _tensor(weight, "weight", x.shape[2:], torch.float32, dev)
    y, yp = _output(out, "out", x, x.shape, x.dtype)
    _run("ssd_gated_norm", dev, ctypes.byref(tok), xp, xs, zp, zs, w, ngroups, eps,
         1 if norm_before_gate else 0, yp)
    return y


def gated_norm_backward(x, z, weight, dy, *, eps=1e-5, ngroups=1, norm_before_gate=False):
    """Gradients of gated_norm for dy (x's dtype and shape). Returns a dict: dx, dz (x's dtype; dz
    None without z), dweight (float32)."""
    _io(x)
    dev = x.device
    tok, _ = _tokens(x)
    xp, xs = _rows(x, "x", x.shape, x.dtype, dev)
    zp, zs = _rows(z, "z", x.shape, x.dtype, dev)
    w = _tensor(weight, "weight", x.shape[2:], torch.float32, dev)
    dyp = _tensor(dy, "dy", x.shape, x.dtype, dev)
    g = dict(dx=torch.empty(x.shape, dtype=x.dtype, device=dev),
             dz=None if z is None else torch.empty(x.shape, dtype=x.dtype, device=dev),
             dweight=torch.empty(x.shape[2:], dtype=torch.float32, device=dev))
    t = ctypes.byref(tok)
    ws, wp, n = _workspace("ssd_gated_norm_backward_workspace", dev, t, ngroups)
    _run("ssd_gated_norm_backward", dev, t, xp, xs, zp, zs, w, ngroups, eps,
         1 if norm_before_gate else 0, dyp, *(None if v is None else v.data_ptr()
                                              for v in g.values()), wp, n)
    return g


def _res_dtype(t, name, x):
    if t.dtype not in (x.dtype, torch.float32):
        raise ValueError(f"{name} must be {x.dtype} or float32, got {t.dtype}")
    return t.dtype


def residual_norm(x, residual, weight, *, scale=None, eps=1e-5, residual_dtype=None, out=None,
                  residual_out=None):
    """Residual sum r = residual + scale x and the RMS norm of the next block, y = weight r /
    sqrt(mean r^2 + eps). x [Bt, L, C]; residual the same in x's dtype or float32, None for the
    first block (r = scale x, kept in residual_dtype, by default x's); scale [C] f32 (None: 1);
    C a multiple of 8 up to 8192. Returns (y, r)."""
    _io(x)
    dev = x.device
    tok, _ = _tokens(x)
    xp, xs = _rows(x, "x", x.shape, x.dtype, dev)
    if residual is not None:
        rt = _res_dtype(residual, "residual", x)
        if residual_dtype not in (None, rt):
            raise ValueError(f"residual_dtype must be residual's, {rt}")
    else:
        rt = x.dtype if residual_dtype is None else residual_dtype
        if rt not in (x.dtype, torch.float32):
            raise ValueError(f"residual_dtype must be {x.dtype} or float32, got {rt}")
    rp = _tensor(residual, "residual", x.shape, rt, dev)
    w = _tensor(weight, "weight", x.shape[2:], torch.float32, dev)
    sc = _tensor(scale, "scale", x.shape[2:], torch.float32, dev)
    y, yp = _output(out, "out", x, x.shape, x.dtype)
    r, op = _output(residual_out, "residual_out", x, x.shape, rt)
    _run("ssd_residual_norm", dev, ctypes.byref(tok), xp, xs, rp, DTYPES[rt], sc, w, eps, yp, op)
    return y, r


def residual_norm_backward(x, residual_sum, weight, dy, dres=None, *, scale=None, eps=1e-5,
                           want_residual_grad=True):
    """Gradients of residual_norm from what it returned: residual_sum is its r, dy the gradient of
    y, dres that of r (r's dtype, None: zero). Without a scale x gives only its shape, dtype and
    device. Returns a dict: dx (x's dtype), dresidual (r's dtype; the same tensor as dx where there
    is no scale and the two dtypes agree; None unless want_residual_grad), dweight and dscale
    (float32; dscale None without a scale)."""
    _io(x)
    dev = x.device
    tok, _ = _tokens(x)
    xp, xs = (None, 0) if scale is None else _rows(x, "x", x.shape, x.dtype, dev)
    rt = _res_dtype(residual_sum, "residual_sum", x)
    rp = _tensor(residual_sum, "residual_sum", x.shape, rt, dev)
    w = _tensor(weight, "weight", x.shape[2:], torch.float32, dev)
    sc = _tensor(scale, "scale", x.shape[2:], torch.float32, dev)
    dyp = _tensor(dy, "dy", x.shape, x.dtype, dev)
    drp = _tensor(dres, "dres", x.shape, rt, dev)
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
    same = scale is None and rt == x.dtype
    dr = torch.empty(x.shape, dtype=rt, device=dev) if want_residual_grad and not same else None
    f32 = dict(dtype=torch.float32, device=dev)
    dw = torch.empty(x.shape[2:], **f32)
    ds = None if scale is None else torch.empty(x.shape[2:], **f32)
    t = ctypes.byref(tok)
    ws, wp, n = _workspace("ssd_residual_norm_backward_workspace", dev, t)
    _run("ssd_residual_norm_backward", dev, t, rp, DTYPES[rt], xp, xs, sc, w, eps, dyp, drp,
         dx.data_ptr(), None if dr is None else dr.data_ptr(), dw.data_ptr(),
         None if ds is None else ds.data_ptr(), wp, n)
    return dict(dx=dx, dresidual=dx if want_residual_grad and same else dr, dweight=dw, dscale=ds)
