"""Float64 CPU oracle of the operators around the scan, from their formulas (test infrastructure
only): causal convolution, selective scan, gated norm, residual norm, forward and backward.

Every function takes a list of (first, end) token ranges, the sequences of one flat row axis
(dense batches are ranges of equal length), and arrays [rows, ...]. With ``absolute`` True the
same sums run over the absolute values of their terms: what fp32 rounding errors are relative to.
"""

from __future__ import annotations

import numpy as np


def sigmoid(v):
    return 0.5 * (1.0 + np.tanh(0.5 * np.asarray(v, np.float64)))


def silu(v):
    return v * sigmoid(v)


def dsilu(v):
    s = sigmoid(v)
    return s * (1.0 + v * (1.0 - s))


def softplus(v):
    return np.logaddexp(0.0, v)


def _f64(*arrays):
    return [None if a is None else np.asarray(a, np.float64) for a in arrays]


# ---- convolution ---------------------------------------------------------------------------------

def conv(x, w, bias, seqs, init=None, act=True, absolute=False):
    """(y, final [nseq, W - 1, C]); rows of no sequence stay zero."""
    x, w, bias, init = _f64(x, w, bias, init)
    C, W = w.shape
    if absolute:
        x, w = np.abs(x), np.abs(w)
        bias = None if bias is None else np.abs(bias)
        init = None if init is None else np.abs(init)
    v, final = np.zeros_like(x), np.zeros((len(seqs), W - 1, C))
    for s, (a, b) in enumerate(seqs):
        u = np.concatenate([np.zeros((W - 1, C)) if init is None else init[s], x[a:b]])
        final[s] = u[b - a:]
        for k in range(W):
            v[a:b] += w[:, k] * u[k:k + b - a]
        if bias is not None:
            v[a:b] += bias
    return (silu(v) if act and not absolute else v), final


def conv_backward(x, w, bias, dy, seqs, init=None, dfinal=None, act=True, absolute=False):
    """dict(dx, dw, db, dinit). absolute: with |x|, |w|, |dv| in every sum, dv as it is (its own
    factors bounded by |dy| 1.1)."""
    x, w, bias, dy, init, dfinal = _f64(x, w, bias, dy, init, dfinal)
    C, W = w.shape
    v, _ = conv(x, w, bias, seqs, init, act=False)
    if act:
        vabs, _ = conv(x, w, bias, seqs, init, act=False, absolute=True)
        dv = dy * dsilu(v)
        if absolute:  # silu' has slope below 1/2: the error of v enters through it
            dv = np.abs(dy) * (1.1 + 0.5 * vabs)
    else:
        dv = dy.copy()
    if absolute:
        x, w, dv = np.abs(x), np.abs(w), np.abs(dv)
        init, dfinal = (None if t is None else np.abs(t) for t in (init, dfinal))
    out = dict(dx=np.zeros_like(x), dw=np.zeros_like(w), db=np.zeros(C),
               dinit=np.zeros((len(seqs), W - 1, C)))
    for s, (a, b) in enumerate(seqs):
        u = np.concatenate([np.zeros((W - 1, C)) if init is None else init[s], x[a:b]])
        du = np.zeros_like(u)
        for k in range(W):
            du[k:k + b - a] += w[:, k] * dv[a:b]
            out["dw"][:, k] += (u[k:k + b - a] * dv[a:b]).sum(0)
        if dfinal is not None:
            du[b - a:] += dfinal[s]
        out["db"] += dv[a:b].sum(0)
        out["dinit"][s], out["dx"][a:b] = du[:W - 1], du[W - 1:]
    return out


# ---- selective scan --------------------------------------------------------------------------------

def _delta(dt, dt_bias, soft):
    raw = dt if dt_bias is None else dt + dt_bias
    return raw, softplus(raw) if soft else raw


def selective(x, dt, A, B, C, D, z, seqs, h0=None, dt_bias=None, soft=False, absolute=False):
    """dict(y, final, h: the state after every row, pre: y before the gate). B, C [rows, G, N]."""
    x, dt, A, B, C, D, z, h0, dt_bias = _f64(x, dt, A, B, C, D, z, h0, dt_bias)
    R, Dm = x.shape
    N = A.shape[1]
    _, dl = _delta(dt, dt_bias, soft)
    if absolute:
        x, B, C = np.abs(x), np.abs(B), np.abs(C)
        D, h0 = (None if t is None else np.abs(t) for t in (D, h0))
    per = Dm // B.shape[1]
    Bd, Cd = (np.repeat(m, per, axis=1) for m in (B, C))  # [rows, Dm, N]
    h = np.zeros((R, Dm, N))
    final = np.zeros((len(seqs), Dm, N))
    weight = np.abs(dl) if absolute else dl
    for s, (a, b) in enumerate(seqs):
        state = np.zeros((Dm, N)) if h0 is None else h0[s].copy()
        for t in range(a, b):
            state = np.exp(dl[t][:, None] * A) * state + (weight[t] * x[t])[:, None] * Bd[t]
            h[t] = state
        final[s] = state
    pre = (h * Cd).sum(-1) + (0 if D is None else D * x)
    y = pre if z is None else pre * (np.abs(silu(z)) if absolute else silu(z))
    return dict(y=y, final=final, h=h, pre=pre)


def selective_backward(x, dt, A, B, C, D, z, dy, seqs, h0=None, dfinal=None, dt_bias=None,
                       soft=False, absolute=False):
    """dict(dx, ddt, dz, dB, dC, dA, dD, ddt_bias, dinit)."""
    f = selective(x, dt, A, B, C, D, z, seqs, h0, dt_bias, soft, absolute)
    x, dt, A, B, C, D, z, dy, h0, dfinal, dt_bias = _f64(x, dt, A, B, C, D, z, dy, h0, dfinal,
                                                         dt_bias)
    R, Dm = x.shape
    G, N = B.shape[1:]
    per = Dm // G
    raw, dl = _delta(dt, dt_bias, soft)
    ab = np.abs if absolute else (lambda t: t)
    decay = np.exp(dl[:, :, None] * A)
    x, B, C, dy = ab(x), ab(B), ab(C), ab(dy)
    h0, dfinal, D = (None if t is None else ab(t) for t in (h0, dfinal, D))
    Aw, dlw = ab(A), ab(dl)
    gate = 1.0 if z is None else ab(silu(z))
    e = dy * gate
    Bd, Cd = (np.repeat(m, per, axis=1) for m in (B, C))
    Gt, prev = np.zeros((R, Dm, N)), np.zeros((R, Dm, N))
    dinit = np.zeros((len(seqs), Dm, N))
    for s, (a, b) in enumerate(seqs):
        g = np.zeros((Dm, N)) if dfinal is None else dfinal[s].copy()
        for t in range(b - 1, a - 1, -1):
            g = g + e[t][:, None] * Cd[t]
            Gt[t] = g
            prev[t] = f["h"][t - 1] if t > a else (0.0 if h0 is None else h0[s])
            g = decay[t] * g
        dinit[s] = g
    q = (Gt * Bd).sum(-1)
    w = Gt * decay * prev
    ddl = x * q + (w * Aw).sum(-1)
    inside = np.zeros((R, 1))
    for a, b in seqs:
        inside[a:b] = 1.0
    slope = sigmoid(raw) if soft else 1.0
    ddt = ddl * slope * inside
    over = lambda t: t.reshape(R, G, per, N).sum(2)  # noqa: E731
    if z is not None:
        # silu'(z) = s (1 + z (1 - s)) cancels for z < 0 (it is zero near z = -1.28), so its
        # rounding errors are relative to the sum of its terms' absolute values, not to itself
        sz = sigmoid(z)
        gslope = sz * (1.0 + ab(z) * (1.0 - sz))
    return dict(dx=((0 if D is None else D * e) + dlw * q) * inside, ddt=ddt,
                dz=None if z is None else dy * f["pre"] * gslope * inside,
                dB=over(Gt * (dlw * x)[:, :, None]), dC=over(f["h"] * e[:, :, None]),
                dA=(w * dlw[:, :, None]).sum(0), dD=(e * x * inside).sum(0),
                ddt_bias=ddt.sum(0), dinit=dinit)


# ---- norms -----------------------------------------------------------------------------------------

def _rms(v, groups, eps):
    g = v.reshape(*v.shape[:-1], groups, -1)
    return np.broadcast_to(1.0 / np.sqrt((g * g).mean(-1, keepdims=True) + eps), g.shape).reshape(
        v.shape)


def _group_mean(v, groups):
    g = v.reshape(*v.shape[:-1], groups, -1)
    return np.broadcast_to(g.mean(-1, keepdims=True), g.shape).reshape(v.shape)


def gated_norm(x, z, w, groups=1, eps=1e-5, before=False):
    x, z, w = _f64(x, z, w)
    gate = 1.0 if z is None else silu(z)
    v = x if before else x * gate
    y = w * v * _rms(v, groups, eps)
    return y * gate if before else y


def gated_norm_backward(x, z, w, dy, groups=1, eps=1e-5, before=False):
    """dict(dx, dz, dw) and, beside each, what its fp32 errors are relative to (key + "_abs")."""
    x, z, w, dy = _f64(x, z, w, dy)
    gate, slope = (1.0, 0.0) if z is None else (silu(z), dsilu(z))
    v = x if before else x * gate
    r = _rms(v, groups, eps)
    n = v * r
    dn = w * dy * gate if before else w * dy
    m, mabs = _group_mean(dn * n, groups), _group_mean(np.abs(dn * n), groups)
    dv, dvabs = r * (dn - n * m), r * (np.abs(dn) + np.abs(n) * mabs)
    if before:
        dx, dxa = dv, dvabs
        dz, dwt = dy * w * n * slope, dy * n * gate
        dza = np.abs(dy * w * n)
    else:
        dx, dxa = dv * gate, dvabs * np.abs(gate)
        dz, dza = dv * x * slope, dvabs * np.abs(x)
        dwt = dy * n
    return dict(dx=dx, dx_abs=dxa, dz=None if z is None else dz, dz_abs=1.1 * dza,
                dw=dwt.reshape(-1, w.size).sum(0), dw_abs=np.abs(dwt).reshape(-1, w.size).sum(0))


def residual_norm(x, res, w, scale=None, eps=1e-5):
    x, res, w, scale = _f64(x, res, w, scale)
    r = (x if scale is None else scale * x) + (0.0 if res is None else res)
    return w * r * _rms(r, 1, eps), r


def residual_norm_backward(x, r, w, dy, dres=None, scale=None, eps=1e-5):
    """dict(dx, dr, dw, ds), each with its "_abs"; r is the sum that the forward returned."""
    x, r, w, dy, dres, scale = _f64(x, r, w, dy, dres, scale)
    g = gated_norm_backward(r, None, w, dy, 1, eps)
    dr = g["dx"] + (0.0 if dres is None else dres)
    dra = g["dx_abs"] + (0.0 if dres is None else np.abs(dres))
    sc = 1.0 if scale is None else scale
    flat = lambda t: t.reshape(-1, w.size).sum(0)  # noqa: E731
    return dict(dr=dr, dr_abs=dra, dx=dr * sc, dx_abs=dra * np.abs(sc), dw=g["dw"],
                dw_abs=g["dw_abs"], ds=flat(dr * x), ds_abs=flat(dra * np.abs(x)))
