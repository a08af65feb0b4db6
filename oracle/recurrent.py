"""Float64 CPU oracle of the operators of layers of linear recurrence, from their formulas (test
infrastructure only): gated linear recurrence, rotation of B and C, group norm, each forward and
backward. Sequences are (first, end) ranges of one flat row axis, as in block.py.

Each function returns its results and, for each, a bound of what fp32 arithmetic may be off, in units
of 2^-24: the relative errors of a token's factors are followed through the sums and the recurrence.
Counts of roundings (first order): sigmoid(v) from its exponential's argument 2 |v|, the exponential,
sum, reciprocal and product 8: 2 |v| + 8; the factor sharpness softplus(decay) 8; what follows from
them at each place below.
"""

from __future__ import annotations

import numpy as np

from .block import _f64, dsilu, silu, softplus


def sigmoid(v):
    """To a few roundings of itself where it is small, too."""
    return np.exp(-np.logaddexp(0.0, -np.asarray(v, np.float64)))


# ---- gated linear recurrence ---------------------------------------------------------------------

def _token(gate, decay, sharpness):
    """Factors of every element and the relative errors of them, in roundings."""
    r, no = sigmoid(gate), sigmoid(-gate)
    kr = 2 * np.abs(gate) + 8
    if decay is None:
        return dict(r=r, no=no, kr=kr, a=r, m=no, ka=kr, km=kr, u=None, tiny=0.0)
    u = sharpness * softplus(decay) * r
    ku = kr + 9
    a = np.exp(-u)
    ka = u * (ku + 2) + 2
    # 1 - exp(-2u): u's own error enters at most once; the series has 8 roundings, the difference (from
    # 2u = 1/4 on, where it is at least 0.22) two times those of a, (0.184 (ku + 2) + 3) / 0.22 at
    # most; a square root halves them and adds 4
    km = (1.7 * (ku + 2) + 28) / 2 + 4
    # below fp32's range: where 1 - a^2 is under 2^-126, m lies under 2^-63 and what is computed does,
    # too, as u / m and (r / m) softplus(decay) sharpness = sqrt(u / 2) do; where r is, they lie under
    # 2^-63 sqrt(2 k). (Absolute, in units of 2^-24.)
    sq, k = -np.expm1(-2 * u), sharpness * softplus(decay)
    tiny = np.where(np.minimum(sq, r) < 2.0 ** -126, 2.0 ** -39 * np.maximum(1, np.sqrt(2 * k)), 0.0)
    return dict(r=r, no=no, kr=kr, a=a, m=np.sqrt(sq), ka=ka, km=km, u=u, ku=ku, tiny=tiny)


def _inputs(x, gate, decay, input_gate, seqs, init, sharpness):
    f = _token(gate, decay, sharpness)
    f["si"], f["ks"] = (1.0, 0.0) if input_gate is None else (sigmoid(input_gate),
                                                             2 * np.abs(input_gate) + 8)
    f["v"] = f["si"] * x
    f["kb"] = f["km"] + f["ks"] + 2
    f["off"] = f["tiny"] * np.abs(f["v"])
    C = x.shape[1]
    h = np.zeros_like(x)      # states, sums of absolute values, errors; and those before each row
    S, E = np.zeros_like(x), np.zeros_like(x)
    before = [np.zeros_like(x) for _ in range(3)]
    final = [np.zeros((len(seqs), C)) for _ in range(3)]
    for s, (a, b) in enumerate(seqs):
        now = np.zeros(C) if init is None else init[s].copy()
        size, err = np.abs(now), np.zeros(C)
        for t in range(a, b):
            for d, v in zip(before, (now, size, err)):
                d[t] = v
            bt = f["m"][t] * f["v"][t]
            err = f["a"][t] * (err + (f["ka"][t] + 4) * size)
            now = f["a"][t] * now + bt
            size = f["a"][t] * size + np.abs(bt)
            err = err + f["kb"][t] * np.abs(bt) + 2 * size + f["off"][t]
            h[t], S[t], E[t] = now, size, err
        for d, v in zip(final, (now, size, err)):
            d[s] = v
    f.update(h=h, S=S, E=E, before=before, final=final)
    return f


def recurrence(x, gate, decay, input_gate, seqs, init=None, sharpness=8.0):
    """dict name -> (values, bound): y, final."""
    f = _inputs(*_f64(x, gate, decay, input_gate), seqs, *_f64(init), sharpness)
    return dict(y=(f["h"], f["E"]), final=(f["final"][0], f["final"][2]))


def recurrence_backward(x, gate, decay, input_gate, dy, seqs, init=None, dfinal=None,
                        sharpness=8.0):
    """dict name -> (values, bound): dx, dgate, dinput_gate, ddecay, dinitial_state."""
    x, gate, decay, input_gate, dy, init, dfinal = _f64(x, gate, decay, input_gate, dy, init, dfinal)
    f = _inputs(x, gate, decay, input_gate, seqs, init, sharpness)
    C = x.shape[1]
    lam, size, err = (np.zeros_like(x) for _ in range(3))
    dinit = [np.zeros((len(seqs), C)) for _ in range(2)]
    inside = np.zeros(len(x), bool)
    for s, (a, b) in enumerate(seqs):
        inside[a:b] = True
        c = np.zeros(C) if dfinal is None else dfinal[s].copy()  # what comes from the right
        cs, ce = np.abs(c), np.zeros(C)
        for t in range(b - 1, a - 1, -1):
            lam[t], size[t] = dy[t] + c, np.abs(dy[t]) + cs
            err[t] = ce + 2 * size[t]
            c, cs = f["a"][t] * lam[t], f["a"][t] * size[t]
            ce = f["a"][t] * (err[t] + (f["ka"][t] + 4) * size[t])
        dinit[0][s], dinit[1][s] = c, ce
    lam[~inside] = 0
    h, hs, he = f["before"]
    v, si, m, a = f["v"], f["si"], f["m"], f["a"]
    av, k = np.abs(v), f["km"] + f["ks"] + 6
    out = dict(dx=(lam * m * si, si * (m * (err + size * k) + size * f["tiny"])),
               dinitial_state=tuple(dinit))
    if input_gate is not None:
        no = sigmoid(-input_gate)
        out["dinput_gate"] = (lam * m * v * no, av * no * (m * (err + size * (k + f["ks"])) +
                                                           size * f["tiny"]))
    if decay is None:
        t, ts = h - v, hs + av
        te = he + (f["ks"] + 2) * ts
        out["dgate"] = (lam * t * a * m, a * m * (err * ts + size * (te + ts * (2 * f["kr"] + 6))))
        return out
    w, r, u = f["u"] / m, f["r"], f["u"]
    # dlog a = lam (a h - a^2 / m v)
    q = lam * (a * h - a * a / m * v)
    ks = f["ku"] + 2 * f["ka"] + f["km"] + f["ks"] + f["kr"] + 12
    terms = a * a / m * av + a * hs
    bound = err * terms + size * (ks * terms + a * he)
    off = size * a * a * f["off"]
    out["dgate"] = (-q * u * f["no"], f["no"] * (u * bound + off))
    slope = sharpness * sigmoid(decay)
    rows = max(1, int(inside.sum()))
    # added up by a wave, its block, and groups of 16 of those
    adds = 16 + 8 + 16 + rows / 16 / 16 + 2 * np.abs(decay) + 12
    out["ddecay"] = ((-q * r)[inside].sum(0) * slope,
                     (r * (bound + adds * size * terms))[inside].sum(0) * slope +
                     off[inside].sum(0))
    return out


# ---- rotation ------------------------------------------------------------------------------------

def rotate(x, positions, frequencies, sections, interleaved=False, inverse=False):
    """(values, bound) of x [rows, G, N] turned; positions [axes, rows]."""
    x, freq = np.asarray(x, np.float64), np.asarray(frequencies, np.float64)
    axis = np.repeat(np.arange(len(sections)), sections)
    angle = np.asarray(positions)[axis].T.astype(np.float64) * freq  # exact up to 2^29 (29 and 24 bits)
    angle = angle[:, None, :] * (-1.0 if inverse else 1.0)
    n = len(freq)
    p, q = (np.arange(0, 2 * n, 2), np.arange(1, 2 * n, 2)) if interleaved else \
        (np.arange(n), np.arange(n, 2 * n))
    out, bound = x.copy(), np.zeros_like(x)
    cos, sin = np.cos(angle), np.sin(angle)
    out[..., p] = x[..., p] * cos - x[..., q] * sin
    out[..., q] = x[..., p] * sin + x[..., q] * cos
    # what is left of a turn: 2 roundings to 24 bits and 2^-52 of the whole angle; sine and cosine 4
    # roundings each, products and sum 2
    e = (np.abs(x[..., p]) + np.abs(x[..., q])) * (8 + np.abs(angle) * 2.0 ** -28)
    bound[..., p] = bound[..., q] = e
    return out, bound


# ---- group norm ----------------------------------------------------------------------------------

def group_stats(x, seqs, G, eps):
    """(stats [nseq, G, 2], bound)."""
    x = np.asarray(x, np.float64)
    stats, bound = np.zeros((len(seqs), G, 2)), np.zeros((len(seqs), G, 2))
    stats[..., 1] = 0.0 if eps == 0 else eps ** -0.5
    bound[..., 1] = 4 * stats[..., 1]
    for s, (a, b) in enumerate(seqs):
        if a == b:
            continue
        t = x[a:b].reshape(b - a, G, -1)
        mean = t.mean((0, 2))
        dev = (t - mean[:, None]) ** 2
        var = dev.mean((0, 2))
        # a thread adds up to 64 values, its group's up to 256 threads (or the strips, in 64 bits)
        adds = 64 + min(256, t.shape[2] // 8 + 8)
        kmean = adds * np.abs(t).mean((0, 2)) + 4 * np.abs(mean)
        # squares about a row of the data: their sum is the variance's and that row's own deviation
        about = 1 + np.max(dev.mean(2), 0) / np.maximum(var, 1e-300)
        kvar = (adds + 8) * about * var + 2.0 ** -24 * kmean ** 2
        stats[s, :, 0], stats[s, :, 1] = mean, 1 / np.sqrt(var + eps)
        bound[s, :, 0] = kmean
        bound[s, :, 1] = stats[s, :, 1] * (0.5 * kvar / (var + eps) + 6)
    return stats, bound


def _spread(v, C):
    return np.repeat(v, C // v.shape[-1], -1)


def group_norm(x, weight, bias, seqs, G, eps, act):
    """(y, bound, stats, bound of stats)."""
    x, weight, bias = _f64(x, weight, bias)
    C = x.shape[1]
    w, b = np.ones(C) if weight is None else weight, np.zeros(C) if bias is None else bias
    stats, kst = group_stats(x, seqs, G, eps)
    y, bound = np.zeros_like(x), np.zeros_like(x)
    for s, (i, j) in enumerate(seqs):
        mean, rstd = _spread(stats[s, :, 0], C), _spread(stats[s, :, 1], C)
        kmean, krstd = _spread(kst[s, :, 0], C), _spread(kst[s, :, 1], C)
        d = x[i:j] - mean
        v = d * rstd * w + b
        e = np.abs(w) * (np.abs(d) * krstd + rstd * (kmean + 3 * np.abs(d))) + 2 * np.abs(b) + \
            2 * np.abs(v)
        y[i:j], bound[i:j] = v, e
        if act:  # slope at most 1.1
            y[i:j], bound[i:j] = silu(v), 1.1 * e + np.abs(silu(v)) * (2 * np.abs(v) + 10)
    return y, bound, stats, kst


def group_norm_backward(x, weight, bias, stats, dy, seqs, G, act):
    """dict name -> (values, bound): dx, dweight, dbias, with the stats as given."""
    x, weight, bias, stats, dy = _f64(x, weight, bias, stats, dy)
    C = x.shape[1]
    w, b = np.ones(C) if weight is None else weight, np.zeros(C) if bias is None else bias
    dx, kdx = np.zeros_like(x), np.zeros_like(x)
    dw, db, kdw, kdb = (np.zeros(C) for _ in range(4))
    for s, (i, j) in enumerate(seqs):
        if i == j:
            continue
        mean, rstd = _spread(stats[s, :, 0], C), _spread(stats[s, :, 1], C)
        n = (x[i:j] - mean) * rstd
        v = n * w + b
        ev = np.abs(n * w) * 4 + np.abs(b) + np.abs(v)
        slope = dsilu(v) if act else np.ones_like(v)
        dv = dy[i:j] * slope
        # the slope's own derivative is at most 1/2, its terms at most 1 + |v|
        kdv = np.abs(dy[i:j]) * ((0.5 * ev + (2 * np.abs(v) + 12) * (1 + np.abs(v))) if act else 1)
        rows, cg = j - i, C // G
        # a thread adds 8 tokens' vectors or 16 rows, a block its waves or threads, the rest in 64 bits;
        # walkers of short sequences and the sum over sequences: a few hundred
        adds = 300
        terms = [np.abs(dv), np.abs(dv * n)]
        kdb += (kdv + adds * terms[0]).sum(0)
        kdw += (kdv * np.abs(n) + (adds + 4) * terms[1]).sum(0)
        db += dv.sum(0)
        dw += (dv * n).sum(0)

        def mean_of(t):
            return _spread(t.reshape(rows, G, cg).mean((0, 2)), C)

        g, kg = dv * w, (kdv + 2 * np.abs(dv)) * np.abs(w)
        m1, m2 = mean_of(g), mean_of(g * n)
        k1 = mean_of(kg + adds * np.abs(g))
        k2 = mean_of(kg * np.abs(n) + (adds + 4) * np.abs(g * n))
        dx[i:j] = rstd * (g - m1 - n * m2)
        kdx[i:j] = rstd * (kg + k1 + np.abs(n) * k2 + 4 * (np.abs(g) + np.abs(m1) +
                                                           3 * np.abs(n * m2)))
    return dict(dx=(dx, kdx), dweight=(dw, kdw), dbias=(db, kdb))
