"""The selective scan and its gradients against error bounds that follow each rounding through the
recurrence, so that a loss of a few bits is seen; on the GPU, and on the CPU for a float32 evaluation of
the formulas, once as it should be (inside the bounds) and with single values kept in fewer bits (outside).

With u = 2^-24 and first-order terms only (second-order ones are covered by the factor 1.01), every
quantity q has a bound E[q] on its error and a size S[q], the same sum over its terms' absolute values:

- delta: the sum with the bias is one rounding of raw, which softplus passes on with its slope; softplus
  itself, max(v, 0) + log(1 + e) with e = exp(-|v|): the exponential's argument has two roundings and the
  instruction one unit in the last place (2 u), so e is off by (2 |v| + 2) u e; logarithm, its factor
  and the sums add 5 u of delta, the term left out less than u e;
- decay a = exp(delta A): three roundings of the argument, 2 u of the instruction, and delta's error; a
  chunk's decay comes from a sum of up to M deltas, which adds M u |A delta|;
- state: h = a h + delta x B, a rounding for each product and sum, and one more where a chunk's own part
  and the entering state's are joined: 2 u S[h] a token;
- sums over n entries pass at most n + 2 roundings, sums over rows 64 in a chunk, then one partial a
  chunk in 16 groups; sums over channels four in a wave, three over the waves and one a tile;
- a sigmoid 1 / (1 + exp(-v)): the exponential's (2 |v| + 2) u reaches it by the factor sigmoid(-v),
  sum and reciprocal add 3 u;
- the gradient of the entering state of a chunk is a sum over its rows with up to M roundings of the
  whole: (M + 2) u S[G] where a chunk begins.
Outputs in bf16 add half a step of their value."""

import numpy as np
import pytest
import torch

import mamba_ssd_chunked_cumsum_amd as ssd
from oracle.block import sigmoid, softplus

from gpu_util import DEV, note

U = 2.0 ** -24
M = 64  # rows of a chunk
HALF = {"f32": 0.0, "bf16": 2.0 ** -8}


def slope_of(v):
    """Error bound of the kernels' sigmoid, relative."""
    return (sigmoid(-v) * (2 * np.abs(v) + 2) + 3) * U


def bounds(p, seqs):
    """name -> (value, error bound, size) of every output, from float64 arrays x, dt, z, dy [R, Dm], B, C
    [R, G, N], A [Dm, N], D, dt_bias [Dm], h0, dfinal [S, Dm, N]; softplus on."""
    x, dt, z, dy, A, D, bias = (p[k] for k in ("x", "dt", "z", "dy", "A", "D", "dt_bias"))
    R, Dm = x.shape
    G, N = p["B"].shape[1:]
    per = Dm // G
    B, C = (np.repeat(p[k], per, axis=1) for k in ("B", "C"))
    raw = dt + bias
    dl, far = softplus(raw), np.exp(-np.abs(raw))
    e_dl = U * (sigmoid(raw) * np.abs(raw) + 5 * dl + (2 * np.abs(raw) + 3) * far)
    du = dl * x
    e_du = np.abs(x) * e_dl + U * np.abs(du)
    v = du[..., None] * B
    e_v = np.abs(B) * e_du[..., None] + U * np.abs(v)
    a = np.exp(dl[..., None] * A)
    r_a = (3 + M) * U * np.abs(dl[..., None] * A) + np.abs(A) * e_dl[..., None] + 2 * U

    h, e_h, s_h, prev, e_prev, s_prev = (np.zeros((R, Dm, N)) for _ in range(6))
    out_h, out_g = ([np.zeros((len(seqs), Dm, N)) for _ in range(3)] for _ in range(2))
    for s, (first, end) in enumerate(seqs):
        st, er, si = p["h0"][s].copy(), np.zeros((Dm, N)), np.abs(p["h0"][s])
        for t in range(first, end):
            prev[t], e_prev[t], s_prev[t] = st, er, si
            st, er = a[t] * st + v[t], a[t] * (er + si * r_a[t]) + e_v[t]
            si = a[t] * si + np.abs(v[t])
            er = er + 2 * U * si
            h[t], e_h[t], s_h[t] = st, er, si
        for o, w in zip(out_h, (st, er, si)):
            o[s] = w

    g = z * sigmoid(z)
    r_g = slope_of(z) + U
    pre = (C * h).sum(-1) + D * x
    s_pre = (np.abs(C) * s_h).sum(-1) + np.abs(D * x)
    e_pre = (np.abs(C) * e_h).sum(-1) + (N + 2) * U * s_pre
    y = pre * g
    e_y = np.abs(g) * (e_pre + s_pre * (r_g + U))
    e = dy * g
    e_e = np.abs(e) * (r_g + U)

    Gv, e_G, s_G = (np.zeros((R, Dm, N)) for _ in range(3))
    for s, (first, end) in enumerate(seqs):
        st, er, si = p["dfinal"][s].copy(), np.zeros((Dm, N)), np.abs(p["dfinal"][s])
        for t in range(end - 1, first - 1, -1):
            st, si = st + e[t][:, None] * C[t], si + np.abs(e[t][:, None] * C[t])
            er = er + np.abs(C[t]) * e_e[t][:, None] + 2 * U * si
            Gv[t], e_G[t], s_G[t] = st, er, si
            er = a[t] * (er + si * (r_a[t] + U))
            st, si = a[t] * st, a[t] * si
            if t % M == 0:
                er = er + (M + 2) * U * si
        for o, w in zip(out_g, (st, er, si)):
            o[s] = w

    q, s_q = (Gv * B).sum(-1), (s_G * np.abs(B)).sum(-1)
    e_q = (np.abs(B) * e_G).sum(-1) + (N + 2) * U * s_q
    w, s_w = a * Gv * prev, a * s_G * s_prev
    e_w = a * (e_G + s_G * (r_a + 2 * U)) * s_prev + a * s_G * e_prev
    sa, s_sa = (w * A).sum(-1), (s_w * np.abs(A)).sum(-1)
    e_sa = (np.abs(A) * e_w).sum(-1) + (N + 5) * U * s_sa
    De = D * e
    s_dx = dl * s_q + np.abs(De)
    e_dx = dl * e_q + s_q * e_dl + np.abs(D) * e_e + U * np.abs(De) + U * s_dx
    dd, s_dd = x * q + sa, np.abs(x) * s_q + s_sa
    e_dd = np.abs(x) * e_q + e_sa + U * s_dd
    sl = sigmoid(raw)
    r_sl = slope_of(raw) + sigmoid(-raw) * np.abs(raw) * U
    ddt, s_ddt = dd * sl, s_dd * sl
    e_ddt = sl * (e_dd + s_dd * (r_sl + U))
    sg, r_sg = sigmoid(z), slope_of(z)
    s_gs = sg * (1 + np.abs(z) * (1 - sg))
    gs = sg * (1 + z * (1 - sg))
    e_gs = sg * np.abs(z) * (sg * r_sg + U * (1 - sg)) + s_gs * (r_sg + 2 * U)
    dz, s_dz = dy * pre * gs, np.abs(dy) * s_pre * s_gs
    e_dz = np.abs(dy) * (e_pre * np.abs(gs) + s_pre * e_gs) + 2 * U * s_dz

    def over(m):  # the channels of a group
        return m.reshape(R, G, per, N).sum(2)

    n_ch = 8 + -(-per // 16)
    chunks = -(-R // M)
    n_row = M + 16 + -(-chunks // 16) + 16
    adu = np.abs(du)[..., None]
    s_dB = over(s_G * adu)
    e_dB = over(e_G * adu + s_G * (e_du[..., None] + U * adu)) + n_ch * U * s_dB
    ae = np.abs(e)[..., None]
    s_dC = over(s_h * ae)
    e_dC = over(e_h * ae + s_h * (e_e[..., None] + U * ae)) + n_ch * U * s_dC
    s_dA = (s_w * dl[..., None]).sum(0)
    e_dA = (e_w * dl[..., None] + s_w * e_dl[..., None]).sum(0) + n_row * U * s_dA
    s_dD = np.abs(e * x).sum(0)
    e_dD = (e_e * np.abs(x)).sum(0) + n_row * U * s_dD
    s_db = s_ddt.sum(0)
    return dict(
        y=(y, e_y, s_pre * np.abs(g)), final=tuple(out_h), dx=(q * dl + De, e_dx, s_dx),
        ddt=(ddt, e_ddt, s_ddt), dz=(dz, e_dz, s_dz),
        dB=(over(Gv * du[..., None]), e_dB, s_dB), dC=(over(h * e[..., None]), e_dC, s_dC),
        dA=((w * dl[..., None]).sum(0), e_dA, s_dA), dD=((e * x).sum(0), e_dD, s_dD),
        ddt_bias=(ddt.sum(0), e_ddt.sum(0) + n_row * U * s_db, s_db), dinitial_state=tuple(out_g))


IO = ("y", "dx", "ddt", "dz", "dB", "dC")


def worst(got, want, io):
    """name -> the largest error as a share of its bound."""
    r = {}
    for k, (value, error, _) in want.items():
        half = HALF[io] if k in IO else 0.0
        err = np.abs(np.asarray(got[k], np.float64).reshape(value.shape) - value)
        r[k] = float(np.max(err / (1.01 * (half * (np.abs(value) + error) + error) + 1e-30)))
    return r


def draw(seed, lens, Dm, N, G, io):
    rng = np.random.default_rng(seed)
    at = np.concatenate([[0], np.cumsum(lens)])
    seqs, R, S = list(zip(at[:-1].tolist(), at[1:].tolist())), int(at[-1]), len(lens)

    def f32(m):
        return m.astype(np.float32)

    def act(*shape):
        t = torch.from_numpy(f32(rng.standard_normal(shape)))
        return t.to(torch.bfloat16).float().numpy() if io == "bf16" else t.numpy()

    p = dict(x=act(R, Dm), dt=act(R, Dm), z=act(R, Dm), dy=act(R, Dm), B=act(R, G, N), C=act(R, G, N),
             A=f32(-rng.uniform(0.05, 8.0, (Dm, N))), D=f32(rng.standard_normal(Dm)),
             dt_bias=f32(rng.uniform(-5.0, 0.0, Dm)), h0=f32(rng.standard_normal((S, Dm, N))),
             dfinal=f32(rng.standard_normal((S, Dm, N))))
    return p, seqs, at


# dense batches (equal lengths given as such) and packed ones; every number of lanes a channel
CASES = [
    ((1,), 16, 4, 1, "f32", False), ((130, 130), 72, 16, 1, "f32", False),
    ((261,), 40, 16, 1, "f32", True), ((5, 0, 64, 1, 200, 63), 80, 8, 2, "f32", True),
    ((100, 33), 136, 20, 1, "f32", True), ((150,), 48, 64, 1, "f32", False),
    ((192, 192), 64, 16, 1, "bf16", False), ((40, 77), 32, 40, 2, "bf16", True)]


def case_name(c):
    return f"{'x'.join(map(str, c[0]))}-C{c[1]}-N{c[2]}-G{c[3]}-{c[4]}"


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=case_name)
def test_selective_scan_stays_inside_its_rounding_bounds(case):
    lens, Dm, N, G, io, packed = case
    note(f"selective rounding {case_name(case)}")
    p, seqs, at = draw(71, lens, Dm, N, G, io)
    R, lead = int(at[-1]), (1, int(at[-1])) if packed else (len(lens), lens[0])
    t = {k: torch.from_numpy(m).to(DEV) for k, m in p.items()}
    for k in ("x", "dt", "z", "dy", "B", "C"):
        t[k] = t[k].to(torch.bfloat16 if io == "bf16" else torch.float32).unflatten(0, lead)
    kw = dict(dt_bias=t["dt_bias"], dt_softplus=True,
              cu_seqlens=torch.tensor(at, dtype=torch.int32, device=DEV) if packed else None)
    args = [t[k] for k in ("x", "dt", "A", "B", "C", "D", "z")]
    y, final = ssd.selective_scan(*args, t["h0"], **kw)
    got = ssd.selective_backward(*args, t["dy"], t["h0"], t["dfinal"], **kw)
    got = {k: m.double().cpu().numpy() for k, m in dict(got, y=y, final=final).items()}
    want = bounds({k: m.astype(np.float64) for k, m in p.items()}, seqs)
    shares = worst(got, want, io)
    assert R and max(shares.values()) <= 1.0, shares


def evaluate(p, seqs, coarse=None):
    """The formulas in float32, token by token; `coarse` names one value that is kept to 12 bits."""
    f = np.float32

    def keep(name, m):
        m = np.asarray(m, f)
        if name != coarse:
            return m
        k = f(2.0 ** 12 + 1)  # (Dekker's splitting: the upper 12 bits)
        return f(k * m) - f(f(k * m) - m)

    x, dt, z, dy, A, D, bias = (p[k] for k in ("x", "dt", "z", "dy", "A", "D", "dt_bias"))
    R, Dm = x.shape
    G, N = p["B"].shape[1:]
    per = Dm // G
    B, C = (np.repeat(p[k], per, axis=1) for k in ("B", "C"))
    raw = dt + bias
    dl = keep("delta", np.maximum(raw, 0) + np.log1p(np.exp(-np.abs(raw))))
    a = keep("decay", np.exp(dl[..., None] * A))
    du = dl * x
    sg, sl = (f(1) / (f(1) + np.exp(-m)) for m in (z, raw))
    g = keep("gate", z * sg)
    h, prev, Gv = (np.zeros((R, Dm, N), f) for _ in range(3))
    S = len(seqs)
    final, dinit, dA = np.zeros((S, Dm, N), f), np.zeros((S, Dm, N), f), np.zeros((Dm, N), f)
    e = dy * g
    for s, (first, end) in enumerate(seqs):
        st = p["h0"][s]
        for t in range(first, end):
            prev[t] = st
            st = h[t] = keep("state", a[t] * st + du[t][:, None] * B[t])
        final[s] = st
        st = p["dfinal"][s]
        for t in range(end - 1, first - 1, -1):
            Gv[t] = keep("adjoint", st + e[t][:, None] * C[t])
            st = a[t] * Gv[t]
        dinit[s] = st
    w = a * Gv * prev
    for t in range(R):
        dA = keep("sum of dA", dA + w[t] * dl[t][:, None])
    pre = keep("sum over the states", (h * C).sum(-1)) + D * x
    q = (Gv * B).sum(-1)
    ddt = (x * q + (w * A).sum(-1)) * sl

    def over(m):
        return m.reshape(R, G, per, N).sum(2)

    return dict(y=pre * g, final=final, dx=dl * q + D * e, ddt=ddt, dz=dy * pre * (sg * (1 + z * (1 - sg))),
                dB=over(Gv * du[..., None]), dC=over(h * e[..., None]), dA=dA, dD=(e * x).sum(0),
                ddt_bias=ddt.sum(0), dinitial_state=dinit)


@pytest.mark.parametrize("case", [c for c in CASES if c[4] == "f32"], ids=case_name)
def test_float32_stays_inside_the_bounds_and_fewer_bits_do_not(case):
    lens, Dm, N, G, io, _ = case
    p, seqs, _ = draw(72, lens, Dm, N, G, io)
    want = bounds({k: m.astype(np.float64) for k, m in p.items()}, seqs)
    shares = worst(evaluate(p, seqs), want, io)
    assert max(shares.values()) <= 1.0, shares
    for coarse in ("delta", "decay", "gate", "state", "adjoint", "sum of dA", "sum over the states"):
        if coarse == "sum of dA" and max(lens) < 100:
            continue
        shares = worst(evaluate(p, seqs, coarse), want, io)
        assert max(shares.values()) > 1.0, (coarse, shares)
