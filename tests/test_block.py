"""The operators around the scan on the GPU against their float64 oracle, element by element.

Bound of every comparison: |g - r| <= half a step of the output's type |r| (its one rounding;
nothing for float32 outputs, whose roundings are counted below) + 2^-24 k S, where S is the oracle's
sum of the absolute values of the terms that make the element (for activations times the slope's
bound) and k counts the fp32 roundings a term passes:

- convolution: W products and sums, the sigmoid (exp, add, reciprocal: 8) and its product: k = 32;
  sums over rows pass one rounding a row, at most 64 + 16 + 256 of them in a partial: k = 512;
- selective scan: a term of the state passes two roundings a token, a decay's own error is (2 |delta
  A| + 2) roundings, and x exp(-x) < 0.4 bounds what the argument's part adds over any number of
  tokens; delta has 16 (softplus), the sum of delta over a chunk one a token; then the sums over
  dstate. k = 8 (L + N + 16) forward; backward a term passes as many again, sums over tokens (dA,
  dD, ddt_bias) one a row, sums over channels (dB, dC) one a channel: k = 16 (L + N + C + 16);
- norms: the sum of squares over n channels enters by half its relative error, in at most n / 64 + 64
  additions a lane and a few waves: k = n / 32 + 64; sums over rows one a row.
"""

import ctypes

import numpy as np
import pytest
import torch

import mamba_ssd_chunked_cumsum_amd as ssd
from mamba_ssd_chunked_cumsum_amd import block as block_binding
from oracle import block

from gpu_util import DEV, note

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


def half_step(t):
    return torch.finfo(t.dtype).eps / 2 if t.dtype != torch.float32 else 0.0


def check(got, want, size, k, name):
    g = got.detach().double().cpu().numpy().reshape(np.shape(want))
    bound = half_step(got) * np.abs(want) * (1 + U) + U * k * np.abs(size) + 1e-30
    err = np.abs(g - want)
    bad = ~(err <= bound)
    assert not bad.any(), (name, int(bad.sum()), float(np.max(err / bound)),
                           np.argwhere(bad)[:3].tolist())


def value(rng, shape, io="f32", scale=1.0):
    """A device tensor and its exact float64 values."""
    t = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(TORCH[io])
    return t.to(DEV), t.double().numpy()


def sliced(rng, lead, width, io, pad):
    """The same, standing behind `pad` other values (NaN) in each row."""
    t, v = value(rng, (*lead, width), io)
    wide = torch.full((*lead, pad + width + 8), float("nan"), dtype=t.dtype, device=DEV)
    wide[..., pad:pad + width] = t
    return wide[..., pad:pad + width], v


def ranges(lens=None, batch=None, L=None):
    if lens is None:
        return [(i * L, (i + 1) * L) for i in range(batch)], None
    at = np.concatenate([[0], np.cumsum(lens)])
    return [(int(a), int(b)) for a, b in zip(at, at[1:])], torch.tensor(at, dtype=torch.int32,
                                                                        device=DEV)


# (batch, seqlen) or packed lengths with rows behind the last sequence
LAYOUTS = [
    dict(batch=1, L=1), dict(batch=3, L=2), dict(batch=2, L=17), dict(batch=1, L=130),
    dict(batch=2, L=261),
    dict(lens=[5, 0, 1, 2, 40, 0], spare=0), dict(lens=[0, 0, 3], spare=7),
    dict(lens=[64, 64, 1, 63, 130], spare=70), dict(lens=[0], spare=5),
]


def layout(d):
    if "lens" in d:
        seqs, cu = ranges(lens=d["lens"])
        return (1, sum(d["lens"]) + d["spare"]), seqs, cu
    seqs, _ = ranges(batch=d["batch"], L=d["L"])
    return (d["batch"], d["L"]), seqs, None


def name_of(d):
    return "x".join(map(str, d["lens"])) + f"+{d['spare']}" if "lens" in d else \
        f"{d['batch']}x{d['L']}"


def inside(seqs, rows):
    m = np.zeros(rows, bool)
    for a, b in seqs:
        m[a:b] = True
    return m


FILL = 7.0  # what given outputs hold before a call: rows of no sequence keep it


# ---- convolution -----------------------------------------------------------------------------------

@pytest.mark.parametrize("io,W,C,split,pad,act,bias,init", [
    ("f32", 4, 40, None, 0, "silu", True, True), ("bf16", 4, 600, (520, 40, 40), 24, "silu", True, False),
    ("bf16", 2, 8, None, 8, None, False, True), ("bf16", 3, 72, (8, 64), 0, "silu", False, True),
    ("f32", 3, 264, (8, 248, 8), 8, None, True, False)])
@pytest.mark.parametrize("lay", LAYOUTS, ids=name_of)
def test_conv(lay, io, W, C, split, pad, act, bias, init):
    rng = np.random.default_rng(11)
    lead, seqs, cu = layout(lay)
    S, rows = len(seqs), lead[0] * lead[1]
    note(f"conv {name_of(lay)} {io} W{W} C{C}")
    x, xv = sliced(rng, lead, C, io, pad)
    w, wv = value(rng, (C, W))
    b, bv = value(rng, (C,)) if bias else (None, None)
    h, hv = value(rng, (S, W - 1, C), io) if init else (None, None)
    sizes = split or (C,)
    out = tuple(torch.full((*lead, n), FILL, dtype=x.dtype, device=DEV) for n in sizes)
    y, f = ssd.conv(x, w, b, h, activation=act, split=split, cu_seqlens=cu,
                    out=out if split else out[0])
    xv = xv.reshape(rows, C)
    want, wf = block.conv(xv, wv, bv, seqs, hv, act is not None)
    size, _ = block.conv(xv, wv, bv, seqs, hv, False, absolute=True)
    got = torch.cat([t.reshape(rows, -1) for t in out], 1)
    m = inside(seqs, rows)
    check(got[torch.from_numpy(m).to(DEV)], want[m], size[m], 32, "y")
    assert torch.all(got[torch.from_numpy(~m).to(DEV)] == FILL)
    check(f, wf, wf, 0, "final")

    # backward: dy in the io type, or in float32
    for dyt in {io, "f32"}:
        dy, dyv = value(rng, (*lead, C), dyt)
        df, dfv = value(rng, (S, W - 1, C))
        dyv = dyv.reshape(rows, C) * m[:, None]
        parts = tuple(t.contiguous() for t in dy.split(sizes, -1))
        g = ssd.conv_backward(x, w, b, parts if split else parts[0], h, df, activation=act,
                              cu_seqlens=cu)
        wg = block.conv_backward(xv, wv, bv, dyv, seqs, hv, dfv, act is not None)
        ag = block.conv_backward(xv, wv, bv, dyv, seqs, hv, dfv, act is not None, absolute=True)
        mt = torch.from_numpy(m).to(DEV)
        check(g["dx"].reshape(rows, C)[mt], wg["dx"][m], ag["dx"][m], 64, "dx")
        assert torch.all(g["dx"].reshape(rows, C)[~mt] == 0)
        check(g["dweight"], wg["dw"], ag["dw"], 512, "dweight")
        if bias:
            check(g["dbias"], wg["db"], ag["db"], 512, "dbias")
        else:
            assert g["dbias"] is None
        check(g["dinitial_state"], wg["dinit"], ag["dinit"], 64, "dinitial_state")
    g = ssd.conv_backward(x, w, b, parts if split else parts[0], h, activation=act,
                          cu_seqlens=cu, want_initial_grad=False)
    wg = block.conv_backward(xv, wv, bv, dyv, seqs, hv, None, act is not None)
    check(g["dx"].reshape(rows, C)[mt], wg["dx"][m], ag["dx"][m], 64, "dx without dfinal")
    assert g["dinitial_state"] is None


@pytest.mark.parametrize("io,W,C,split", [("f32", 4, 40, None), ("bf16", 3, 600, (520, 40, 40)),
                                          ("bf16", 2, 8, None)])
def test_conv_steps_continue_a_prompt(io, W, C, split):
    rng = np.random.default_rng(12)
    Bt, L = 3, 21
    note(f"conv_step {io} W{W} C{C}")
    x, xv = sliced(rng, (Bt, L), C, io, 8)
    w, wv = value(rng, (C, W))
    b, bv = value(rng, (C,))
    seqs, _ = ranges(batch=Bt, L=L)
    want, wf = block.conv(xv.reshape(-1, C), wv, bv, seqs)
    size, _ = block.conv(xv.reshape(-1, C), wv, bv, seqs, None, False, absolute=True)
    want, size = want.reshape(Bt, L, C), size.reshape(Bt, L, C)
    with pytest.raises(ValueError, match="evenly spaced"):  # rows of a shorter batch are not
        ssd.conv(x[:, :10], w, b)
    _, state = ssd.conv(x[:, :10].contiguous(), w, b)
    for t in range(10, L):
        before = state.clone()
        y2, s2 = ssd.conv_step(state, x[:, t], w, b, split=split)
        assert torch.equal(state, before)
        y, s = ssd.conv_step(state, x[:, t], w, b, split=split, out_state=state)  # in place
        assert s.data_ptr() == state.data_ptr() and torch.equal(s, s2)
        y = torch.cat(y, -1) if split else y
        assert torch.equal(y, torch.cat(y2, -1) if split else y2)
        check(y, want[:, t], size[:, t], 32, t)
    check(state, wf, wf, 0, "state")


# ---- selective scan --------------------------------------------------------------------------------

def selective_inputs(rng, lead, S, Dm, N, G, io, pad, gate, init, skip, bias):
    t, v = {}, {}
    for k in ("x", "dt") + (("z",) if gate else ()):
        t[k], v[k] = sliced(rng, lead, Dm, io, pad)
    if not bias:  # given as they are: positive
        t["dt"] = t["dt"].abs() * 0.5
        v["dt"] = t["dt"].double().cpu().numpy()
    bc = [sliced(rng, lead, G * N, io, pad) for _ in range(2)]
    t["B"], t["C"] = (m.unflatten(-1, (G, N)) for m, _ in bc)
    v["B"], v["C"] = (m.reshape(-1, G, N) for _, m in bc)
    t["A"] = -torch.from_numpy(rng.uniform(0.0, 4.0, (Dm, N)).astype(np.float32)).to(DEV)
    t["A"][0] = 0.0  # a channel that forgets nothing
    v["A"] = t["A"].double().cpu().numpy()
    t["D"], v["D"] = value(rng, (Dm,)) if skip else (None, None)
    t["dt_bias"], v["dt_bias"] = value(rng, (Dm,), scale=3.0) if bias else (None, None)
    t["h0"], v["h0"] = value(rng, (S, Dm, N)) if init else (None, None)
    t.setdefault("z"), v.setdefault("z")
    rows = lead[0] * lead[1]
    for k in ("x", "dt", "z"):
        v[k] = None if v[k] is None else v[k].reshape(rows, Dm)
    return t, v


NAMES = ("x", "dt", "A", "B", "C", "D", "z")


@pytest.mark.parametrize("io,Dm,N,G,pad,gate,init,skip,soft", [
    ("f32", 72, 16, 1, 0, True, True, True, True), ("bf16", 136, 16, 1, 8, True, False, True, True),
    ("bf16", 16, 4, 2, 0, False, True, False, False), ("f32", 80, 8, 2, 8, False, False, True, True),
    ("f32", 48, 20, 1, 0, True, True, True, False), ("bf16", 40, 64, 1, 24, True, True, True, True)])
@pytest.mark.parametrize("lay", LAYOUTS, ids=name_of)
def test_selective(lay, io, Dm, N, G, pad, gate, init, skip, soft):
    rng = np.random.default_rng(13)
    lead, seqs, cu = layout(lay)
    S, rows, L = len(seqs), lead[0] * lead[1], max(b - a for a, b in seqs)
    note(f"selective {name_of(lay)} {io} Dm{Dm} N{N} G{G}")
    t, v = selective_inputs(rng, lead, S, Dm, N, G, io, pad, gate, init, skip, soft)
    kw = dict(dt_bias=t["dt_bias"], dt_softplus=soft, cu_seqlens=cu)
    out = torch.full((*lead, Dm), FILL, dtype=TORCH[io], device=DEV)
    y, f = ssd.selective_scan(*(t[k] for k in NAMES), t["h0"], out=out, **kw)
    args = [v[k] for k in NAMES]
    want = block.selective(*args, seqs, v["h0"], v["dt_bias"], soft)
    size = block.selective(*args, seqs, v["h0"], v["dt_bias"], soft, absolute=True)
    m = inside(seqs, rows)
    mt = torch.from_numpy(m).to(DEV)
    k = 8 * (L + N + 16)
    check(y.reshape(rows, Dm)[mt], want["y"][m], size["y"][m], k, "y")
    assert torch.all(y.reshape(rows, Dm)[~mt] == FILL)
    check(f, want["final"], size["final"], k, "final")
    y2, none = ssd.selective_scan(*(t[k] for k in NAMES), t["h0"], want_final=False, **kw)
    assert none is None and torch.equal(y2.reshape(rows, Dm)[mt], y.reshape(rows, Dm)[mt])

    dy, dyv = value(rng, (*lead, Dm), io)
    df, dfv = value(rng, (S, Dm, N))
    dyv = dyv.reshape(rows, Dm) * m[:, None]
    k = 16 * (L + N + Dm + 16)
    for final in (True, False):
        g = ssd.selective_backward(*(t[n] for n in NAMES), dy, t["h0"], df if final else None, **kw)
        more = (dyv, seqs, v["h0"], dfv if final else None, v["dt_bias"], soft)
        wg = block.selective_backward(*args, *more)
        ag = block.selective_backward(*args, *more, absolute=True)
        for n in ("dx", "ddt", "dB", "dC") + (("dz",) if gate else ()):
            check(g[n].flatten(0, 1)[mt], wg[n][m], ag[n][m], k, (n, final))
            assert torch.all(g[n].flatten(0, 1)[~mt] == 0)
        check(g["dA"], wg["dA"], ag["dA"], k + 16 * rows, "dA")
        if skip:
            check(g["dD"], wg["dD"], ag["dD"], k + 16 * rows, "dD")
        if soft:
            check(g["ddt_bias"], wg["ddt_bias"], ag["ddt_bias"], k + 16 * rows, "ddt_bias")
        check(g["dinitial_state"], wg["dinit"], ag["dinit"], k, "dinitial_state")
        assert (g["dz"] is None) == (not gate) and (g["dD"] is None) == (not skip)


@pytest.mark.parametrize("io,Dm,N,lay", [
    ("f32", 64, 16, dict(batch=1, L=1700)), ("bf16", 32, 40, dict(batch=2, L=900)),
    ("f32", 64, 8, dict(lens=[700, 0, 1, 650, 300], spare=33)),
    ("bf16", 320, 16, dict(lens=[1400], spare=0))])
def test_selective_long(io, Dm, N, lay):
    """Long sequences of few channels: the rows are cut into chunks that are chained."""
    test_selective(lay, io, Dm, N, 1, 0, True, True, True, True)


@pytest.mark.parametrize("io,Dm,N,G,gate", [("f32", 72, 16, 1, True), ("bf16", 80, 8, 2, False),
                                            ("bf16", 24, 52, 1, True), ("f32", 16, 4, 1, False),
                                            ("f32", 24, 28, 1, True)])
def test_selective_steps_continue_a_prompt(io, Dm, N, G, gate):
    rng = np.random.default_rng(14)
    Bt, L, cut = 3, 23, 11
    note(f"selective_step {io} Dm{Dm} N{N}")
    t, v = selective_inputs(rng, (Bt, L), Bt, Dm, N, G, io, 0, gate, True, True, True)
    seqs, _ = ranges(batch=Bt, L=L)
    args = [v[k] for k in NAMES]
    want = block.selective(*args, seqs, v["h0"], v["dt_bias"], True)
    size = block.selective(*args, seqs, v["h0"], v["dt_bias"], True, absolute=True)
    k = 8 * (L + N + 16)
    head = [t[n] if n in "AD" or t[n] is None else t[n][:, :cut].contiguous() for n in NAMES]
    kw = dict(dt_bias=t["dt_bias"], dt_softplus=True)
    _, state = ssd.selective_scan(*head, t["h0"], **kw)
    for i in range(cut, L):
        one = [t[n] if n in "AD" or t[n] is None else t[n][:, i] for n in NAMES]
        before = state.clone()
        y2, s2 = ssd.selective_step(state, *one, **kw)
        assert torch.equal(state, before)
        y, s = ssd.selective_step(state, *one, out_state=state, **kw)
        assert s.data_ptr() == state.data_ptr() and torch.equal(s, s2) and torch.equal(y, y2)
        check(y, want["y"].reshape(Bt, L, Dm)[:, i], size["y"].reshape(Bt, L, Dm)[:, i], k, i)
    check(state, want["final"], size["final"], k, "state")


def test_selective_extremes():
    """Decays that underflow, a large step, softplus at both ends; a NaN reaches its own channel
    from its token on and nothing else."""
    rng = np.random.default_rng(15)
    Bt, L, Dm, N = 1, 70, 64, 16
    note("selective extremes")
    t, v = selective_inputs(rng, (Bt, L), Bt, Dm, N, 1, "f32", 0, False, True, True, True)
    t["dt"][0, 5] = 60.0
    t["dt"][0, 6] = -100.0
    v["dt"] = t["dt"].double().cpu().numpy().reshape(L, Dm)
    t["A"][3] = -1e4
    v["A"] = t["A"].double().cpu().numpy()
    seqs, _ = ranges(batch=1, L=L)
    kw = dict(dt_bias=t["dt_bias"], dt_softplus=True)
    y, f = ssd.selective_scan(*(t[k] for k in NAMES), t["h0"], **kw)
    args = [v[k] for k in NAMES]
    want = block.selective(*args, seqs, v["h0"], v["dt_bias"], True)
    size = block.selective(*args, seqs, v["h0"], v["dt_bias"], True, absolute=True)
    k = 8 * (L + N + 16)
    check(y[0], want["y"], size["y"], k, "y")
    check(f, want["final"], size["final"], k, "final")
    t["x"] = t["x"].clone()
    t["x"][0, 40, 9] = float("nan")
    y2, f2 = ssd.selective_scan(*(t[k] for k in NAMES), t["h0"], **kw)
    assert torch.isnan(y2[0, 40:, 9]).all() and torch.isnan(f2[0, 9]).all()
    keep = torch.ones(L, Dm, dtype=torch.bool, device=DEV)
    keep[40:, 9] = False
    assert torch.equal(y2[0][keep], y[0][keep])
    keep = torch.arange(Dm, device=DEV) != 9
    assert torch.equal(f2[0][keep], f[0][keep])


@pytest.mark.parametrize("lens", [(70, 90, 60), (64, 128, 64), (3, 1, 2), (130, 640, 700)])
def test_a_sequence_of_nan_stays_alone(lens):
    """NaN in every input of the middle sequence: the others' outputs, states and gradients are those
    of a call without it, bit for bit."""
    rng = np.random.default_rng(19)
    L, Dm, N = sum(lens), 72, 16
    note(f"a sequence of NaN, {lens}")
    t, _ = selective_inputs(rng, (1, L), 3, Dm, N, 1, "f32", 0, True, True, True, True)
    dy, _ = value(rng, (1, L, Dm))
    df, _ = value(rng, (3, Dm, N))
    w, _ = value(rng, (Dm, 4))
    cs, _ = value(rng, (3, 3, Dm))
    _, cu = ranges(lens=lens)
    mid = slice(lens[0], lens[0] + lens[1])
    kw = dict(dt_bias=t["dt_bias"], dt_softplus=True, cu_seqlens=cu)
    x = t["x"].contiguous()

    def calls():
        y, f = ssd.selective_scan(*(t[k] for k in NAMES), t["h0"], **kw)
        g = ssd.selective_backward(*(t[k] for k in NAMES), dy, t["h0"], df, **kw)
        cy, cf = ssd.conv(x, w, None, cs, cu_seqlens=cu)
        cg = ssd.conv_backward(x, w, None, dy, cs, cs.float(), cu_seqlens=cu)
        rows = [y, cy, cg["dx"]] + [g[k].flatten(2) for k in ("dx", "ddt", "dz", "dB", "dC")]
        return [v.clone() for v in rows], [v.clone() for v in (
            f, g["dinitial_state"], cf, cg["dinitial_state"])]

    rows, states = calls()
    for k in ("x", "dt", "B", "C", "z"):
        t[k] = t[k].clone()
        t[k][:, mid] = float("nan")
    x[:, mid] = float("nan")
    for v in (dy[0], ):
        v[mid] = float("nan")
    for v in (t["h0"], df, cs):
        v[1] = float("nan")
    rows2, states2 = calls()
    for a, b in zip(rows, rows2):
        assert torch.equal(a[:, :mid.start], b[:, :mid.start])
        assert torch.equal(a[:, mid.stop:], b[:, mid.stop:])
    for a, b in zip(states, states2):
        assert torch.equal(a[::2], b[::2])


# ---- norms -----------------------------------------------------------------------------------------

NORMS = [(8, 1), (40, 1), (1024, 1), (1032, 1), (2048, 2), (2560, 1), (4104, 1), (5120, 1),
         (6144, 1), (8192, 1), (8192, 8), (24, 3)]


@pytest.mark.parametrize("C,G", NORMS)
@pytest.mark.parametrize("io,pad,gate,before", [("f32", 0, True, False), ("bf16", 24, True, True),
                                                ("bf16", 0, False, False), ("f32", 8, True, True),
                                                ("bf16", 8, True, False)])
def test_gated_norm(C, G, io, pad, gate, before):
    rng = np.random.default_rng(16)
    for lead in ((1, 1), (3, 13)):
        n = C // G
        note(f"gated_norm {lead} C{C} G{G} {io}")
        x, xv = sliced(rng, lead, C, io, pad)
        z, zv = sliced(rng, lead, C, io, pad) if gate else (None, None)
        w, wv = value(rng, (C,))
        kw = dict(eps=1e-5, ngroups=G, norm_before_gate=before)
        y = ssd.gated_norm(x, z, w, **kw)
        want = block.gated_norm(xv, zv, wv, G, 1e-5, before)
        k = n / 32 + 64
        check(y, want, want, k, "y")
        dy, dyv = value(rng, (*lead, C), io)
        g = ssd.gated_norm_backward(x, z, w, dy, **kw)
        wg = block.gated_norm_backward(xv, zv, wv, dyv, G, 1e-5, before)
        check(g["dx"], wg["dx"], wg["dx_abs"], k, "dx")
        if gate:
            check(g["dz"], wg["dz"], wg["dz_abs"], k, "dz")
        else:
            assert g["dz"] is None
        check(g["dweight"], wg["dw"], wg["dw_abs"], k + 64, "dweight")


@pytest.mark.parametrize("C", [8, 264, 1024, 1032, 2560, 5120, 8192])
@pytest.mark.parametrize("io,res,pad,scaled,first", [("f32", "f32", 0, True, False),
                                                     ("bf16", "f32", 8, False, False),
                                                     ("bf16", "bf16", 0, True, False),
                                                     ("bf16", "bf16", 24, False, False),
                                                     ("bf16", "f32", 8, True, True)])
def test_residual_norm(C, io, res, pad, scaled, first):
    rng = np.random.default_rng(17)
    for lead in ((1, 1), (2, 19)):
        note(f"residual_norm {lead} C{C} {io} {res}")
        x, xv = sliced(rng, lead, C, io, pad)
        r, rv = (None, None) if first else value(rng, (*lead, C), res, 3.0)
        w, wv = value(rng, (C,))
        s, sv = value(rng, (C,)) if scaled else (None, None)
        y, total = ssd.residual_norm(x, r, w, scale=s, residual_dtype=TORCH[res])
        want, wt = block.residual_norm(xv, rv, wv, sv)
        terms = np.abs(xv if sv is None else sv * xv) + (0 if rv is None else np.abs(rv))
        k = C / 32 + 64
        # the sum's own rounding is relative to its terms, and reaches y through weight / rms
        rms = np.sqrt((wt * wt).mean(-1, keepdims=True) + 1e-5)
        check(y, want, np.abs(want) + np.abs(wv) * terms / rms, k, "y")
        check(total, wt, terms, 2, "residual")
        tv = total.double().cpu().numpy()
        dy, dyv = value(rng, (*lead, C), io)
        for with_res in (True, False):
            dr, drv = value(rng, (*lead, C), res) if with_res else (None, None)
            g = ssd.residual_norm_backward(x, total, w, dy, dr, scale=s)
            wg = block.residual_norm_backward(xv, tv, wv, dyv, drv, sv)
            check(g["dx"], wg["dx"], wg["dx_abs"], k, "dx")
            check(g["dresidual"], wg["dr"], wg["dr_abs"], k, "dresidual")
            check(g["dweight"], wg["dw"], wg["dw_abs"], k + 64, "dweight")
            if scaled:
                check(g["dscale"], wg["ds"], wg["ds_abs"], k + 64, "dscale")
            else:
                assert g["dscale"] is None
        same = not scaled and io == res
        assert (g["dresidual"].data_ptr() == g["dx"].data_ptr()) == same
        assert ssd.residual_norm_backward(x, total, w, dy, scale=s,
                                          want_residual_grad=False)["dresidual"] is None


def test_norms_of_zeros_and_many_rows():
    note("norms of zeros, many rows")
    w = torch.ones(64, device=DEV)
    zero = torch.zeros(2, 3, 64, device=DEV)
    assert torch.all(ssd.gated_norm(zero, zero, w) == 0)
    y, r = ssd.residual_norm(zero, zero, w)
    assert torch.all(y == 0) and torch.all(r == 0)
    g = ssd.gated_norm_backward(zero, zero, w, torch.ones_like(zero))
    assert all(torch.isfinite(v).all() for v in g.values())
    rng = np.random.default_rng(18)  # more rows than walkers
    x, xv = value(rng, (1, 33000, 64))
    z, zv = value(rng, (1, 33000, 64))
    dy, dyv = value(rng, (1, 33000, 64))
    g = ssd.gated_norm_backward(x, z, w, dy)
    wg = block.gated_norm_backward(xv, zv, np.ones(64), dyv)
    check(g["dx"], wg["dx"], wg["dx_abs"], 66, "dx")
    check(g["dweight"], wg["dw"], wg["dw_abs"], 66 + 512, "dweight")


# ---- together --------------------------------------------------------------------------------------

def block_inputs(rng, Bt, L, H, P, N, io):
    Dm = H * P
    t, v = {}, {}
    t["proj"], v["proj"] = value(rng, (Bt, L, 2 * Dm + 2 * N), io)  # z, then x, B, C
    t["w"], v["w"] = value(rng, (Dm + 2 * N, 4), scale=0.5)
    t["b"], v["b"] = value(rng, (Dm + 2 * N,), scale=0.1)
    t["nw"], v["nw"] = value(rng, (Dm,))
    t["dt"] = torch.from_numpy(rng.uniform(0.01, 0.3, (Bt, L, H)).astype(np.float32)).to(DEV)
    t["A"] = torch.from_numpy(-rng.uniform(0.5, 4, H).astype(np.float32)).to(DEV)
    t["D"] = torch.ones(H, device=DEV)
    for k in ("dt", "A", "D"):
        v[k] = t[k].double().cpu().numpy()
    return t, v


def test_a_block_forward_and_backward():
    """convolution over x, B and C of one projection, the SSD scan on its three outputs, gated norm
    with the projection's z, residual norm; and the gradients back to the projection. fp32, held to
    the fp32 bar of the scan's own tests (1e-4 of the largest value)."""
    from oracle import ssd_recurrence
    from oracle.backward import ssd_backward
    rng = np.random.default_rng(21)
    Bt, L, H, P, N = 2, 96, 2, 32, 16
    Dm = H * P
    note("a block, forward and backward")
    t, v = block_inputs(rng, Bt, L, H, P, N, "f32")
    res, resv = value(rng, (Bt, L, Dm))
    z, xbc = t["proj"][..., :Dm], t["proj"][..., Dm:]
    (x, B, C), _ = ssd.conv(xbc, t["w"], t["b"], split=(Dm, N, N))
    x4, B4, C4 = x.view(Bt, L, H, P), B.view(Bt, L, 1, N), C.view(Bt, L, 1, N)
    y, _ = ssd.forward(x4, t["dt"], t["A"], B4, C4, t["D"], 64)
    n = ssd.gated_norm(y.view(Bt, L, Dm), z, t["nw"])
    out, total = ssd.residual_norm(n, res, t["nw"])

    seqs, _ = ranges(batch=Bt, L=L)
    xbcv = v["proj"][..., Dm:].reshape(Bt * L, -1)
    zv = v["proj"][..., :Dm]
    cv, _ = block.conv(xbcv, v["w"], v["b"], seqs)
    cv = cv.reshape(Bt, L, -1)
    xv, Bv, Cv = cv[..., :Dm].reshape(Bt, L, H, P), cv[..., Dm:Dm + N], cv[..., Dm + N:]
    Bv, Cv = Bv[:, :, None], Cv[:, :, None]
    yv, _ = ssd_recurrence(xv, v["dt"], v["A"], Bv, Cv, v["D"])
    yv = yv.reshape(Bt, L, Dm)
    nv = block.gated_norm(yv, zv, v["nw"])
    ov, tv = block.residual_norm(nv, resv, v["nw"])

    def near(g, w):
        g = g.double().cpu().numpy().reshape(w.shape)
        assert np.abs(g - w).max() <= 1e-4 * np.abs(w).max(), np.abs(g - w).max()

    near(out, ov)
    near(total, tv)
    dout, doutv = value(rng, (Bt, L, Dm))
    gr = ssd.residual_norm_backward(n, total, t["nw"], dout)
    gn = ssd.gated_norm_backward(y.view(Bt, L, Dm), z, t["nw"], gr["dx"])
    gs = ssd.backward(x4, t["dt"], t["A"], B4, C4, t["D"], gn["dx"].view(Bt, L, H, P), 64)
    gc = ssd.conv_backward(xbc, t["w"], t["b"],
                           (gs["dx"].view(Bt, L, Dm), gs["dB"].view(Bt, L, N),
                            gs["dC"].view(Bt, L, N)))
    wr = block.residual_norm_backward(nv, tv, v["nw"], doutv)
    wn = block.gated_norm_backward(yv, zv, v["nw"], wr["dx"])
    ws = ssd_backward(xv, v["dt"], v["A"], Bv, Cv, v["D"], wn["dx"].reshape(xv.shape))
    dcv = np.concatenate([ws["dx"].reshape(Bt, L, Dm), ws["dB"].reshape(Bt, L, N),
                          ws["dC"].reshape(Bt, L, N)], -1).reshape(Bt * L, -1)
    wc = block.conv_backward(xbcv, v["w"], v["b"], dcv, seqs)
    near(gn["dz"], wn["dz"])
    near(gc["dx"], wc["dx"].reshape(Bt, L, -1))
    near(gc["dweight"], wc["dw"])
    near(gc["dbias"], wc["db"])


def test_decoding_a_block_continues_its_prompt():
    """Tokens one at a time (conv_step, step, gated_norm) give what the prompt run over all of them
    gives, bf16 and fp32: to two roundings of the output type plus the fp32 bar."""
    rng = np.random.default_rng(22)
    Bt, L, H, P, N, cut = 2, 40, 2, 32, 16, 33
    Dm = H * P
    note("decoding a block")
    t, _ = block_inputs(rng, Bt, L, H, P, N, "f32")

    def prompt(upto):
        xbc, z = t["proj"][:, :upto, Dm:].contiguous(), t["proj"][:, :upto, :Dm].contiguous()
        (x, B, C), cs = ssd.conv(xbc, t["w"], t["b"], split=(Dm, N, N))
        y, hs = ssd.forward(x.view(Bt, upto, H, P), t["dt"][:, :upto].contiguous(), t["A"],
                            B.view(Bt, upto, 1, N), C.view(Bt, upto, 1, N), t["D"], 64)
        return ssd.gated_norm(y.view(Bt, upto, Dm), z, t["nw"]), cs, hs

    whole, _, _ = prompt(L)
    _, cs, hs = prompt(cut)
    for i in range(cut, L):
        (x, B, C), _ = ssd.conv_step(cs, t["proj"][:, i, Dm:], t["w"], t["b"], split=(Dm, N, N),
                                     out_state=cs)
        y, _ = ssd.step(hs, x.view(Bt, H, P), t["dt"][:, i].contiguous(), t["A"],
                        B.view(Bt, 1, N), C.view(Bt, 1, N), t["D"], out_state=hs)
        o = ssd.gated_norm(y.view(Bt, 1, Dm), t["proj"][:, i:i + 1, :Dm], t["nw"])
        w = whole[:, i:i + 1]
        assert (o - w).abs().max() <= 1e-4 * w.abs().max()


def every_call(rng, io="bf16", L=600, Dm=64, N=16):
    """name -> a call of each entry point on inputs of its own."""
    t, _ = selective_inputs(rng, (1, L), 1, Dm, N, 1, io, 0, True, True, True, True)
    kw = dict(dt_bias=t["dt_bias"], dt_softplus=True)
    w, _ = value(rng, (Dm, 4))
    nw, _ = value(rng, (Dm,))
    state, _ = value(rng, (1, 3, Dm), io)
    dy, _ = value(rng, (1, L, Dm), io)
    x, z = t["x"].contiguous(), t["z"].contiguous()
    first = [t[k] if k in "AD" else t[k][:, 0].contiguous() for k in NAMES]
    return {
        "conv": lambda: ssd.conv(x, w, nw, state),
        "conv_step": lambda: ssd.conv_step(state, x[:, 0], w, nw),
        "conv_backward": lambda: ssd.conv_backward(x, w, nw, dy, state),
        "selective_scan": lambda: ssd.selective_scan(*(t[k] for k in NAMES), t["h0"], **kw),
        "selective_step": lambda: ssd.selective_step(t["h0"], *first, **kw),
        "selective_backward": lambda: ssd.selective_backward(*(t[k] for k in NAMES), dy, t["h0"],
                                                             **kw),
        "gated_norm": lambda: ssd.gated_norm(x, z, nw),
        "gated_norm_backward": lambda: ssd.gated_norm_backward(x, z, nw, dy),
        "residual_norm": lambda: ssd.residual_norm(x, z, nw, scale=nw),
        "residual_norm_backward": lambda: ssd.residual_norm_backward(x, z, nw, dy, scale=nw),
    }


def tensors(r):
    if isinstance(r, torch.Tensor):
        return [r]
    if isinstance(r, dict):
        r = [r[k] for k in sorted(r)]
    return [t for v in r if v is not None for t in tensors(v)]


CALLS = ["conv", "conv_step", "conv_backward", "selective_scan", "selective_step",
         "selective_backward", "gated_norm", "gated_norm_backward", "residual_norm",
         "residual_norm_backward"]


@pytest.mark.parametrize("name", CALLS)
def test_repeats_streams_and_graphs(name):
    """The same bits again, on another stream, and from a captured graph replayed with eager calls
    and synchronisations between."""
    note(f"{name}: repeats, streams, graphs")
    call = every_call(np.random.default_rng(23))[name]
    want = [t.clone() for t in tensors(call())]
    assert all(torch.equal(a, b) for a, b in zip(tensors(call()), want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = tensors(call())
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = tensors(call())
    for _ in range(3):
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
        assert all(torch.equal(a, b) for a, b in zip(tensors(call()), want))


def test_two_graphs_do_not_share_a_workspace():
    note("two graphs at once")
    calls = [every_call(np.random.default_rng(s), L=1500) for s in (24, 25)]
    names = ("selective_scan", "selective_backward", "conv_backward", "gated_norm_backward")
    want = [[t.clone() for n in names for t in tensors(c[n]())] for c in calls]
    torch.cuda.synchronize()
    graphs, held = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append([t for n in names for t in tensors(c[n]())])
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for h, w in zip(held, want):
            assert all(torch.equal(a, b) for a, b in zip(h, w))


def test_offsets_that_break_the_contract_stay_inside():
    """Offsets beyond the rows, negative or decreasing: no result is promised, but every access
    stays inside the tensors (the offsets are clamped where they are read)."""
    note("bad offsets")
    rng = np.random.default_rng(26)
    x, _ = value(rng, (1, 50, 64))
    w, _ = value(rng, (64, 4))
    t, _ = selective_inputs(rng, (1, 50), 3, 64, 16, 1, "f32", 0, True, True, True, True)
    for bad in ([0, 20, 40, 10 ** 9], [-5, 20, 30, 50], [0, 40, 10, 50], [60, 70, 80, 90]):
        cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
        ssd.conv(x, w, cu_seqlens=cu)
        ssd.conv_backward(x, w, None, x, cu_seqlens=cu)
        ssd.selective_scan(*(t[k] for k in NAMES), t["h0"], cu_seqlens=cu)
        ssd.selective_backward(*(t[k] for k in NAMES), x, t["h0"], cu_seqlens=cu)
        torch.cuda.synchronize()


def test_refusals_write_nothing():
    note("refusals")
    x = torch.zeros(1, 8, 64, device=DEV)
    w = torch.zeros(64, 4, device=DEV)
    out = torch.full_like(x, FILL)
    wide = torch.zeros(1, 8, 100, device=DEV)
    for bad in (lambda: ssd.conv(x, w, out=x),                                  # y on x
                lambda: ssd.conv(wide[..., 2:66], w, out=out),                  # 8-byte offset
                lambda: ssd.conv(wide[..., 4:68], w, out=out),                  # row stride 100
                lambda: ssd.conv(x, torch.zeros(64, 5, device=DEV), out=out),   # width 5
                lambda: ssd.gated_norm(x, x, w[:, 0].contiguous(), ngroups=16, out=out),
                lambda: ssd.residual_norm(x, x, w[:, 0].contiguous(), residual_out=x, out=out)):
        with pytest.raises(ssd.SSDError):
            bad()
    torch.cuda.synchronize()
    assert torch.all(out == FILL)


# ---- the variants that only large sizes take -------------------------------------------------------

def test_large_batches_equal_their_parts():
    """Many rows or sequences take longer strips, stores past the caches and several sequences a
    thread: bit for bit what the sequences give one batch at a time."""
    note("large batches against their parts")
    rng = np.random.default_rng(27)
    w, _ = value(rng, (1024, 4))
    x = torch.randn(3, 11003, 1024, device=DEV).to(torch.bfloat16)
    state = torch.randn(3, 3, 1024, device=DEV).to(torch.bfloat16)
    y, f = ssd.conv(x, w, None, state)
    for i in range(3):
        part = x[i:i + 1, :4000].contiguous()
        yi, fi = ssd.conv(part, w, None, state[i:i + 1].contiguous())
        assert torch.equal(y[i:i + 1, :4000], yi) and torch.equal(fi, part[:, -3:])
    assert torch.equal(f, x[:, -3:])
    for Bt, Dm, N, G in ((67, 4104, 16, 1), (19, 2048, 40, 2)):
        t, _ = selective_inputs(rng, (Bt, 1), Bt, Dm, N, G, "bf16", 8, True, True, True, True)
        one = [t[k] if k in "AD" else t[k][:, 0] for k in NAMES]
        kw = dict(dt_bias=t["dt_bias"], dt_softplus=True)
        y, s = ssd.selective_step(t["h0"], *one, **kw)
        for i in (0, 3, Bt - 1):
            few = [v if k in "AD" else v[i:i + 1] for k, v in zip(NAMES, one)]
            yi, si = ssd.selective_step(t["h0"][i:i + 1].contiguous(), *few, **kw)
            assert torch.equal(y[i:i + 1], yi) and torch.equal(s[i:i + 1], si)


def test_which_scans_are_cut_into_chunks():
    """A long sequence of few channels needs a workspace (its rows are cut into chunks), many short
    sequences of many channels none."""
    note("scan plans")
    rng = np.random.default_rng(28)
    sizes = []
    for Bt, L, Dm in ((1, 4096, 64), (64, 32, 4096)):
        t, _ = selective_inputs(rng, (Bt, L), Bt, Dm, 16, 1, "bf16", 0, False, False, False, False)
        q = block_binding._selective(t["x"], t["dt"], t["A"], t["B"], t["C"], None, None, None, None,
                                     False, Bt, (Bt, L), t["x"].device)
        tok, _ = block_binding._tokens(t["x"])
        ws, _, n = block_binding._workspace("ssd_selective_scan_workspace", t["x"].device,
                                            ctypes.byref(tok), ctypes.byref(q))
        sizes.append(n)
    assert sizes[0] > 0 and sizes[1] == 0


def test_offsets_beyond_32_bits():
    """Tensors of more than 2^31 elements: the last sequence is what it is alone. The selective scan
    may be cut differently there, so its outputs are held to two roundings of bf16 of the largest
    value; the others are equal bit for bit."""
    note("offsets beyond 32 bits")
    S, L, C, N = 2701, 100, 8192, 4
    assert S * L * C > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(29)

    def act():
        t = torch.empty(S, L, C, dtype=torch.bfloat16, device=DEV)
        return t.normal_(generator=g)

    def last(t):
        return t[-1:].contiguous()

    x, z, dy = act(), act(), act()
    w = torch.randn(C, 4, device=DEV, generator=g)
    nw = torch.randn(C, device=DEV, generator=g)
    A = -torch.rand(C, N, device=DEV, generator=g)
    B = torch.empty(S, L, 1, N, dtype=torch.bfloat16, device=DEV).normal_(generator=g)
    pairs = [
        (lambda x, z, dy: ssd.conv(x, w, nw)[0], True),
        (lambda x, z, dy: ssd.conv_backward(x, w, nw, dy)["dx"], True),
        (lambda x, z, dy: ssd.gated_norm(x, z, nw), True),
        (lambda x, z, dy: ssd.gated_norm_backward(x, z, nw, dy)["dz"], True),
        (lambda x, z, dy: ssd.residual_norm(x, z, nw)[1], True),
        (lambda x, z, dy: ssd.residual_norm_backward(x, z, nw, dy)["dx"], True),
        (lambda x, z, dy: ssd.selective_scan(x, z, A, B[-x.shape[0]:], B[-x.shape[0]:], nw, z,
                                             dt_softplus=True, want_final=False)[0], False),
        (lambda x, z, dy: ssd.selective_backward(x, z, A, B[-x.shape[0]:], B[-x.shape[0]:], nw, z,
                                                 dy, dt_softplus=True)["ddt"], False),
    ]
    for i, (call, same) in enumerate(pairs):
        got = last(call(x, z, dy))
        want = call(last(x), last(z), last(dy))
        if same:
            assert torch.equal(got, want), i
        else:
            err = (got.float() - want.float()).abs().max()
            assert err <= 2 * torch.finfo(got.dtype).eps * want.float().abs().max(), (i, err)
        del got, want
    del x, z, dy, B, pairs
    torch.cuda.empty_cache()


@pytest.mark.parametrize("lens", [None, (96, 1, 700, 64, 0, 2000, 979)])
def test_selective_backward_of_many_channels_equals_its_parts(lens):
    """Many channels (chunks with and without sequence boundaries in launches of their own) against a
    call with a few of them, which are independent but for dB and dC: to 2^-17 of the largest
    value, some tens of fp32 roundings."""
    note("selective backward, many channels")
    rng = np.random.default_rng(30)
    C, N, few = 4096, 16, slice(1984, 2112)
    Bt, L = (40, 96) if lens is None else (1, sum(lens))
    seqs, cu = ranges(batch=Bt, L=L) if lens is None else ranges(lens=lens)
    S = len(seqs)
    t, _ = selective_inputs(rng, (Bt, L), S, C, N, 1, "f32", 0, True, True, True, True)
    dy, _ = value(rng, (Bt, L, C))
    df, _ = value(rng, (S, C, N))
    kw = dict(dt_softplus=True, cu_seqlens=cu)
    g = ssd.selective_backward(*(t[k] for k in NAMES), dy, t["h0"], df, dt_bias=t["dt_bias"], **kw)

    def cut(v):
        return v[..., few].contiguous()

    p = ssd.selective_backward(cut(t["x"]), cut(t["dt"]), t["A"][few].contiguous(), t["B"], t["C"],
                               cut(t["D"]), cut(t["z"]), cut(dy), t["h0"][:, few].contiguous(),
                               df[:, few].contiguous(), dt_bias=cut(t["dt_bias"]), **kw)
    for k in ("dx", "ddt", "dz", "dD", "ddt_bias", "dA", "dinitial_state"):
        whole = g[k][few] if k == "dA" else g[k][:, few] if k == "dinitial_state" else cut(g[k])
        err = (whole - p[k]).abs().max()
        assert err <= 2.0 ** -17 * p[k].abs().max(), (k, err)


@pytest.mark.parametrize("lens", [None, (96, 1, 700, 64, 0, 300, 579)])
def test_selective_backward_of_many_groups_equals_its_parts(lens):
    """Many waves (chunks with and without sequence boundaries in launches of their own) against calls
    with one group, which shares nothing with the others: to 2^-17 of the largest value, some tens
    of fp32 roundings."""
    note("selective backward, many groups")
    rng = np.random.default_rng(31)
    G, cg, N = 128, 8, 64
    Bt, L = (5, 350) if lens is None else (1, sum(lens))
    seqs, cu = ranges(batch=Bt, L=L) if lens is None else ranges(lens=lens)
    S, C = len(seqs), G * cg
    t, _ = selective_inputs(rng, (Bt, L), S, C, N, G, "f32", 0, True, True, True, True)
    dy, _ = value(rng, (Bt, L, C))
    df, _ = value(rng, (S, C, N))
    kw = dict(dt_softplus=True, cu_seqlens=cu)
    g = ssd.selective_backward(*(t[k] for k in NAMES), dy, t["h0"], df, dt_bias=t["dt_bias"], **kw)
    for i in (0, 77, G - 1):
        few = slice(i * cg, (i + 1) * cg)

        def cut(k, v):
            if k in ("B", "C", "dB", "dC"):
                return v[:, :, i:i + 1].contiguous()
            if k in ("A", "dA"):
                return v[few].contiguous()
            return v[:, few].contiguous() if k in ("h0", "dinitial_state") else v[..., few].contiguous()

        p = ssd.selective_backward(*(cut(k, t[k]) for k in NAMES), cut("dy", dy), cut("h0", t["h0"]),
                                   cut("h0", df), dt_bias=cut("dt_bias", t["dt_bias"]), **kw)
        for k in p:
            err = (cut(k, g[k]) - p[k]).abs().max()
            assert err <= 2.0 ** -17 * p[k].abs().max(), (i, k, err)
