"""The operators of layers of linear recurrence on the GPU against their float64 oracle, element by
element: |g - r| <= half a step of the output's type |r| (its one rounding) + 2^-24 times the bound that
the oracle follows through each value's roundings (oracle/recurrent.py)."""

import numpy as np
import pytest
import torch

import mamba_ssd_chunked_cumsum_amd as ssd
from oracle import block, recurrent

from gpu_util import DEV, note
from test_block import (FILL, LAYOUTS, TORCH, U, half_step, inside, layout, name_of, ranges, sliced,
                        tensors, value)

pytestmark = pytest.mark.gpu

# chunks of 128 rows, strips of 64: sequences that end on, before and behind their borders
LONG = [dict(batch=3, L=700), dict(batch=2, L=128), dict(batch=9, L=16), dict(batch=11, L=8),
        dict(lens=[128, 0, 128, 1, 127, 256, 0], spare=0), dict(lens=[300, 5, 400], spare=200)]


def check(got, want, name):
    want, bound = want
    g = got.detach().double().cpu().numpy().reshape(np.shape(want))
    limit = half_step(got) * np.abs(want) * (1 + U) + U * 1.01 * bound + 1e-36
    err = np.abs(g - want)
    bad = ~(err <= limit)
    assert not bad.any(), (name, int(bad.sum()), float(np.max(err / limit)),
                           np.argwhere(bad)[:3].tolist())


def pick(pair, m):
    return pair[0][m], pair[1][m]


# ---- recurrence ------------------------------------------------------------------------------------

def recurrence_inputs(rng, lead, S, C, io, pad, decay, gated, init):
    t, v = {}, {}
    rows = lead[0] * lead[1]
    for k in ("x", "gate") + (("input_gate",) if gated else ()):
        t[k], v[k] = sliced(rng, lead, C, io, pad)
        v[k] = v[k].reshape(rows, C)
    t["decay"] = v["decay"] = None
    if decay:  # a forgets between 1e-5 and 1/2 of the state where the gate is open
        d = torch.from_numpy(rng.uniform(-13, -2, C).astype(np.float32))
        t["decay"], v["decay"] = d.to(DEV), d.double().numpy()
    t["init"], v["init"] = value(rng, (S, C)) if init else (None, None)
    t.setdefault("input_gate"), v.setdefault("input_gate")
    return t, v


IN = ("x", "gate", "decay", "input_gate")


def run_recurrence(lay, io, C, pad, decay, gated, init, seed=61):
    rng = np.random.default_rng(seed)
    lead, seqs, cu = layout(lay)
    S, rows = len(seqs), lead[0] * lead[1]
    note(f"recurrence {name_of(lay)} {io} C{C} decay{decay} gated{gated}")
    t, v = recurrence_inputs(rng, lead, S, C, io, pad, decay, gated, init)
    out = torch.full((*lead, C), FILL, dtype=TORCH[io], device=DEV)
    y, f = ssd.recurrence(*(t[k] for k in IN), t["init"], cu_seqlens=cu, out=out)
    want = recurrent.recurrence(*(v[k] for k in IN), seqs, v["init"])
    m = inside(seqs, rows)
    mt = torch.from_numpy(m).to(DEV)
    check(y.reshape(rows, C)[mt], pick(want["y"], m), "y")
    assert torch.all(y.reshape(rows, C)[~mt] == FILL)
    check(f, want["final"], "final")
    y2, none = ssd.recurrence(*(t[k] for k in IN), t["init"], cu_seqlens=cu, want_final=False)
    assert none is None and torch.equal(y2.reshape(rows, C)[mt], y.reshape(rows, C)[mt])

    dy, dyv = value(rng, (*lead, C), io)
    df, dfv = value(rng, (S, C))
    dyv = dyv.reshape(rows, C) * m[:, None]
    for final in (True, False):
        g = ssd.recurrence_backward(*(t[k] for k in IN), dy, t["init"], df if final else None,
                                    cu_seqlens=cu, want_initial_grad=final)
        wg = recurrent.recurrence_backward(*(v[k] for k in IN), dyv, seqs, v["init"],
                                           dfv if final else None)
        for n in ("dx", "dgate") + (("dinput_gate",) if gated else ()):
            check(g[n].reshape(rows, C)[mt], pick(wg[n], m), (n, final))
            assert torch.all(g[n].reshape(rows, C)[~mt] == 0)
        if decay:
            check(g["ddecay"], wg["ddecay"], "ddecay")
        if final:
            check(g["dinitial_state"], wg["dinitial_state"], "dinitial_state")
        assert (g["ddecay"] is None) == (not decay)
        assert (g["dinput_gate"] is None) == (not gated)
        assert (g["dinitial_state"] is None) == (not final)


@pytest.mark.parametrize("io,C,pad,decay,gated,init", [
    ("f32", 72, 0, True, True, True), ("bf16", 136, 8, True, True, False),
    ("bf16", 8, 0, True, False, True), ("f32", 16, 8, False, True, False),
    ("bf16", 264, 24, False, False, True)])
@pytest.mark.parametrize("lay", LAYOUTS + LONG, ids=name_of)
def test_recurrence(lay, io, C, pad, decay, gated, init):
    run_recurrence(lay, io, C, pad, decay, gated, init)


# around the backward's blocks: four waves of 7 (fp32 12) rows, sixteen, several sequences in one; and the
# forward's: sixteen waves of 16 rows
@pytest.mark.parametrize("io,lay", [
    ("bf16", dict(batch=1, L=28)), ("bf16", dict(batch=1, L=29)), ("bf16", dict(batch=7, L=29)),
    ("bf16", dict(batch=3, L=112)), ("bf16", dict(batch=1, L=113)), ("f32", dict(batch=1, L=48)),
    ("f32", dict(batch=5, L=49)), ("f32", dict(batch=1, L=192)), ("f32", dict(batch=2, L=193)),
    ("bf16", dict(lens=[40, 0, 1, 60], spare=11)), ("bf16", dict(lens=[40, 0, 1, 60], spare=12)),
    ("f32", dict(lens=[0, 99, 93], spare=0)), ("f32", dict(lens=[0, 99, 94], spare=0)),
    ("bf16", dict(batch=3, L=256)), ("f32", dict(batch=2, L=257)),
    ("bf16", dict(lens=[100, 0, 150], spare=6)), ("f32", dict(lens=[100, 0, 150], spare=7))],
    ids=lambda v: v if isinstance(v, str) else name_of(v))
@pytest.mark.parametrize("decay,gated", [(True, True), (False, False)])
def test_recurrence_of_one_block(io, lay, decay, gated):
    run_recurrence(lay, io, 136, 8, decay, gated, True)


@pytest.mark.parametrize("io,decay,lay", [
    ("f32", True, dict(batch=1, L=5000)), ("bf16", False, dict(batch=2, L=3000)),
    ("f32", True, dict(lens=[1700, 0, 1, 2650, 300], spare=33))])
def test_recurrence_long(io, decay, lay):
    run_recurrence(lay, io, 24, 0, decay, True, True)


@pytest.mark.parametrize("io,decay,gated", [("f32", True, True), ("bf16", False, False),
                                            ("bf16", True, False), ("f32", False, True)])
def test_recurrence_steps_continue_a_prompt(io, decay, gated):
    rng = np.random.default_rng(62)
    Bt, L, C, cut = 3, 29, 40, 17
    note(f"recurrence_step {io} decay{decay}")
    t, v = recurrence_inputs(rng, (Bt, L), Bt, C, io, 8, decay, gated, True)
    seqs, _ = ranges(batch=Bt, L=L)
    want = recurrent.recurrence(*(v[k] for k in IN), seqs, v["init"])
    y64, e64 = (a.reshape(Bt, L, C) for a in want["y"])
    head = [t[k] if k == "decay" or t[k] is None else t[k][:, :cut].contiguous() for k in IN]
    _, state = ssd.recurrence(*head, t["init"])
    for i in range(cut, L):
        one = [t[k] if k == "decay" or t[k] is None else t[k][:, i] for k in IN]
        before = state.clone()
        y2, s2 = ssd.recurrence_step(state, *one)
        assert torch.equal(state, before)
        y, s = ssd.recurrence_step(state, *one, out_state=state)
        assert s.data_ptr() == state.data_ptr() and torch.equal(s, s2) and torch.equal(y, y2)
        check(y, (y64[:, i], e64[:, i]), i)
    check(state, want["final"], "state")


def test_recurrence_extremes():
    """Gates that are shut and wide open, a decay parameter whose softplus is zero in fp32 or the
    parameter itself, other sharpnesses; gradients stay finite."""
    rng = np.random.default_rng(63)
    L, C = 150, 64
    note("recurrence extremes")
    for sharp in (8.0, 0.25, 200.0):
        t, v = recurrence_inputs(rng, (1, L), 1, C, "f32", 0, True, True, True)
        t["gate"], t["input_gate"] = t["gate"].clone(), t["input_gate"].clone()
        for k, rows in (("gate", (3, 4, 5, 6, 140)), ("input_gate", (7, 8, 9, 10, 141))):
            for r, x in zip(rows, (-200.0, 200.0, -40.0, 30.0, -87.0)):
                t[k][0, r] = x
        t["decay"][:4] = torch.tensor([-200.0, 25.0, -100.0, 3.0])
        for k in IN:
            v[k] = t[k].double().cpu().numpy().reshape(-1, C) if k != "decay" else \
                t[k].double().cpu().numpy()
        seqs = [(0, L)]
        dy, dyv = value(rng, (1, L, C))
        y, f = ssd.recurrence(*(t[k] for k in IN), t["init"], sharpness=sharp)
        g = ssd.recurrence_backward(*(t[k] for k in IN), dy, t["init"], sharpness=sharp)
        for k in g:
            assert torch.isfinite(g[k]).all(), k
        args = [v[k] for k in IN]
        with np.errstate(all="ignore"):
            want = recurrent.recurrence(*args, seqs, v["init"], sharp)
            wg = recurrent.recurrence_backward(*args, dyv[0], seqs, v["init"], sharpness=sharp)
        check(y[0], want["y"], "y")
        check(f, want["final"], "final")
        # where 1 / m overflows in the oracle there is nothing to compare with; fp32 underflows there
        for k in ("dx", "dgate", "dinput_gate", "dinitial_state"):
            m = np.isfinite(wg[k][0]) & np.isfinite(wg[k][1])
            assert m.mean() > 0.9, k
            check(g[k].reshape(wg[k][0].shape)[torch.from_numpy(m).to(DEV)], pick(wg[k], m), k)
        m = np.isfinite(wg["ddecay"][0]) & np.isfinite(wg["ddecay"][1])
        assert m.sum() >= C - 2
        check(g["ddecay"][torch.from_numpy(m).to(DEV)], pick(wg["ddecay"], m), "ddecay")


def test_recurrence_infinite_decays():
    """An infinite decay parameter forgets all and takes the input whole, one of minus infinity keeps all
    and takes nothing; gates at both infinities; NaN stays NaN; gradients are finite but for NaN's."""
    note("recurrence infinite decays")
    inf, L, C = float("inf"), 40, 64
    g = torch.Generator(DEV).manual_seed(68)
    x, gate, dy = (torch.randn(1, L, C, device=DEV, generator=g) for _ in range(3))
    decay = torch.zeros(C, device=DEV)
    decay[0], decay[1], decay[2] = inf, -inf, float("nan")
    gate[0, :, 3], gate[0, :, 4] = inf, -inf
    h0 = torch.randn(1, C, device=DEV, generator=g)
    y, f = ssd.recurrence(x, gate, decay, None, h0)
    assert torch.equal(y[0, :, 0], x[0, :, 0]) and torch.equal(f[0, 0], x[0, -1, 0])
    assert torch.all(y[0, :, 1] == h0[0, 1]) and torch.all(y[0, :, 4] == h0[0, 4])
    a = 2.0 ** -8  # softplus(0) = log 2, the gate wide open
    want, w64 = torch.empty(L, dtype=torch.float64), h0[0, 3].double().cpu()
    for t in range(L):
        w64 = a * w64 + (1 - a * a) ** 0.5 * x[0, t, 3].double().cpu()
        want[t] = w64
    assert torch.all((y[0, :, 3].double().cpu() - want).abs() <= 2.0 ** -24 * 64 * want.abs().max())
    assert torch.isnan(y[0, :, 2]).all() and torch.isnan(y).sum() == L
    grads = ssd.recurrence_backward(x, gate, decay, None, dy, h0)
    for k in ("dx", "dgate", "ddecay", "dinitial_state"):
        v = grads[k].reshape(-1, C)
        assert torch.isnan(v[:, 2]).all() and torch.isnan(v).sum() == v.shape[0], k


def test_recurrence_nan_and_infinity_stay_in_their_channel():
    rng = np.random.default_rng(64)
    L, C = 400, 64
    note("recurrence NaN")
    t, _ = recurrence_inputs(rng, (1, L), 1, C, "f32", 0, True, True, True)
    y, f = ssd.recurrence(*(t[k] for k in IN), t["init"])
    for bad in (float("nan"), float("inf")):
        t["x"] = t["x"].clone()
        t["x"][0, 40, 9] = bad
        y2, f2 = ssd.recurrence(*(t[k] for k in IN), t["init"])
        assert not torch.isfinite(y2[0, 40:, 9]).any() and not torch.isfinite(f2[0, 9]).any()
        keep = torch.ones(L, C, dtype=torch.bool, device=DEV)
        keep[40:, 9] = False
        assert torch.equal(y2[0][keep], y[0][keep])


FILLS = (0.0, float("nan"), float("inf"), -float("inf"))


@pytest.mark.parametrize("io,decay", [("f32", True), ("bf16", False)])
@pytest.mark.parametrize("first,lens,spare", [
    (0, [10], 54), (0, [64], 64), (20, [44], 0), (70, [30, 100, 0, 90], 100),
    (130, [5, 0, 64, 1, 130], 147), (130, [0], 9), (0, [128, 128], 200)])
def test_rows_outside_sequences_have_no_part(first, lens, spare, io, decay):
    """Whatever rows of no sequence hold: the same bits in every output, what was there before in
    forward outputs, zero in gradients."""
    rng = np.random.default_rng(65)
    C, G = 64, 4
    at = first + np.concatenate([[0], np.cumsum(lens)])
    rows, S = int(at[-1]) + spare, len(lens)
    cu = torch.tensor(at, dtype=torch.int32, device=DEV)
    m = torch.zeros(rows, dtype=torch.bool, device=DEV)
    m[int(at[0]):int(at[-1])] = True
    note(f"rows outside {first}+{lens}+{spare} {io}")
    t, _ = recurrence_inputs(rng, (1, rows), S, C, io, 8, decay, True, True)
    dy, _ = value(rng, (1, rows, C), io)
    df, _ = value(rng, (S, C))
    w, _ = value(rng, (C,))
    stats = torch.rand(S, G, 2, device=DEV)
    clean = None
    for fill in FILLS:
        for k in ("x", "gate", "input_gate"):
            t[k][:, ~m] = fill
        dy[:, ~m] = fill
        out = [torch.full((1, rows, C), FILL, dtype=TORCH[io], device=DEV) for _ in range(2)]
        y, f = ssd.recurrence(*(t[k] for k in IN), t["init"], cu_seqlens=cu, out=out[0])
        n, st = ssd.group_norm(t["x"], w, w, ngroups=G, cu_seqlens=cu, out=out[1])
        g = ssd.recurrence_backward(*(t[k] for k in IN), dy, t["init"], df, cu_seqlens=cu)
        h = ssd.group_norm_backward(t["x"], w, w, stats, dy, ngroups=G, cu_seqlens=cu)
        got = dict(g, y=y, f=f, n=n, st=st, **{"gn_" + k: v for k, v in h.items()})
        clean = clean or {k: v.clone() for k, v in got.items() if v is not None}
        for k, v in clean.items():
            assert torch.equal(got[k], v), (k, fill)
        assert all(torch.all(o[0, ~m] == FILL) for o in out)
        for k in ("dx", "dgate", "dinput_gate", "gn_dx"):
            assert torch.all(got[k][0, ~m] == 0), k


@pytest.mark.parametrize("lens", [(70, 90, 60), (128, 128, 128), (3, 1, 2), (130, 640, 700)])
def test_a_sequence_of_nan_stays_alone(lens):
    """NaN in every input of the middle sequence: the others' results are those of a call without it,
    bit for bit."""
    rng = np.random.default_rng(66)
    L, C, G = sum(lens), 72, 3
    note(f"a sequence of NaN, {lens}")
    _, cu = ranges(lens=lens)
    mid = slice(lens[0], lens[0] + lens[1])
    for decay in (True, False):
        t, _ = recurrence_inputs(rng, (1, L), 3, C, "f32", 0, decay, True, True)
        dy, _ = value(rng, (1, L, C))
        df, _ = value(rng, (3, C))

        def calls():
            y, f = ssd.recurrence(*(t[k] for k in IN), t["init"], cu_seqlens=cu)
            g = ssd.recurrence_backward(*(t[k] for k in IN), dy, t["init"], df, cu_seqlens=cu)
            n, st = ssd.group_norm(t["x"], ngroups=G, cu_seqlens=cu)
            h = ssd.group_norm_backward(t["x"], None, None, st, dy, ngroups=G, cu_seqlens=cu)
            return ([y, n, h["dx"]] + [g[k] for k in ("dx", "dgate", "dinput_gate")],
                    [f, g["dinitial_state"], st])

        rows, states = calls()
        for k in ("x", "gate", "input_gate"):
            t[k] = t[k].clone()
            t[k][:, mid] = float("nan")
        dy[:, mid] = float("nan")
        for v in (t["init"], df):
            v[1] = float("nan")
        rows2, states2 = calls()
        for a, b in zip(rows, rows2):
            assert torch.equal(a[:, :mid.start], b[:, :mid.start])
            assert torch.equal(a[:, mid.stop:], b[:, mid.stop:])
            assert torch.isnan(b[:, mid]).all()
        for a, b in zip(states, states2):
            assert torch.equal(a[::2], b[::2])


# ---- rotation --------------------------------------------------------------------------------------

@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("io,lead,G,N,nf,sections,pad,far", [
    ("bf16", (2, 33), 1, 128, 64, (64,), 0, 10 ** 6), ("bf16", (3,), 2, 48, 20, (4, 9, 7), 8, 9),
    ("f32", (1, 70), 5, 16, 8, (0, 8), 24, 2 ** 31 - 1), ("f32", (2, 3), 9, 24, 4, (1, 1, 1, 1), 0, 500),
    ("bf16", (1, 1), 8, 256, 64, (16, 24, 24), 0, 20000), ("f32", (130,), 1, 8, 4, (4,), 8, 3000),
    ("bf16", (5,), 4, 16, 8, (3, 5), 0, 10 ** 6)])
def test_rotate(io, lead, G, N, nf, sections, pad, far, interleaved, inverse):
    rng = np.random.default_rng(71)
    note(f"rotate {io} {lead} G{G} N{N} nf{nf} {sections}")
    rows = int(np.prod(lead))
    t, v = {}, {}
    for k in "BC":
        t[k], v[k] = sliced(rng, lead, G * N, io, pad)
        t[k], v[k] = t[k].unflatten(-1, (G, N)), v[k].reshape(rows, G, N)
    pos = torch.from_numpy(rng.integers(-far, far, (len(sections), *lead)).astype(np.int32))
    freq = torch.from_numpy((10000.0 ** -(np.arange(nf) / nf)).astype(np.float32))
    call = ssd.rotate_backward if inverse else ssd.rotate
    kw = dict(sections=sections, interleaved=interleaved)
    args = pos.to(DEV), freq.to(DEV)
    got = call(t["B"], t["C"], *args, **kw)
    for g, k in zip(got, "BC"):
        assert g.shape == t[k].shape and g.dtype == t[k].dtype and g.is_contiguous()
        check(g, recurrent.rotate(v[k], pos.reshape(len(sections), rows).numpy(), freq.numpy(),
                                  sections, interleaved, inverse), k)
        assert torch.equal(g[..., 2 * nf:], t[k][..., 2 * nf:])
    alone, none = call(t["B"], None, *args, **kw)
    assert none is None and torch.equal(alone, got[0])
    out = torch.empty_like(got[0]), torch.empty_like(got[1])
    given = call(t["B"], t["C"], *args, out=out, **kw)
    assert all(a is b and torch.equal(a, c) for a, b, c in zip(given, out, got))


def test_rotate_position_zero_and_nan():
    """Position zero changes nothing; a NaN stays in its pair."""
    note("rotate zero, NaN")
    B = torch.randn(1, 4, 2, 16, device=DEV)
    freq = torch.rand(8, device=DEV)
    pos = torch.zeros(1, 1, 4, dtype=torch.int32, device=DEV)
    got, _ = ssd.rotate(B, None, pos, freq)
    assert torch.equal(got, B)
    pos += 7
    want, _ = ssd.rotate(B, None, pos, freq)
    B[0, 2, 1, 3] = float("nan")
    got, _ = ssd.rotate(B, None, pos, freq)
    bad = torch.zeros_like(B, dtype=torch.bool)
    bad[0, 2, 1, 3] = bad[0, 2, 1, 11] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])


def test_rotated_scan_has_decays_with_a_phase():
    """forward over rotated B and C against the recurrence with complex decays exp(dt A + i angle
    difference) that it stands for, and step from its final state; the gradients of B and C through both
    against differences. fp32 bar of the scan: 1e-4 of the largest value."""
    rng = np.random.default_rng(72)
    Bt, L, H, P, N, nf = 1, 70, 2, 16, 16, 8
    note("rotated scan")
    x, xv = value(rng, (Bt, L, H, P))
    B, Bv = value(rng, (Bt, L, 1, N))
    C, Cv = value(rng, (Bt, L, 1, N))
    dt = torch.from_numpy(rng.uniform(0.01, 0.2, (Bt, L, H)).astype(np.float32)).to(DEV)
    A = torch.tensor([-1.0, -0.3], device=DEV)
    D = torch.zeros(H, device=DEV)
    pos = torch.from_numpy(rng.integers(0, 9, (2, Bt, L)).cumsum(-1).astype(np.int32)).to(DEV)
    freq = torch.from_numpy(rng.uniform(0.01, 1, nf).astype(np.float32)).to(DEV)
    kw = dict(sections=(5, 3))
    Br, Cr = ssd.rotate(B, C, pos, freq, **kw)
    y, h = ssd.forward(x, dt, A, Br, Cr, D, 64)

    axis = np.repeat([0, 1], (5, 3))
    angle = pos.cpu().numpy()[axis, 0].T * freq.double().cpu().numpy()  # [L, nf]
    dtv, Av = dt.double().cpu().numpy()[0], A.double().cpu().numpy()

    def scan(Bv, Cv):
        b, c = (m[0, :, 0, :nf] + 1j * m[0, :, 0, nf:] for m in (Bv, Cv))
        s, out = np.zeros((H, P, nf), complex), np.zeros((L, H, P))
        for t in range(L):
            turn = np.exp(1j * (angle[t - 1] - angle[t])) if t else np.ones(nf)
            s = np.exp(dtv[t] * Av)[:, None, None] * turn * s + \
                (dtv[t][:, None] * xv[0, t])[..., None] * b[t]
            out[t] = (s * c[t].conj()).sum(-1).real
        return out

    want = scan(Bv, Cv)
    bar = 1e-4 * np.abs(want).max()
    assert np.abs(y[0].double().cpu().numpy() - want).max() <= bar
    # the last token again, as a step from the state before it
    _, h = ssd.forward(*(v[:, :-1].contiguous() if v.dim() > 1 else v for v in (x, dt, A, Br, Cr, D)), 64)
    b1, c1 = ssd.rotate(B[:, -1], C[:, -1], pos[:, :, -1].contiguous(), freq, **kw)
    assert torch.equal(b1, Br[:, -1]) and torch.equal(c1, Cr[:, -1])
    y1, _ = ssd.step(h, x[:, -1].contiguous(), dt[:, -1].clone(), A, b1, c1, D)
    assert np.abs(y1[0].double().cpu().numpy() - want[-1]).max() <= bar

    dy, dyv = value(rng, (Bt, L, H, P))
    g = ssd.backward(x, dt, A, Br, Cr, D, dy, 64)
    dB, dC = ssd.rotate_backward(g["dB"], g["dC"], pos, freq, **kw)
    for got, k in ((dB, 0), (dC, 1)):
        got = got.double().cpu().numpy()
        for _ in range(6):
            at = (0, int(rng.integers(L)), 0, int(rng.integers(N)))
            two = []
            for step in (1e-5, -1e-5):
                bc = [Bv.copy(), Cv.copy()]
                bc[k][at] += step
                two.append((scan(*bc) * dyv[0]).sum())
            assert abs((two[0] - two[1]) / 2e-5 - got[at]) <= 1e-4 * np.abs(got).max()


# ---- group norm ------------------------------------------------------------------------------------

def run_group_norm(lay, io, C, G, pad, act, affine, shift=0.0, eps=1e-5):
    rng = np.random.default_rng(81)
    lead, seqs, cu = layout(lay)
    S, rows = len(seqs), lead[0] * lead[1]
    note(f"group_norm {name_of(lay)} {io} C{C} G{G}")
    x, _ = sliced(rng, lead, C, io, pad)
    x += shift
    xv = x.double().cpu().numpy().reshape(rows, C)
    w, wv = value(rng, (C,)) if affine != "bias" else (None, None)
    b, bv = value(rng, (C,)) if affine else (None, None)
    if affine is None:
        w, wv = None, None
    m = inside(seqs, rows)
    mt = torch.from_numpy(m).to(DEV)
    out = torch.full((*lead, C), FILL, dtype=TORCH[io], device=DEV)
    kw = dict(ngroups=G, activation="silu" if act else None, cu_seqlens=cu)
    y, st = ssd.group_norm(x, w, b, eps=eps, out=out, **kw)
    want, bound, stats, kst = recurrent.group_norm(xv, wv, bv, seqs, G, eps, act)
    check(y.reshape(rows, C)[mt], (want[m], bound[m]), "y")
    assert torch.all(y.reshape(rows, C)[~mt] == FILL)
    check(st, (stats, kst), "stats")
    y2, none = ssd.group_norm(x, w, b, eps=eps, want_stats=False, **kw)
    assert none is None and torch.equal(y2.reshape(rows, C)[mt], y.reshape(rows, C)[mt])

    dy, dyv = value(rng, (*lead, C), io)
    dyv = dyv.reshape(rows, C) * m[:, None]
    given = torch.from_numpy(stats.astype(np.float32)).to(DEV)
    g = ssd.group_norm_backward(x, w, b, given, dy, **kw)
    wg = recurrent.group_norm_backward(xv, wv, bv, given.double().cpu().numpy(), dyv, seqs, G, act)
    check(g["dx"].reshape(rows, C)[mt], pick(wg["dx"], m), "dx")
    assert torch.all(g["dx"].reshape(rows, C)[~mt] == 0)
    for k, p in (("dweight", w), ("dbias", b)):
        assert (g[k] is None) == (p is None)
        if p is not None:
            check(g[k], wg[k], k)


@pytest.mark.parametrize("io,C,G,pad,act,affine", [
    ("f32", 64, 8, 0, True, "both"), ("bf16", 40, 4, 8, True, "both"), ("bf16", 2080, 1, 0, False, None),
    ("f32", 24, 24, 8, False, "bias"), ("bf16", 5120, 80, 0, True, "both"), ("f32", 600, 3, 0, True, "both")])
@pytest.mark.parametrize("lay", LAYOUTS + [LONG[0], LONG[3], LONG[5], dict(batch=70, L=1)], ids=name_of)
def test_group_norm(lay, io, C, G, pad, act, affine):
    run_group_norm(lay, io, C, G, pad, act, affine)


# groups of fewer vectors than lanes, of a wave and one vector more, of several waves, of the widest block
# and one vector more, for one token and for several; more tokens than one round of threads takes
@pytest.mark.parametrize("io,C,G", [("bf16", 72, 3), ("f32", 40, 1), ("bf16", 512, 1), ("f32", 1040, 2),
                                    ("bf16", 4104, 3), ("f32", 4096, 1), ("bf16", 4104, 1),
                                    ("f32", 8192, 1), ("bf16", 8200, 1)])
@pytest.mark.parametrize("lay", [dict(batch=3, L=1), dict(batch=7, L=5), dict(batch=2, L=8),
                                 dict(batch=2, L=9)], ids=name_of)
def test_group_norm_of_a_few_tokens(lay, io, C, G):
    run_group_norm(lay, io, C, G, 8, True, "both")


@pytest.mark.parametrize("tokens,C,G", [(1031, 8192, 8), (2051, 4096, 1), (9001, 1000, 25), (33001, 24, 3)])
def test_group_norm_of_many_single_tokens(tokens, C, G):
    run_group_norm(dict(batch=tokens, L=1), "bf16", C, G, 0, False, "both")


@pytest.mark.parametrize("lay", [dict(batch=5, L=2), dict(batch=2, L=200), dict(lens=[90, 3, 40], spare=5)],
                         ids=name_of)
def test_group_norm_of_values_far_from_zero(lay):
    """A mean of 1000 standard deviations: the variance is taken about values of the data."""
    run_group_norm(lay, "f32", 96, 6, 0, False, "both", shift=1000.0)


@pytest.mark.parametrize("lay", [dict(batch=5, L=2), dict(batch=2, L=200)], ids=name_of)
def test_group_norm_of_equal_values(lay):
    """No variance: the bias alone, and finite gradients."""
    note("group_norm of equal values")
    x = torch.full((lay["batch"], lay["L"], 64), 3.25, device=DEV)
    b = torch.randn(64, device=DEV)
    y, st = ssd.group_norm(x, b, b, ngroups=8, eps=1e-5, activation=None)
    assert torch.equal(y, b.expand_as(y))
    assert torch.all(st[..., 0] == 3.25)
    assert torch.allclose(st[..., 1], torch.tensor(1e-5 ** -0.5, device=DEV), rtol=1e-6)
    g = ssd.group_norm_backward(x, b, b, st, torch.randn_like(x), ngroups=8)
    assert all(torch.isfinite(v).all() for v in g.values())


# ---- calls -----------------------------------------------------------------------------------------

def every_call(seed, io="bf16", L=600, C=64):
    rng = np.random.default_rng(seed)
    t, _ = recurrence_inputs(rng, (1, L), 1, C, io, 0, True, True, True)
    dy, _ = value(rng, (1, L, C), io)
    w, _ = value(rng, (C,))
    bc = [value(rng, (1, L, 2, 32), io)[0] for _ in range(2)]
    pos = torch.arange(L, dtype=torch.int32, device=DEV).view(1, 1, L)
    freq = torch.rand(16, device=DEV, generator=torch.Generator(DEV).manual_seed(seed))
    stats = torch.rand(1, 8, 2, device=DEV, generator=torch.Generator(DEV).manual_seed(seed))
    one = [t[k] if k == "decay" else t[k][:, 0].contiguous() for k in IN]
    heads = t["x"].contiguous().view(L, 1, C)
    hstats = stats.expand(L, 8, 2).contiguous()
    return {
        "recurrence": lambda: ssd.recurrence(*(t[k] for k in IN), t["init"]),
        "recurrence_step": lambda: ssd.recurrence_step(t["init"], *one),
        "recurrence_backward": lambda: ssd.recurrence_backward(*(t[k] for k in IN), dy, t["init"]),
        "rotate": lambda: ssd.rotate(*bc, pos, freq),
        "rotate_backward": lambda: ssd.rotate_backward(*bc, pos, freq, interleaved=True),
        "group_norm": lambda: ssd.group_norm(t["x"], w, w, ngroups=8),
        "group_norm_backward": lambda: ssd.group_norm_backward(t["x"], w, w, stats, dy, ngroups=8),
        "group_norm_heads": lambda: ssd.group_norm(heads, w, w, ngroups=8),
        "group_norm_heads_backward": lambda: ssd.group_norm_backward(
            heads, w, w, hstats, dy.view(L, 1, C), ngroups=8),
    }


CALLS = list(["recurrence", "recurrence_step", "recurrence_backward", "rotate", "rotate_backward",
              "group_norm", "group_norm_backward", "group_norm_heads", "group_norm_heads_backward"])


@pytest.mark.parametrize("name", CALLS)
def test_repeats_streams_and_graphs(name):
    note(f"{name}: repeats, streams, graphs")
    call = every_call(91)[name]
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
    calls = [every_call(s, L=1500) for s in (92, 93)]
    want = [[t.clone() for n in CALLS for t in tensors(c[n]())] for c in calls]
    torch.cuda.synchronize()
    graphs, held = [], []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append([t for n in CALLS for t in tensors(c[n]())])
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
    note("bad offsets")
    rng = np.random.default_rng(94)
    t, _ = recurrence_inputs(rng, (1, 150), 3, 64, "f32", 0, True, True, True)
    stats = torch.rand(3, 8, 2, device=DEV)
    for bad in ([0, 20, 40, 10 ** 9], [-5, 20, 130, 150], [0, 140, 10, 150], [160, 170, 180, 190],
                [0, 150, 0, 150], [-9, -8, -7, -6]):
        cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
        ssd.recurrence(*(t[k] for k in IN), t["init"], cu_seqlens=cu)
        ssd.recurrence_backward(*(t[k] for k in IN), t["x"].contiguous(), t["init"], cu_seqlens=cu)
        ssd.group_norm(t["x"], ngroups=8, cu_seqlens=cu)
        ssd.group_norm_backward(t["x"], None, None, stats, t["x"].contiguous(), ngroups=8, cu_seqlens=cu)
        torch.cuda.synchronize()


def test_refusals_write_nothing():
    note("refusals")
    x = torch.zeros(1, 8, 64, device=DEV)
    w = torch.zeros(64, device=DEV)
    out = torch.full_like(x, FILL)
    wide = torch.zeros(1, 8, 100, device=DEV)
    bc = torch.zeros(1, 8, 4, 16, device=DEV)
    pos, f = torch.zeros(1, 1, 8, dtype=torch.int32, device=DEV), torch.zeros(8, device=DEV)
    two = out.view(1, 8, 4, 16), torch.full_like(bc, FILL)
    for bad in (lambda: ssd.recurrence(x, x, out=x),
                lambda: ssd.recurrence(wide[..., 2:66], x, out=out),
                lambda: ssd.recurrence(x, wide[..., 4:68], out=out),
                lambda: ssd.recurrence(x, x, w, sharpness=0.0, out=out),
                lambda: ssd.rotate(bc, bc, pos, f, out=(two[0], two[0])),
                lambda: ssd.rotate(bc, bc, pos, f, out=(two[0], bc)),
                lambda: ssd.rotate(bc, bc, pos, f[:6].contiguous(), out=two),
                lambda: ssd.group_norm(x, w, ngroups=5, out=out),
                lambda: ssd.group_norm(x, w, ngroups=0, out=out),
                lambda: ssd.group_norm(x, w, ngroups=8, eps=-1.0, out=out),
                lambda: ssd.group_norm(x, w, ngroups=8, out=x)):
        with pytest.raises(ssd.SSDError):
            bad()
    torch.cuda.synchronize()
    assert torch.all(out == FILL) and torch.all(two[1] == FILL)


def test_offsets_beyond_32_bits():
    """Tensors of more than 2^31 elements: the last sequences are what they are alone, bit for bit; the
    group norm's strips may be cut differently there, so its outputs, sums in another order rounded to
    bf16, are held to one step of that type, twice the half step each may be off."""
    note("offsets beyond 32 bits")
    S, L, C = 2701, 100, 8192
    assert S * L * C > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(95)

    def act():
        return torch.empty(S, L, C, dtype=torch.bfloat16, device=DEV).normal_(generator=g)

    def last(t):
        return t[-1:].contiguous()

    x, gate, dy = act(), act(), act()
    w = torch.randn(C, device=DEV, generator=g)
    stats = torch.rand(S, 64, 2, device=DEV, generator=g)
    freq = torch.rand(64, device=DEV, generator=g)
    pos = torch.randint(0, 1000, (1, S, L), device=DEV, generator=g).to(torch.int32)

    def heads(t):
        return t.view(t.shape[0] * L, 1, C)

    pairs = [
        lambda x, gate, dy: ssd.recurrence(x, gate, w, gate, want_final=False)[0],
        lambda x, gate, dy: ssd.recurrence_backward(x, gate, w, gate, dy)["dgate"],
        lambda x, gate, dy: ssd.group_norm(x, w, w, ngroups=64)[0],
        lambda x, gate, dy: ssd.group_norm_backward(x, w, w, stats[-x.shape[0]:], dy,
                                                    ngroups=64)["dx"],
        lambda x, gate, dy: ssd.group_norm(heads(x), w, w, ngroups=64)[0].view(x.shape),
        lambda x, gate, dy: ssd.rotate(x.view(-1, L, 64, 128), dy.view(-1, L, 64, 128),
                                       pos[:, -x.shape[0]:], freq)[1].view(x.shape),
    ]
    for i, call in enumerate(pairs):
        got = last(call(x, gate, dy))
        want = call(last(x), last(gate), last(dy))
        if i in (2, 3):
            step = torch.finfo(torch.bfloat16).eps * want.float().abs() + 2.0 ** -20
            assert torch.all((got.float() - want.float()).abs() <= step), i
        else:
            assert torch.equal(got, want), i
        del got, want
    del x, gate, dy
    torch.cuda.empty_cache()


def test_many_empty_sequences():
    """A million packed sequences, all but three empty: states pass through, the rest is what the three
    give alone; the group norm's rows are divided otherwise there, so its sums of some hundred values are
    in another order: to 2^-17 of the largest value, some tens of fp32 roundings."""
    note("many empty sequences")
    S, C, rows = 1_000_003, 64, 300
    ends = [100, 250, 300]
    cu = torch.zeros(S + 1, dtype=torch.int32, device=DEV)
    at = [17, 500_000, S - 1]  # the sequences that have rows
    for s, e in zip(at, ends):
        cu[s + 1:] = e
    few = torch.tensor([0, *ends], dtype=torch.int32, device=DEV)
    rng = np.random.default_rng(96)
    t, _ = recurrence_inputs(rng, (1, rows), 3, C, "f32", 0, True, False, True)
    dy, _ = value(rng, (1, rows, C))
    big = torch.randn(S, C, device=DEV)
    big[at] = t["init"]
    ins = [t[k] for k in IN]
    y, f = ssd.recurrence(*ins, big, cu_seqlens=cu)
    y2, f2 = ssd.recurrence(*ins, t["init"], cu_seqlens=few)
    g = ssd.recurrence_backward(*ins, dy, big, big, cu_seqlens=cu)
    g2 = ssd.recurrence_backward(*ins, dy, t["init"], t["init"], cu_seqlens=few)
    keep = torch.ones(S, dtype=torch.bool, device=DEV)
    keep[at] = False
    assert torch.equal(y, y2) and torch.equal(f[at], f2) and torch.equal(f[keep], big[keep])
    assert torch.equal(g["dinitial_state"][at], g2["dinitial_state"])
    assert torch.equal(g["dinitial_state"][keep], big[keep])
    assert all(torch.equal(g[k], g2[k]) for k in ("dx", "dgate", "ddecay"))
    n, st = ssd.group_norm(t["x"], ngroups=8, cu_seqlens=cu)
    n2, st2 = ssd.group_norm(t["x"], ngroups=8, cu_seqlens=few)
    for a, b in ((n, n2), (st[at], st2)):
        assert (a - b).abs().max() <= 2.0 ** -17 * b.abs().max()


# ---- together --------------------------------------------------------------------------------------

def test_a_layer_runs_together():
    """A layer of gated recurrence over packed prompts: convolution, recurrence, group norm, and their
    gradients back through it, against the oracles one after another; then a token of decoding. fp32,
    to 1e-4 of each result's largest value (sums of some hundred terms, three operators deep)."""
    rng = np.random.default_rng(97)
    C, G, lens = 64, 4, [150, 0, 61, 300]
    lead, seqs, cu = layout(dict(lens=lens, spare=0))
    rows, S = lead[1], len(lens)
    note("a layer together")

    def near(got, want):
        want = np.asarray(want)
        err = np.abs(got.double().cpu().numpy().reshape(want.shape) - want)
        assert err.max() <= 1e-4 * np.abs(want).max()

    proj, pv = value(rng, (1, rows, 3 * C))
    w, wv = value(rng, (C, 4), scale=0.5)
    decay = torch.from_numpy(rng.uniform(-8, -3, C).astype(np.float32)).to(DEV)
    lam = decay.double().cpu().numpy()
    nw, nwv = value(rng, (C,))
    xin, gate, ig = proj.split(C, -1)
    xv, gv, iv = (pv[0, :, i * C:(i + 1) * C] for i in range(3))
    u, cs = ssd.conv(xin, w, None, cu_seqlens=cu)
    h, hs = ssd.recurrence(u, gate, decay, ig, cu_seqlens=cu)
    y, st = ssd.group_norm(h, nw, nw, ngroups=G, cu_seqlens=cu)
    uv, _ = block.conv(xv, wv, None, seqs)
    hv = recurrent.recurrence(uv, gv, lam, iv, seqs)["y"][0]
    yv, _, stv, _ = recurrent.group_norm(hv, nwv, nwv, seqs, G, 1e-5, True)
    near(u, uv)
    near(h, hv)
    near(y, yv)
    dy, dyv = value(rng, (1, rows, C))
    gn = ssd.group_norm_backward(h, nw, nw, st, dy, ngroups=G, cu_seqlens=cu)
    gr = ssd.recurrence_backward(u, gate, decay, ig, gn["dx"], cu_seqlens=cu)
    gc = ssd.conv_backward(xin, w, None, gr["dx"], cu_seqlens=cu)
    wn = recurrent.group_norm_backward(hv, nwv, nwv, stv, dyv[0], seqs, G, True)
    wr = recurrent.recurrence_backward(uv, gv, lam, iv, wn["dx"][0], seqs)
    wc = block.conv_backward(xv, wv, None, wr["dx"][0], seqs)
    for k in ("dx", "dweight", "dbias"):
        near(gn[k], wn[k][0])
    for k in ("dx", "dgate", "dinput_gate", "ddecay", "dinitial_state"):
        near(gr[k], wr[k][0])
    near(gc["dx"], wc["dx"])
    near(gc["dweight"], wc["dw"])
    # one more token for each sequence, as rows of a batch
    new, newv = value(rng, (S, 3 * C))
    u1, cs = ssd.conv_step(cs, new[:, :C], w, None, out_state=cs)
    h1, hs1 = ssd.recurrence_step(hs, u1, new[:, C:2 * C], decay, new[:, 2 * C:])
    y1, _ = ssd.group_norm(h1.view(S, 1, C), nw, nw, ngroups=G)
    more = [(a + i, b + i + 1) for i, (a, b) in enumerate(seqs)]
    put = np.concatenate([np.concatenate([pv[0, a:b], newv[i:i + 1]]) for i, (a, b) in enumerate(seqs)])
    uv, _ = block.conv(put[:, :C], wv, None, more)
    hv = recurrent.recurrence(uv, put[:, C:2 * C], lam, put[:, 2 * C:], more)["y"][0]
    last = np.array([b - 1 for _, b in more])
    near(h1, hv[last])
    ends = [(i, i + 1) for i in range(S)]
    near(y1, recurrent.group_norm(hv[last], nwv, nwv, ends, G, 1e-5, True)[0])
