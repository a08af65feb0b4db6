"""Packed rows outside every sequence (behind the last, in front of the first) on the GPU: whatever
lies there, no output, state or gradient of a sequence depends on it. The rows are filled with NaN or
infinities in every input; results are held to the float64 oracle with the bounds derived in
test_block.py, and bit for bit to those of a call whose outside rows are zero."""

import numpy as np
import pytest
import torch

import mamba_ssd_chunked_cumsum_amd as ssd
from oracle import block

from gpu_util import DEV, note
from test_block import FILL, NAMES, TORCH, check, inside, selective_inputs, value

pytestmark = pytest.mark.gpu

FILLS = (float("nan"), float("inf"), -float("inf"))

# rows before the first sequence, lengths, rows behind the last
GAPS = [(0, [10], 54), (0, [40], 24), (0, [64], 64), (20, [44], 0), (70, [30], 100),
        (33, [5, 0, 64, 1, 130], 47), (0, [1], 15), (130, [0], 9)]


def gap_name(v):
    return f"{v[0]}+{'x'.join(map(str, v[1]))}+{v[2]}"


def packed(gap):
    first, lens, spare = gap
    at = first + np.concatenate([[0], np.cumsum(lens)])
    seqs = [(int(a), int(b)) for a, b in zip(at, at[1:])]
    return int(at[-1]) + spare, seqs, torch.tensor(at, dtype=torch.int32, device=DEV)


def fill_outside(mask, tensors, fill):
    for t in tensors:
        if t is not None:
            t[:, ~mask] = fill


# (the last three: 16 and 8 state entries a lane in the backward's first pass, with chunks that have
# events in the one launch or in one of their own)
@pytest.mark.parametrize("gap,io,Dm,N,G", [
    *((gap, io, Dm, N, G) for gap in GAPS for io, Dm, N, G in (
        ("f32", 72, 16, 1), ("bf16", 40, 64, 1), ("f32", 80, 8, 2), ("bf16", 48, 20, 1),
        ("f32", 16, 4, 2))),
    ((70, [300, 1, 50], 100), "f32", 1024, 64, 128),
    ((33, [700, 300], 567), "f32", 1024, 64, 128),
    ((70, [300, 1, 50], 100), "bf16", 4096, 8, 512)],
    ids=lambda v: gap_name(v) if isinstance(v, tuple) else str(v))
def test_selective_rows_outside_sequences(gap, io, Dm, N, G):
    rng = np.random.default_rng(41)
    rows, seqs, cu = packed(gap)
    S, L = len(seqs), max(b - a for a, b in seqs)
    note(f"selective outside rows {gap_name(gap)} {io} Dm{Dm} N{N} G{G}")
    t, v = selective_inputs(rng, (1, rows), S, Dm, N, G, io, 8, True, True, True, True)
    dy, dyv = value(rng, (1, rows, Dm), io)
    df, dfv = value(rng, (S, Dm, N))
    m = inside(seqs, rows)
    mt = torch.from_numpy(m).to(DEV)
    kw = dict(dt_bias=t["dt_bias"], dt_softplus=True, cu_seqlens=cu)

    def calls():
        out = torch.full((1, rows, Dm), FILL, dtype=TORCH[io], device=DEV)
        y, f = ssd.selective_scan(*(t[k] for k in NAMES), t["h0"], out=out, **kw)
        g = ssd.selective_backward(*(t[k] for k in NAMES), dy, t["h0"], df, **kw)
        return dict(g, y=y, final=f)

    held = [t[k] for k in ("x", "dt", "B", "C", "z")] + [dy]
    fill_outside(mt, held, 0.0)
    clean = calls()
    for fill in FILLS:
        fill_outside(mt, held, fill)
        got = calls()
        for k in got:
            assert torch.equal(got[k], clean[k]), (k, fill)
    assert torch.all(got["y"][0, ~mt] == FILL)
    if Dm > 100:  # (too much for the oracle)
        return
    args = [v[k] for k in NAMES]
    more = (dyv.reshape(rows, Dm) * m[:, None], seqs, v["h0"], dfv, v["dt_bias"], True)
    want = block.selective_backward(*args, *more)
    size = block.selective_backward(*args, *more, absolute=True)
    k = 16 * (L + N + Dm + 16)
    for n in ("dx", "ddt", "dz", "dB", "dC"):
        check(got[n].flatten(0, 1)[mt], want[n][m], size[n][m], k, n)
        assert torch.all(got[n].flatten(0, 1)[~mt] == 0)
    for n in ("dA", "dD", "ddt_bias"):
        check(got[n], want[n], size[n], k + 16 * rows, n)
    check(got["dinitial_state"], want["dinit"], size["dinit"], k, "dinitial_state")


def test_selective_state_that_overflows_at_the_last_token():
    """The state after the last token has no part in dA, infinite or not: the gradients are those of a
    call that ends with the sequence."""
    note("selective state that overflows at a sequence's last token")
    rng = np.random.default_rng(42)
    L, R, Dm, N = 40, 64, 72, 16
    t, _ = selective_inputs(rng, (1, R), 1, Dm, N, 1, "f32", 0, False, True, True, False)
    dy, _ = value(rng, (1, R, Dm))
    t["x"][0, L - 1] = 3e38
    t["dt"][0, L - 1] = 4.0
    cu = torch.tensor([0, L], dtype=torch.int32, device=DEV)
    g = ssd.selective_backward(*(t[k] for k in NAMES), dy, t["h0"], cu_seqlens=cu)
    cut = [t[k] if k in "AD" or t[k] is None else t[k][:, :L] for k in NAMES]
    w = ssd.selective_backward(*cut, dy[:, :L], t["h0"], cu_seqlens=cu)
    assert torch.isfinite(w["dA"]).all()
    assert torch.equal(g["dA"], w["dA"])
    assert torch.equal(g["dinitial_state"], w["dinitial_state"])


@pytest.mark.parametrize("io,W,C", [("f32", 4, 40), ("bf16", 3, 72), ("bf16", 2, 8)])
@pytest.mark.parametrize("gap", GAPS, ids=gap_name)
def test_conv_rows_outside_sequences(gap, io, W, C):
    rng = np.random.default_rng(43)
    rows, seqs, cu = packed(gap)
    S = len(seqs)
    note(f"conv outside rows {gap_name(gap)} {io} W{W} C{C}")
    x, xv = value(rng, (1, rows, C), io)
    dy, dyv = value(rng, (1, rows, C), "f32")
    w, wv = value(rng, (C, W))
    b, bv = value(rng, (C,))
    h, hv = value(rng, (S, W - 1, C), io)
    df, dfv = value(rng, (S, W - 1, C))
    m = inside(seqs, rows)
    mt = torch.from_numpy(m).to(DEV)

    def calls():
        out = torch.full((1, rows, C), FILL, dtype=x.dtype, device=DEV)
        y, f = ssd.conv(x, w, b, h, cu_seqlens=cu, out=out)
        g = ssd.conv_backward(x, w, b, dy, h, df, cu_seqlens=cu)
        return dict(g, y=y, final=f)

    fill_outside(mt, [x, dy], 0.0)
    clean = calls()
    for fill in FILLS:
        fill_outside(mt, [x, dy], fill)
        got = calls()
        for k in got:
            assert torch.equal(got[k], clean[k]), (k, fill)
    assert torch.all(got["y"][0, ~mt] == FILL) and torch.all(got["dx"][0, ~mt] == 0)
    more = (xv.reshape(rows, C), wv, bv, dyv.reshape(rows, C) * m[:, None], seqs, hv, dfv)
    want, size = block.conv_backward(*more), block.conv_backward(*more, absolute=True)
    check(got["dx"][0, mt], want["dx"][m], size["dx"][m], 64, "dx")
    check(got["dweight"], want["dw"], size["dw"], 512, "dweight")
    check(got["dbias"], want["db"], size["db"], 512, "dbias")
    check(got["dinitial_state"], want["dinit"], size["dinit"], 64, "dinitial_state")
