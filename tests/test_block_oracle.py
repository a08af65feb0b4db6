"""The float64 oracle of the operators around the scan, on the CPU: its backward formulas against
central differences of its forward, and its forward against hand-worked values.

A central difference with step d has an error of d^2 / 6 times the third derivative (O(1) values:
below 1e-9 at d = 1e-5... 1e-4) and 2^-53 / d times the loss's terms (1e-11 at 1e-5, a sum of a few
hundred terms: 1e-9); 1e-6 of the gradient's largest value is far above both."""

import numpy as np
import pytest

from oracle import block

STEP, TOL = 1e-5, 1e-6


def differences(loss, arrays, names, grads):
    for name in names:
        a, g = arrays[name], grads[name]
        flat, want = a.reshape(-1), g.reshape(-1)
        scale = max(np.abs(want).max(), 1.0)
        rng = np.random.default_rng(0)
        for i in rng.choice(flat.size, size=min(flat.size, 25), replace=False):
            keep = flat[i]
            flat[i] = keep + STEP
            up = loss()
            flat[i] = keep - STEP
            down = loss()
            flat[i] = keep
            got = (up - down) / (2 * STEP)
            assert abs(got - want[i]) <= TOL * scale, (name, i, got, want[i])


SEQS = [(0, 5), (5, 5), (5, 6), (6, 8)]  # an empty one, ones shorter than the window; row 8 in none


@pytest.mark.parametrize("act", [True, False])
def test_conv_gradients(act):
    r = np.random.default_rng(1)
    a = dict(x=r.standard_normal((9, 3)), w=r.standard_normal((3, 4)), b=r.standard_normal(3),
             init=r.standard_normal((4, 3, 3)))
    dy, df = r.standard_normal((9, 3)), r.standard_normal((4, 3, 3))
    dy[8] = 0

    def loss():
        y, f = block.conv(a["x"], a["w"], a["b"], SEQS, a["init"], act)
        return (y * dy)[:8].sum() + (f * df).sum()

    g = block.conv_backward(a["x"], a["w"], a["b"], dy, SEQS, a["init"], df, act)
    differences(loss, a, ("x", "w", "b", "init"),
                dict(x=g["dx"], w=g["dw"], b=g["db"], init=g["dinit"]))


@pytest.mark.parametrize("gate,soft", [(True, True), (False, False)])
def test_selective_gradients(gate, soft):
    r = np.random.default_rng(2)
    n = r.standard_normal
    a = dict(x=n((9, 4)), dt=np.abs(n((9, 4))) * 0.5, A=-np.abs(n((4, 3))), B=n((9, 2, 3)),
             C=n((9, 2, 3)), D=n(4), z=n((9, 4)), h0=n((4, 4, 3)), tb=n(4) * 0.1)
    dy, df = n((9, 4)), n((4, 4, 3))

    def args():
        return (a["x"], a["dt"], a["A"], a["B"], a["C"], a["D"], a["z"] if gate else None)

    def loss():
        f = block.selective(*args(), SEQS, a["h0"], a["tb"], soft)
        return (f["y"] * dy)[:8].sum() + (f["final"] * df).sum()

    g = block.selective_backward(*args(), dy, SEQS, a["h0"], df, a["tb"], soft)
    for k in ("dB", "dC"):
        g[k][8] = 0
    names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", D="dD", h0="dinit", tb="ddt_bias")
    if gate:
        names["z"] = "dz"
    differences(loss, a, names, {k: g[v] for k, v in names.items()})


@pytest.mark.parametrize("before", [False, True])
def test_gated_norm_gradients(before):
    r = np.random.default_rng(3)
    a = dict(x=r.standard_normal((5, 8)), z=r.standard_normal((5, 8)), w=r.standard_normal(8))
    dy = r.standard_normal((5, 8))
    g = block.gated_norm_backward(a["x"], a["z"], a["w"], dy, 2, 1e-5, before)
    differences(lambda: (block.gated_norm(a["x"], a["z"], a["w"], 2, 1e-5, before) * dy).sum(), a,
                ("x", "z", "w"), dict(x=g["dx"], z=g["dz"], w=g["dw"]))


def test_residual_norm_gradients():
    r = np.random.default_rng(4)
    a = dict(x=r.standard_normal((5, 8)), res=r.standard_normal((5, 8)),
             w=r.standard_normal(8), s=r.standard_normal(8))
    dy, dr = r.standard_normal((5, 8)), r.standard_normal((5, 8))

    def loss():
        y, s = block.residual_norm(a["x"], a["res"], a["w"], a["s"])
        return (y * dy).sum() + (s * dr).sum()

    _, total = block.residual_norm(a["x"], a["res"], a["w"], a["s"])
    g = block.residual_norm_backward(a["x"], total, a["w"], dy, dr, a["s"])
    differences(loss, a, ("x", "res", "w", "s"),
                dict(x=g["dx"], res=g["dr"], w=g["dw"], s=g["ds"]))


def test_conv_by_hand():
    # weights 1, 10, 100: y_t = x_{t-2} + 10 x_{t-1} + 100 x_t + 0.5, inputs -1, -2 before
    y, f = block.conv(np.array([[3.0], [4.0]]), np.array([[1.0, 10.0, 100.0]]), np.array([0.5]),
                      [(0, 2)], np.array([[[-1.0], [-2.0]]]), act=False)
    assert y.ravel().tolist() == [-1 - 20 + 300 + 0.5, -2 + 30 + 400 + 0.5]
    assert f.ravel().tolist() == [3.0, 4.0]


def test_selective_by_hand():
    # decay exp(-ln 2) = 1/2 a token: h = 1/2 * 8 + 1 * 3 * 2 = 10, then 5 + 1 * 1 * 2 = 7
    A = np.array([[-np.log(2.0)]])
    one = np.ones((2, 1))
    f = block.selective(np.array([[3.0], [1.0]]), one, A, 2 * np.ones((2, 1, 1)),
                        np.array([[[1.0]], [[10.0]]]), np.array([0.5]), None, [(0, 2)],
                        np.array([[[8.0]]]))
    assert np.allclose(f["h"].ravel(), [10.0, 7.0], rtol=1e-15)
    assert np.allclose(f["y"].ravel(), [10 + 1.5, 70 + 0.5], rtol=1e-15)


def test_selective_equals_the_ssd_recurrence():
    """One decay for every state entry of a head: the scan of the SSD form."""
    from oracle import ssd_recurrence
    r = np.random.default_rng(5)
    H, P, N, L = 2, 3, 4, 6
    x, dt = r.standard_normal((1, L, H, P)), r.uniform(0.1, 0.5, (1, L, H))
    A, D = -r.uniform(1, 4, H), r.standard_normal(H)
    B, C = r.standard_normal((1, L, 1, N)), r.standard_normal((1, L, 1, N))
    y, fin = ssd_recurrence(x, dt, A, B, C, D)
    f = block.selective(x.reshape(L, H * P), np.repeat(dt[0], P, axis=1),
                        np.repeat(A, P)[:, None] * np.ones(N), B[0], C[0], np.repeat(D, P), None,
                        [(0, L)])
    assert np.allclose(f["y"], y.reshape(L, H * P), atol=1e-12)
    assert np.allclose(f["final"].reshape(H, P, N), fin[0], atol=1e-12)
