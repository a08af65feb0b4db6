"""The float64 oracle of the operators of layers of linear recurrence, on the CPU: its backward
formulas against central differences of its forward (bounds as in test_block_oracle.py), and its
forward against values worked by hand."""

import numpy as np
import pytest

from oracle import recurrent
from test_block_oracle import SEQS, differences


@pytest.mark.parametrize("decay", [True, False])
@pytest.mark.parametrize("gated", [True, False])
def test_recurrence_gradients(decay, gated):
    r = np.random.default_rng(1)
    n = r.standard_normal
    a = dict(x=n((9, 3)), gate=n((9, 3)), decay=n(3) - 2 if decay else None,
             input_gate=n((9, 3)) if gated else None, init=n((4, 3)))
    dy, df = n((9, 3)), n((4, 3))
    dy[8] = 0

    def args():
        return a["x"], a["gate"], a["decay"], a["input_gate"]

    def loss():
        f = recurrent.recurrence(*args(), SEQS, a["init"])
        return (f["y"][0] * dy)[:8].sum() + (f["final"][0] * df).sum()

    g = recurrent.recurrence_backward(*args(), dy, SEQS, a["init"], df)
    names = ["x", "gate", "init"] + ["decay"] * decay + ["input_gate"] * gated
    grads = {k: g["dinitial_state" if k == "init" else "d" + k][0] for k in names}
    differences(loss, a, names, grads)


@pytest.mark.parametrize("act", [True, False])
@pytest.mark.parametrize("affine", [True, False])
def test_group_norm_gradients(act, affine):
    r = np.random.default_rng(2)
    n = r.standard_normal
    a = dict(x=n((9, 12)) + 0.5, w=n(12) if affine else None, b=n(12) if affine else None)
    dy = n((9, 12))
    dy[8] = 0

    def loss():
        return (recurrent.group_norm(a["x"], a["w"], a["b"], SEQS, 3, 1e-3, act)[0] * dy)[:8].sum()

    stats, _ = recurrent.group_stats(a["x"], SEQS, 3, 1e-3)
    g = recurrent.group_norm_backward(a["x"], a["w"], a["b"], stats, dy, SEQS, 3, act)
    names = ["x", "w", "b"] if affine else ["x"]
    differences(loss, a, names, dict(x=g["dx"][0], w=g["dweight"][0], b=g["dbias"][0]))


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotation_is_orthogonal_and_relative(interleaved):
    """Turned back it is the input; products of two rows depend on the difference of their positions."""
    r = np.random.default_rng(3)
    x, f = r.standard_normal((6, 2, 12)), np.array([1.0, 0.3, 0.01, 1e-3])
    pos = np.array([[0, 1, 7, -3, 100000, 2], [5, 5, 0, 2, 1, 9]])
    kw = dict(sections=(3, 1), interleaved=interleaved)
    y, _ = recurrent.rotate(x, pos, f, **kw)
    back, _ = recurrent.rotate(y, pos, f, inverse=True, **kw)
    assert np.allclose(back, x, atol=1e-14)
    assert np.array_equal(y[..., 8:], x[..., 8:])
    far, _ = recurrent.rotate(x, pos + 1234, f, **kw)
    products = [np.einsum("tgn,sgn->tsg", v, v) for v in (y, far)]
    assert np.allclose(*products, atol=1e-10)


def test_values_by_hand():
    # a = sigmoid(0) = 1/2: h = 1/2 x, then 1/2 h + 1/2 x
    f = recurrent.recurrence(np.array([[2.0], [4.0]]), np.zeros((2, 1)), None, None, [(0, 2)])
    assert np.allclose(f["y"][0][:, 0], [1.0, 2.5]) and np.allclose(f["final"][0], 2.5)
    # softplus(decay) = log 2, sigmoid(gate) = 1/2, sharpness 2: a = 1/2, m = sqrt(3)/2
    f = recurrent.recurrence(np.array([[2.0], [4.0]]), np.zeros((2, 1)), np.zeros(1), None,
                             [(0, 2)], np.array([[8.0]]), 2.0)
    m = np.sqrt(0.75)
    assert np.allclose(f["y"][0][:, 0], [4 + 2 * m, 2 + 5 * m])
    y, _ = recurrent.rotate(np.array([[[1.0, 0.0]]]), np.array([[3]]), np.array([np.pi / 2]), (1,))
    assert np.allclose(y, [[[0.0, -1.0]]])
    x = np.array([[1.0, 3.0, 5.0, 5.0]])
    y, _, stats, _ = recurrent.group_norm(x, None, None, [(0, 1)], 2, 0.0 + 1e-12, False)
    assert np.allclose(y, [[-1, 1, 0, 0]], atol=1e-5) and np.allclose(stats[0, :, 0], [2, 5])
