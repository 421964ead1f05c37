"""Pins of the oracle in oracle/moe_ref.py: hand-made cases, and its gradients
against differences of its own forward passes."""
import math

import numpy as np

from oracle import moe_ref as R


def test_sort_by_hand():
    offsets, order, place, bad = R.sort([[2, 0], [0, -1], [2, 2], [1, 0]], 3)
    assert offsets.tolist() == [0, 3, 4, 7] and order.tolist() == [1, 2, 7, 6, 0, 4, 5]
    assert place.tolist() == [[4, 0], [1, -1], [5, 6], [3, 2]] and not bad
    offsets, order, place, bad = R.sort([[2, 0], [0, 3]], 3, rows=1)
    assert offsets.tolist() == [0, 1, 1, 1] and order.tolist() == [1] and bad
    assert place.tolist() == [[-1, 0], [-1, -1]]
    assert R.sort([[9, 1]], 2, mask=[False])[3] is False


def test_dispatch_and_combine_by_hand():
    place = np.array([[1, -1], [0, 2]])
    xs = R.dispatch([[1.0], [5.0]], place, 4)
    assert xs[:3, 0].tolist() == [5.0, 1.0, 5.0] and math.isnan(xs[3, 0])
    out, mass = R.combine([[2.0], [3.0], [-4.0], [math.nan]], place, [[0.5, math.nan], [1.0, 2.0]])
    assert out[:, 0].tolist() == [1.5, -6.0] and mass[:, 0].tolist() == [1.5, 10.0]


def test_gradients_against_differences():
    """The forward pass is linear in ys and in the weights: differences are exact."""
    rng = np.random.default_rng(0)
    place = np.array([[3, 0], [-1, 1], [2, 4]])
    ys, w, dout = rng.normal(size=(5, 6)), rng.normal(size=(3, 2)), rng.normal(size=(3, 6))
    dys, dw, _ = R.combine_grad(dout, ys, w, place)
    f = lambda ys, w: float(np.sum(dout * R.combine(ys, place, w)[0]))
    for grad, arg, g in ((dys, ys, lambda a: f(a, w)), (dw, w, lambda a: f(ys, a))):
        for i in np.ndindex(arg.shape):
            up, down = arg.copy(), arg.copy()
            up[i] += 1.0
            down[i] -= 1.0
            assert abs((g(up) - g(down)) / 2 - grad[i]) < 1e-12
    # dispatch's gradient is the sum over a token's rows
    x, d = rng.normal(size=(3, 6)), rng.normal(size=(5, 6))
    y = R.dispatch(x, place, 5)
    assert abs(np.sum(d * y) - np.sum(R.combine(d, place)[0] * x)) < 1e-12


def test_norm_by_hand():
    assert R.grad_norm([[3.0], [[4.0]]], 10.0) == (5.0, 1.0)
    assert R.grad_norm([[3.0], [4.0]], 1.0) == (5.0, 1.0 / (5.0 + 1e-6))
    n, s = R.grad_norm([[math.inf], [1.0]], 1.0)
    assert n == math.inf and math.isnan(s)
