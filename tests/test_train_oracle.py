"""Oracle of the balance loss, 8-bit checkpoints, gated activation and weight
gradients: worked cases, properties, and gradients against differences."""
import math

import numpy as np
import pytest

from oracle import train_ref as R


def test_balance_of_an_even_router_is_its_coefficient():
    """Every expert chosen equally often and equally probable: loss = coef."""
    T, E, K = 12, 4, 2
    chosen = np.array([[t % E, (t + 1) % E] for t in range(T)])
    for score in ("softmax", "sigmoid"):
        r = R.balance(np.zeros((T, E)), chosen, score=score, coef=0.5)
        assert math.isclose(r["loss"], 0.5) and r["counts"].tolist() == [6, 6, 6, 6]
        assert np.allclose(r["grad"], 0.0)


def test_balance_by_hand():
    """Two tokens, two experts, top-1, both sent to expert 0: f = (2, 0),
    loss = coef/2 * 2 * (p_00 + p_10)."""
    x = np.array([[math.log(3.0), 0.0], [0.0, 0.0]])
    r = R.balance(x, np.array([[0], [0]]), coef=1.0)
    assert math.isclose(r["loss"], 0.75 + 0.5)
    # token 1: p = (1/2, 1/2), load = (1, 0): grad = p (load - 1/2)
    assert np.allclose(r["grad"][1], [0.25, -0.25])


def test_balance_disabled_experts_and_padding():
    x = np.array([[0.0, -np.inf, 1.0], [-np.inf] * 3, [5.0, 2.0, 1.0]])
    r = R.balance(x, np.array([[2], [-1], [0]]), mask=[1, 1, 0], coef=1.0)
    assert r["grad"][0, 1] == 0 and not r["grad"][1].any() and not r["grad"][2].any()
    assert r["counts"].tolist() == [0, 0, 1]
    assert np.isfinite(r["loss"])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_gradient_against_differences(score):
    rng = np.random.default_rng(5)
    T, E, K = 11, 5, 2
    x = rng.normal(size=(T, E))
    chosen = np.argsort(-x, axis=1)[:, :K]
    kw = dict(chosen=chosen, seq_begin=[0, 4, 4, 9], mask=rng.random(T) > 0.2, score=score, coef=0.3)
    g = R.balance(x, **kw)["grad"]
    h = 1e-6
    for t in range(T):
        for e in range(E):
            d = np.zeros_like(x)
            d[t, e] = h
            num = (R.balance(x + d, **kw)["loss"] - R.balance(x - d, **kw)["loss"]) / (2 * h)
            assert abs(num - g[t, e]) < 1e-9


def test_act8_worked_blocks():
    """amax 127 * 2^-3 exactly -> e = -3; a hair more -> e = -2; ties to even."""
    x = np.zeros((3, 40))
    x[0, :3] = [127 / 8, 0.5 / 8, 1.5 / 8]
    x[1, 0] = np.nextafter(np.float32(127 / 8), np.float32(1e9))
    x[2, 35] = -3.0
    codes, exps = R.act8_encode(x)
    assert exps[0, 0] == 127 - 3 and codes[0, :3].tolist() == [127, 0, 2]
    assert exps[1, 0] == 127 - 2 and codes[1, 0] == 64
    assert exps[2, 0] == 1 and exps[2, 1] == 127 - 5 and codes[2, 35] == -96
    assert codes.shape == (3, 64) and not codes[:, 40:].any()


def test_act8_error_and_range():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(20, 77)) * np.exp2(rng.integers(-40, 40, size=(20, 1)))
    codes, exps = R.act8_encode(x)
    back = R.act8_decode(codes, exps, 77)
    step = np.repeat(np.ldexp(1.0, exps.astype(int) - 127), 32, axis=1)[:, :77]
    assert np.all(np.abs(back - x) <= step / 2)
    assert np.max(np.abs(codes)) <= 127
    big = float(np.finfo(np.float32).max)
    c, e = R.act8_encode(np.array([[big, -big, 1.0]]))
    assert np.all(np.isfinite(R.act8_decode(c, e, 3).astype(np.float32)))
    c, e = R.act8_encode(np.array([[1.0, np.inf] + [0.0] * 31 + [2.0]]))
    v = R.act8_decode(c, e, 34)
    assert np.all(np.isnan(v[0, :32])) and v[0, 33] == 2.0


def test_swiglu_gradient_against_differences():
    rng = np.random.default_rng(2)
    g, u, d = rng.normal(size=(3, 200)) * 3
    dg, du = R.swiglu_grad(d, g, u)
    h = 1e-6
    assert np.allclose(dg, d * (R.swiglu(g + h, u) - R.swiglu(g - h, u)) / (2 * h), atol=1e-7)
    assert np.allclose(du, d * (R.swiglu(g, u + h) - R.swiglu(g, u - h)) / (2 * h), atol=1e-7)


def test_weight_grads_against_differences():
    """G is the gradient of sum_t dy_t . (W_e x_t)."""
    rng = np.random.default_rng(3)
    dy, x = rng.normal(size=(9, 3)), rng.normal(size=(9, 4))
    off = [0, 2, 2, 9]
    g, _ = R.weight_grads(dy, x, off)
    assert not g[1].any()
    W = rng.normal(size=(3, 3, 4))
    f = lambda W: sum(float(dy[t] @ (W[e] @ x[t])) for e in range(3) for t in range(off[e], off[e + 1]))
    h = 1e-5
    for e, o, i in [(0, 1, 2), (1, 0, 0), (2, 2, 3), (2, 0, 1)]:
        d = np.zeros_like(W)
        d[e, o, i] = h
        assert abs((f(W + d) - f(W - d)) / (2 * h) - g[e, o, i]) < 1e-8
