"""Pins of the operators' oracle: worked examples, invariances, and gradients against central
differences of the forward definitions."""

import numpy as np
import pytest

from oracle import operators as P


def test_linear_worked_example():
    out, mag = P.linear([[1.0, -2.0]], [[3.0, 4.0], [0.5, -1.0]])
    assert out.tolist() == [[-5.0, 2.5]] and mag.tolist() == [[11.0, 2.5]]


def test_moe_ffn_worked_example():
    # one feature: g = 2, u = 3, h = 3 * 2 / (1 + e^-2); two slots on one expert, one dropped
    x = np.array([[1.0, 1.0]])
    w1 = np.array([[[1.0, 1.0], [2.0, 1.0]]])
    w2 = np.array([[[1.0], [-2.0]]])
    h = 6.0 / (1.0 + np.exp(-2.0))
    out, bound = P.moe_ffn(x, np.array([[0, -1, 0]]), np.array([[0.25, 9.0, 0.5]]), w1, w2)
    np.testing.assert_allclose(out, [[0.75 * h, -1.5 * h]], rtol=1e-14)
    assert (bound > 0).all() and (bound < 1e-2 * np.abs(out)).all()
    out, _ = P.moe_ffn(x, np.array([[5, -1]]), np.ones((1, 2)), w1, w2)
    assert (out == 0).all()


def test_balance_even_and_concentrated_loads():
    T, E, k = 8, 4, 1
    z = np.zeros((T, E))
    ids = np.arange(T)[:, None] % E
    loss, counts, tokens, grad = P.balance(z, ids, 0.5)
    assert loss == pytest.approx(0.5) and counts.tolist() == [[2, 2, 2, 2]] and tokens[0] == T
    assert np.abs(grad).max() < 1e-17  # an even load has no gradient at even probabilities
    # every token on expert 0 with probability 1: f = (E, 0, 0, 0), P = (1, 0, 0, 0)
    z[:, 0] = 1e3
    loss, counts, _, _ = P.balance(z, np.zeros((T, 1), int), 0.5)
    assert loss == pytest.approx(0.5 * E) and counts.tolist() == [[T, 0, 0, 0]]


def test_balance_ignores_masked_tokens_and_rows_outside():
    rng = np.random.default_rng(0)
    z, ids = rng.normal(size=(9, 5)), rng.integers(-1, 5, size=(9, 2))
    keep = [1, 2, 4, 5, 6]
    mask = np.isin(np.arange(9), keep)
    a = P.balance(z, ids, 1.0, offs=[1, 4, 4, 7], mask=mask)
    b = P.balance(z[keep], ids[keep], 1.0, offs=[0, 2, 2, 5])
    assert a[0] == pytest.approx(b[0], rel=1e-15) and (a[1] == b[1]).all() and (a[2] == b[2]).all()
    np.testing.assert_allclose(a[3][keep], b[3], rtol=1e-14)
    assert (a[3][~mask] == 0).all()


def test_balance_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(1)
    z, ids = rng.normal(size=(7, 6)), rng.integers(0, 6, size=(7, 2))
    z[3, 2] = -np.inf
    z[5] = -np.inf
    offs = [0, 3, 7]
    grad = P.balance(z, ids, 0.3, offs, dloss=1.7)[3]
    assert grad[3, 2] == 0 and (grad[5] == 0).all()
    d = np.where(np.isfinite(z), rng.normal(size=z.shape), 0.0)
    eps = 1e-5
    up, dn = P.balance(z + eps * d, ids, 0.3, offs)[0], P.balance(z - eps * d, ids, 0.3, offs)[0]
    assert float((grad * d).sum()) == pytest.approx(1.7 * (up - dn) / (2 * eps), rel=1e-6)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
def test_residual_norm_gradient_is_the_difference_quotient(gate, post):
    rng = np.random.default_rng(2)
    T, H = 4, 10
    shape = {"none": None, "channel": (1, H), "token": (T, 1), "full": (T, H)}[gate]
    v = dict(r=rng.normal(size=(T, H)), y=rng.normal(size=(T, H)),
             gate=1.0 if shape is None else rng.normal(size=shape), pre_gamma=rng.normal(size=H),
             post_gamma=rng.normal(size=H) if post else None)
    dr_new, dn = rng.normal(size=(T, H)), rng.normal(size=(T, H))

    def value(v):
        rn, n = P.residual_norm(scale=0.7, eps=1e-3, **v)[:2]
        return float((dr_new * rn).sum() + (dn * n).sum())

    g = P.residual_norm_grad(dr_new, dn, scale=0.7, eps=1e-3, **v)
    names = {"r": "dr", "y": "dy", "pre_gamma": "dpre_gamma"}
    if post:
        names["post_gamma"] = "dpost_gamma"
    if shape is not None:
        names["gate"] = "dgate"
    for name, key in names.items():
        d = rng.normal(size=np.shape(v[name]))
        up, dn_ = dict(v), dict(v)
        up[name], dn_[name] = v[name] + 1e-6 * d, v[name] - 1e-6 * d
        val, mag = g[key]
        assert (mag >= np.abs(val) * (1 - 1e-12)).all()
        # the gate's gradient is elementwise: the product broadcasts and sums it
        assert float((val * d).sum()) == pytest.approx((value(up) - value(dn_)) / 2e-6, rel=1e-6)


def test_residual_norm_of_a_constant_row():
    rn, n, rs_y, rs_r, _ = P.residual_norm(np.zeros((1, 4)), np.full((1, 4), 3.0), np.ones(4),
                                           pre_gamma=np.ones(4), scale=2.0, eps=0.0)
    np.testing.assert_allclose(rn, 2.0)
    np.testing.assert_allclose(n, 1.0)
    assert rs_y[0, 0] == pytest.approx(1 / 3) and rs_r[0, 0] == pytest.approx(0.5)
