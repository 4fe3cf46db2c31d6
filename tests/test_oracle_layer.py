"""Pins of the 64-bit gated block and losses (oracle/layer.py): closed forms and
differences (CPU)."""
import math

import numpy as np
import pytest

from oracle import layer

KINDS = ["silu", "gelu", "gelu_tanh"]


@pytest.mark.parametrize("kind,at_1", [("silu", 1 / (1 + math.exp(-1))),
                                       ("gelu", 0.8413447460685429),
                                       ("gelu_tanh", 0.8411919906082768)])
def test_activation_values(kind, at_1):
    g = np.array([0.0, 1.0, -1.0, 40.0, -40.0])
    a, da = layer.act(g, kind)
    assert a[0] == 0 and da[0] == 0.5
    assert abs(a[1] - at_1) < 1e-15 and abs(a[2] - (at_1 - 1)) < 1e-15
    assert abs(a[3] - 40) < 1e-12 and abs(a[4]) < 1e-12 and abs(da[3] - 1) < 1e-12


@pytest.mark.parametrize("kind", KINDS)
def test_activation_slopes_are_differences(kind):
    g = np.linspace(-6, 6, 241)
    h = 1e-5
    up, down = layer.act(g + h, kind)[0], layer.act(g - h, kind)[0]
    # third derivatives are below 4, so differences are off by h^2 and by 2^-52 / h
    assert np.abs(layer.act(g, kind)[1] - (up - down) / (2 * h)).max() < 4 * h * h + 1e-9


def _difference(f, v, at, h):
    old = v[at]
    v[at] = old + h
    up = f()
    v[at] = old - h
    down = f()
    v[at] = old
    return (up - down) / (2 * h)


@pytest.mark.parametrize("kind", KINDS)
def test_gated_gradients_are_differences(kind):
    rng = np.random.default_rng(0)
    x, w, do = (rng.standard_normal(s) for s in ((3, 5), (8, 5), (3, 4)))
    out, g, u = layer.gated(x, w, kind)
    assert np.allclose(out, layer.act(x @ w[:4].T, kind)[0] * (x @ w[4:].T), rtol=1e-15)
    dx, dw = layer.gated_grad(do, x, g, u, w, kind)

    def f():
        return (layer.gated(x, w, kind)[0] * do).sum()

    for v, d in ((x, dx), (w, dw)):
        for at in np.ndindex(v.shape):
            assert abs(_difference(f, v, at, 1e-5) - d[at]) < 1e-7


def _losses(rng, t=4, d=3, v=7):
    x, w = rng.standard_normal((t, d)), rng.standard_normal((v, d))
    weights = rng.random(t) + 0.5
    targets = np.array([2, -1, 6, 2])
    ids = np.array([[1, 4, -1], [-1, -1, -1], [6, 0, 6], [3, -1, 5]])
    logits = rng.standard_normal(ids.shape)
    return x, w, weights, targets, ids, logits


def test_cross_entropy_against_the_definition():
    x, w, weights, targets, _, _ = _losses(np.random.default_rng(1))
    loss, d, dx, dw = layer.vocab_loss(x, w, targets, weights, 3.0)
    z = x @ w.T
    for t in (0, 2, 3):
        want = weights[t] * (math.log(np.exp(z[t]).sum()) - z[t, targets[t]])
        assert abs(loss[t] - want) < 1e-14
        assert abs(d[t].sum()) < 1e-14
    assert loss[1] == 0 and not d[1].any() and not dx[1].any()

    def f():
        return 3.0 * layer.vocab_loss(x, w, targets, weights)[0].sum()

    for v, g in ((x, dx), (w, dw)):
        for at in np.ndindex(v.shape):
            assert abs(_difference(f, v, at, 1e-5) - g[at]) < 1e-7


@pytest.mark.parametrize("tau", [1.0, 2.5])
def test_distillation_against_the_definition(tau):
    x, w, weights, _, ids, logits = _losses(np.random.default_rng(2))
    loss, d, dx, dw = layer.distill_loss(x, w, ids, logits, tau, weights, 2.0)
    assert loss[1] == 0 and not dx[1].any()
    # row 2 has id 6 twice: the dense target adds its shares
    q = np.zeros((4, 7))
    for r in (0, 2, 3):
        e = {j: math.exp(logits[r, j] / tau) for j in range(3) if ids[r, j] >= 0}
        for j, s in e.items():
            q[r, ids[r, j]] += s / sum(e.values())
    z = x @ w.T / tau
    p = np.exp(z) / np.exp(z).sum(1, keepdims=True)
    for r in (0, 2, 3):
        assert np.allclose(d[r], weights[r] * (p[r] - q[r]), atol=1e-15)

    def f():
        return 2.0 * layer.distill_loss(x, w, ids, logits, tau, weights)[0].sum()

    for v, g in ((x, dx), (w, dw)):
        for at in np.ndindex(v.shape):
            assert abs(_difference(f, v, at, 1e-5) - g[at]) < 1e-7


def test_one_entry_is_cross_entropy():
    x, w, weights, targets, _, _ = _losses(np.random.default_rng(3))
    a = layer.vocab_loss(x, w, targets, weights)
    b = layer.distill_loss(x, w, targets[:, None], np.full((4, 1), 5.0), 1.0, weights)
    for u, v in zip(a, b):
        assert np.allclose(u, v, atol=1e-14)


def test_a_teacher_that_agrees_has_no_gradient():
    rng = np.random.default_rng(4)
    x, w = rng.standard_normal((2, 3)), rng.standard_normal((5, 3))
    ids = np.tile(np.arange(5), (2, 1))
    loss, d, dx, dw = layer.distill_loss(x, w, ids, x @ w.T, 3.0)
    for v in (loss, d, dx, dw):
        assert np.abs(v).max() < 1e-14


def test_left_out_rows_may_hold_anything():
    x, w, weights, targets, _, _ = _losses(np.random.default_rng(5))
    want = layer.vocab_loss(x, w, targets, weights)
    x[1] = np.nan
    for a, b in zip(want, layer.vocab_loss(x, w, targets, weights)):
        assert np.array_equal(a, b)
