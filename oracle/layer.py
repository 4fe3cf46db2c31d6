"""A gated feed-forward block and the losses over a vocabulary, in 64 bits.

    gated(x, w, act)           g = x wg^T, u = x wu^T, out = act(g) . u;  w = [wg; wu]
    gated_grad(...)            its gradients
    vocab_loss(...)            softmax cross entropy of x w^T and its gradients
    distill_loss(...)          KL divergence from a teacher's top logits, likewise

Gradients are those of scale * sum(loss).
"""
from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


def share(g, kind: str):
    """(p, dp/dg) of act(g) = g p(g)."""
    g = np.asarray(g, np.float64)
    if kind == "silu":
        with np.errstate(over="ignore"):
            p = 1.0 / (1.0 + np.exp(-g))
        return p, p * (1.0 - p)
    if kind == "gelu":
        return (0.5 * (1.0 + _erf(g / math.sqrt(2.0))),
                np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi))
    c = math.sqrt(2.0 / math.pi)
    h = np.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * (1.0 + h), 0.5 * (1.0 - h * h) * c * (1.0 + 3 * 0.044715 * g * g)


def act(g, kind: str):
    """(act(g), act'(g))."""
    p, slope = share(g, kind)
    return g * p, p + g * slope


def gated(x, w, kind: str):
    """(out, g, u)."""
    f = w.shape[0] // 2
    g, u = x @ w[:f].T, x @ w[f:].T
    return act(g, kind)[0] * u, g, u


def gated_slopes(dout, g, u, kind: str):
    """[dg du]."""
    a, da = act(g, kind)
    return np.concatenate([dout * u * da, dout * a], axis=1)


def gated_grad(dout, x, g, u, w, kind: str):
    """(dx, dw) from the block's input x and its held projections g and u."""
    d = gated_slopes(dout, g, u, kind)
    return d @ w, d.T @ x


def _softmax(z):
    z = z - z.max(axis=1, keepdims=True)
    e = np.exp(z)
    return e / e.sum(axis=1, keepdims=True)


def _log_softmax(z):
    z = z - z.max(axis=1, keepdims=True)
    return z - np.log(np.exp(z).sum(axis=1, keepdims=True))


def _grads(d, x, w, scale):
    return scale * (d @ w), scale * (d.T @ x)


def vocab_loss(x, w, targets, weights=None, scale=1.0):
    """(loss, d, dx, dw): d is the gradient of sum(loss) by the logits."""
    t = x.shape[0]
    weight = np.ones(t) if weights is None else np.asarray(weights, np.float64)
    loss, d = np.zeros(t), np.zeros((t, w.shape[0]))
    on = np.flatnonzero((targets >= 0) & (weight != 0))
    if on.size:
        z = x[on] @ w.T
        y = targets[on]
        loss[on] = -weight[on] * _log_softmax(z)[np.arange(on.size), y]
        p = _softmax(z)
        p[np.arange(on.size), y] -= 1.0
        d[on] = weight[on, None] * p
    safe = np.where((d != 0).any(axis=1)[:, None], x, 0.0)     # left-out rows add nothing
    return loss, d, *_grads(d, safe, w, scale)


def shares_of(ids, logits, tau):
    """A teacher's shares q [t, top]: the softmax over a row's entries (0 without)."""
    q = np.zeros(ids.shape)
    for r in range(ids.shape[0]):
        there = ids[r] >= 0
        if there.any():
            q[r, there] = _softmax(logits[r:r + 1, there] / tau)[0]
    return q


def distill_loss(x, w, ids, logits, tau=1.0, weights=None, scale=1.0):
    """(loss, d, dx, dw): d is the gradient of sum(loss) / tau by the logits."""
    t = x.shape[0]
    weight = np.ones(t) if weights is None else np.asarray(weights, np.float64)
    loss, d = np.zeros(t), np.zeros((t, w.shape[0]))
    q = shares_of(ids, logits, tau)
    for r in range(t):
        there = np.flatnonzero(ids[r] >= 0)
        if there.size == 0 or weight[r] == 0:
            continue
        z = (x[r:r + 1] @ w.T) / tau
        log_p = _log_softmax(z)[0]
        d[r] = np.exp(log_p)
        for j in there:
            if q[r, j] > 0:
                loss[r] += q[r, j] * (math.log(q[r, j]) - log_p[ids[r, j]])
            d[r, ids[r, j]] -= q[r, j]
        loss[r] *= weight[r] * tau ** 2
        d[r] *= weight[r]
    safe = np.where((d != 0).any(axis=1)[:, None], x, 0.0)
    return loss, d, *_grads(d, safe, w, scale * tau)
