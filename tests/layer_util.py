"""Error bounds of the gated block's and the losses' tests, written down before their
first run (act_util has the outputs' own rounding).

u = 2^-24 is half a step of fp32, e(t) that of a 16-bit type.  A product's sums of n
exact products are off by at most 2 n u times the sum of magnitudes (n additions of at
most u each, twice that for an accumulation that truncates), and n + 16 covers what
joins splits.
"""
import numpy as np

from act_util import EPS, TINY, U
from oracle import layer


def product(n, mag):
    return 2 * (n + 16) * U * mag


def share_roundings(g, kind):
    """Roundings, in u, of the share p that passes: a few of exp, reciprocal and erfc,
    and those of the argument, which exp turns into |y| as many (erfc: 2 y^2, y^2 =
    g^2 / 2)."""
    a = np.abs(g)
    if kind == "gelu":
        return 16 + 2 * a * a
    if kind == "silu":
        return 16 + 4 * a
    return 16 + 8 * 1.6 * a * (1 + 0.0447 * a * a)


# A share below what exp holds in fp32 becomes 0.
SMALL = 2.0 ** -125


def gated_bound(x, w, kind):
    """Bounds of g, u and out before their rounding."""
    f = w.shape[0] // 2
    out, g, u = layer.gated(x, w, kind)
    dg, du = (product(x.shape[1], np.abs(x) @ np.abs(v).T) for v in (w[:f], w[f:]))
    a = np.abs(layer.act(g, kind)[0])
    # |act'| <= 1.13
    do = (1.13 * dg * (np.abs(u) + du) + a * du + share_roundings(g, kind) * U * np.abs(out)
          + SMALL * np.abs(g * u))
    return dg, du, do


def slopes_bound(dout, g, u, kind, dtype):
    """Bound of the rounded [dg du]."""
    p, slope = layer.share(g, kind)
    d = layer.gated_slopes(dout, g, u, kind)
    k = share_roundings(g, kind) * U * np.abs(dout)
    # 1 - p is off by u, whatever is left of it
    far = (1 + np.abs(g)) * np.maximum(p, SMALL)
    if kind != "silu":                      # the slope's factor (1 + g^2) of its own
        far = far * (1 + np.abs(g)) ** 2
    err = np.concatenate([k * np.abs(u) * far, k * np.abs(g) * np.maximum(p, SMALL)], axis=1)
    return d, err + EPS[dtype] * (np.abs(d) + err) + TINY[dtype]


def loss_bounds(x, w, d, loss, weights, tau, scale, dtype, top_weight, q=None):
    """Bounds of (loss, dx, dw) of a loss whose oracle gave d (and for distillation the
    dense shares q); rows that are left out have d = 0."""
    on = (d != 0).any(axis=1)
    xs = np.where(on[:, None], x, 0.0)
    wt = np.where(on, np.abs(weights), 0.0)[:, None]
    z = xs @ w.T / tau
    dz = product(x.shape[1], np.abs(xs) @ np.abs(w).T) / tau + 2 * U * np.abs(z)
    dz = dz.max(axis=1, keepdims=True)
    far = z.max(axis=1, keepdims=True) - z
    # relative error of p: the logits twice (its own, the sum's), exp's argument, the
    # sum over 512 threads' parts and their join
    rel = 2 * dz + (w.shape[0] / 512 + 80 + 4 * np.minimum(far, 90.0)) * U
    p = np.exp(-far)
    p = p / p.sum(axis=1, keepdims=True)
    err = wt * (p * rel + 2 * U * (p + (0 if q is None else 24 * q) + np.abs(d) / np.maximum(wt, 1e-300)))
    held = 2.0 ** -13 * top_weight          # fp16: d comes 2^14 / 2^e times as large
    err = err + EPS[dtype] * (np.abs(d) + err) + TINY[dtype] * (held if dtype == "fp16" else 1)
    err = np.where(on[:, None], err, 0.0)
    gap = np.abs(z).max(axis=1) + np.log(w.shape[0]) + 1
    loss_err = (wt[:, 0] * tau ** 2 * (2 * dz[:, 0] + (w.shape[0] / 512 + 80) * U + 16 * U * gap)
                + 16 * U * np.abs(loss))
    c = abs(scale) * tau
    mag = np.abs(d) + err
    dx = c * (err @ np.abs(w) + product(w.shape[0], mag @ np.abs(w)))
    dw = c * (err.T @ np.abs(xs) + product(x.shape[0], mag.T @ np.abs(xs)))
    return loss_err, dx * (1 + 4 * U), dw * (1 + 4 * U)
