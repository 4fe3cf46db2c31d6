"""The gated block's gradients against differences of its own forward, at inputs whose
projections the 8-bit checkpoints hold exactly, so that nothing but the difference's own
error and 16-bit roundings stands between them.

x holds whole numbers and w multiples of 1/16, so g, u are multiples of 1/16, below 8 in
magnitude: int8's step in a block of 32 is at most 2^-4 (its largest value below 8).  The
direction is the gradient's sign, the step 2^-4 (2^-6 for w), which 16 bits hold on both
sides.  Along a direction with projections rg, ru the third derivative of
act(g + s rg) (u + s ru) is act3 rg^3 (u + s ru) + 3 act2 rg^2 ru, with act's second and
third derivatives.  A token's input moves its own outputs only, and a unit's two weight
rows only that unit's: one direction gives a difference for each of them."""
import numpy as np
import pytest
import torch

import zero_sharded_mixed_bucketed_amd as Z
from act_util import EPS, f64
from gpu_util import need_gpu
from oracle import layer

T, D, F, H = 9, 12, 40, 2.0 ** -4
ACT = {"silu": Z.ACT_SILU, "gelu": Z.ACT_GELU, "gelu_tanh": Z.ACT_GELU_TANH}


def _inputs():
    rng = np.random.default_rng(11)
    x = rng.choice([-1.0, 1.0], (T, D))
    w = rng.integers(-10, 11, (2 * F, D)) / 16.0
    c = rng.integers(-8, 9, (T, F)) / 8.0
    return x, w, c


def _direction(grad, of_w):
    return np.where(grad < 0, -1.0, 1.0) / (4 if of_w else 1)


def _along(grad, r, of_w):
    """The derivative along r, of each token (x) or of each unit (w)."""
    return (grad * r).reshape(2, F, D).sum((0, 2)) if of_w else (grad * r).sum(1)


def _difference(forward, x, w, c, r, of_w):
    """(the difference along r, the larger sum of its terms' magnitudes) of each."""
    ends = []
    for s in (H, -H):
        out = (forward(x, w + s * r) if of_w else forward(x + s * r, w)) * c
        ends.append((out.sum(0 if of_w else 1), np.abs(out).sum(0 if of_w else 1)))
    (up, mag), (down, more) = ends
    return (up - down) / (2 * H), np.maximum(mag, more)


def _largest_derivatives(kind):
    """The largest second and third derivatives of act, from differences of the definition
    on a fine grid (0.1% between its points)."""
    g = np.linspace(-12, 12, 24001)
    a, step = layer.act(g, kind)[0], g[1] - g[0]
    return [1.001 * np.abs(np.diff(a, n)).max() / step ** n for n in (2, 3)]


def _slack(x, w, c, r, of_w, kind, mag):
    """Bound of |difference - derivative along r|, of each."""
    g, u = x @ w[:F].T, x @ w[F:].T
    rg, ru = (np.abs(x @ r[:F].T), np.abs(x @ r[F:].T)) if of_w else \
        (np.abs(r @ w[:F].T), np.abs(r @ w[F:].T))
    second, third = _largest_derivatives(kind)
    cut = H * H / 6 * (np.abs(c) * (third * rg ** 3 * (np.abs(u) + H * ru)
                                    + 3 * second * rg ** 2 * ru)).sum(0 if of_w else 1)
    # out is rounded on both sides, its sums' own error far below; dg, du and the result
    d = np.abs(layer.gated_slopes(c, g, u, kind))
    along = _along(d.T @ np.abs(x) if of_w else d @ np.abs(w), np.abs(r), of_w)
    return cut + mag * EPS["fp16"] * 1.05 / H + 2 * EPS["fp16"] * 1.05 * along


def _mistakes(x, w, c, of_w, kind):
    """Gradients with one mistake each: a sign, act' left out, act' without its second
    term, one projection's share left out, the shares exchanged."""
    g, u = x @ w[:F].T, x @ w[F:].T
    a, da = layer.act(g, kind)
    for dg, du in ((-c * u * da, -c * a), (c * u, c * a), (c * u * layer.share(g, kind)[0], c * a),
                   (c * u * da, 0 * a), (0 * a, c * a), (c * a, c * u * da)):
        d = np.concatenate([dg, du], axis=1)
        yield d.T @ x if of_w else d @ w


@pytest.mark.parametrize("kind", sorted(ACT))
@pytest.mark.parametrize("of_w", [False, True])
def test_the_bound_tells_a_mistake_from_the_gradient(kind, of_w):
    """In 64 bits: the differences lie within the bound of the derivatives, the bound is
    small beside them, and a gradient with a mistake is twice as far off somewhere."""
    x, w, c = _inputs()
    g, u = x @ w[:F].T, x @ w[F:].T
    assert max(np.abs(g).max(), np.abs(u).max()) < 8
    grad = layer.gated_grad(c, x, g, u, w, kind)[of_w]
    r = _direction(grad, of_w)
    far, mag = _difference(lambda a, b: layer.gated(a, b, kind)[0], x, w, c, r, of_w)
    got, slack = _along(grad, r, of_w), _slack(x, w, c, r, of_w, kind, mag)
    assert (np.abs(far - got) < slack).all() and slack.sum() < 0.05 * got.sum()
    for bad in _mistakes(x, w, c, of_w, kind):
        assert (np.abs(far - _along(bad, r, of_w)) > 2 * slack).any()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", sorted(ACT))
def test_gated_gradients_are_differences_of_the_forward(kind):
    need_gpu()
    x, w, c = _inputs()

    def dev(v):
        assert np.array_equal(v.astype(np.float16), v)
        return torch.from_numpy(v).half().cuda()

    def forward(a, b):
        out = torch.empty((T, F), dtype=torch.float16, device="cuda")
        Z.gated_ffn(dev(a), dev(b), out, ACT[kind])
        return f64(out)

    kx, kg, ku = (Z.ckpt_empty(T, n) for n in (D, F, F))
    Z.ckpt_write(dev(x), kx)
    Z.gated_ffn(dev(x), dev(w), None, ACT[kind], ckpt_gate=kg, ckpt_up=ku)
    for k, want in ((kx, x), (kg, x @ w[:F].T), (ku, x @ w[F:].T)):
        held = torch.empty((T, k.cols), device="cuda")
        Z.ckpt_read(k, held)
        assert np.array_equal(f64(held), want)
    dx = torch.empty((T, D), dtype=torch.float16, device="cuda")
    dw = torch.empty((2 * F, D), dtype=torch.float16, device="cuda")
    Z.gated_ffn_grad(dev(c), kg, ku, dev(w), ACT[kind], dx=dx, ckpt_x=kx, dw=dw)
    for grad, of_w in ((f64(dx), False), (f64(dw), True)):
        r = _direction(grad, of_w)
        far, mag = _difference(forward, x, w, c, r, of_w)
        got, slack = _along(grad, r, of_w), _slack(x, w, c, r, of_w, kind, mag)
        assert (np.abs(far - got) < slack).all() and slack.sum() < 0.05 * got.sum()
