"""What the rounding of the losses' gradients by the logits leaves out at a token's entries
is kept where at most 64 tokens have a loss, whatever the number of rows they are given in.

Inputs whose logits are exact: x holds multiples of 1/8 and w of 1/8, so that fp32 sums of
their products are the sums.  What is left of an entry's error are the few roundings of its
fp32 value, and a rounding of the rest: EPS^2 of the value.  Without the rests it is EPS of
it.  dw is taken in fp32.  For dx, whose own rounding is EPS of the result: all words have a
part in common, which the gradient's zero sum over them takes out of the result, not out of
the error."""
import numpy as np
import pytest
import torch

import zero_sharded_mixed_bucketed_amd as Z
from act_util import EPS, TINY, TORCH, U, close, f64
from gpu_util import need_gpu
from layer_util import product
from oracle import layer

D = 16
# (tokens with a loss, rows)
COUNTS = [(1, 1), (5, 5), (14, 14), (14, 40), (33, 64), (64, 64), (64, 65), (10, 66), (3, 127),
          (14, 128), (64, 300), (1, 3000), (40, 5000)]


def _inputs(n, rows, v, k, seed, tau):
    rng = np.random.default_rng(seed)
    x = rng.integers(-8, 9, (rows, D)) / 8.0
    w = rng.integers(-1, 2, (v, D)) / 8.0 + 6.0 * rng.choice([-1, 1], D)
    x[:, -1] = -(x[:, :-1] * w[0, :-1].round()).sum(1) / w[0, -1].round()   # the common part: 0
    x = np.round(x * 8) / 8
    ids = np.full((rows, k), -1)
    at = np.sort(rng.permutation(rows)[:n])
    ids[at] = np.stack([rng.permutation(v)[:k] for _ in range(n)])
    top = rng.integers(-16, 17, (rows, k)) / 8.0 * tau
    weights = rng.random(rows) + 0.5
    return x, w, ids, top, weights.astype(np.float32).astype(np.float64)


def _errors(x, w, d, weights, tau, dtype, q, rests):
    """Bound of the held gradient by the logits, rows with a loss; rests: True where they
    are kept."""
    on = (d != 0).any(axis=1)
    wt = np.where(on, weights, 0.0)[:, None]
    z = x @ w.T / tau
    far = z.max(axis=1, keepdims=True) - z
    p = np.exp(-far) / np.exp(-far).sum(axis=1, keepdims=True)
    # the logits are exact but for their scaling; exp's argument, the sum and its join
    rel = 4 * U * np.abs(z).max(axis=1, keepdims=True) + (w.shape[0] / 512 + 80
                                                          + 4 * np.minimum(far, 90.0)) * U
    err = wt * (p * rel + 2 * U * (p + 24 * q + np.abs(d) / np.maximum(wt, 1e-300)))
    held = 2.0 ** -13 * weights[on].max() if dtype == "fp16" else 1
    err = err + np.where(rests, EPS[dtype], 1) * EPS[dtype] * (np.abs(d) + err) \
        + TINY[dtype] * held
    return np.where(on[:, None], err, 0.0)


def _want(x, w, ids, top, weights, tau, scale):
    want = layer.distill_loss(x, w, ids, top, tau, weights, scale)
    q = np.zeros(want[1].shape)
    shares = layer.shares_of(ids, top, tau)
    for r, j in zip(*np.nonzero(ids >= 0)):
        q[r, ids[r, j]] += shares[r, j]
    return want, q


def _bounds(x, w, err, d, tau, scale):
    c, mag = abs(scale) * tau, np.abs(d) + err
    n = np.count_nonzero((d != 0).any(axis=1))
    return (c * (err @ np.abs(w) + product(2 * w.shape[0], mag @ np.abs(w))) * (1 + 4 * U),
            c * (err.T @ np.abs(x) + product(2 * n, mag.T @ np.abs(x))) * (1 + 4 * U))


def _without(d, weights, dtype):
    """d with one rounding to dtype, as the products would take it without rests."""
    on = (d != 0).any(axis=1)
    e = np.frexp(np.float32(weights[on].max()))[1]
    held = 2.0 ** (14 - e)
    return torch.from_numpy(d * held).to(TORCH[dtype]).double().numpy() / held


def _case(n, rows, dtype, v, k, tau):
    """(inputs, oracle, error bound of d, bounds of dx and dw, scale)."""
    seed = n * 1000 + rows
    x, w, ids, top, weights = _inputs(n, rows, v, k, seed, tau)
    scale = 2.0 ** -4
    want, q = _want(x, w, ids, top, weights, tau, scale)
    err = _errors(x, w, want[1], weights, tau, dtype, q, q > 0)
    return (x, w, ids, top, weights), want, err, _bounds(x, w, err, want[1], tau, scale), scale


CASES = [("fp16", 8, 8, 1.0), ("bf16", 8, 8, 2.0), ("fp16", 200, 1, 1.0), ("bf16", 200, 3, 2.0)]


@pytest.mark.parametrize("n,rows", COUNTS)
@pytest.mark.parametrize("dtype,v,k,tau", CASES)
def test_the_bounds_need_the_rests(n, rows, dtype, v, k, tau):
    """In 64 bits: products with gradients that are rounded once lie outside the bounds (dw
    everywhere; dx where all words are entries)."""
    (x, w, _, _, weights), want, _, bounds, scale = _case(n, rows, dtype, v, k, tau)
    for m in (x, w):
        assert np.array_equal(torch.from_numpy(m).to(TORCH[dtype]).double().numpy(), m)
    d = _without(want[1], weights, dtype)
    off = np.abs(scale * tau * (d.T @ x) - want[3])
    assert (off > 1.5 * bounds[1]).any()
    if k == v:
        off = np.abs(scale * tau * (d @ w) - want[2])
        assert (off > 2 * (bounds[0] + EPS[dtype] * np.abs(want[2]) + TINY[dtype])).any()


@pytest.mark.gpu
@pytest.mark.parametrize("n,rows", COUNTS)
@pytest.mark.parametrize("dtype,v,k,tau", CASES)
def test_few_tokens_keep_their_entries_rests_in_any_number_of_rows(n, rows, dtype, v, k, tau):
    need_gpu()
    print(flush=True)
    (x, w, ids, top, weights), want, _, bounds, scale = _case(n, rows, dtype, v, k, tau)
    dev = [torch.from_numpy(m).to(TORCH[dtype]).cuda() for m in (x, w)]
    loss, dx = torch.empty(rows, device="cuda"), torch.empty_like(dev[0])
    dw = torch.empty((v, D), device="cuda")
    wt = torch.from_numpy(weights).float().cuda()
    Z.distill_loss(*dev, torch.from_numpy(ids).cuda(), torch.from_numpy(top).float().cuda(), loss,
                   temperature=tau, weights=wt, scale=scale, dx=dx, dw=dw)
    close(f64(dx), want[2], bounds[0], dtype, "dx")
    close(f64(dw), want[3], bounds[1], "fp32", "dw")
    if k == 1:                                         # one entry is cross entropy
        loss2, dx2, dw2 = torch.empty_like(loss), torch.empty_like(dx), torch.empty_like(dw)
        Z.vocab_loss(*dev, torch.from_numpy(ids[:, 0].copy()).cuda(), loss2, weights=wt,
                     scale=scale, dx=dx2, dw=dw2)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
