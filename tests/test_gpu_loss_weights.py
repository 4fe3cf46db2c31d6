"""Weights of the losses' rows at the ends of their range: one that is not finite leaves the
other rows as they are, and any finite ones keep fp16's range (bounds of layer_util)."""
import math

import numpy as np
import pytest
import torch

import zero_sharded_mixed_bucketed_amd as Z
from act_util import TORCH, close, f64
from gpu_util import need_gpu
from layer_util import loss_bounds
from oracle import layer

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    print(flush=True)


def _inputs(t, d, v, dtype, seed):
    rng = np.random.default_rng(seed)
    w = torch.from_numpy(2 * d ** -0.5 * rng.standard_normal((v, d))).to(TORCH[dtype]).cuda()
    x = torch.from_numpy(rng.standard_normal((t, d))).to(TORCH[dtype]).cuda()
    return rng, x, w, rng.integers(0, v, t)


def _run(x, w, targets, weights, scale, distil, dw_dtype):
    t, (v, d) = x.shape[0], w.shape
    loss, dx = torch.empty(t, device="cuda"), torch.empty_like(x)
    dw = torch.empty((v, d), dtype=dw_dtype, device="cuda")
    y, wt = torch.from_numpy(targets).cuda(), torch.from_numpy(weights.astype(np.float32)).cuda()
    if distil:
        Z.distill_loss(x, w, y[:, None], torch.zeros((t, 1), device="cuda"), loss, weights=wt,
                       scale=scale, dx=dx, dw=dw)
    else:
        Z.vocab_loss(x, w, y, loss, weights=wt, scale=scale, dx=dx, dw=dw)
    return loss, dx, dw


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("distil", [False, True])
@pytest.mark.parametrize("t", [40, 1100])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_a_weight_that_is_not_finite_stays_in_its_row(bad, distil, t, dtype):
    """Next to weights of 1000, whose gradients need their power of two taken out; rows 5
    and 1029 are the same thread's."""
    rng, x, w, targets = _inputs(t, 48, 300, dtype, 3)
    weights = rng.random(t) + 0.5
    weights[t - 71 if t > 100 else 30] = 1000.0
    weights[5] = bad
    scale = 1 / 64
    loss, dx, dw = _run(x, w, targets, weights, scale, distil, torch.float32)
    rest = np.arange(t) != 5
    # visible where it belongs: an infinite weight's products with x stay infinite in dw
    assert not np.isfinite(f64(loss)[5]) and np.isnan(f64(dx)[5]).any()
    assert not dw.isfinite().all()
    weights[5] = 0.0                                   # the others' results do without it
    want = layer.vocab_loss(f64(x), f64(w), targets, weights.astype(np.float32), scale)
    bounds = loss_bounds(f64(x), f64(w), want[1], want[0],
                         weights.astype(np.float32).astype(np.float64), 1.0, scale, dtype, 1000.0)
    close(f64(loss)[rest], want[0][rest], bounds[0][rest], "fp32", "loss")
    close(f64(dx)[rest], want[2][rest], bounds[1][rest], dtype, "dx")


@pytest.mark.parametrize("spread", [2.0 ** -105, 2.0 ** 105, 2.0 ** 120])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_weights_far_from_one(spread, dtype):
    rng, x, w, targets = _inputs(40, 64, 700, dtype, 4)
    weights = spread * (0.25 + rng.random(40))
    scale = 2.0 / spread
    loss, dx, dw = _run(x, w, targets, weights, scale, False, torch.float32)
    w32 = weights.astype(np.float32).astype(np.float64)
    want = layer.vocab_loss(f64(x), f64(w), targets, w32, scale)
    bounds = loss_bounds(f64(x), f64(w), want[1], want[0], w32, 1.0, scale, dtype, w32.max())
    close(f64(loss), want[0], bounds[0], "fp32", "loss")
    close(f64(dx), want[2], bounds[1], dtype, "dx")
    close(f64(dw), want[3], bounds[2], "fp32", "dw")
