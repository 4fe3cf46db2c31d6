"""Helpers of the activation tests: inputs in 16 bits, their float64 values, and
error bounds.

Bounds are sums of two parts, written down before the first run:
* the output's own rounding, at most half a step: finfo(t).eps / 2 of the value
  (plus half the smallest step of fp16, 2^-25, or of bf16, 2^-134);
* the fp32 arithmetic before it: K * 2^-24 times the expression's value with
  every term replaced by its magnitude, where K counts the roundings on the way
  to one output.
"""
import numpy as np
import torch

TORCH = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
EPS = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
TINY = {"fp16": 2.0 ** -25, "bf16": 2.0 ** -134, "fp32": 2.0 ** -150}
U = 2.0 ** -24


def f64(t):
    return t.detach().cpu().double().numpy()


def strided(shape, dtype, pad=0, offset=0, device="cuda", fill=None):
    """A [t, h] view into a larger buffer: rows h + pad apart, `offset` elements
    in.  The buffer is returned too, to check that nothing else was written."""
    t, h = shape
    buf = torch.full((offset + max(t, 1) * (h + pad) + 8,), 7.0 if fill is None else fill,
                     dtype=torch.float32).to(dtype).to(device)
    return buf.as_strided((t, h), (h + pad, 1), offset), buf


def acts(rng, t, h, dtype, pad=0, offset=0, device="cuda", sigma=1.0):
    x = rng.standard_normal((t, h)) * sigma
    x *= np.where(rng.random(h) < 0.02, 12.0, 1.0)
    view, _ = strided((t, h), TORCH[dtype], pad, offset, device)
    view.copy_(torch.from_numpy(x).to(TORCH[dtype]))
    return view


def close(got, want, bound, dtype, what):
    """|got - want| <= bound + the rounding to `dtype`; NaN and infinities of a
    want that the type does not hold must agree."""
    got, want, bound = (np.asarray(v, np.float64) for v in (got, want, bound))
    assert got.shape == want.shape, what
    tol = bound * (1 + EPS[dtype]) + EPS[dtype] * np.abs(want) + TINY[dtype]
    bad = ~(np.abs(got - want) <= tol) & ~(np.isnan(got) & np.isnan(want))
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} off; first at "
                           f"{np.argwhere(bad)[0]}: got {got[bad][0]} want {want[bad][0]} "
                           f"tolerance {tol[bad][0]}")
