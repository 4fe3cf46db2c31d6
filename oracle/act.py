"""Activations kept in 8 bits, the weight gradient from them, and the norms
around a block, in 64 bits.

The checkpoint format, per row and block of 32 columns (a scale byte b stands
for 2^(b - 127), 255 for NaN):

* int8: the scale is 2^(floor(log2 amax) - 6), codes are whole numbers nearest
  to x / scale (ties to even) and within +-127;
* e4m3: x is held to +-1.875 * 2^E (E = 15 for fp16, 127 for bf16) and the
  scale is the least power of two with amax / scale <= 448; codes are the
  nearest e4m3 values (ties to even).

Scales are at least 2^-126 (int8) and 2^-117 (e4m3).  A block with a value that
is not finite is NaN.
"""
from __future__ import annotations

import numpy as np

BLOCK = 32
E_MAX = {"fp16": 15, "bf16": 127}


def e4m3_value(code: int) -> float:
    """The value of an e4m3 code (bias 7, no infinities, S.1111.111 is NaN)."""
    sign = -1.0 if code & 0x80 else 1.0
    e, m = (code >> 3) & 15, code & 7
    if e == 15 and m == 7:
        return float("nan")
    return sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))


def _nearest_e4m3(y: float) -> int:
    """The code nearest to y (|y| <= 464), ties to the even mantissa."""
    best, code = None, 0
    for c in range(0x7F):
        d = abs(abs(y) - e4m3_value(c))
        if best is None or d < best or (d == best and c % 2 == 0):
            best, code = d, c
    return code | (0x80 if np.signbit(y) else 0)


_E4M3 = np.array([e4m3_value(c) for c in range(0x7F)])
_E4M3_ALL = np.array([e4m3_value(c) for c in range(256)])


def _encode_e4m3(y: np.ndarray) -> np.ndarray:
    a = np.abs(y)
    hi = np.searchsorted(_E4M3, a).clip(0, 0x7E)       # first value >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _E4M3[lo], _E4M3[hi] - a
    down = (dl < dh) | ((dl == dh) & (lo % 2 == 0))
    code = np.where(down, lo, hi)
    return (code | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)


def _padded(x, fill=0.0):
    t, h = x.shape
    nb = -(-h // BLOCK)
    out = np.full((t, nb * BLOCK), fill, dtype=x.dtype)
    out[:, :h] = x
    return out.reshape(t, nb, BLOCK)


def store(x: np.ndarray, fmt: str, dtype: str):
    """(codes uint8 [t, h], scale bytes uint8 [t, ceil(h / 32)]) of float64 x."""
    t, h = x.shape
    xb = _padded(np.asarray(x, np.float64))
    finite = np.isfinite(xb).all(axis=2)
    xb = np.where(finite[..., None], xb, 0.0)
    if fmt == "e4m3":
        top = 1.875 * 2.0 ** E_MAX[dtype]
        xb = np.clip(xb, -top, top)
    amax = np.abs(xb).max(axis=2)
    m, k = np.frexp(amax)                              # amax = m 2^k, m in [0.5, 1)
    if fmt == "int8":
        e = np.where(amax > 0, np.maximum(k - 7, -126), -126)
        codes = np.clip(np.rint(np.ldexp(xb, -e[..., None])), -127, 127)
        codes = codes.astype(np.int8).view(np.uint8)
    else:
        e = np.where(amax > 0, np.maximum(np.where(m > 0.875, k - 8, k - 9), -117), -117)
        codes = _encode_e4m3(np.ldexp(xb, -e[..., None]))
    codes = np.where(finite[..., None], codes, 0).astype(np.uint8)
    scales = np.where(finite, e + 127, 255).astype(np.uint8)
    return codes.reshape(t, -1)[:, :h].copy(), scales


def held(codes: np.ndarray, scales: np.ndarray, fmt: str) -> np.ndarray:
    """float64 values of a checkpoint."""
    t, h = codes.shape
    v = codes.view(np.int8).astype(np.float64) if fmt == "int8" else _E4M3_ALL[codes]
    b = scales.astype(np.int64)
    s = np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))
    return v * np.repeat(s, BLOCK, axis=1)[:, :h]


def weight_grad(dy: np.ndarray, x: np.ndarray) -> np.ndarray:
    """dW[n, k] = sum over t of dy[t, n] x[t, k]."""
    return dy.astype(np.float64).T @ x.astype(np.float64)


def stats(x: np.ndarray, kind: str, eps: float):
    """(mean, 1 / deviation) per row; (0, 1) without a norm, mean 0 for rms."""
    t = x.shape[0]
    if kind == "none":
        return np.zeros((t, 1)), np.ones((t, 1))
    m = x.mean(axis=1, keepdims=True) if kind == "layer" else np.zeros((t, 1))
    return m, 1.0 / np.sqrt(np.mean((x - m) ** 2, axis=1, keepdims=True) + eps)


def _or(v, other):
    return other if v is None else np.asarray(v, np.float64)


def block_norm(h, b, post, pre, gate=None, scale=1.0):
    """(h', z, stats [t, 4]); post and pre are (kind, eps, weight, bias); b None:
    h' = h."""
    t = h.shape[0]
    m2, r2 = np.zeros((t, 1)), np.ones((t, 1))
    out = np.asarray(h, np.float64)
    if b is not None:
        m2, r2 = stats(b, post[0], post[1])
        o = (b - m2) * r2 * _or(post[2], 1.0) + _or(post[3], 0.0)
        out = out + scale * (_or(gate, 1.0) * o)
    m1, r1 = stats(out, pre[0], pre[1])
    z = (out - m1) * r1 * _or(pre[2], 1.0) + _or(pre[3], 0.0)
    return out, z, np.concatenate([m2, r2, m1, r1], axis=1)


def _through(q, xn, r, kind):
    """The gradient of x from q, that of the normalised xn."""
    if kind == "none":
        return q
    d = q - xn * np.mean(q * xn, axis=1, keepdims=True)
    if kind == "layer":
        d = d - np.mean(q, axis=1, keepdims=True)
    return r * d


def block_norm_grad(dout, dz, x_out, x_block, st, post, pre, gate=None, scale=1.0):
    """Gradients of block_norm as a dict, from values x_out of h' and x_block of b
    and the statistics st; dgate is per token (sum it for a broadcast gate)."""
    m2, r2, m1, r1 = (st[:, i:i + 1].astype(np.float64) for i in range(4))
    d = 0.0 if dout is None else np.asarray(dout, np.float64)
    g = {}
    if pre[0] != "none":
        x1 = (x_out - m1) * r1
        d = d + _through(dz * _or(pre[2], 1.0), x1, r1, pre[0])
        g["dw_pre"], g["db_pre"] = (dz * x1).sum(axis=0), dz.sum(axis=0)
    g["dres"] = d
    u = scale * d
    p = u * _or(gate, 1.0)
    v = p * _or(post[2], 1.0)
    if x_block is not None:
        x2 = (x_block - m2) * r2
        g["dgate"] = u * (x2 * _or(post[2], 1.0) + _or(post[3], 0.0))
        if post[0] != "none":
            g["dw_post"], g["db_post"] = (p * x2).sum(axis=0), p.sum(axis=0)
        v = _through(v, x2, r2, post[0])
    g["dblock"] = v
    return g
