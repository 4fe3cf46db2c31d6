"""The gated block and the losses over a vocabulary on the GPU against the 64-bit
oracle, within bounds that count the roundings (layer_util)."""
import math

import numpy as np
import pytest
import torch

import zero_sharded_mixed_bucketed_amd as Z
from act_util import EPS, TORCH, acts, close, f64, strided
from gpu_util import need_gpu
from layer_util import gated_bound, loss_bounds, product, slopes_bound
from oracle import act as oact
from oracle import layer

pytestmark = pytest.mark.gpu

FMT = {"int8": Z.CKPT_INT8, "e4m3": Z.CKPT_E4M3}
ACT = {"silu": Z.ACT_SILU, "gelu": Z.ACT_GELU, "gelu_tanh": Z.ACT_GELU_TANH}
KINDS = sorted(ACT)


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    print(flush=True)


def _matrix(rng, t, h, dtype, pad=0, off=0, sigma=1.0):
    view, _ = strided((t, h), TORCH[dtype], pad, off)
    view.copy_(torch.from_numpy(rng.standard_normal((t, h)) * sigma).to(TORCH[dtype]))
    return view


def _kept(buf, view, before):
    """Nothing beside the view's rows was written."""
    after = buf.clone()
    after.as_strided(view.shape, view.stride(), view.storage_offset()).copy_(
        before.as_strided(view.shape, view.stride(), view.storage_offset()))
    return torch.equal(after.view(torch.uint8), before.view(torch.uint8))


def _stored(x, fmt, dtype):
    codes, scales = oact.store(x, fmt, dtype)
    k = Z.Ckpt(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), FMT[fmt])
    return k, oact.held(codes, scales, fmt)


# ---------------------------------------------------------------- the gated block

SHAPES = [(1, 1, 1, 0, 0), (1, 8, 32, 0, 0), (1, 300, 500, 3, 1), (3, 7, 5, 1, 0),
          (31, 64, 33, 0, 0), (33, 70, 40, 8, 8), (64, 128, 96, 0, 0), (130, 200, 129, 1, 3),
          (257, 1032, 300, 0, 0), (300, 72, 1000, 2, 1)]
LARGE = [(2048, 64, 4096, 0, 0), (1025, 136, 4099, 1, 1)]


@pytest.mark.parametrize("t,d,f,pad,off", SHAPES + LARGE)
@pytest.mark.parametrize("kind,dtype", [("silu", "bf16"), ("gelu", "fp16"),
                                        ("gelu_tanh", "fp16"), ("silu", "fp16"),
                                        ("gelu_tanh", "bf16"), ("gelu", "bf16")])
def test_gated_ffn(t, d, f, pad, off, kind, dtype):
    rng = np.random.default_rng(t * 31 + d + f)
    x = acts(rng, t, d, dtype, pad, off)
    w = _matrix(rng, 2 * f, d, dtype, pad, off, 1.5 / math.sqrt(d))
    out, buf = strided((t, f), TORCH[dtype], pad, off)
    before = buf.clone()
    Z.gated_ffn(x, w, out, ACT[kind])
    want = layer.gated(f64(x), f64(w), kind)[0]
    close(f64(out), want, gated_bound(f64(x), f64(w), kind)[2], dtype, "out")
    assert _kept(buf, out, before)


@pytest.mark.parametrize("kind", KINDS)
def test_gated_ffn_over_the_range_of_the_gate(kind):
    """Gates from -65504 to 65504, and infinite and NaN ones: products of one term."""
    g = np.concatenate([np.linspace(-12, 12, 481), [-65504, -1000, -100, -90, -20, 20, 90, 100,
                                                    1000, 65504, -0.0, 6e-8]])
    x = torch.from_numpy(g[:, None]).half().cuda()
    w = torch.tensor([[1.0], [1.0]], dtype=torch.float16, device="cuda")
    out = torch.empty((g.size, 1), dtype=torch.float16, device="cuda")
    # u = g too: act(g) g
    Z.gated_ffn(x, w, out, ACT[kind])
    want = layer.gated(f64(x), f64(w), kind)[0]
    bound = gated_bound(f64(x), f64(w), kind)[2]
    want = torch.from_numpy(want).half().double().numpy() if np.abs(want).max() > 65504 else want
    fine = np.isfinite(want)
    close(np.where(fine, f64(out), 0), np.where(fine, want, 0), bound * fine + 2.0 ** -11 *
          np.abs(np.where(fine, want, 0)), "fp16", "out")
    assert np.array_equal(f64(out)[~fine], want[~fine])
    x = torch.tensor([[math.nan], [math.inf]], dtype=torch.float16, device="cuda")
    Z.gated_ffn(x, w, out[:2], ACT[kind])
    assert np.isnan(f64(out)[0, 0]) and f64(out)[1, 0] == math.inf


@pytest.mark.parametrize("t,d,f", [(5, 16, 33), (70, 64, 257), (40, 40, 96), (1100, 16, 4100)])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_emitted_checkpoints_are_those_of_the_rounded_projections(t, d, f, fmt, dtype):
    """Small whole numbers: sums are exact, so codes have to be the oracle's."""
    rng = np.random.default_rng(t + f)
    x = torch.from_numpy(rng.integers(-3, 4, (t, d))).to(TORCH[dtype]).cuda()
    w = torch.from_numpy(rng.integers(-3, 4, (2 * f, d))).to(TORCH[dtype]).cuda()
    ks = [Z.ckpt_empty(t, f, FMT[fmt]) for _ in range(3)]
    for k in ks:
        k.codes.fill_(0x55)
    out = torch.empty((t, f), dtype=TORCH[dtype], device="cuda")
    Z.gated_ffn(x, w, out, Z.ACT_SILU, *ks)
    _, g, u = layer.gated(f64(x), f64(w), "silu")
    for k, v in zip(ks, (g, u, f64(out))):
        v = f64(torch.from_numpy(v).to(TORCH[dtype]))
        codes, scales = oact.store(v, fmt, dtype)
        assert np.array_equal(k.codes.cpu().numpy(), codes)
        assert np.array_equal(k.scales.cpu().numpy(), scales)
    # alone, and without out
    alone = Z.ckpt_empty(t, f, FMT[fmt])
    Z.gated_ffn(x, w, None, Z.ACT_SILU, ckpt_up=alone)
    assert torch.equal(alone.codes, ks[1].codes) and torch.equal(alone.scales, ks[1].scales)


@pytest.mark.parametrize("t,d,f,pad,off", SHAPES + [(4096, 4096, 64, 0, 0), (1025, 4100, 65, 1, 1)])
@pytest.mark.parametrize("kind,fmt,dtype,out,acc", [
    ("silu", "int8", "bf16", "bf16", False), ("gelu", "e4m3", "fp16", "fp16", True),
    ("gelu_tanh", "int8", "fp16", "fp32", True), ("silu", "e4m3", "bf16", "fp32", False)])
def test_gated_ffn_grad(t, d, f, pad, off, kind, fmt, dtype, out, acc):
    rng = np.random.default_rng(t * 17 + d + f)
    kx, x = _stored(f64(acts(rng, t, d, dtype)), fmt, dtype)
    kg, g = _stored(f64(acts(rng, t, f, dtype)), fmt, dtype)
    ku, u = _stored(f64(acts(rng, t, f, dtype)), fmt, dtype)
    w = _matrix(rng, 2 * f, d, dtype, pad, off, 1 / math.sqrt(d))
    dout = _matrix(rng, t, f, dtype, pad, off, 0.1)
    dx, dx_buf = strided((t, d), TORCH[dtype], pad, off)
    dw, dw_buf = strided((2 * f, d), TORCH[out], pad, off)
    old = f64(dw) if acc else 0.0
    dx0, dw0 = dx_buf.clone(), dw_buf.clone()
    Z.gated_ffn_grad(dout, kg, ku, w, ACT[kind], dx=dx, ckpt_x=kx, dw=dw, accumulate=acc)
    d0, err = slopes_bound(f64(dout), g, u, kind, dtype)
    mag = np.abs(d0) + err
    wv = f64(w)
    close(f64(dx), d0 @ wv, err @ np.abs(wv) + product(2 * f, mag @ np.abs(wv)), dtype, "dx")
    bound = err.T @ np.abs(x) + product(t, mag.T @ np.abs(x) + np.abs(old))
    close(f64(dw), d0.T @ x + old, bound, out, "dw")
    assert _kept(dx_buf, dx, dx0) and _kept(dw_buf, dw, dw0)
    # each alone gives the same bits
    only, _ = strided((t, d), TORCH[dtype], pad, off)
    Z.gated_ffn_grad(dout, kg, ku, w, ACT[kind], dx=only)
    assert torch.equal(only, dx)
    if not acc:
        only, _ = strided((2 * f, d), TORCH[out], pad, off)
        Z.gated_ffn_grad(dout, kg, ku, None, ACT[kind], ckpt_x=kx, dw=only)
        assert torch.equal(only, dw)


def test_gated_gradients_are_differences():
    """Along a direction of the input: inputs on a grid that 16 bits hold on both sides.
    The loss is sum(out . c); its third difference is below 2 |r_g|^3 |u| + ... <= 40 a
    term here, so a step of 2^-6 is off by 40 h^2 / 6 a term."""
    rng = np.random.default_rng(11)
    t, d, f, h = 9, 16, 24, 2.0 ** -6
    x = rng.integers(-64, 65, (t, d)) / 64.0
    w = rng.integers(-64, 65, (2 * f, d)) / 256.0
    r = rng.choice([-1.0, 1.0], (t, d))
    c = rng.integers(-8, 9, (t, f)) / 8.0

    def dev(v):
        return torch.from_numpy(v).half().cuda()

    def value(v):
        out = torch.empty((t, f), dtype=torch.float16, device="cuda")
        Z.gated_ffn(dev(v), dev(w), out, Z.ACT_GELU)
        return (f64(out) * c).sum(), np.abs(f64(out) * c).sum()

    (up, mag), (down, _) = value(x + h * r), value(x - h * r)
    kx, kg, ku = (Z.ckpt_empty(t, n) for n in (d, f, f))
    Z.ckpt_write(dev(x), kx)
    Z.gated_ffn(dev(x), dev(w), None, Z.ACT_GELU, ckpt_gate=kg, ckpt_up=ku)
    dx = torch.empty((t, d), dtype=torch.float16, device="cuda")
    Z.gated_ffn_grad(dev(c), kg, ku, dev(w), Z.ACT_GELU, dx=dx)
    got = (f64(dx) * r).sum()
    # int8 holds g and u to 2^-7 of a block's largest (below 8 here)
    slack = (40 * h * h / 6 * np.abs(c).sum() + 2 * mag * EPS["fp16"] / (2 * h)
             + 8 * 2.0 ** -7 * 1.2 * 2 * (np.abs(c) @ (np.abs(w[:f]) + np.abs(w[f:]))).sum())
    assert abs((up - down) / (2 * h) - got) < slack
    assert abs(got) > 0 and slack < 40 * np.abs(c).sum()


def test_gated_gradients_without_rows():
    w = torch.ones((8, 16), dtype=torch.float16, device="cuda")
    dout = torch.empty((0, 4), dtype=torch.float16, device="cuda")
    k, kx = Z.ckpt_empty(0, 4), Z.ckpt_empty(0, 16)
    dw = torch.full((8, 16), 3.0, dtype=torch.float16, device="cuda")
    Z.gated_ffn_grad(dout, k, k, w, ckpt_x=kx, dw=dw, accumulate=True)
    assert (dw == 3).all()
    Z.gated_ffn_grad(dout, k, k, w, ckpt_x=kx, dw=dw)
    assert (dw == 0).all()
    Z.gated_ffn(torch.empty((0, 16), dtype=torch.float16, device="cuda"), w, dout)


def test_nan_tokens_stay_in_their_rows_of_the_gated_block():
    rng = np.random.default_rng(3)
    x, w = acts(rng, 70, 48, "fp16"), _matrix(rng, 200, 48, "fp16")
    outs, ks = [], []
    for bad in (False, True):
        if bad:
            x[17, 5], x[40, 0] = math.nan, math.inf
        out = torch.empty((70, 100), dtype=torch.float16, device="cuda")
        k = Z.ckpt_empty(70, 100)
        Z.gated_ffn(x, w, out, ckpt_gate=k)
        outs.append(out)
        ks.append(k)
    rest = [i for i in range(70) if i not in (17, 40)]
    assert torch.equal(outs[0][rest], outs[1][rest]) and outs[1][17].isnan().all()
    assert torch.equal(ks[0].codes[rest], ks[1].codes[rest])
    assert (ks[1].scales[17] == 255).all() and (ks[1].scales[40] == 255).any()


def test_gated_block_past_32_bits():
    """Rows more than 2^31 elements apart in every operand."""
    t, d, f, stride = 3, 40, 24, (1 << 30) + 8
    big = torch.empty(2 * f * stride, dtype=torch.float16, device="cuda")
    far = [big.as_strided((n, h), (s, 1), o) for n, h, s, o in
           ((t, d, 3 * stride, 0), (2 * f, d, stride, 64), (t, f, 3 * stride, 128),
            (t, d, 3 * stride, 256), (t, f, 3 * stride, 320))]
    rng = np.random.default_rng(1)
    for v in far:
        v.copy_(torch.from_numpy(rng.standard_normal(v.shape)).half())
    x, w, out, dx, dout = far
    near = [v.clone() for v in far]
    k = [Z.ckpt_empty(t, f) for _ in range(4)]
    Z.gated_ffn(x, w, out, ckpt_gate=k[0], ckpt_up=k[1])
    Z.gated_ffn(near[0], near[1], near[2], ckpt_gate=k[2], ckpt_up=k[3])
    assert torch.equal(out, near[2]) and torch.equal(k[0].codes, k[2].codes)
    Z.gated_ffn_grad(dout, k[0], k[1], w, dx=dx)
    Z.gated_ffn_grad(near[4], k[2], k[3], near[1], dx=near[3])
    assert torch.equal(dx, near[3])


# ---------------------------------------------------------------- the losses

def _loss_inputs(rng, t, d, v, dtype, pad, off, left_out, weights):
    w = _matrix(rng, v, d, dtype, pad, off, 2.0 / math.sqrt(d))
    targets = rng.integers(0, v, t)
    lift = 3.0 * rng.random((t, 1)) * (rng.random((t, 1)) < 0.5)
    x = _matrix(rng, t, d, dtype, pad, off)
    x.copy_(torch.from_numpy(rng.standard_normal((t, d)) + lift * f64(w)[targets]).to(x.dtype))
    targets[rng.random(t) < left_out] = -100
    wt = rng.random(t) + 0.25 if weights else None
    if weights and t > 2:
        wt[t // 2], wt[t // 3] = 0.0, -1.5
    return x, w, targets, wt


def _dev(v, dt=torch.float32):
    return None if v is None else torch.from_numpy(v).to(dt).cuda()


def _check_loss(x, w, wt, call, want, tau, scale, dtype, out, acc, pad, off, q=None):
    """call(loss, **outputs) against want = (loss, d, dx, dw)."""
    t, v, d = x.shape[0], w.shape[0], x.shape[1]
    loss, buf = strided((1, t), torch.float32, 0, 1)
    dx, dx_buf = strided((t, d), TORCH[dtype], pad, off)
    dw, dw_buf = strided((v, d), TORCH[out], pad, off)
    old = f64(dw) if acc else 0.0
    dx0, dw0, loss0 = dx_buf.clone(), dw_buf.clone(), buf.clone()
    call(loss[0], dx=dx, dw=dw, accumulate=acc, scale=scale)
    weights = np.ones(t) if wt is None else wt.astype(np.float32).astype(np.float64)
    on = (want[1] != 0).any(axis=1)
    top = np.abs(weights).max(initial=0.0, where=on) if wt is not None else 1.0
    bounds = loss_bounds(f64(x), f64(w), want[1], want[0], weights, tau, scale, dtype, top, q)
    close(f64(loss[0]), want[0], bounds[0], "fp32", "loss")
    close(f64(dx), want[2], bounds[1], dtype, "dx")
    close(f64(dw), want[3] + old, bounds[2] + product(1, np.abs(old)), out, "dw")
    assert (f64(loss[0])[~on] == 0).all() and (f64(dx)[~on] == 0).all()
    assert _kept(buf, loss, loss0) and _kept(dx_buf, dx, dx0) and _kept(dw_buf, dw, dw0)
    # parts of it give the same bits
    loss2, dx2 = torch.empty(t, device="cuda"), torch.empty((t, d), dtype=x.dtype, device="cuda")
    call(loss2, scale=scale)
    assert torch.equal(loss2, loss[0])
    call(loss2, dx=dx2, scale=scale)
    assert torch.equal(dx2, dx) and torch.equal(loss2, loss[0])
    if not acc:
        dw2 = torch.empty((v, d), dtype=TORCH[out], device="cuda")
        call(loss2, dw=dw2, scale=scale)
        assert torch.equal(dw2, dw)


LOSS_SHAPES = [(1, 1, 1, 0, 0), (1, 8, 3, 0, 0), (2, 33, 128, 1, 1), (5, 64, 100, 0, 0),
               (33, 72, 1000, 8, 8), (70, 130, 513, 3, 1), (129, 64, 4097, 0, 0),
               (300, 136, 2050, 2, 1), (40, 1032, 700, 0, 0)]
LOSS_LARGE = [(2048, 64, 8192, 0, 0), (128, 4096, 4096, 0, 0), (1000, 100, 9001, 1, 1)]


@pytest.mark.parametrize("t,d,v,pad,off", LOSS_SHAPES + LOSS_LARGE)
@pytest.mark.parametrize("dtype,out,acc,left_out,weights,ids", [
    ("bf16", "bf16", False, 0.0, False, torch.int64),
    ("fp16", "fp16", True, 0.4, True, torch.int32),
    ("fp16", "fp32", False, 0.2, True, torch.int64),
    ("bf16", "fp32", True, 0.6, False, torch.int32)])
def test_vocab_loss(t, d, v, pad, off, dtype, out, acc, left_out, weights, ids):
    rng = np.random.default_rng(t * 7 + d + v)
    x, w, targets, wt = _loss_inputs(rng, t, d, v, dtype, pad, off, left_out, weights)
    scale = 64.0 / t
    w32 = None if wt is None else wt.astype(np.float32)
    want = layer.vocab_loss(f64(x), f64(w), targets, w32, scale)

    def call(loss, **kw):
        Z.vocab_loss(x, w, _dev(targets, ids), loss, weights=_dev(wt), **kw)

    _check_loss(x, w, wt, call, want, 1.0, scale, dtype, out, acc, pad, off)


def _top(rng, t, v, k, left_out):
    ids = np.stack([rng.permutation(v)[:k] if v >= k else rng.integers(0, v, k)
                    for _ in range(t)])
    ids[rng.random((t, k)) < left_out] = -1
    ids[rng.random(t) < left_out] = -5
    if k > 2:
        ids[:, 2] = np.where(rng.random(t) < 0.5, ids[:, 0], ids[:, 2])   # the same id twice
    logits = 3.0 * rng.standard_normal((t, k))
    if k > 3:
        logits[rng.random(t) < 0.3, 1] = -np.inf
    return ids, logits


@pytest.mark.parametrize("t,d,v,pad,off,k", [
    s + (k,) for s, k in zip(LOSS_SHAPES + LOSS_LARGE, (1, 2, 5, 64, 17, 100, 256, 8, 600, 33, 16,
                                                        50))] + [(6, 40, 3000, 0, 0, 1024)])
@pytest.mark.parametrize("dtype,out,acc,left_out,weights,top,tau", [
    ("bf16", "bf16", False, 0.0, False, "fp32", 1.0),
    ("fp16", "fp16", True, 0.4, True, "bf16", 2.0),
    ("fp16", "fp32", False, 0.2, False, "fp16", 0.7)])
def test_distill_loss(t, d, v, pad, off, k, dtype, out, acc, left_out, weights, top, tau):
    rng = np.random.default_rng(t * 7 + d + v + k)
    x, w, _, wt = _loss_inputs(rng, t, d, v, dtype, pad, off, 0.0, weights)
    ids, logits = _top(rng, t, v, k, left_out)
    if t > 1:
        # -infinity alone is refused by the result, not here: one entry at least
        logits[(ids >= 0).sum(1) == 1] = 1.0
    s_ids, _ = strided((t, k), torch.float32, pad, off)
    ids_dev = torch.empty_strided(s_ids.shape, s_ids.stride(), dtype=torch.int32, device="cuda")
    ids_dev.copy_(torch.from_numpy(ids))
    top_dev = _matrix(rng, t, k, top, pad, off)
    top_dev.copy_(torch.from_numpy(logits).to(TORCH[top]))
    scale = 64.0 / t
    w32 = None if wt is None else wt.astype(np.float32)
    want = layer.distill_loss(f64(x), f64(w), ids, f64(top_dev), float(np.float32(tau)), w32,
                              scale)
    dense = np.zeros((t, v))
    shares = layer.shares_of(ids, f64(top_dev), tau)
    for r in range(t):
        for j in np.flatnonzero(ids[r] >= 0):
            dense[r, ids[r, j]] += shares[r, j]

    def call(loss, **kw):
        Z.distill_loss(x, w, ids_dev, top_dev, loss, temperature=tau, weights=_dev(wt), **kw)

    _check_loss(x, w, wt, call, want, tau, scale, dtype, out, acc, pad, off, dense)


def test_a_token_that_is_learnt_keeps_its_gradient():
    """p at the target within 1e-4 .. 1 of 1: what is left is far below a 16-bit step of
    p, and has to be exact to its own."""
    rng = np.random.default_rng(8)
    t, d, v = 64, 64, 500
    x, w, targets, _ = _loss_inputs(rng, t, d, v, "bf16", 0, 0, 0.0, False)
    lift = np.linspace(1, 5, t)[:, None]
    x.copy_(torch.from_numpy(lift * f64(w)[targets]).to(x.dtype))
    want = layer.vocab_loss(f64(x), f64(w), targets, None, 1.0)
    assert (np.abs(want[1][np.arange(t), targets]) < 1e-3).any()
    call = lambda loss, **kw: Z.vocab_loss(x, w, _dev(targets, torch.int64), loss, **kw)  # noqa: E731
    _check_loss(x, w, None, call, want, 1.0, 1.0, "bf16", "bf16", False, 0, 0)


def test_left_out_tokens_may_hold_anything():
    rng = np.random.default_rng(9)
    t, d, v = 300, 72, 900
    x, w, targets, _ = _loss_inputs(rng, t, d, v, "fp16", 0, 0, 0.5, False)
    wt = np.where(rng.random(t) < 0.2, 0.0, 1.0)
    off = (targets < 0) | (wt == 0)
    got = []
    for fill in (0.0, math.nan, math.inf, -65504.0):
        x[torch.from_numpy(off).cuda()] = fill
        loss, dx, dw = (torch.full(s, 9.0, dtype=dt, device="cuda") for s, dt in
                        (((t,), torch.float32), ((t, d), torch.float16), ((v, d), torch.float16)))
        Z.vocab_loss(x, w, _dev(targets, torch.int64), loss, weights=_dev(wt), dx=dx, dw=dw)
        got.append((loss, dx, dw))
        ids = torch.from_numpy(targets[:, None]).int().cuda()
        dist = [torch.empty_like(v) for v in got[-1]]
        Z.distill_loss(x, w, ids, torch.full((t, 1), math.pi, device="cuda"), dist[0],
                       weights=_dev(wt), dx=dist[1], dw=dist[2])
        # one entry is cross entropy: log 1 = 0 is added
        assert torch.equal(dist[1], dx) and torch.equal(dist[2], dw)
        assert torch.allclose(dist[0], loss, rtol=2.0 ** -21, atol=2.0 ** -20)
    assert (got[0][0][torch.from_numpy(off).cuda()] == 0).all()
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)


def test_no_token_with_a_loss():
    x, w = (torch.ones((n, 24), dtype=torch.bfloat16, device="cuda") for n in (70, 300))
    targets = torch.full((70,), -1, device="cuda")
    loss, dx, dw = (torch.full(s, 9.0, dtype=dt, device="cuda") for s, dt in
                    (((70,), torch.float32), ((70, 24), x.dtype), ((300, 24), x.dtype)))
    Z.vocab_loss(x, w, targets, loss, dx=dx, dw=dw, accumulate=True)
    assert (loss == 0).all() and (dx == 0).all() and (dw == 9).all()
    Z.vocab_loss(x, w, targets, loss, dx=dx, dw=dw)
    assert (dw == 0).all()
    # and no token at all
    none = torch.empty((0, 24), dtype=x.dtype, device="cuda")
    dw.fill_(9)
    Z.vocab_loss(none, w, targets[:0], loss[:0], dw=dw, accumulate=True)
    assert (dw == 9).all()
    Z.vocab_loss(none, w, targets[:0], loss[:0], dx=none, dw=dw)
    assert (dw == 0).all()
    Z.distill_loss(none, w, targets[:0, None].expand(0, 3).contiguous(),
                   torch.empty((0, 3), device="cuda"), loss[:0], dx=none)


@pytest.mark.parametrize("bad", [1000, 1001, 2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 62])
def test_ids_past_the_vocabulary_are_visible_and_read_nothing(bad):
    rng = np.random.default_rng(10)
    x, w, targets, _ = _loss_inputs(rng, 50, 40, 1000, "fp16", 0, 0, 0.0, False)
    good = [torch.empty(s, dtype=dt, device="cuda") for s, dt in
            (((50,), torch.float32), ((50, 40), torch.float16))]
    Z.vocab_loss(x, w, _dev(targets, torch.int64), good[0], dx=good[1])
    targets[7] = bad
    loss, dx, dw = torch.empty_like(good[0]), torch.empty_like(good[1]), torch.empty_like(w)
    rest = [i for i in range(50) if i != 7]
    Z.vocab_loss(x, w, _dev(targets, torch.int64), loss, dx=dx, dw=dw)
    ids = torch.from_numpy(targets[:, None]).cuda().repeat(1, 2)
    ids[:, 1] = -1
    for _ in range(2):
        assert loss[7].isnan() and dx[7].isnan().all() and dw.isnan().all()
        assert torch.allclose(loss[rest], good[0][rest], rtol=2.0 ** -21, atol=2.0 ** -20)
        assert torch.equal(dx[rest], good[1][rest])
        Z.distill_loss(x, w, ids, torch.zeros((50, 2), device="cuda"), loss, dx=dx, dw=dw)


def test_teachers_without_a_softmax_are_visible():
    rng = np.random.default_rng(12)
    x, w, _, _ = _loss_inputs(rng, 4, 40, 100, "bf16", 0, 0, 0.0, False)
    ids = torch.tensor([[1, 2], [3, 4], [5, 6], [7, -1]], device="cuda")
    top = torch.tensor([[math.nan, 0.0], [math.inf, 0.0], [-math.inf, -math.inf],
                        [0.0, math.nan]], device="cuda")
    loss, dx = torch.empty(4, device="cuda"), torch.empty_like(x)
    Z.distill_loss(x, w, ids, top, loss, dx=dx)
    assert loss[:3].isnan().all() and dx[:3].isnan().any(1).all()
    assert loss[3].isfinite() and dx[3].isfinite().all()      # its NaN is no entry


@pytest.mark.parametrize("spread", [1e-6, 1.0, 3e4])
def test_weights_of_any_size(spread):
    """fp16's range: the largest weight's power of two is taken out before the rounding."""
    rng = np.random.default_rng(13)
    t, d, v = 40, 64, 700
    x, w, targets, _ = _loss_inputs(rng, t, d, v, "fp16", 0, 0, 0.1, False)
    wt = spread * (0.25 + rng.random(t))
    scale = 100.0 / spread / t
    want = layer.vocab_loss(f64(x), f64(w), targets, wt.astype(np.float32), scale)
    call = lambda loss, **kw: Z.vocab_loss(x, w, _dev(targets, torch.int64), loss,  # noqa: E731
                                           weights=_dev(wt), **kw)
    _check_loss(x, w, wt, call, want, 1.0, scale, "fp16", "fp16", False, 0, 0)


def _reference(x, w, targets, scale):
    """(loss, dx, dw) in 64 bits on the device, 512 tokens at a time."""
    x, w = x.double(), w.double()
    loss, dx, dw = x.new_zeros(x.shape[0]), torch.zeros_like(x), torch.zeros_like(w)
    on = torch.nonzero(targets >= 0)[:, 0]
    for at in on.split(512):
        z = x[at] @ w.t()
        log_p = z - torch.logsumexp(z, 1, keepdim=True)
        y = targets[at, None]
        loss[at] = -log_p.gather(1, y)[:, 0]
        dz = torch.exp(log_p).scatter_add_(1, y, -torch.ones_like(y, dtype=torch.float64))
        dx[at] = scale * (dz @ w)
        dw += scale * (dz.t().contiguous() @ x[at])
    return loss, dx, dw


@pytest.mark.parametrize("left_out", [0.0, 0.3])
def test_several_pieces_of_tokens(left_out):
    """More logits than a piece holds: the pieces' sums of dw are joined in fp32."""
    t, d, v = 27000, 48, 131075
    assert t * v * 4 > 2 * 6 * 2 ** 30
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    x = torch.randn((t, d), generator=gen, device="cuda").bfloat16()
    w = (0.3 * torch.randn((v, d), generator=gen, device="cuda")).bfloat16()
    targets = torch.randint(0, v, (t,), generator=gen, device="cuda")
    targets[torch.rand(t, generator=gen, device="cuda") < left_out] = -1
    dw0 = torch.randn((v, d), generator=gen, device="cuda").bfloat16()
    loss, dx, dw = torch.empty(t, device="cuda"), torch.empty_like(x), dw0.clone()
    Z.vocab_loss(x, w, targets, loss, scale=0.5, dx=dx, dw=dw, accumulate=True)
    want = _reference(x, w, targets, 0.5)
    # products of 48 terms of about 0.3, a sum over v of equal ones: far inside these
    assert (loss.double() - want[0]).abs().max() < 2e-5
    # |d| <= 1: half a step of bf16 of it, and of the result
    for got, ref, mag in ((dx, want[1], 0.5 * 2 * 0.3 * 6), (dw, want[2] + dw0.double(), 0.5 * 5)):
        assert ((got.double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + mag)).all()
    rel = (dw.double() - want[2] - dw0.double()).norm() / (want[2] + dw0.double()).norm()
    assert rel < 2.0 ** -8


def test_losses_past_32_bits():
    """Rows more than 2^31 bytes apart in x, w, dx and dw."""
    t, d, v, stride = 3, 40, 50, (1 << 30) + 8
    big = torch.empty(v * stride + 4096, dtype=torch.float16, device="cuda")
    far = [big.as_strided((n, d), (s, 1), o) for n, s, o in
           ((t, 9 * stride, 0), (v, stride, 64), (t, 9 * stride, 128), (v, stride, 192))]
    rng = np.random.default_rng(1)
    for m in far:
        m.copy_(torch.from_numpy(rng.standard_normal(m.shape) * 0.3).half())
    near = [m.clone() for m in far]
    targets = torch.tensor([4, -1, 49], device="cuda")
    got = []
    for x, w, dx, dw in (far, near):
        loss = torch.empty(t, device="cuda")
        Z.vocab_loss(x, w, targets, loss, dx=dx, dw=dw, accumulate=True)
        got.append((loss, dx, dw))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_loss_gradients_are_differences():
    """Along a direction of x and of w whose steps 16 bits hold exactly.  A token's loss
    has third derivatives of at most 2 (its logits' largest change)^3."""
    rng = np.random.default_rng(14)
    t, d, v, h = 12, 16, 60, 2.0 ** -6
    x, w = rng.integers(-64, 65, (t, d)) / 64.0, rng.integers(-64, 65, (v, d)) / 128.0
    rx, rw = rng.choice([-1.0, 1.0], (t, d)), rng.choice([-0.5, 0.5], (v, d))
    targets, scale = rng.integers(0, v, t), 4.0

    def dev(m):
        return torch.from_numpy(m).half().cuda()

    def value(a, b):
        loss = torch.empty(t, device="cuda")
        Z.vocab_loss(dev(a), dev(b), _dev(targets, torch.int64), loss)
        return scale * f64(loss).sum()

    loss, dx, dw = torch.empty(t, device="cuda"), dev(x), dev(w)
    Z.vocab_loss(dev(x), dev(w), _dev(targets, torch.int64), loss, scale=scale, dx=dx, dw=dw)
    for g, r, up, down, change in (
            (dx, rx, (x + h * rx, w), (x - h * rx, w), rx @ w.T),
            (dw, rw, (x, w + h * rw), (x, w - h * rw), x @ rw.T)):
        got = (f64(g) * r).sum()
        third = 2 * np.abs(2 * change).max(axis=1) ** 3
        slack = (scale * third.sum() * h * h / 6 + 2 * scale * t * 64 * 2.0 ** -24 * 8 / (2 * h)
                 + 2 * EPS["fp16"] * 4 * np.abs(f64(g) * r).sum() + 1e-3)
        assert abs((value(*up) - value(*down)) / (2 * h) - got) < slack


def test_the_same_bits_each_time():
    rng = np.random.default_rng(15)
    x, w, targets, wt = _loss_inputs(rng, 700, 264, 5003, "fp16", 0, 0, 0.3, True)
    got = []
    for _ in range(3):
        loss, dx, dw = torch.empty(700, device="cuda"), torch.empty_like(x), torch.empty_like(w)
        Z.vocab_loss(x, w, _dev(targets, torch.int64), loss, weights=_dev(wt), dx=dx, dw=dw)
        got.append((loss, dx, dw))
    for other in got[1:]:
        for a, b in zip(got[0], other):
            assert torch.equal(a, b)


def test_infinite_and_nan_logits_are_visible():
    rng = np.random.default_rng(16)
    x, w, targets, _ = _loss_inputs(rng, 20, 40, 300, "bf16", 0, 0, 0.0, False)
    x[3, 0], x[11, 5] = math.nan, math.inf
    loss, dx = torch.empty(20, device="cuda"), torch.empty_like(x)
    Z.vocab_loss(x, w, _dev(targets, torch.int64), loss, dx=dx)
    rest = [i for i in range(20) if i not in (3, 11)]
    assert loss[3].isnan() and loss[11].isnan() and dx[3].isnan().all()
    assert loss[rest].isfinite().all() and dx[rest].isfinite().all()
