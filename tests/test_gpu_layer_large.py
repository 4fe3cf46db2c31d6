"""The gated block and the losses at sizes whose products take whole large tiles, several of
them a workgroup, and splits by the rows that are counted, against 64-bit results on the
device.  Bounds as in layer_util."""
import pytest
import torch

import zero_sharded_mixed_bucketed_amd as Z
from act_util import EPS, TINY, TORCH, U
from gpu_util import need_gpu
from layer_util import product

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    print(flush=True)


def _normal(gen, shape, dtype, sigma=1.0, pad=0):
    full = torch.empty((shape[0], shape[1] + pad), dtype=TORCH[dtype], device="cuda")
    view = full[:, :shape[1]]
    view.copy_(sigma * torch.randn(shape, generator=gen, device="cuda"))
    return view


def _rounded(ref, err, dtype):
    """The bound of a result that is rounded to dtype."""
    return err + EPS[dtype] * (ref.abs() + err) + TINY[dtype] if dtype != "fp32" else err + U * ref.abs()


def _check(got, ref, bound):
    off = (got.double() - ref).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (int(bad.sum()), torch.nonzero(bad)[0], off[bad][0], bound[bad][0])


# (tokens, cols, words): the logits in tiles of 256, 128, 128, 32 and 256 rows; dx of 128 with
# splits, 256, 128 with splits, 32 with splits and 128; dw of 256, 256 with splits, 256, 128
# and 128 with splits
@pytest.mark.parametrize("t,d,v", [(3000, 512, 20000), (8192, 2048, 4104), (1300, 1024, 16384),
                                   (100, 512, 8192), (9000, 2056, 1024)])
@pytest.mark.parametrize("dtype,out,acc,left_out,weights,pad", [
    ("bf16", "bf16", False, 0.0, False, 0), ("fp16", "fp32", True, 0.7, True, 8),
    ("fp16", "fp16", True, 0.2, False, 0), ("bf16", "fp32", False, 0.97, True, 16)])
def test_vocab_loss_of_large_products(t, d, v, dtype, out, acc, left_out, weights, pad):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(t + v)
    scale = 0.75
    x, w = _normal(gen, (t, d), dtype, 1.0, pad), _normal(gen, (v, d), dtype, 2 * d ** -0.5, pad)
    y = torch.randint(0, v, (t,), generator=gen, device="cuda")
    y[torch.rand(t, generator=gen, device="cuda") < left_out] = -1
    wt = torch.randn(t, generator=gen, device="cuda").abs() + 0.1 if weights else None
    dw0 = _normal(gen, (v, d), out, 0.5, pad) if acc else torch.full((v, d), float("nan"),
                                                                     dtype=TORCH[out], device="cuda")
    loss = torch.full((t,), float("nan"), device="cuda")
    dx = torch.full((t, d + pad), float("nan"), dtype=TORCH[dtype], device="cuda")[:, :d]
    dw = dw0.clone()
    Z.vocab_loss(x, w, y, loss, weights=wt, scale=scale, dx=dx, dw=dw, accumulate=acc)

    on = torch.nonzero(y >= 0)[:, 0]
    x64, w64, yo = x[on].double(), w.double(), y[on, None]
    w1 = (wt[on].double() if weights else torch.ones(len(on), device="cuda", dtype=torch.float64))[:, None]
    z = x64 @ w64.t()
    lse = torch.logsumexp(z, 1, keepdim=True)
    loss64 = w1[:, 0] * (lse - z.gather(1, yo))[:, 0]
    p = torch.exp(z - lse)
    d64 = (w1 * p).scatter_add_(1, yo, -w1)
    dz = (product(d, x64.abs() @ w64.abs().t()) + 2 * U * z.abs()).amax(1, keepdim=True)
    far = z.amax(1, keepdim=True) - z
    rel = 2 * dz + (v / 512 + 80 + 4 * far.clamp(max=90.0)) * U
    err = w1 * (p * rel + 2 * U * (p + d64.abs() / w1))
    held = 2.0 ** -13 * (wt.max().item() if weights else 1.0) if dtype == "fp16" else 1.0
    err = err + EPS[dtype] * (d64.abs() + err) + TINY[dtype] * held
    loss_err = (w1[:, 0] * (2 * dz[:, 0] + (v / 512 + 80) * U
                            + 16 * U * (z.abs().amax(1) + torch.log(torch.tensor(float(v))).item() + 1))
                + 16 * U * loss64.abs())
    mag = d64.abs() + err
    off = y < 0
    assert (loss[off] == 0).all() and (dx[off] == 0).all()
    _check(loss[on], loss64, loss_err)
    ref = scale * (d64 @ w64)
    bound = scale * (err @ w64.abs() + product(v, mag @ w64.abs()))
    _check(dx[on], ref, _rounded(ref, bound * (1 + 4 * U), dtype))
    ref = scale * (d64.t().contiguous() @ x64)
    bound = scale * (err.t().contiguous() @ x64.abs() + product(len(on), mag.t().contiguous() @ x64.abs()))
    if acc:
        ref += dw0.double()
    _check(dw, ref, _rounded(ref, bound * (1 + 4 * U) + U * ref.abs(), out))


@pytest.mark.parametrize("t,d,f", [(2304, 520, 4112), (1024, 2048, 4096), (32, 2056, 5000)])
@pytest.mark.parametrize("dtype,out,acc", [("bf16", "fp32", True), ("fp16", "fp16", False),
                                           ("bf16", "bf16", True)])
def test_gated_block_of_large_products(t, d, f, dtype, out, acc):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(t + f)
    x, w = _normal(gen, (t, d), dtype), _normal(gen, (2 * f, d), dtype, d ** -0.5)
    a = torch.empty((t, f), dtype=TORCH[dtype], device="cuda")
    kx, kg, ku = (Z.ckpt_empty(t, c) for c in (d, f, f))
    Z.ckpt_write(x, kx)
    Z.gated_ffn(x, w, a, Z.ACT_SILU, ckpt_gate=kg, ckpt_up=ku)
    x64, w64 = x.double(), w.double()
    g, u = x64 @ w64[:f].t(), x64 @ w64[f:].t()
    s = torch.sigmoid(g)
    dg, du = (product(d, x64.abs() @ m.abs().t()) for m in (w64[:f], w64[f:]))
    ref = g * s * u
    err = (1.13 * dg * (u.abs() + du) + (g * s).abs() * du + (16 + 4 * g.abs()) * U * ref.abs()
           + 2.0 ** -125 * (g * u).abs())
    _check(a, ref, _rounded(ref, err, dtype))

    # the backward, from what the checkpoints hold
    held = []
    for k in (kx, kg, ku):
        scale = torch.ldexp(torch.ones((), device="cuda", dtype=torch.float64), k.scales.int() - 127)
        held.append(k.codes.view(torch.int8).double() * scale.repeat_interleave(32, 1)[:, :k.cols])
    xh, g, u = held
    dout = _normal(gen, (t, f), dtype)
    dw0 = _normal(gen, (2 * f, d), out, 0.5)
    dx, dw = torch.empty_like(x), dw0.clone()
    Z.gated_ffn_grad(dout, kg, ku, w, Z.ACT_SILU, dx=dx, ckpt_x=kx, dw=dw, accumulate=acc)
    d64, s = dout.double(), torch.sigmoid(g)
    slopes = torch.cat([d64 * u * (s + g * s * (1 - s)), d64 * g * s], 1)
    k = (16 + 4 * g.abs()) * U * d64.abs()
    err = torch.cat([k * u.abs() * (1 + g.abs()) * s, k * g.abs() * s], 1)
    err = err + EPS[dtype] * (slopes.abs() + err) + TINY[dtype]
    mag = slopes.abs() + err
    ref = slopes @ w64
    _check(dx, ref, _rounded(ref, err @ w64.abs() + product(2 * f, mag @ w64.abs()), dtype))
    ref = slopes.t().contiguous() @ xh
    bound = err.t().contiguous() @ xh.abs() + product(t, mag.t().contiguous() @ xh.abs())
    if acc:
        ref += dw0.double()
    _check(dw, ref, _rounded(ref, bound + U * ref.abs(), out))
