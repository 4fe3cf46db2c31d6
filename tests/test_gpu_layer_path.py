"""The gated block and the losses together with the rest of a rank's step: a layer's
forward with 8-bit checkpoints, the loss over the vocabulary, the backward through the
norms and the block into the local gradients, then the reduce and Adam; streams,
captured graphs and calls that the binding refuses."""
import numpy as np
import pytest
import torch

import zero_sharded_mixed_bucketed_amd as Z
from act_util import acts, f64
from gpu_util import assert_bits, f32, need_gpu, u16
from oracle import act as oact
from oracle import adam as oadam
from oracle import layer as olayer
from oracle import reduce as ored
from zero_sharded_mixed_bucketed_amd import rank as zr

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    print(flush=True)


T, H, F, V = 96, 160, 200, 1000
PLACES = {"w_pre": (0, H), "w_ffn": (H, 2 * F * H), "w_down": (H + 2 * F * H, H * F),
          "w_last": (H + 3 * F * H, H), "w_vocab": (2 * H + 3 * F * H, V * H)}
PSI = 2 * H + 3 * F * H + V * H


def _param(flat, name, *shape):
    lo, n = PLACES[name]
    return flat[lo:lo + n].view(*shape) if shape else flat[lo:lo + n]


def _params(rng):
    p = torch.from_numpy(rng.standard_normal(PSI)).half()
    for name, sigma in (("w_ffn", H ** -0.5), ("w_down", F ** -0.5), ("w_vocab", 2 * H ** -0.5)):
        _param(p, name).mul_(sigma)
    for name in ("w_pre", "w_last"):
        _param(p, name).mul_(0.1).add_(1.0)
    return p.cuda()


def _buffers(st):
    def new(*shape):
        return torch.empty(shape, dtype=torch.float16, device="cuda")

    s = {n: new(T, H) for n in ("h1", "z1", "h2", "z2", "y", "dz2", "dh", "dz1", "dblock", "dh0")}
    s.update(a=new(T, F), da=new(T, F), stats1=torch.empty((T, 4), device="cuda"),
             stats2=torch.empty((T, 4), device="cuda"), loss=torch.empty(T, device="cuda"))
    for n, width in (("kh1", H), ("kz1", H), ("kg", F), ("ku", F), ("ka", F), ("ky", H),
                     ("kh2", H)):
        s[n] = st.checkpoint(T, width)
    return s


def _step(st, s, p, h0, targets, bucket=None, teacher=None):
    """h1 = h0; z1 = rms(h1); a = gated(z1); y = a Wd^T; h2 = h1 + y; z2 = rms(h2); the
    loss of z2; and back, with every parameter's gradient in the local gradient."""
    pre, last = (Z.Norm(Z.NORM_RMS, 1e-5, _param(p, n)) for n in ("w_pre", "w_last"))
    w_ffn, w_down = _param(p, "w_ffn", 2 * F, H), _param(p, "w_down", H, F)
    w_vocab = _param(p, "w_vocab", V, H)
    Z.block_norm(h0, None, s["h1"], s["z1"], s["stats1"], pre=pre, ckpt_out=s["kh1"],
                 ckpt_z=s["kz1"])
    Z.gated_ffn(s["z1"], w_ffn, s["a"], Z.ACT_SILU, s["kg"], s["ku"], s["ka"])
    s["y"].copy_(s["a"].float() @ w_down.float().t())
    Z.block_norm(s["h1"], s["y"], s["h2"], s["z2"], s["stats2"], pre=last, ckpt_out=s["kh2"])
    if teacher is None:
        st.loss_grad(PLACES["w_vocab"][0], s["z2"], w_vocab, targets, s["loss"], dx=s["dz2"],
                     bucket=bucket, scale=8.0)
    else:
        st.distill_grad(PLACES["w_vocab"][0], s["z2"], w_vocab, *teacher, s["loss"], dx=s["dz2"],
                        bucket=bucket, scale=8.0, temperature=2.0)
    st.norm_grad({"dw_pre": PLACES["w_last"][0]}, None, s["dz2"], s["kh2"], None, s["stats2"],
                 bucket=bucket, pre=last, dres=s["dh"])
    st.linear_grad(PLACES["w_down"][0], s["ka"], s["dh"], bucket=bucket)
    s["da"].copy_(s["dh"].float() @ w_down.float())
    st.gated_grad(PLACES["w_ffn"][0], s["da"], s["kg"], s["ku"], s["kz1"], w_ffn, Z.ACT_SILU,
                  dx=s["dz1"], bucket=bucket)
    st.norm_grad({"dw_pre": PLACES["w_pre"][0]}, s["dh"], s["dz1"], s["kh1"], None, s["stats1"],
                 bucket=bucket, pre=pre, dres=s["dh0"])


def _inputs(rng):
    h0 = acts(rng, T, H, "fp16")
    targets = torch.from_numpy(rng.integers(0, V, T)).cuda()
    targets[rng.random(T) < 0.3] = -1
    ids = torch.from_numpy(rng.permuted(np.tile(np.arange(V), (T, 1)), axis=1)[:, :20].copy()).cuda()
    ids[targets < 0] = -1
    return h0, targets, (ids, torch.from_numpy(rng.standard_normal((T, 20))).half().cuda())


def _held(k, fmt="int8"):
    return oact.held(k.codes.cpu().numpy(), k.scales.cpu().numpy(), fmt)


def _near(got, want, what):
    """Each stage from the inputs that the kernel had: one rounding to fp16 of an
    intermediate and one of the result, and fp32 sums whose roundings (2^-24 a term, a
    thousand terms) stay below 2^-14 of the largest value."""
    err = np.abs(f64(got) - want)
    tol = 2.0 ** -10 * np.abs(want) + 2.0 ** -12 * np.abs(want).max() + 2.0 ** -24
    assert (err <= tol).all(), (what, float((err / tol).max()))


@pytest.mark.parametrize("stage,distil", [(1, False), (2, True), (3, False)])
def test_a_layer_and_its_loss_into_the_local_gradients_then_reduce_and_adam(stage, distil):
    nd, rank = 3, 1
    rng = np.random.default_rng(20 + stage)
    p = _params(rng)
    rows = torch.zeros((nd, PSI), dtype=torch.int16, device="cuda")
    st = zr.RankState(PSI, nd, rank, stage, local_grad=rows[rank] if stage == 1 else None)
    for k in range(nd):
        peer = st if k == rank else zr.RankState(PSI, nd, k, stage,
                                                 local_grad=rows[k] if stage == 1 else None)
        h0, targets, teacher = _inputs(rng)
        s = _buffers(peer)
        _step(peer, s, p, h0, targets, bucket=None if stage == 1 else rows[k],
              teacher=teacher if distil else None)
        torch.cuda.synchronize()
        g = rows[k].view(torch.float16)
        w_ffn, w_vocab = f64(_param(p, "w_ffn", 2 * F, H)), f64(_param(p, "w_vocab", V, H))
        out, gate, up = olayer.gated(f64(s["z1"]), w_ffn, "silu")
        _near(s["a"], out, "a")
        for kk, v in ((s["kg"], gate), (s["ku"], up), (s["ka"], out)):
            # int8 codes: half a step of a block's largest, 2^-7 of it at most, and fp16's own
            assert (np.abs(_held(kk) - v) <= 2.0 ** -7 * np.abs(v).max(1, keepdims=True) * 1.01
                    + 2.0 ** -11 * np.abs(v)).all()
        if distil:
            want = olayer.distill_loss(f64(s["z2"]), w_vocab, teacher[0].cpu().numpy(),
                                       f64(teacher[1]), 2.0, None, 8.0)
        else:
            want = olayer.vocab_loss(f64(s["z2"]), w_vocab, targets.cpu().numpy(), None, 8.0)
        assert np.abs(f64(s["loss"]) - want[0]).max() < 1e-4
        _near(s["dz2"], want[2], "dz2")
        _near(_param(g, "w_vocab", V, H), want[3], "w_vocab")
        dx, dw = olayer.gated_grad(f64(s["da"]), _held(s["kz1"]), _held(s["kg"]), _held(s["ku"]),
                                   w_ffn, "silu")
        _near(s["dz1"], dx, "dz1")
        _near(_param(g, "w_ffn", 2 * F, H), dw, "w_ffn")
        assert (g != 0).float().mean() > 0.95
    lo, n = st.geom.offset, st.geom.len
    local = u16(rows)
    st.master.copy_(p[lo:lo + n])
    st.reduce_bucket(0, PSI, rows)
    st.adam_step(1e-3, 0.9, 0.999, 1e-8, 1)
    torch.cuda.synchronize()
    g16 = ored.reduce_values(local[:, lo:lo + n], nd).astype(np.float16)
    assert_bits(u16(st.grad), g16.view(np.uint16), "reduced gradient")
    z = np.zeros(n, np.float32)
    th = oadam.step_values(f32(p[lo:lo + n]), z, z, g16.astype(np.float32),
                           oadam.scalars(1e-3, 0.9, 0.999, 1e-8, 1))[0]
    assert_bits(f32(st.master), th, "master")


@pytest.mark.parametrize("distil", [False, True])
def test_captured_steps_replay_as_the_eager_step(distil):
    """Two graphs of the same buffers, replayed in turn with other work between."""
    rng = np.random.default_rng(30)
    p = _params(rng)
    st = zr.RankState(PSI, 2, 0, 1)
    h0, targets, teacher = _inputs(rng)
    s = _buffers(st)
    args = (st, s, p, h0, targets, None, teacher if distil else None)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _step(*args)
    side.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _step(*args)
        graphs.append(g)
    for i in range(6):
        h0.copy_(acts(rng, T, H, "fp16"))
        targets.copy_(torch.from_numpy(rng.integers(-50, V, T)).cuda())
        _step(*args)
        torch.cuda.synchronize()
        want = [st.local_grad.clone(), s["loss"].clone(), s["dh0"].clone()]
        for v in (st.local_grad, s["loss"], s["dh0"]):
            v.zero_()
        graphs[i % 2].replay()
        _ = torch.randn(1000, device="cuda").sum().item()
        for a, b in zip(want, (st.local_grad, s["loss"], s["dh0"])):
            assert torch.equal(a, b)


def test_two_streams_at_once_match_one_after_the_other():
    rng = np.random.default_rng(31)
    t, d, v = 1500, 256, 6000
    xs = [acts(rng, t, d, "fp16") for _ in range(2)]
    w = torch.from_numpy(0.1 * rng.standard_normal((v, d))).half().cuda()
    targets = torch.from_numpy(rng.integers(-1000, v, t)).cuda()
    w2 = torch.from_numpy(0.1 * rng.standard_normal((2 * d, d))).half().cuda()

    def run(x, stream):
        loss = torch.empty(t, device="cuda")
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        ks = [Z.ckpt_empty(t, d) for _ in range(3)]
        out, dx2, dw2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w2)
        torch.cuda.synchronize()
        Z.vocab_loss(x, w, targets, loss, dx=dx, dw=dw, stream=stream)
        Z.ckpt_write(x, ks[0], stream=stream)
        Z.gated_ffn(x, w2, out, Z.ACT_GELU, ks[1], ks[2], stream=stream)
        Z.gated_ffn_grad(dx, ks[1], ks[2], w2, Z.ACT_GELU, dx=dx2, ckpt_x=ks[0], dw=dw2,
                         stream=stream)
        return loss, dx, dw, out, dx2, dw2

    want = [run(x, None) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        got = [run(x, s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_given_workspaces_are_used_and_small_ones_refused():
    rng = np.random.default_rng(32)
    x, w = acts(rng, 60, 64, "fp16"), acts(rng, 500, 64, "fp16")
    targets = torch.from_numpy(rng.integers(0, 500, 60)).cuda()
    need = Z.loss_workspace(60, 64, 500)
    ws = torch.zeros(need + 64, dtype=torch.uint8, device="cuda")
    loss, dx, dw = torch.empty(60, device="cuda"), torch.empty_like(x), torch.empty_like(w)
    Z.vocab_loss(x, w, targets, loss, dx=dx, dw=dw, workspace=ws[:need])
    assert ws[:need].any() and not ws[need:].any()
    with pytest.raises(ValueError):
        Z.vocab_loss(x, w, targets, loss, dx=dx, dw=dw, workspace=ws[:need - 1])
    with pytest.raises(ValueError):
        Z.vocab_loss(x, w, targets, loss, dx=dx, dw=dw, workspace=ws[:need].cpu())
    k, kx = [Z.ckpt_empty(60, 32) for _ in range(2)], Z.ckpt_empty(60, 64)
    Z.ckpt_write(x, kx)
    out = torch.empty((60, 32), dtype=torch.float16, device="cuda")
    Z.gated_ffn(x, w[:64], out, ckpt_gate=k[0], ckpt_up=k[1])
    need = Z.gated_ffn_grad_workspace(60, 64, 32)
    ws.zero_()
    Z.gated_ffn_grad(out, *k, w[:64], dx=dx, ckpt_x=kx, dw=dw[:64], workspace=ws[:need])
    assert ws[:need].any() and not ws[need:].any()
    with pytest.raises(ValueError):
        Z.gated_ffn_grad(out, *k, w[:64], dx=dx, workspace=ws[:need - 1])


def test_binding_refuses_what_the_kernels_do_not_take():
    def m(t, h, dt=torch.float16):
        return torch.zeros((t, h), dtype=dt, device="cuda")

    x, w, out = m(4, 8), m(12, 8), m(4, 6)
    loss, ids = torch.zeros(4, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    k = Z.ckpt_empty(4, 6)
    bad_gated = [(m(4, 8, torch.float32), w, out), (x, m(12, 8, torch.bfloat16), out),
                 (x, m(11, 8), out), (x, m(12, 9), out), (x, w, m(4, 7)), (x, w, m(5, 6)),
                 (x.t(), w, out), (x[0], w, out)]
    for args in bad_gated:
        with pytest.raises((ValueError, Z.ZeroError)):
            Z.gated_ffn(*args)
    for kw in (dict(act=7), dict(ckpt_gate=Z.ckpt_empty(4, 7)),
               dict(ckpt_gate=k, ckpt_up=Z.ckpt_empty(4, 6, Z.CKPT_E4M3))):
        with pytest.raises(Z.ZeroError):
            Z.gated_ffn(x, w, out, **kw)
    for kw in (dict(), dict(dx=m(4, 9)), dict(dx=x.float()), dict(dw=m(12, 8, torch.bfloat16))):
        with pytest.raises((ValueError, Z.ZeroError)):
            Z.gated_ffn_grad(out, k, k, w, **kw)
    with pytest.raises(ValueError):
        Z.gated_ffn_grad(out, k, k, None, dx=m(4, 8))
    for args in ((x, m(9, 7), ids, loss), (x, w, ids[:3], loss), (x, w, ids, loss[:3]),
                 (x, w, ids.float(), loss), (x, w, ids.cpu(), loss), (x, w, ids, loss.double()),
                 (x.float(), w, ids, loss), (x, w, ids[None], loss)):
        with pytest.raises(ValueError):
            Z.vocab_loss(*args)
    for kw in (dict(weights=loss[:3]), dict(weights=loss.double()), dict(dx=m(4, 9)),
               dict(dw=m(11, 8)), dict(dw=m(12, 8, torch.bfloat16))):
        with pytest.raises(ValueError):
            Z.vocab_loss(x, w, ids, loss, **kw)
    two, top = ids[:, None].repeat(1, 2), m(4, 2)
    for args in ((x, w, two[:3], top[:3], loss), (x, w, two, m(4, 3), loss),
                 (x, w, two, top.double(), loss), (x, w, ids, top, loss)):
        with pytest.raises(ValueError):
            Z.distill_loss(*args)
    for kw in (dict(temperature=0.0), dict(temperature=float("nan")), dict(scale=float("inf"))):
        with pytest.raises(Z.ZeroError):
            Z.distill_loss(x, w, two, top, loss, **kw)
