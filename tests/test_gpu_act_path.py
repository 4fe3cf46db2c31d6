"""The activation entry points together and with the rest of a rank's step: a
layer's forward that keeps 8-bit checkpoints, its backward from them into the Nd
ranks' local gradients, then the reduce and Adam; checkpoints partitioned over a
group; streams, captured graphs and calls that the binding refuses."""
import numpy as np
import pytest
import torch

import zero_sharded_mixed_bucketed_amd as Z
from act_util import EPS, U, acts, close, f64
from gpu_util import assert_bits, f32, need_gpu, u16
from oracle import act as oact
from oracle import adam as oadam
from oracle import reduce as ored
from zero_sharded_mixed_bucketed_amd import rank as zr

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    print(flush=True)


T, H, N = 96, 160, 224
TENSORS = {"w_post": H, "w_pre": H, "linear": N * H}         # flat, in this order
PSI = sum(TENSORS.values())
FLAT = {"w_post": 0, "w_pre": H, "linear": 2 * H}


def _layer(st, rng, params, bucket=None, fmt=Z.CKPT_INT8):
    """One rank's forward and backward of out = h + post(b), z = pre(out), y = z W^T
    with a random upstream gradient; the parameters' gradients go to the local
    gradient.  Returns what the oracle needs."""
    h, b = acts(rng, T, H, "fp16"), acts(rng, T, H, "fp16")
    out, z = torch.empty_like(h), torch.empty_like(h)
    stats = torch.empty((T, 4), dtype=torch.float32, device="cuda")
    norms = dict(post=Z.Norm(Z.NORM_RMS, 1e-5, params[:H]),
                 pre=Z.Norm(Z.NORM_RMS, 1e-5, params[H:2 * H]))
    ks = {n: st.checkpoint(T, H, fmt) for n in ("ckpt_block", "ckpt_out", "ckpt_z")}
    Z.block_norm(h, b, out, z, stats, **norms, **ks)
    dy = acts(rng, T, N, "fp16", sigma=0.02)
    dout = acts(rng, T, H, "fp16", sigma=0.02)
    dz = (dy.float() @ params[2 * H:].view(N, H).float()).half()
    dres, dblock = torch.empty_like(h), torch.empty_like(h)
    st.linear_grad(FLAT["linear"], ks["ckpt_z"], dy, bucket=bucket)
    st.norm_grad({"dw_post": FLAT["w_post"], "dw_pre": FLAT["w_pre"]}, dout, dz, ks["ckpt_out"],
                 ks["ckpt_block"], stats, bucket=bucket, dres=dres, dblock=dblock, **norms)
    return dict(h=h, b=b, out=out, z=z, stats=stats, dy=dy, dout=dout, dz=dz, dres=dres,
                dblock=dblock, ks=ks)


def _held(x, fmt="int8"):
    return oact.held(*oact.store(f64(x), fmt, "fp16"), fmt)


@pytest.mark.parametrize("stage", [1, 2, 3])
def test_layer_into_the_local_gradients_then_reduce_and_adam(stage):
    nd, rank = 3, 1
    rng = np.random.default_rng(stage)
    params = torch.from_numpy(1 + 0.1 * rng.standard_normal(PSI)).half().cuda()
    params[2 * H:] *= 0.05
    rows = torch.zeros((nd, PSI), dtype=torch.int16, device="cuda")
    st = zr.RankState(PSI, nd, rank, stage, local_grad=rows[rank] if stage == 1 else None)
    for k in range(nd):
        peer = st if k == rank else zr.RankState(PSI, nd, k, stage,
                                                 local_grad=rows[k] if stage == 1 else None)
        r = _layer(peer, rng, params, bucket=None if stage == 1 else rows[k])
        torch.cuda.synchronize()
        g = rows[k].view(torch.float16)
        hz, dyv = _held(r["z"]), f64(r["dy"])
        close(f64(g[2 * H:].view(N, H)), oact.weight_grad(dyv, hz),
              (T + 32) * 2 * U * (np.abs(dyv).T @ np.abs(hz)), "fp16", "linear")
        norm = {n: ("rms", 1e-5, f64(params[FLAT["w_" + n]:FLAT["w_" + n] + H]), None)
                for n in ("post", "pre")}
        want = oact.block_norm_grad(f64(r["dout"]), f64(r["dz"]), _held(r["out"]),
                                    _held(r["b"]), f64(r["stats"]), norm["post"], norm["pre"])
        # 16-bit outputs: their half step covers the fp32 arithmetic unless terms
        # cancel, for which 2^-14 of the largest value is 2^10 fp32 roundings
        for name, got in (("dres", r["dres"]), ("dblock", r["dblock"]),
                          ("dw_post", g[:H]), ("dw_pre", g[H:2 * H])):
            close(f64(got), want[name], 2.0 ** -14 * np.abs(want[name]).max(), "fp16", name)
    # the owner's reduce and Adam on what the backward left
    lo, n = st.geom.offset, st.geom.len
    local = u16(rows)
    st.master.copy_(params[lo:lo + n])
    st.reduce_bucket(0, PSI, rows)
    st.adam_step(1e-3, 0.9, 0.999, 1e-8, 1)
    torch.cuda.synchronize()
    g16 = ored.reduce_values(local[:, lo:lo + n], nd).astype(np.float16)
    assert_bits(u16(st.grad), g16.view(np.uint16), "reduced gradient")
    z = np.zeros(n, np.float32)
    th, m, v, p16 = oadam.step_values(f32(params[lo:lo + n]), z, z, g16.astype(np.float32),
                                      oadam.scalars(1e-3, 0.9, 0.999, 1e-8, 1))
    assert_bits(f32(st.master), th, "master")
    assert_bits(f32(st.m), m, "m")


def test_accumulating_micro_batches_equals_their_sum():
    rng = np.random.default_rng(5)
    dw = torch.zeros((40, 96), dtype=torch.float32, device="cuda")
    row = torch.zeros(96, dtype=torch.float32, device="cuda")
    want, mag = 0.0, 0.0
    for _ in range(3):
        x, dy = acts(rng, 50, 96, "bf16"), acts(rng, 50, 40, "bf16")
        k = Z.ckpt_empty(50, 96, Z.CKPT_E4M3)
        Z.ckpt_write(x, k)
        Z.ckpt_weight_grad(k, dy, dw, accumulate=True)
        hx = oact.held(*oact.store(f64(x), "e4m3", "bf16"), "e4m3")
        want = want + oact.weight_grad(f64(dy), hx)
        mag = mag + np.abs(f64(dy)).T @ np.abs(hx)
        st = torch.tensor([[0.0, 1.0, 0.0, 1.0]], device="cuda").repeat(50, 1)
        Z.block_norm_grad(None, x, k, None, st, pre=Z.Norm(Z.NORM_RMS, 1e-5), dw_pre=row,
                          accumulate=True)
    close(f64(dw), want, 200 * 2 * U * mag, "fp32", "dw")
    assert (row != 0).any()


@pytest.mark.parametrize("h", [96, 1100, 9000])
@pytest.mark.parametrize("grad", ["fp32", "bf16"])
def test_norm_gradients_accumulated_over_micro_batches_equal_their_sum(h, grad):
    """Each call adds its rows' sums once to what is there and replaces nothing."""
    rng = np.random.default_rng(h)
    t, calls = 50, 3
    dt = torch.float32 if grad == "fp32" else torch.bfloat16
    got = {n: torch.from_numpy(rng.standard_normal(h)).to(dt).cuda() for n in ("dw_pre", "db_pre")}
    want = {n: f64(v) for n, v in got.items()}
    mag = {n: np.abs(v) for n, v in want.items()}
    kept = {n: 0.0 for n in got}                       # roundings between the calls
    for i in range(calls):
        x, dz = acts(rng, t, h, "bf16"), acts(rng, t, h, "bf16")
        k = Z.ckpt_empty(t, h, Z.CKPT_E4M3)
        Z.ckpt_write(x, k)
        st = torch.tensor([[0.0, 1.0, 0.0, 1.0]], device="cuda").repeat(t, 1)
        Z.block_norm_grad(None, dz, k, None, st, pre=Z.Norm(Z.NORM_RMS, 1e-5), accumulate=True,
                          **got)
        hx, d = oact.held(*oact.store(f64(x), "e4m3", "bf16"), "e4m3"), f64(dz)
        for n, s in (("dw_pre", d * hx), ("db_pre", d)):
            want[n], mag[n] = want[n] + s.sum(0), mag[n] + np.abs(s).sum(0)
            if i + 1 < calls and grad == "bf16":
                kept[n] = kept[n] + EPS["bf16"] * np.abs(want[n])
    for n, v in got.items():
        # in fp32: at most two roundings of a product, one addition a token, 16 in the
        # join and one a call; a kept value's rounding may itself be of one off by that
        bound = (t + 2 + 16 + calls) * U * mag[n]
        close(f64(v), want[n], bound + kept[n] * (1 + EPS["bf16"]) + 2 * EPS["bf16"] * bound,
              grad, n)


@pytest.mark.parametrize("tokens,group", [(96, 4), (50, 7)])
def test_checkpoint_partitioned_over_a_group(tokens, group):
    """Each rank of a group stores its own tokens of one activation; the parts in
    rank order are the whole checkpoint."""
    rng = np.random.default_rng(tokens)
    x = acts(rng, tokens, 300, "fp16")
    whole = Z.ckpt_empty(tokens, 300, Z.CKPT_INT8)
    for r in range(group):
        g = Z.shard_geometry(tokens, group, r)
        part = whole.row_range(g.offset, g.offset + g.len)
        Z.ckpt_write(x[g.offset:g.offset + g.len], part)
    c, s = oact.store(f64(x), "int8", "fp16")
    assert np.array_equal(whole.codes.cpu().numpy(), c)
    assert np.array_equal(whole.scales.cpu().numpy(), s)


OUTPUTS = ("out", "z", "stats", "back", "dres", "dblock", "dw", "dw_pre", "dw_post", "db_pre",
           "db_post", "dgate")


def _step_buffers(rng, dtype="bf16", t=300, h=264, n=200):
    dt = {"fp16": torch.float16, "bf16": torch.bfloat16}[dtype]

    def mat(c):
        return torch.empty((t, c), dtype=dt, device="cuda")

    b = dict(h=acts(rng, t, h, dtype), b=acts(rng, t, h, dtype), dout=acts(rng, t, h, dtype),
             dz=acts(rng, t, h, dtype), dy=acts(rng, t, n, dtype), out=mat(h), z=mat(h),
             dres=mat(h), dblock=mat(h), back=mat(h),
             stats=torch.empty((t, 4), dtype=torch.float32, device="cuda"),
             dw=torch.empty((n, h), dtype=torch.float32, device="cuda"),
             gate=torch.rand(h, device="cuda").to(dt), w=torch.rand(h, device="cuda").to(dt),
             k=[Z.ckpt_empty(t, h, Z.CKPT_INT8) for _ in range(4)])
    for name in ("dw_pre", "dw_post", "db_pre", "db_post", "dgate"):
        b[name] = torch.empty(h, dtype=torch.float32, device="cuda")
    return b


def _step(b, stream=None, ws=None):
    norms = dict(post=Z.Norm(Z.NORM_LAYER, 1e-5, b["w"], b["gate"]),
                 pre=Z.Norm(Z.NORM_LAYER, 1e-5, b["w"], b["gate"]), gate=b["gate"], scale=0.5,
                 stream=stream)
    kb, ko, kz, kx = b["k"]
    w1, w2 = ws or (None, None)
    Z.block_norm(b["h"], b["b"], b["out"], b["z"], b["stats"], ckpt_block=kb, ckpt_out=ko,
                 ckpt_z=kz, **norms)
    Z.ckpt_write(b["z"], kx, stream=stream)
    Z.ckpt_read(kx, b["back"], stream=stream)
    Z.block_norm_grad(b["dout"], b["dz"], ko, kb, b["stats"], workspace=w1,
                      **{k: b[k] for k in ("dres", "dblock", "dw_pre", "dw_post", "db_pre",
                                           "db_post", "dgate")}, **norms)
    Z.ckpt_weight_grad(kz, b["dy"], b["dw"], workspace=w2, stream=stream)
    return [b[k] for k in OUTPUTS]


def _bits(ts):
    return [t.clone().view(torch.int16 if t.element_size() == 2 else torch.int32) for t in ts]


@pytest.mark.parametrize("own_workspace", [False, True])
def test_captured_step_replays_equal_the_eager_step(own_workspace):
    rng = np.random.default_rng(8)
    b = _step_buffers(rng, t=1500)
    ws = None
    if own_workspace:
        ws = (torch.empty(Z.block_norm_grad_workspace(1500, 264), dtype=torch.uint8,
                          device="cuda"),
              torch.empty(max(1, Z.ckpt_weight_grad_workspace(1500, 264, 200)),
                          dtype=torch.uint8, device="cuda"))
    first = _bits(_step(b, ws=ws))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        _step(b, stream=side, ws=ws)
    noise = torch.randn(1 << 20, device="cuda")
    for i in range(4):
        for t in (b["h"], b["b"], b["dz"], b["dy"]):      # new inputs for every replay
            t.copy_(t.roll(1, 0) * 0.5 + 0.25)
        want = _bits(_step(b, ws=ws))
        for k in ("out", "z", "dres", "dblock", "dw", "dgate", "dw_pre"):
            b[k].zero_()
        torch.cuda.synchronize()
        graph.replay()
        noise = noise * 1.0001 + 1.0
        torch.cuda.synchronize()
        for name, y in zip(OUTPUTS, want):
            assert torch.equal(_bits([b[name]])[0], y), (i, name)
        assert not torch.equal(want[0], first[0])


def test_two_streams_at_once_match_one_after_the_other():
    """The workspaces the binding takes are the calls' own, on the calls' streams."""
    bufs = [_step_buffers(np.random.default_rng(20 + i), t=2000) for i in range(2)]
    want = [_bits(_step(b)) for b in bufs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bufs]
    for b in bufs:
        for k in ("out", "z", "dres", "dblock", "dw"):
            b[k].zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for b, s in zip(bufs, streams):
            _step(b, stream=s)
    torch.cuda.synchronize()
    for b, w in zip(bufs, want):
        got = _bits([b[k] for k in OUTPUTS])
        for x, y in zip(got, w):
            assert torch.equal(x, y)


def test_binding_refuses_what_the_kernels_do_not_take():
    t, h = 8, 64
    x = torch.zeros((t, h), dtype=torch.float16, device="cuda")
    k = Z.ckpt_empty(t, h, Z.CKPT_INT8)
    w = torch.ones(h, dtype=torch.float16, device="cuda")
    n = Z.Norm(Z.NORM_RMS, 1e-5, w)
    st = torch.zeros((t, 4), dtype=torch.float32, device="cuda")
    f = torch.zeros(h, dtype=torch.float32, device="cuda")
    bad = [
        lambda: Z.ckpt_write(x.float(), k), lambda: Z.ckpt_write(x[:7], k),
        lambda: Z.ckpt_write(x.t(), k), lambda: Z.ckpt_read(k, x.int()),
        lambda: Z.ckpt_read(k, x[:, :63]), lambda: Z.ckpt_write(x[0], k),
        lambda: Z.ckpt_weight_grad(k, x[:7], torch.empty((h, h), device="cuda")),
        lambda: Z.ckpt_weight_grad(k, x, torch.empty((h, h), device="cuda").bfloat16()),
        lambda: Z.ckpt_weight_grad(k, x, torch.empty((h, 63), device="cuda")),
        lambda: Z.block_norm(x, x.bfloat16(), x, x, st, pre=n),
        lambda: Z.block_norm(x, x, x, x, st[:7], pre=n),
        lambda: Z.block_norm(x, x, x, x, st, pre=Z.Norm(Z.NORM_RMS, 1e-5, w.float())),
        lambda: Z.block_norm(x, x, x, x, st, pre=n, gate=w[:63]),
        lambda: Z.block_norm(x, x, x, x, st, pre=n, gate=w.expand(t, h)),
        lambda: Z.block_norm_grad(x, x, k, k, st, pre=n, dres=x, dgate=f),
        lambda: Z.block_norm_grad(x, x, k, k, st, pre=n, dw_pre=f.int()),
        lambda: Z.block_norm_grad(x, x, k, k, st, pre=n, post=n, dw_pre=f, dw_post=w),
        lambda: Z.block_norm_grad(x, x, k, k, st, pre=n, dw_pre=f,
                                  workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(Z.ZeroError) as e:
        Z.block_norm(x, x, x, None, st, pre=n)
    assert e.value.code == Z.ZERO_E_INVAL
    with pytest.raises(Z.ZeroError) as e:
        Z.ckpt_read(k, x[:1].expand(t, h))
    assert e.value.code == Z.ZERO_E_RANGE


def test_rank_refuses_places_outside_the_local_gradient():
    st = zr.RankState(1000, 2, 0, 2)
    row = torch.zeros(400, dtype=torch.int16, device="cuda")
    assert st.grad_slot(600, 400, row, 600).numel() == 400
    for args in ((0, 10), (599, 10, row, 600), (601, 400, row, 600), (900, 200, row, 850),
                 (0, 10, row.float()), (0, 10, row[::2])):
        with pytest.raises(ValueError):
            st.grad_slot(*args)
