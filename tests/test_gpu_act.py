"""The activation entry points on the GPU against the 64-bit oracle: 8-bit
checkpoints bit for bit, the weight gradient and the norms within bounds that
count the roundings (act_util)."""
import numpy as np
import pytest
import torch

import zero_sharded_mixed_bucketed_amd as Z
from act_util import EPS, TORCH, U, acts, close, f64, strided
from gpu_util import need_gpu
from oracle import act as oact

pytestmark = pytest.mark.gpu

FMT = {"int8": Z.CKPT_INT8, "e4m3": Z.CKPT_E4M3}
KIND = {"none": Z.NORM_NONE, "rms": Z.NORM_RMS, "layer": Z.NORM_LAYER}


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    print(flush=True)


def _ckpt(t, h, fmt, code_pad=0, code_off=0, scale_pad=0):
    nb = -(-h // 32)
    codes = torch.full((code_off + max(t, 1) * (h + code_pad) + 8,), 0x55, dtype=torch.uint8,
                       device="cuda")
    scales = torch.full((max(t, 1) * (nb + scale_pad) + 8,), 0xAA, dtype=torch.uint8,
                        device="cuda")
    return Z.Ckpt(codes.as_strided((t, h), (h + code_pad, 1), code_off),
                  scales.as_strided((t, nb), (nb + scale_pad, 1)), FMT[fmt]), codes, scales


def _stored(x, fmt, dtype):
    """A device checkpoint with the oracle's codes, and the held values."""
    codes, scales = oact.store(f64(x), fmt, dtype)
    k = Z.Ckpt(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), FMT[fmt])
    return k, oact.held(codes, scales, fmt)


# ---------------------------------------------------------------- checkpoints

SHAPES = [(1, 1, 0, 0), (1, 31, 0, 0), (3, 32, 0, 0), (2, 33, 0, 1), (5, 8, 8, 0), (7, 100, 3, 0),
          (130, 1024, 0, 0), (33, 2056, 8, 8), (17, 4099, 1, 3), (3, 40000, 0, 0),
          (1500, 24, 0, 0)]


@pytest.mark.parametrize("t,h,pad,off", SHAPES)
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_write_and_read_match_the_oracle_bits(t, h, pad, off, fmt, dtype):
    rng = np.random.default_rng(t * 131 + h)
    x = acts(rng, t, h, dtype, pad, off)
    k, cbuf, sbuf = _ckpt(t, h, fmt, pad, off, pad)
    Z.ckpt_write(x, k)
    want_c, want_s = oact.store(f64(x), fmt, dtype)
    assert np.array_equal(k.codes.cpu().numpy(), want_c)
    assert np.array_equal(k.scales.cpu().numpy(), want_s)
    # nothing beside the rows was written
    mask = torch.ones_like(cbuf, dtype=torch.bool)
    mask.as_strided((t, h), (h + pad, 1), off).fill_(False)
    assert (cbuf[mask] == 0x55).all()
    mask = torch.ones_like(sbuf, dtype=torch.bool)
    mask.as_strided(k.scales.shape, k.scales.stride()).fill_(False)
    assert (sbuf[mask] == 0xAA).all()
    held = oact.held(want_c, want_s, fmt)
    for out_t in (dtype, "fp32"):
        out, buf = strided((t, h), TORCH[out_t], pad, off)
        before = buf.clone()
        Z.ckpt_read(k, out)
        assert np.array_equal(f64(out), held)          # exact in the type
        out.copy_(before.as_strided(out.shape, out.stride(), off))
        assert torch.equal(buf, before)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_write_over_the_whole_range_of_the_type(fmt, dtype):
    """Every 16-bit pattern as a block's largest value beside smaller ones, and
    blocks of arbitrary patterns: subnormals, the type's largest values,
    infinities and NaN."""
    bits = np.arange(65536, dtype=np.uint16)
    rng = np.random.default_rng(4)
    rows = np.zeros((65536, 32), np.uint16)
    rows[:, 5] = bits
    rows[:, 6] = (bits & 0x7FFF) - np.minimum(bits & 0x7FFF, rng.integers(0, 2000, 65536))
    rows[:, 7] = bits ^ 0x8000
    mixed = rng.integers(0, 65536, size=(4096, 32)).astype(np.uint16)
    near = (rng.integers(0, 65536, size=(65536, 1)) ^ rng.integers(0, 2048, size=(65536, 32)))
    allr = np.concatenate([rows, mixed, near.astype(np.uint16)])
    x = torch.from_numpy(allr.view(np.int16)).cuda().view(TORCH[dtype])
    k = Z.ckpt_empty(allr.shape[0], 32, FMT[fmt])
    Z.ckpt_write(x, k)
    want_c, want_s = oact.store(f64(x), fmt, dtype)
    got_s = k.scales.cpu().numpy()
    bad = np.flatnonzero(got_s[:, 0] != want_s[:, 0])
    assert bad.size == 0, (bad[:4], got_s[bad[:4], 0], want_s[bad[:4], 0], f64(x)[bad[:1]])
    got = oact.held(k.codes.cpu().numpy(), got_s, fmt)
    assert np.array_equal(got, oact.held(want_c, want_s, fmt), equal_nan=True)
    out = torch.empty_like(x)
    Z.ckpt_read(k, out)
    assert np.array_equal(f64(out), got, equal_nan=True)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_read_every_code_and_scale(fmt):
    """All 256 codes under all 256 scale bytes, into each type, each value rounded
    to nearest even; overflow gives infinities."""
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 8, axis=1)
    k = Z.Ckpt(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), FMT[fmt])
    held = torch.from_numpy(oact.held(codes, scales, fmt))
    for dt in (torch.float16, torch.bfloat16, torch.float32):
        out = torch.empty((256, 256), dtype=dt, device="cuda")
        Z.ckpt_read(k, out)
        want = held.to(torch.float32).to(dt)           # fp32 first: 2^(e-9) may be below it
        assert np.array_equal(f64(out), want.double().numpy(), equal_nan=True), dt


def test_checkpoint_past_32_bits():
    """Rows 2^31 + 8 elements apart: byte offsets beyond 2^32 on both sides."""
    h, stride = 200, (1 << 31) + 8
    x = torch.empty(2 * stride + h, dtype=torch.float16, device="cuda").as_strided(
        (3, h), (stride, 1))
    x.copy_(torch.randn((3, h), device="cuda"))
    codes = torch.empty(2 * stride + h, dtype=torch.uint8, device="cuda").as_strided(
        (3, h), (stride, 1))
    k = Z.Ckpt(codes, torch.empty((3, 7), dtype=torch.uint8, device="cuda"), Z.CKPT_INT8)
    Z.ckpt_write(x, k)
    want_c, want_s = oact.store(f64(x), "int8", "fp16")
    assert np.array_equal(codes.cpu().numpy(), want_c)
    assert np.array_equal(k.scales.cpu().numpy(), want_s)
    out = torch.empty((3, h), dtype=torch.float16, device="cuda")
    Z.ckpt_read(k, out)
    assert np.array_equal(f64(out), oact.held(want_c, want_s, "int8"))
    # the weight gradient reads both operands at those offsets
    dy = x[:, :40]
    dw = torch.empty((40, h), dtype=torch.float32, device="cuda")
    Z.ckpt_weight_grad(k, dy, dw)
    d, hx = f64(dy), oact.held(want_c, want_s, "int8")
    close(f64(dw), oact.weight_grad(d, hx), 16 * U * (np.abs(d).T @ np.abs(hx)), "fp32", "dw")


def test_many_rows_past_32_bits():
    """2^26 + 5 rows of 72 columns: more than 2^32 elements in dense rows."""
    t, h = (1 << 26) + 5, 72
    x = torch.zeros((t, h), dtype=torch.float16, device="cuda")
    rows = torch.tensor([0, 1, (1 << 26) // 3, (1 << 26) - 1, t - 1], device="cuda")
    x[rows] = torch.randn((5, h), device="cuda").half()
    k = Z.ckpt_empty(t, h, Z.CKPT_E4M3)
    Z.ckpt_write(x, k)
    want_c, want_s = oact.store(f64(x[rows]), "e4m3", "fp16")
    assert np.array_equal(k.codes[rows].cpu().numpy(), want_c)
    assert np.array_equal(k.scales[rows].cpu().numpy(), want_s)
    assert int(k.codes.count_nonzero()) == int(np.count_nonzero(want_c))
    Z.ckpt_read(k, x)
    assert np.array_equal(f64(x[rows]), oact.held(want_c, want_s, "e4m3"))


# ---------------------------------------------------------------- weight gradient

WSHAPES = [  # t, k, n, dy pad, dw pad
    (1, 1, 1, 0, 0), (1, 200, 3, 0, 0), (5, 32, 129, 0, 0), (31, 128, 128, 0, 0),
    (32, 136, 64, 8, 8), (33, 127, 130, 1, 3), (64, 256, 256, 0, 0), (100, 1032, 77, 3, 0),
    (257, 513, 260, 0, 1), (1000, 96, 520, 8, 0), (3001, 264, 136, 0, 0), (4096, 64, 40, 0, 0)]
# enough output for tiles of 256 x 256: whole ones, ragged edges, lengths around the
# tokens of a turn, and odd strides
WLARGE = [(1, 2048, 4096, 0, 0), (200, 2080, 4100, 0, 0), (64, 4096, 2304, 8, 0),
          (193, 2313, 2561, 1, 1), (320, 2560, 2048, 0, 0)]


@pytest.mark.parametrize("t,k,n,pad,wpad", WSHAPES)
@pytest.mark.parametrize("fmt,dtype,out", [("int8", "fp16", "fp16"), ("int8", "bf16", "fp32"),
                                           ("e4m3", "fp16", "fp32"), ("e4m3", "bf16", "bf16")])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_grad(t, k, n, pad, wpad, fmt, dtype, out, accumulate):
    rng = np.random.default_rng(t + 7 * k + 13 * n)
    x, hx = _stored(acts(rng, t, k, dtype), fmt, dtype)
    dy = acts(rng, t, n, dtype, pad, pad, sigma=0.05)
    dw, buf = strided((n, k), TORCH[out], wpad, wpad)
    dw.copy_(torch.from_numpy(rng.standard_normal((n, k))))
    old, before = f64(dw), buf.clone()
    Z.ckpt_weight_grad(x, dy, dw, accumulate=accumulate)
    d = f64(dy)
    want = oact.weight_grad(d, hx) + (old if accumulate else 0.0)
    mag = np.abs(d).T @ np.abs(hx) + (np.abs(old) if accumulate else 0.0)
    # t additions in any order (of partial sums too), each within 2^-23 should the
    # matrix unit cut instead of rounding; the products are exact
    close(f64(dw), want, (t + 32) * 2 * U * mag, out, "dw")
    dw.copy_(before.as_strided(dw.shape, dw.stride(), wpad))
    assert torch.equal(buf, before)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_weight_grad_reads_every_code_and_scale(fmt, dtype):
    """One token with a unit gradient: dw is the held row, rounded to dy's type."""
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(1, 256)
    one = torch.ones((1, 1), dtype=TORCH[dtype], device="cuda")
    dw = torch.empty((1, 256), dtype=torch.float32, device="cuda")
    for b in range(256):
        scales = torch.full((1, 8), b, dtype=torch.uint8, device="cuda")
        Z.ckpt_weight_grad(Z.Ckpt(codes, scales, FMT[fmt]), one, dw)
        held = oact.held(codes.cpu().numpy(), scales.cpu().numpy(), fmt)
        want = torch.from_numpy(held).float().to(TORCH[dtype]).double().numpy()
        assert np.array_equal(f64(dw), want, equal_nan=True), b


@pytest.mark.parametrize("t,k,n,pad,wpad", WLARGE)
@pytest.mark.parametrize("fmt,dtype,out,accumulate", [
    ("int8", "fp16", "fp16", False), ("int8", "bf16", "fp32", True),
    ("e4m3", "fp16", "fp32", False), ("e4m3", "bf16", "bf16", True)])
def test_weight_grad_large_tiles(t, k, n, pad, wpad, fmt, dtype, out, accumulate):
    test_weight_grad(t, k, n, pad, wpad, fmt, dtype, out, accumulate)


def test_weight_grad_without_tokens():
    x = Z.ckpt_empty(0, 70, Z.CKPT_INT8)
    dy = torch.empty((0, 33), dtype=torch.float16, device="cuda")
    dw = torch.ones((33, 70), dtype=torch.float16, device="cuda")
    Z.ckpt_weight_grad(x, dy, dw, accumulate=True)
    assert (dw == 1).all()
    Z.ckpt_weight_grad(x, dy, dw)
    assert (dw == 0).all()


@pytest.mark.parametrize("t", [40, 700])
def test_weight_grad_keeps_infinities_and_nan_where_they_belong(t):
    """A NaN block reaches its own columns, an infinite gradient its own row; a
    padded row or column of a tile reaches nothing."""
    rng = np.random.default_rng(t)
    a = acts(rng, t, 130, "fp16")
    a[3, 40] = float("inf")
    x, hx = _stored(a, "int8", "fp16")
    dy = acts(rng, t, 67, "fp16")
    dy[t - 1, 5] = float("inf")
    dy[0, 66] = float("nan")
    dw = torch.empty((67, 130), dtype=torch.float32, device="cuda")
    Z.ckpt_weight_grad(x, dy, dw)
    with np.errstate(invalid="ignore"):
        got, want = f64(dw), np.einsum("tn,tk->nk", f64(dy), hx)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.isinf(got), np.isinf(want))
    assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])


def test_weight_grad_overflow_is_infinite():
    x, hx = _stored(torch.full((64, 32), 6e4, dtype=torch.float16, device="cuda"), "int8", "fp16")
    dy = torch.full((64, 8), 2.0, dtype=torch.float16, device="cuda")
    dw = torch.empty((8, 32), dtype=torch.float16, device="cuda")
    Z.ckpt_weight_grad(x, dy, dw)
    assert torch.isinf(dw).all() and (dw > 0).all()


def test_weight_grad_is_the_same_bits_each_time():
    rng = np.random.default_rng(9)
    x, _ = _stored(acts(rng, 5000, 200, "bf16"), "int8", "bf16")
    dy = acts(rng, 5000, 100, "bf16")
    got = []
    for _ in range(3):
        dw = torch.empty((100, 200), dtype=torch.float32, device="cuda")
        Z.ckpt_weight_grad(x, dy, dw)
        got.append(dw)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


# ---------------------------------------------------------------- norms

K_ROW = 64     # roundings on the way through one row sum (16 in a thread, 6 in a
#                wave, 16 across waves) and the elementwise operations around it


def _norm_inputs(rng, h, dtype, kind):
    w = torch.from_numpy(1 + 0.2 * rng.standard_normal(h)).to(TORCH[dtype]).cuda()
    b = torch.from_numpy(0.2 * rng.standard_normal(h)).to(TORCH[dtype]).cuda()
    return (None, None) if kind == "none" else (w, b if kind == "layer" else None)


def _spec(kind, eps, w, b):
    return (kind, eps, None if w is None else f64(w), None if b is None else f64(b))


def _abs(v, other):
    return other if v is None else np.abs(v)


def _check_forward(got, h, b, post, pre, gate, scale, dtype, what):
    """Bounds: each term's magnitude times K_ROW * 2^-24 a norm."""
    out, z, st = oact.block_norm(h, b, post, pre, gate, scale)
    mag = np.abs(h)
    if b is not None:
        m2, r2 = st[:, 0:1], st[:, 1:2]
        spread = np.abs(b) + (np.mean(np.abs(b), axis=1, keepdims=True)
                              if post[0] == "layer" else 0.0)
        o = spread * r2 * _abs(post[2], 1.0) + _abs(post[3], 0.0)
        mag = mag + abs(scale) * _abs(gate, 1.0) * o
    if got.get("out") is not None:
        close(f64(got["out"]), out, K_ROW * U * mag, dtype, what + " out")
    if got.get("z") is not None:
        r1 = st[:, 3:4]
        big = mag + (np.mean(mag, axis=1, keepdims=True) if pre[0] == "layer" else 0.0)
        # the deviation's own error, from its input's error, moves every value
        rel = np.sqrt(np.mean(big ** 2, axis=1, keepdims=True)) * r1
        zmag = big * r1 * (1 + rel) * _abs(pre[2], 1.0) + _abs(pre[3], 0.0)
        close(f64(got["z"]), z, 2 * K_ROW * U * zmag, dtype, what + " z")
    if got.get("stats") is not None:
        s = f64(got["stats"])
        assert np.array_equal(s[:, 0:1] == 0, st[:, 0:1] == 0)
        if pre[0] != "none":
            assert np.all(np.abs(s[:, 3] - st[:, 3]) <= 4 * K_ROW * U * st[:, 3] * (
                1 + (rel[:, 0])))
    return out, z, st


def _run_forward(rng, t, h, dtype, post, pre, gate, pad=0, ckpts=None, inplace=False, scale=0.75,
                 stream=None):
    w2, c2 = _norm_inputs(rng, h, dtype, post)
    w1, c1 = _norm_inputs(rng, h, dtype, pre)
    res, block = acts(rng, t, h, dtype, pad, pad), acts(rng, t, h, dtype, pad, 0)
    g = None
    if gate == "channel":
        g = torch.from_numpy(rng.random(h)).to(TORCH[dtype]).cuda()
    elif gate == "token":
        g = acts(rng, t, h, dtype, pad)
    hv, bv = f64(res), f64(block)
    out = res if inplace else strided((t, h), TORCH[dtype], pad, pad)[0]
    z = None
    if pre != "none":
        z = block if inplace else strided((t, h), TORCH[dtype], pad, 0)[0]
    stats = torch.empty((t, 4), dtype=torch.float32, device="cuda")
    Z.block_norm(res, block, out, z, stats, post=Z.Norm(KIND[post], 1e-5, w2, c2),
                 pre=Z.Norm(KIND[pre], 1e-5, w1, c1), gate=g, scale=scale, stream=stream,
                 **(ckpts or {}))
    return dict(out=out, z=z, stats=stats, hv=hv, bv=bv, g=g, w=(w2, c2, w1, c1), block=block,
                post=_spec(post, 1e-5, w2, c2), pre=_spec(pre, 1e-5, w1, c1), scale=scale)


NSHAPES = [(1, 1, 0), (2, 7, 0), (1, 8, 0), (3, 33, 1), (5, 100, 3), (4, 512, 0), (67, 520, 8),
           (9, 1024, 0), (6, 1025, 0), (5, 2048, 0), (3, 4100, 4), (2, 8192, 0), (2, 8191, 1),
           (3, 16384, 0), (2, 12345, 0)]


@pytest.mark.parametrize("t,h,pad", NSHAPES)
@pytest.mark.parametrize("post,pre,gate", [("rms", "rms", "channel"), ("layer", "layer", "token"),
                                           ("rms", "layer", "none"), ("none", "rms", "token"),
                                           ("layer", "none", "channel")])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_block_norm(t, h, pad, post, pre, gate, dtype):
    rng = np.random.default_rng(t * 7 + h)
    r = _run_forward(rng, t, h, dtype, post, pre, gate, pad)
    gate_v = None if r["g"] is None else f64(r["g"])
    _check_forward(r, r["hv"], r["bv"], r["post"], r["pre"], gate_v, r["scale"], dtype, "norm")


@pytest.mark.parametrize("t,h", [(9000, 72), (4500, 1040), (2100, 4096)])
def test_block_norm_more_rows_than_workgroups(t, h):
    rng = np.random.default_rng(t)
    r = _run_forward(rng, t, h, "bf16", "rms", "layer", "channel")
    _check_forward(r, r["hv"], r["bv"], r["post"], r["pre"], f64(r["g"]), r["scale"], "bf16",
                   "norm")


def test_block_norm_in_place_and_without_a_block():
    rng = np.random.default_rng(11)
    r = _run_forward(rng, 300, 520, "fp16", "layer", "rms", "channel", inplace=True)
    _check_forward(r, r["hv"], r["bv"], r["post"], r["pre"], f64(r["g"]), r["scale"], "fp16",
                   "in place")
    h = acts(rng, 20, 200, "fp16")
    z, stats = torch.empty_like(h), torch.empty((20, 4), dtype=torch.float32, device="cuda")
    Z.block_norm(h, None, None, z, stats, pre=Z.Norm(Z.NORM_LAYER, 1e-5))
    _check_forward({"z": z, "stats": stats}, f64(h), None, ("none", 0, None, None),
                   ("layer", 1e-5, None, None), None, 1.0, "fp16", "no block")


@pytest.mark.parametrize("h", [40, 1024, 2051, 5120, 9000])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_emitted_checkpoints_are_those_of_the_stored_outputs(h, fmt, dtype):
    rng = np.random.default_rng(h)
    ks = {n: _ckpt(37, h, fmt, 5, 3)[0] for n in ("ckpt_block", "ckpt_out", "ckpt_z")}
    r = _run_forward(rng, 37, h, dtype, "rms", "layer", "channel", ckpts=ks)
    for name, x in (("ckpt_block", r["block"]), ("ckpt_out", r["out"]), ("ckpt_z", r["z"])):
        c, s = oact.store(f64(x), fmt, dtype)
        assert np.array_equal(ks[name].codes.cpu().numpy(), c), name
        assert np.array_equal(ks[name].scales.cpu().numpy(), s), name


def test_block_norm_rows_of_zeros_and_of_nan():
    """A row of zeros gives the bias; NaN and infinities stay in their row."""
    h = 1000
    x = torch.randn((4, h), device="cuda").half()
    x[1] = 0
    x[2, 7] = float("inf")
    b = torch.randn(h, device="cuda").half()
    z = torch.empty_like(x)
    for kind in (Z.NORM_RMS, Z.NORM_LAYER):
        Z.block_norm(x, None, None, z, None, pre=Z.Norm(kind, 1e-6, None, b))
        assert torch.equal(z[1], b)
        assert torch.isfinite(z[0]).all() and torch.isfinite(z[3]).all()
        assert torch.isnan(z[2, 7])


def _run_backward(rng, t, h, dtype, fmt, post, pre, gate, pad=0, grad="fp32", accumulate=False,
                  inplace=False, scale=0.75, dout=True, block=True, stream=None, workspace=None):
    w2, c2 = _norm_inputs(rng, h, dtype, post)
    w1, c1 = _norm_inputs(rng, h, dtype, pre)
    ho, hb = acts(rng, t, h, dtype), acts(rng, t, h, dtype)
    ko, xo = _stored(ho, fmt, dtype)
    kb, xb = _stored(hb, fmt, dtype)
    st = np.concatenate([*oact.stats(f64(hb), post, 1e-5), *oact.stats(f64(ho), pre, 1e-5)],
                        axis=1).astype(np.float32)
    stats = torch.from_numpy(st).cuda()
    g = None
    if gate == "channel":
        g = torch.from_numpy(rng.random(h)).to(TORCH[dtype]).cuda()
    elif gate == "token":
        g = acts(rng, t, h, dtype, pad)
    do = acts(rng, t, h, dtype, pad, pad, sigma=0.1) if dout else None
    dz = acts(rng, t, h, dtype, pad, sigma=0.1) if pre != "none" else None
    dov, dzv = (None if v is None else f64(v) for v in (do, dz))
    outs = {"dres": do if inplace else strided((t, h), TORCH[dtype], pad)[0]}
    if block:
        outs["dblock"] = dz if inplace else strided((t, h), TORCH[dtype], pad, pad)[0]
    names = (["dw_pre", "db_pre"] if pre != "none" else []) + \
        (["dw_post", "db_post"] if post != "none" and block else [])
    if w2 is not None and c2 is None and "db_post" in names:
        names.remove("db_post")
    if w1 is not None and c1 is None and "db_pre" in names:
        names.remove("db_pre")
    if gate == "channel" and block:
        names.append("dgate")
    if gate == "token" and block:
        outs["dgate"] = strided((t, h), TORCH[dtype], pad)[0]
    old = {}
    for n in names:
        outs[n] = torch.from_numpy(rng.standard_normal(h)).to(TORCH[grad]).cuda()
        old[n] = f64(outs[n])
    Z.block_norm_grad(do, dz, ko if pre != "none" else None, kb if block else None, stats,
                      post=Z.Norm(KIND[post], 1e-5, w2, c2), pre=Z.Norm(KIND[pre], 1e-5, w1, c1),
                      gate=g, scale=scale, accumulate=accumulate, stream=stream,
                      workspace=workspace, **outs)
    return dict(outs=outs, old=old, st=st.astype(np.float64), xo=xo, xb=xb if block else None,
                do=dov, dz=dzv, gate=None if g is None else f64(g), mode=gate,
                post=_spec(post, 1e-5, w2, c2), pre=_spec(pre, 1e-5, w1, c1), scale=scale,
                names=names, accumulate=accumulate, grad=grad, dtype=dtype, t=t)


def _check_backward(r, what="norm grad"):
    post, pre, st, dtype = r["post"], r["pre"], r["st"], r["dtype"]
    want = oact.block_norm_grad(r["do"], r["dz"], r["xo"], r["xb"], st, post, pre, r["gate"],
                                r["scale"])

    def through(q, xn, rstd, kind):     # magnitudes of the gradient through a norm
        if kind == "none":
            return q
        d = q + xn * np.mean(q * xn, axis=1, keepdims=True)
        return rstd * (d + (np.mean(q, axis=1, keepdims=True) if kind == "layer" else 0.0))

    m2, r2, m1, r1 = (np.abs(st[:, i:i + 1]) for i in range(4))
    d = 0.0 if r["do"] is None else np.abs(r["do"])
    mag = {}
    if pre[0] != "none":
        x1, dz = (np.abs(r["xo"]) + m1) * r1, np.abs(r["dz"])
        d = d + through(dz * _abs(pre[2], 1.0), x1, r1, pre[0])
        mag["dw_pre"], mag["db_pre"] = (dz * x1).sum(0), dz.sum(0)
    mag["dres"] = d
    u = abs(r["scale"]) * d
    p = u * _abs(r["gate"], 1.0)
    v = p * _abs(post[2], 1.0)
    if r["xb"] is not None:
        x2 = (np.abs(r["xb"]) + m2) * r2
        mag["dgate"] = u * (x2 * _abs(post[2], 1.0) + _abs(post[3], 0.0))
        mag["dw_post"], mag["db_post"] = (p * x2).sum(0), p.sum(0)
        v = through(v, x2, r2, post[0])
    mag["dblock"] = v
    for name, got in r["outs"].items():
        w, m = want[name], mag[name]
        k, dt = 2 * K_ROW, dtype
        if name in r["names"]:
            if name == "dgate":
                w, m = w.sum(0), m.sum(0)
            dt, k = r["grad"], 2 * K_ROW + r["t"]     # and one addition a token
            if r["accumulate"]:
                w, m = w + r["old"][name], m + np.abs(r["old"][name])
        close(f64(got), w, k * U * m, dt, f"{what} {name}")


@pytest.mark.parametrize("t,h,pad", NSHAPES)
@pytest.mark.parametrize("post,pre,gate,grad,acc", [
    ("rms", "rms", "channel", "fp32", False), ("layer", "layer", "token", "own", True),
    ("rms", "layer", "none", "fp32", True), ("none", "rms", "token", "fp32", False),
    ("layer", "none", "channel", "own", False)])
@pytest.mark.parametrize("fmt,dtype", [("int8", "fp16"), ("e4m3", "bf16")])
def test_block_norm_grad(t, h, pad, post, pre, gate, grad, acc, fmt, dtype):
    rng = np.random.default_rng(t * 17 + h)
    _check_backward(_run_backward(rng, t, h, dtype, fmt, post, pre, gate, pad,
                                  grad=dtype if grad == "own" else grad, accumulate=acc))


@pytest.mark.parametrize("t,h", [(9000, 72), (2600, 1040), (1100, 4096), (520, 8200), (515, 16000)])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_block_norm_grad_more_rows_than_streams(t, h, kind):
    rng = np.random.default_rng(t)
    _check_backward(_run_backward(rng, t, h, "bf16", "int8", kind, kind, "channel"))


@pytest.mark.parametrize("h", [7, 100, 512, 2300, 5120, 8191, 10000])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_norms_without_weights_and_with_every_part(h, dtype):
    """No weights (ones, also past the row's end) and a large mean, which would show
    there; then every gradient of layer norms at once."""
    rng = np.random.default_rng(h)
    t = 40
    x = torch.from_numpy(rng.standard_normal((t, h)) + 3.0).to(TORCH[dtype]).cuda()
    k, xv = _stored(x, "int8", dtype)
    st = np.concatenate([*oact.stats(f64(x), "layer", 1e-5)] * 2, axis=1).astype(np.float32)
    stats = torch.from_numpy(st).cuda()
    dz, do = acts(rng, t, h, dtype), acts(rng, t, h, dtype)
    outs = {n: torch.empty(h, dtype=torch.float32, device="cuda")
            for n in ("dw_pre", "db_pre", "dw_post", "db_post")}
    names = list(outs)
    outs["dres"], outs["dblock"] = torch.empty_like(dz), torch.empty_like(dz)
    n = Z.Norm(Z.NORM_LAYER, 1e-5)
    Z.block_norm_grad(do, dz, k, k, stats, post=n, pre=n, scale=1.5, **outs)
    spec = ("layer", 1e-5, None, None)
    _check_backward(dict(outs=outs, names=names, old={}, st=st.astype(np.float64), xo=xv, xb=xv,
                         do=f64(do), dz=f64(dz), gate=None, post=spec, pre=spec, scale=1.5,
                         accumulate=False, grad="fp32", dtype=dtype, t=t))


def test_block_norm_grad_partial_calls():
    rng = np.random.default_rng(21)
    _check_backward(_run_backward(rng, 90, 520, "fp16", "int8", "rms", "layer", "channel",
                                  inplace=True), "in place")
    _check_backward(_run_backward(rng, 90, 520, "fp16", "int8", "rms", "layer", "none",
                                  dout=False), "no dout")
    _check_backward(_run_backward(rng, 90, 520, "fp16", "int8", "none", "rms", "none",
                                  block=False), "no block")


@pytest.mark.parametrize("h", [8208, 9001, 16384])
@pytest.mark.parametrize("kind,gate", [("rms", "channel"), ("layer", "token")])
def test_block_norm_grad_of_wide_rows_in_place(h, kind, gate):
    rng = np.random.default_rng(h)
    _check_backward(_run_backward(rng, 150, h, "bf16", "int8", kind, kind, gate, inplace=True))


def test_norms_past_32_bits():
    """Rows 2^31 + 8 elements apart on every side."""
    h, stride = 264, (1 << 31) + 8
    rng = np.random.default_rng(1)

    def far(fill):
        t = torch.empty(stride + h, dtype=torch.float16, device="cuda").as_strided(
            (2, h), (stride, 1))
        if fill:
            t.copy_(torch.from_numpy(rng.standard_normal((2, h))))
        return t

    res, block, out, z = far(True), far(True), far(False), far(False)
    stats = torch.empty((2, 4), dtype=torch.float32, device="cuda")
    n = Z.Norm(Z.NORM_LAYER, 1e-5)
    Z.block_norm(res, block, out, z, stats, post=n, pre=n)
    spec = ("layer", 1e-5, None, None)
    _check_forward(dict(out=out, z=z, stats=stats), f64(res), f64(block), spec, spec, None, 1.0,
                   "fp16", "far rows")
    ko, xo = _stored(out, "int8", "fp16")
    kb, xb = _stored(block, "int8", "fp16")
    dw = torch.empty(h, dtype=torch.float32, device="cuda")
    w = torch.ones(h, dtype=torch.float16, device="cuda")
    Z.block_norm_grad(res, z, ko, kb, stats, post=n, pre=Z.Norm(Z.NORM_LAYER, 1e-5, w), dres=out,
                      dblock=block, dw_pre=dw)
    _check_backward(dict(outs={"dres": out, "dblock": block, "dw_pre": dw}, names=["dw_pre"],
                         old={}, st=f64(stats), xo=xo, xb=xb, do=f64(res), dz=f64(z), gate=None,
                         post=spec, pre=spec, scale=1.0, accumulate=False, grad="fp32",
                         dtype="fp16", t=2))


def test_block_norm_grad_without_rows():
    w = torch.ones(50, dtype=torch.float16, device="cuda")
    e = torch.empty((0, 50), dtype=torch.float16, device="cuda")
    st = torch.empty((0, 4), dtype=torch.float32, device="cuda")
    k = Z.ckpt_empty(0, 50, Z.CKPT_INT8)
    dw = torch.ones(50, dtype=torch.float32, device="cuda")
    args = dict(pre=Z.Norm(Z.NORM_RMS, 1e-5, w), dres=e, dw_pre=dw)
    Z.block_norm_grad(None, e, k, None, st, accumulate=True, **args)
    assert (dw == 1).all()
    Z.block_norm_grad(None, e, k, None, st, **args)
    assert (dw == 0).all()
    Z.block_norm_grad(e, e, k, k, st, pre=Z.Norm(Z.NORM_RMS, 1e-5, w),
                      post=Z.Norm(Z.NORM_RMS, 1e-5, w), dres=e, dblock=e)
    Z.block_norm(e, None, None, e, None, pre=Z.Norm(Z.NORM_RMS, 1e-5, w))
    Z.ckpt_write(e, k)
    Z.ckpt_read(k, e)


def test_nan_tokens_stay_in_their_rows():
    rng = np.random.default_rng(2)
    t, h = 40, 1000
    x = acts(rng, t, h, "fp16")
    x[7, 100] = float("nan")
    k, _ = _stored(x, "int8", "fp16")
    stats = torch.tensor([[0.0, 1.0, 0.0, 1.0]], device="cuda").repeat(t, 1)
    dz = acts(rng, t, h, "fp16")
    dres = torch.empty_like(dz)
    dw = torch.empty(h, dtype=torch.float32, device="cuda")
    Z.block_norm_grad(None, dz, k, None, stats, pre=Z.Norm(Z.NORM_RMS, 1e-5), dres=dres,
                      dw_pre=dw)
    rows = torch.isnan(dres).any(dim=1)
    assert rows[7] and int(rows.sum()) == 1
    cols = torch.isnan(dw)
    assert cols[96:128].all() and int(cols.sum()) == 32


@pytest.mark.parametrize("h", [100, 1000, 4096, 9000])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_nan_of_a_block_without_a_norm_stays_out_of_its_gradient(h, gate):
    """Without a post norm the gradient of b does not depend on b: values that the
    checkpoint holds as NaN reach the gate's gradient only, 32 columns each."""
    rng = np.random.default_rng(h)
    b = acts(rng, 6, h, "fp16")
    b[2, 5] = float("nan")
    b[4, h - 1] = float("inf")
    kb = _ckpt(6, h, "int8")[0]
    Z.ckpt_write(b, kb)
    g = acts(rng, 1 if gate == "channel" else 6, h, "fp16")
    dout = acts(rng, 6, h, "fp16")
    dblock = torch.empty_like(dout)
    dgate = torch.empty(h, dtype=torch.float32, device="cuda") if gate == "channel" \
        else torch.empty_like(dout)
    Z.block_norm_grad(dout, None, None, kb, None, gate=g[0] if gate == "channel" else g,
                      scale=0.5, dblock=dblock, dgate=dgate)
    want = 0.5 * f64(dout) * f64(g)
    close(f64(dblock), want, 2 * U * np.abs(want), "fp16", "dblock")   # two products
    nan = np.zeros((6, h), bool)
    nan[2, :32] = True
    nan[4, (h - 1) // 32 * 32:] = True
    assert np.array_equal(np.isnan(f64(dgate)), nan.any(axis=0) if gate == "channel" else nan)


@pytest.mark.parametrize("t,h", [(1, 1032), (1100, 1032), (40, 1536), (1000, 1900), (7, 2048),
                                 (300, 4104), (520, 5001), (9, 5632), (600, 6144), (3, 6145)])
@pytest.mark.parametrize("gate", ["channel", "token", "none"])
@pytest.mark.parametrize("inplace", [False, True])
def test_block_norm_grad_without_biases_at_widths_of_one_chunk_a_thread(t, h, gate, inplace):
    rng = np.random.default_rng(h + t)
    _check_backward(_run_backward(rng, t, h, "bf16", "int8", "rms", "rms", gate, inplace=inplace))


@pytest.mark.parametrize("t,h", [(700, 2560), (5, 3584), (260, 4608), (2, 5120), (270, 5632),
                                 (33, 6144)])
@pytest.mark.parametrize("kind,gate", [("rms", "channel"), ("layer", "token"),
                                       ("layer", "channel")])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_block_norm_grad_at_widths_of_whole_waves(t, h, kind, gate, dtype):
    rng = np.random.default_rng(h + t)
    _check_backward(_run_backward(rng, t, h, dtype, "int8", kind, kind, gate, inplace=True))


@pytest.mark.parametrize("t,h", [(2100, 1040), (300, 4095), (260, 8192), (260, 8190)])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_block_norm_grad_of_layer_norms_over_bf16(t, h, gate):
    rng = np.random.default_rng(h + t)
    _check_backward(_run_backward(rng, t, h, "bf16", "e4m3", "layer", "layer", gate))


def test_block_norm_of_more_rows_than_one_launch():
    """2^26 + 5 rows of 72 columns, a wave each: 2^32 threads and more."""
    t, h = (1 << 26) + 5, 72
    res = torch.zeros((t, h), dtype=torch.float16, device="cuda")
    rows = torch.tensor([0, 1, (1 << 26) - 2, (1 << 26) - 1, 1 << 26, t - 1], device="cuda")
    res[rows] = torch.randn((6, h), device="cuda").half()
    b = torch.full((h,), 0.5, dtype=torch.float16, device="cuda")
    z = torch.zeros_like(res)
    stats = torch.empty((t, 4), dtype=torch.float32, device="cuda")
    Z.block_norm(res, None, None, z, stats, pre=Z.Norm(Z.NORM_RMS, 1e-5, None, b))
    spec = ("rms", 1e-5, None, f64(b))
    _check_forward({"z": z[rows], "stats": stats[rows]}, f64(res[rows]), None,
                   ("none", 0, None, None), spec, None, 1.0, "fp16", "long")
    live = torch.zeros(t, dtype=torch.bool, device="cuda")
    live[rows] = True
    bad = 0
    for lo in range(0, t, 1 << 24):            # rows of zeros give the bias
        part = (z[lo:lo + (1 << 24)] != b).any(dim=1)
        bad += int((part & ~live[lo:lo + (1 << 24)]).sum())
    assert bad == 0


def test_checkpoint_of_more_rows_than_one_launch():
    """2^32 + 17 rows of one column, 16 rows a piece of a wave."""
    t = (1 << 32) + 17
    x = torch.zeros((t, 1), dtype=torch.float16, device="cuda")
    rows = torch.tensor([0, 1, (1 << 32) - 257, (1 << 32) - 256, 1 << 32, t - 1], device="cuda")
    x[rows] = torch.randn((6, 1), device="cuda").half()
    codes = torch.full((t, 1), 0x55, dtype=torch.uint8, device="cuda")
    k = Z.Ckpt(codes, torch.full_like(codes, 0xAA), Z.CKPT_INT8)
    Z.ckpt_write(x, k)
    want_c, want_s = oact.store(f64(x[rows]), "int8", "fp16")
    assert np.array_equal(codes[rows].cpu().numpy(), want_c)
    assert np.array_equal(k.scales[rows].cpu().numpy(), want_s)
    for lo in range(0, t, 1 << 30):            # zeros elsewhere, at the least scale
        part = slice(lo, min(t, lo + (1 << 30)))
        inside = int(((rows >= part.start) & (rows < part.stop)).sum())
        assert int((codes[part] != 0).sum()) == inside
        assert int((k.scales[part] != 1).sum()) == inside
    x.fill_(7.0)
    Z.ckpt_read(k, x)
    assert np.array_equal(f64(x[rows]), oact.held(want_c, want_s, "int8"))
    assert sum(int((x[lo:lo + (1 << 30)] != 0).sum()) for lo in range(0, t, 1 << 30)) == 6
