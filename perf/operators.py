"""The cases on which the activation-side operators are measured: 8-bit
activation checkpoints, the weight gradient taken from them, and the norms
before and after a block with its gate and residual scale, forward and
backward.

Where ``own`` is false, ``run`` computes them with elementary torch operations
in 32 bits; where it is true it calls the package's entry points on the same
inputs.  ``exact`` gives the definition's value in 64 bits.

A checkpoint holds rows of 8-bit codes in blocks of 32 columns, each block with
one scale byte b that stands for 2^(b - 127).
"""
import math

import torch

own = False

BLOCK = 32
EPS = 1e-5
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- cases

def _ckpt(name, t, h, dtype, fmt, pad=0):
    return {"name": name, "op": "ckpt", "t": t, "h": h, "dtype": dtype, "fmt": fmt, "pad": pad}


def _wgrad(name, t, k, n, dtype, fmt, out, acc, pad=0):
    return {"name": name, "op": "wgrad", "t": t, "h": k, "n": n, "dtype": dtype, "fmt": fmt,
            "out": out, "acc": acc, "pad": pad}


def _norm(name, op, t, h, dtype, fmt, kind, gate, pad=0):
    return {"name": name, "op": op, "t": t, "h": h, "dtype": dtype, "fmt": fmt, "kind": kind,
            "gate": gate, "pad": pad}


def _step(name, t, h, n, dtype, fmt, kind, gate):
    return {"name": name, "op": "step", "t": t, "h": h, "n": n, "dtype": dtype, "fmt": fmt,
            "kind": kind, "gate": gate, "pad": 0}


def listed():
    return [
        # a short sequence's activations, stored and read back: latency
        _ckpt("ckpt-small", 128, 1024, "fp16", "int8"),
        # one layer input of two sequences of 8192 tokens at hidden 4096
        _ckpt("ckpt-layer", 16384, 4096, "bf16", "int8"),
        # a ragged batch at an odd width inside a wider buffer
        _ckpt("ckpt-odd", 4099, 8205, "fp16", "e4m3", 3),
        # a small projection on a short sequence
        _wgrad("wgrad-small", 256, 1024, 1024, "fp16", "int8", "fp16", False),
        # the widening projection of a hidden-4096 layer, one sequence of 8192 tokens, into
        # the fp16 local gradient
        _wgrad("wgrad-mlp", 8192, 4096, 16384, "fp16", "int8", "fp16", False),
        # a narrow projection over many tokens, summed onto an fp32 gradient over micro-batches:
        # few output tiles, a long sum
        _wgrad("wgrad-long", 16001, 1032, 776, "bf16", "e4m3", "fp32", True),
        # a short sequence through the norms around a block
        _norm("norm-small", "norm", 64, 1024, "fp16", "int8", "rms", "channel"),
        # two sequences of 8192 tokens at hidden 4096, RMS norms, one gate per channel
        _norm("norm-layer", "norm", 16384, 4096, "bf16", "int8", "rms", "channel"),
        # their backward from the 8-bit checkpoints
        _norm("norm-grad-layer", "norm_grad", 16384, 4096, "bf16", "int8", "rms", "channel"),
        # layer norms with biases at an odd width, a gate for every token
        _norm("norm-grad-odd", "norm_grad", 2051, 8190, "fp16", "e4m3", "layer", "token", 2),
        # forward with its checkpoints, then backward and the next projection's weight gradient:
        # a short sequence, and a hidden-4096 layer
        _step("step-small", 200, 1024, 1024, "fp16", "int8", "layer", "none"),
        _step("step-layer", 8192, 4096, 4096, "bf16", "int8", "rms", "channel"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    h = _log(rng, lo, hi)
    how = rng.random()
    return max(lo, h // 64 * 64) if how < 0.5 else max(lo, h // 8 * 8) if how < 0.75 else h


def draw(rng):
    op = rng.choice(["ckpt", "wgrad", "norm", "norm_grad", "step"])
    c = {"op": op, "dtype": rng.choice(["fp16", "bf16"]), "fmt": rng.choice(["int8", "e4m3"]),
         "pad": rng.choice([0, 0, 0, 8, 1])}
    if op == "ckpt":
        c["h"] = _width(rng, 40, 16384)
        c["t"] = _log(rng, 1, min(32768, (1 << 26) // c["h"]))
        return c
    if op == "wgrad":
        c["h"] = _width(rng, 64, 16384)
        c["n"] = _width(rng, 64, min(16384, (1 << 26) // c["h"]))
        c["t"] = _log(rng, 1, min(16384, (1 << 39) // (c["h"] * c["n"])))
        c["out"] = rng.choice([c["dtype"], "fp32"])
        c["acc"] = rng.choice([False, True])
        return c
    c["kind"] = rng.choice(["rms", "layer"])
    c["gate"] = rng.choice(["none", "channel", "token"])
    if op == "step":
        c["pad"] = 0
        c["h"] = _width(rng, 64, 8192)
        c["n"] = _width(rng, 64, 8192)
        c["t"] = _log(rng, 1, min(8192, (1 << 37) // (c["h"] * c["n"])))
        return c
    c["h"] = _width(rng, 64, 16384)
    c["t"] = _log(rng, 1, min(32768, (1 << 26) // c["h"]))
    return c


# ---------------------------------------------------------------- inputs

def _rows(t, h, pad, dtype):
    """A [t, h] view whose rows lie h + pad apart."""
    return torch.empty((t, h + pad), dtype=dtype, device="cuda")[:, :h]


def _act(gen, t, h, pad, dtype):
    """Activations: normal, with a few channels that are much larger."""
    x = torch.randn((t, h), generator=gen, device="cuda")
    big = torch.rand((h,), generator=gen, device="cuda") < 0.01
    x = x * (1.0 + 15.0 * big)
    out = _rows(t, h, pad, dtype)
    out.copy_(x)
    return out


def _grad(gen, t, h, pad, dtype):
    """Gradients as loss scaling leaves them in 16 bits."""
    out = _rows(t, h, pad, dtype)
    out.copy_(0.05 * torch.randn((t, h), generator=gen, device="cuda"))
    return out


def _pack(x, fmt):
    """Codes and scale bytes of the checkpoint of x (what the forward left)."""
    t, h = x.shape
    y, e = _quantise(x.float(), fmt, x.dtype)
    codes = (y.to(torch.int8).view(torch.uint8) if fmt == "int8"
             else y.to(torch.float8_e4m3fn).view(torch.uint8))
    return codes.contiguous(), (e + 127).to(torch.uint8).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t, h, pad, dt = case["t"], case["h"], case["pad"], TYPES[case["dtype"]]
    s = {"case": dict(case)}
    if case["op"] == "ckpt":
        s["x"] = _act(gen, t, h, pad, dt)
        return s
    if case["op"] == "wgrad":
        s["codes"], s["scales"] = _pack(_act(gen, t, h, 0, dt), case["fmt"])
        s["dy"] = _grad(gen, t, case["n"], pad, dt)
        if case["acc"]:
            s["dw0"] = torch.randn((case["n"], h), generator=gen, device="cuda").to(
                TYPES[case["out"]])
        return s
    for name in ("w_pre", "w_post"):
        s[name] = (1.0 + 0.1 * torch.randn(h, generator=gen, device="cuda")).to(dt)
    for name in ("b_pre", "b_post"):
        s[name] = ((0.1 * torch.randn(h, generator=gen, device="cuda")).to(dt)
                   if case["kind"] == "layer" else None)
    s["gate"] = {"none": None,
                 "channel": torch.rand(h, generator=gen, device="cuda").to(dt),
                 "token": _act(gen, t, h, pad, dt) if case["gate"] == "token" else None,
                 }[case["gate"]]
    s["scale"] = 0.5
    if case["op"] in ("norm", "step"):
        s["res"] = _act(gen, t, h, pad, dt)
        s["block"] = _act(gen, t, h, pad, dt)
    if case["op"] in ("norm_grad", "step"):
        s["dout"] = _grad(gen, t, h, pad, dt)
        s["dz"] = _grad(gen, t, h, pad, dt)
    if case["op"] == "norm_grad":
        res, block = _act(gen, t, h, 0, dt), _act(gen, t, h, 0, dt)
        s["stats"] = torch.cat([_stats(block.float(), case["kind"]),
                                _stats(res.float(), case["kind"])], 1).contiguous()
        s["res_codes"], s["res_scales"] = _pack(res, case["fmt"])
        s["block_codes"], s["block_scales"] = _pack(block, case["fmt"])
    if case["op"] == "step":
        s["dy"] = _grad(gen, t, case["n"], 0, dt)
    return s


# ---------------------------------------------------------------- plain form, 32 bits

def _pow2(e):
    """2^e of whole numbers e in [-126, 127], as fp32."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(a):
    """floor(log2 a) of fp32 a > 0 (-127 for 0 and subnormals)."""
    return (a.view(torch.int32) >> 23) - 127


def _blocks(x):
    t, h = x.shape
    nb = -(-h // BLOCK)
    if nb * BLOCK != h:
        x = torch.cat([x, x.new_zeros((t, nb * BLOCK - h))], 1)
    return x.reshape(t, nb, BLOCK)


def _quantise(x, fmt, dtype):
    """fp32 x -> (scaled and rounded values [t, h], block exponents [t, nb])."""
    t, h = x.shape
    if fmt == "e4m3":
        top = 1.875 * 2.0 ** (15 if dtype == torch.float16 else 127)
        x = x.clamp(-top, top)
    xb = _blocks(x)
    a = xb.abs().amax(2)
    if fmt == "int8":
        e = (_exponent(a) - 6).clamp(min=-126)
        y = torch.round(_scaled(xb, -e)).clamp(-127, 127)
    else:
        e = _exponent(a)
        e = (torch.where(a > 1.75 * _pow2(e.clamp(min=-126)), e - 7, e - 8)).clamp(min=-117)
        y = _scaled(xb, -e)
        step = _pow2(_exponent(y.abs()).clamp(min=-6) - 3)
        y = torch.round(y / step) * step
    return y.reshape(t, -1)[:, :h], e


def _scaled(xb, e):
    """x 2^e per block, in two exact steps (e may pass 127)."""
    half = torch.div(e, 2, rounding_mode="floor")
    return xb * _pow2(half)[..., None] * _pow2(e - half)[..., None]


def _through(x, fmt, dtype):
    """x as its checkpoint holds it, fp32."""
    t, h = x.shape
    y, e = _quantise(x, fmt, dtype)
    return (_blocks(y) * _pow2(e)[..., None]).reshape(t, -1)[:, :h]


def _unpack(codes, scales, fmt):
    t, h = codes.shape
    y = codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float()
    return (_blocks(y) * _pow2(scales.to(torch.int32) - 127)[..., None]).reshape(t, -1)[:, :h]


def _stats(x, kind):
    """(mean, 1 / deviation) of each row, fp32 [t, 2]; the mean is 0 for RMS."""
    m = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    r = torch.rsqrt((x - m).square().mean(1, keepdim=True) + EPS)
    return torch.cat([m, r], 1)


def _forward(s):
    c = s["case"]
    h, b = s["res"].float(), s["block"].float()
    s2 = _stats(b, c["kind"])
    o = (b - s2[:, :1]) * s2[:, 1:] * s["w_post"].float()
    if s["b_post"] is not None:
        o = o + s["b_post"].float()
    if s["gate"] is not None:
        o = o * s["gate"].float()
    out = h + s["scale"] * o
    s1 = _stats(out, c["kind"])
    z = (out - s1[:, :1]) * s1[:, 1:] * s["w_pre"].float()
    if s["b_pre"] is not None:
        z = z + s["b_pre"].float()
    dt = s["res"].dtype
    return out.to(dt), z.to(dt), torch.cat([s2, s1], 1)


def _norm_back(q, x, r, kind):
    d = q - x * (q * x).mean(1, keepdim=True)
    if kind == "layer":
        d = d - q.mean(1, keepdim=True)
    return r * d


def _backward(s, res, block, stats):
    c = s["case"]
    dt = s["dz"].dtype
    dz = s["dz"].float()
    x2 = (block - stats[:, 0:1]) * stats[:, 1:2]
    x1 = (res - stats[:, 2:3]) * stats[:, 3:4]
    d = s["dout"].float() + _norm_back(dz * s["w_pre"].float(), x1, stats[:, 3:4], c["kind"])
    u = s["scale"] * d
    p = u if s["gate"] is None else u * s["gate"].float()
    db = _norm_back(p * s["w_post"].float(), x2, stats[:, 1:2], c["kind"])
    got = {"dres": d.to(dt), "dblock": db.to(dt), "dw_pre": (dz * x1).sum(0),
           "dw_post": (p * x2).sum(0)}
    if c["kind"] == "layer":
        got["db_pre"], got["db_post"] = dz.sum(0), p.sum(0)
    if s["gate"] is not None:
        o = x2 * s["w_post"].float()
        if s["b_post"] is not None:
            o = o + s["b_post"].float()
        got["dgate"] = (u * o).sum(0) if c["gate"] == "channel" else (u * o).to(dt)
    return got


def _plain(s):
    c = s["case"]
    if c["op"] == "ckpt":
        return _through(s["x"].float(), c["fmt"], s["x"].dtype).to(s["x"].dtype)
    if c["op"] == "wgrad":
        dw = s["dy"].float().t() @ _unpack(s["codes"], s["scales"], c["fmt"])
        if c["acc"]:
            dw = s["dw0"].float() + dw
        return dw.to(TYPES[c["out"]])
    if c["op"] == "norm":
        return _forward(s)
    if c["op"] == "norm_grad":
        return _backward(s, _unpack(s["res_codes"], s["res_scales"], c["fmt"]),
                         _unpack(s["block_codes"], s["block_scales"], c["fmt"]), s["stats"])
    out, z, stats = _forward(s)
    dt = out.dtype
    got = _backward(s, _through(out.float(), c["fmt"], dt),
                    _through(s["block"].float(), c["fmt"], dt), stats)
    dw = s["dy"].float().t() @ _through(z.float(), c["fmt"], dt)
    # every parameter's gradient in 16 bits, as the local gradient holds it
    return {"out": out, "z": z, "stats": stats, "dw": dw.to(dt),
            **{k: v.to(dt) for k, v in got.items()}}


# ---------------------------------------------------------------- the package's calls

def _norms(Z, s):
    kind = Z.NORM_LAYER if s["case"]["kind"] == "layer" else Z.NORM_RMS
    return {"post": Z.Norm(kind, EPS, s["w_post"], s["b_post"]),
            "pre": Z.Norm(kind, EPS, s["w_pre"], s["b_pre"])}


def _own_forward(Z, s, **ckpts):
    t, h = s["res"].shape
    out = torch.empty((t, h), dtype=s["res"].dtype, device="cuda")
    z = torch.empty_like(out)
    stats = torch.empty((t, 4), dtype=torch.float32, device="cuda")
    Z.block_norm(s["res"], s["block"], out, z, stats, gate=s["gate"], scale=s["scale"],
                 **_norms(Z, s), **ckpts)
    return out, z, stats


def _own_backward(Z, s, ckpt_res, ckpt_block, stats):
    c = s["case"]
    t, h = s["dz"].shape
    dt = s["dz"].dtype

    def row():
        # a step's parameter gradients go to the 16-bit local gradient
        return torch.empty(h, dtype=dt if c["op"] == "step" else torch.float32, device="cuda")

    got = {"dres": torch.empty((t, h), dtype=dt, device="cuda"),
           "dblock": torch.empty((t, h), dtype=dt, device="cuda"),
           "dw_pre": row(), "dw_post": row()}
    if c["kind"] == "layer":
        got["db_pre"], got["db_post"] = row(), row()
    if c["gate"] != "none":
        got["dgate"] = (row() if c["gate"] == "channel"
                        else torch.empty((t, h), dtype=dt, device="cuda"))
    Z.block_norm_grad(s["dout"], s["dz"], ckpt_res, ckpt_block, stats, gate=s["gate"],
                      scale=s["scale"], **_norms(Z, s), **got)
    return got


def _own(s):
    import zero_sharded_mixed_bucketed_amd as Z

    c = s["case"]
    fmt = Z.CKPT_INT8 if c["fmt"] == "int8" else Z.CKPT_E4M3
    t, h = c["t"], c["h"]
    if c["op"] == "ckpt":
        k = Z.ckpt_empty(t, h, fmt)
        Z.ckpt_write(s["x"], k)
        out = torch.empty((t, h), dtype=s["x"].dtype, device="cuda")
        Z.ckpt_read(k, out)
        return out
    if c["op"] == "wgrad":
        if c["acc"]:
            dw = s["dw0"].clone()
        else:
            dw = torch.empty((c["n"], h), dtype=TYPES[c["out"]], device="cuda")
        Z.ckpt_weight_grad(Z.Ckpt(s["codes"], s["scales"], fmt), s["dy"], dw,
                           accumulate=c["acc"])
        return dw
    if c["op"] == "norm":
        return _own_forward(Z, s)
    if c["op"] == "norm_grad":
        return _own_backward(Z, s, Z.Ckpt(s["res_codes"], s["res_scales"], fmt),
                             Z.Ckpt(s["block_codes"], s["block_scales"], fmt), s["stats"])
    kb, kr, kz = (Z.ckpt_empty(t, h, fmt) for _ in range(3))
    out, z, stats = _own_forward(Z, s, ckpt_block=kb, ckpt_out=kr, ckpt_z=kz)
    got = _own_backward(Z, s, kr, kb, stats)
    dw = torch.empty((c["n"], h), dtype=out.dtype, device="cuda")
    Z.ckpt_weight_grad(kz, s["dy"], dw)
    return {"out": out, "z": z, "stats": stats, "dw": dw, **got}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass needs

def work(case):
    t, h = case["t"], case["h"]
    e, held = t * h, 1.0 + 1.0 / BLOCK
    size = 4 if case.get("out") == "fp32" else 2
    rows = (2 if case.get("kind") == "rms" else 4) * h + (h if case.get("gate") == "channel" else 0)
    token = 2 * e if case.get("gate") == "token" else 0
    forward = 8 * e + token + 16 * t + 2 * rows
    backward = 8 * e + 2 * held * e + 2 * token + 16 * t + 6 * rows
    if case["op"] == "ckpt":
        return {"bytes": (4 + 2 * held) * e, "flops": 4 * e}
    if case["op"] == "wgrad":
        n = case["n"]
        return {"bytes": held * e + 2 * t * n + size * n * h * (2 if case["acc"] else 1),
                "flops": 2 * e * n}
    if case["op"] == "norm":
        return {"bytes": forward, "flops": 12 * e}
    if case["op"] == "norm_grad":
        return {"bytes": backward, "flops": 24 * e}
    n = case["n"]
    return {"bytes": forward + backward + 4 * held * e + 2 * t * n + 2 * n * h,
            "flops": 36 * e + 2 * e * n}


# ---------------------------------------------------------------- the definition, 64 bits

def _x_two_to(k):
    """2^k of whole numbers k, exactly: the exponent field of a 64-bit number."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _x_held(x, fmt, dtype):
    """x (64 bits) rounded as the format rounds it, block by block."""
    t, h = x.shape
    nb = -(-h // BLOCK)
    full = torch.zeros((t, nb * BLOCK), dtype=torch.float64, device=x.device)
    full[:, :h] = x
    full = full.view(t, nb, BLOCK)
    if fmt == "int8":
        _, k = torch.frexp(full.abs().max(dim=2, keepdim=True).values)
        q = _x_two_to((k - 7).clamp(min=-126))
        full = torch.round(full / q).clamp(-127, 127) * q
    else:
        top = 1.875 * 2.0 ** (15 if dtype == torch.float16 else 127)
        full = full.clamp(-top, top)
        m, k = torch.frexp(full.abs().max(dim=2, keepdim=True).values)
        e = (k - 9 + (m > 0.875)).clamp(min=-117)
        _, own_k = torch.frexp(full)
        q = _x_two_to(torch.maximum(own_k - 4, e - 9))
        full = torch.round(full / q) * q
    return full.view(t, -1)[:, :h]


def _x_codes(codes, scales, fmt):
    h = codes.shape[1]
    y = codes.view(torch.int8).double() if fmt == "int8" else \
        codes.view(torch.float8_e4m3fn).double()
    return y * _x_two_to(scales.to(torch.int64) - 127).repeat_interleave(BLOCK, dim=1)[:, :h]


def _x_norm(x, kind):
    n = x.shape[1]
    m = x.sum(1, keepdim=True) / n if kind == "layer" else 0 * x[:, :1]
    v = ((x - m) ** 2).sum(1, keepdim=True) / n
    return m, 1 / torch.sqrt(v + EPS)


def _x_forward(s):
    kind = s["case"]["kind"]
    b, w1, w2 = s["block"].double(), s["w_pre"].double(), s["w_post"].double()
    m2, r2 = _x_norm(b, kind)
    c1 = 0 if s["b_pre"] is None else s["b_pre"].double()
    c2 = 0 if s["b_post"] is None else s["b_post"].double()
    g = 1 if s["gate"] is None else s["gate"].double()
    out = s["res"].double() + s["scale"] * g * (w2 * r2 * (b - m2) + c2)
    m1, r1 = _x_norm(out, kind)
    return out, w1 * r1 * (out - m1) + c1, torch.cat([m2, r2, m1, r1], 1)


def _x_backward(s, res, block, stats):
    kind, n = s["case"]["kind"], res.shape[1]
    layer = 1.0 if kind == "layer" else 0.0
    m2, r2, m1, r1 = (stats[:, i:i + 1].double() for i in range(4))
    dz, w1, w2 = s["dz"].double(), s["w_pre"].double(), s["w_post"].double()
    c2 = 0 if s["b_post"] is None else s["b_post"].double()
    g = 1 if s["gate"] is None else s["gate"].double()
    x1, x2 = r1 * (res - m1), r2 * (block - m2)
    q = w1 * dz
    d = s["dout"].double() + r1 * (q - layer * q.sum(1, keepdim=True) / n
                                   - x1 * (q * x1).sum(1, keepdim=True) / n)
    p = s["scale"] * g * d
    v = w2 * p
    db = r2 * (v - layer * v.sum(1, keepdim=True) / n - x2 * (v * x2).sum(1, keepdim=True) / n)
    got = {"dres": d, "dblock": db, "dw_pre": (dz * x1).sum(0), "dw_post": (p * x2).sum(0)}
    if kind == "layer":
        got["db_pre"], got["db_post"] = dz.sum(0), p.sum(0)
    if s["gate"] is not None:
        dg = s["scale"] * d * (w2 * x2 + c2)
        got["dgate"] = dg.sum(0) if s["case"]["gate"] == "channel" else dg
    return got


def exact(case, seed):
    s = prepare(case, seed)
    fmt = case["fmt"]
    if case["op"] == "ckpt":
        return _x_held(s["x"].double(), fmt, s["x"].dtype)
    if case["op"] == "wgrad":
        dw = s["dy"].double().t().contiguous() @ _x_codes(s["codes"], s["scales"], fmt)
        return dw + s["dw0"].double() if case["acc"] else dw
    if case["op"] == "norm":
        return _x_forward(s)
    if case["op"] == "norm_grad":
        return _x_backward(s, _x_codes(s["res_codes"], s["res_scales"], fmt),
                           _x_codes(s["block_codes"], s["block_scales"], fmt), s["stats"])
    out, z, stats = _x_forward(s)
    dt = s["res"].dtype
    # the checkpoints hold the 16-bit outputs
    got = _x_backward(s, _x_held(out.to(dt).double(), fmt, dt),
                      _x_held(s["block"].double(), fmt, dt), stats)
    dw = s["dy"].double().t().contiguous() @ _x_held(z.to(dt).double(), fmt, dt)
    return {"out": out, "z": z, "stats": stats, "dw": dw, **got}
