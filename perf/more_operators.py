"""The cases on which the operators of a layer's gated feed-forward block and of
the loss over the vocabulary are measured: the block's forward (both
projections, the activation and their product), its backward from 8-bit
checkpoints, the softmax cross entropy of a projection onto the vocabulary, and
the distillation from a teacher's top logits, each with the gradients of its
input and its weight.

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
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases

def _ffn(name, op, t, d, f, dtype, act, fmt="int8", pad=0, acc=False):
    return {"name": name, "op": op, "t": t, "d": d, "f": f, "dtype": dtype, "act": act, "fmt": fmt,
            "pad": pad, "acc": acc}


def _loss(name, op, t, d, v, dtype, grad=True, left_out=0.0, weights=False, pad=0, acc=False, k=0,
          tau=1.0):
    return {"name": name, "op": op, "t": t, "d": d, "v": v, "dtype": dtype, "grad": grad,
            "left_out": left_out, "weights": weights, "pad": pad, "acc": acc, "k": k, "tau": tau}


def listed():
    return [
        # one token through a block of hidden 4096: latency, the weights' reading
        _ffn("ffn-one", "ffn", 1, 4096, 16384, "bf16", "silu"),
        # the block of a hidden-4096 layer over one sequence of 8192 tokens
        _ffn("ffn-layer", "ffn", 8192, 4096, 16384, "bf16", "silu"),
        # a short sequence forward with its checkpoints and backward from them
        _ffn("ffn-step-small", "ffn_step", 200, 1024, 2048, "fp16", "gelu"),
        # the block's backward over the long sequence
        _ffn("ffn-grad-layer", "ffn_grad", 8192, 4096, 16384, "bf16", "silu"),
        # a ragged batch at odd widths inside wider buffers, summed onto the local gradient
        _ffn("ffn-grad-odd", "ffn_grad", 2051, 1032, 2730, "fp16", "gelu_tanh", "e4m3", 3, True),
        # the loss of a held-out batch: no gradients
        _loss("xent-loss", "xent", 4096, 2048, 65536, "bf16", grad=False),
        # a short sequence of a small model with a small vocabulary
        _loss("xent-small", "xent", 128, 1024, 32768, "fp16"),
        # one long sequence of a hidden-4096 model with a large vocabulary
        _loss("xent-layer", "xent", 8192, 4096, 131072, "bf16"),
        # answers after prompts that carry no loss, a weight for every token, odd sizes
        _loss("xent-odd", "xent", 3001, 2050, 50001, "fp16", left_out=0.6, weights=True, pad=2,
              acc=True),
        # distillation on a short sequence, at temperature 1
        _loss("distill-small", "distill", 256, 1024, 32768, "bf16", k=16),
        # a long sequence with a large vocabulary, softened
        _loss("distill-layer", "distill", 4096, 4096, 131072, "bf16", k=64, tau=2.0),
        # ragged sets of entries, tokens without any
        _loss("distill-odd", "distill", 1537, 776, 40003, "fp16", left_out=0.3, weights=True, k=50,
              tau=1.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def _width(rng, lo, hi):
    h = _log(rng, lo, hi)
    how = rng.random()
    return max(lo, h // 64 * 64) if how < 0.5 else max(lo, h // 8 * 8) if how < 0.75 else h


def draw(rng):
    op = rng.choice(["ffn", "ffn_grad", "ffn_step", "xent", "distill"])
    c = {"op": op, "dtype": rng.choice(["fp16", "bf16"]), "pad": rng.choice([0, 0, 0, 8, 1]),
         "acc": rng.choice([False, False, True])}
    c["d"] = _width(rng, 64, 8192 if op.startswith("ffn") else 4096)
    if op.startswith("ffn"):
        c["f"] = _width(rng, 64, min(16384, (1 << 26) // c["d"]))
        c["t"] = _log(rng, 1, min(8192, (1 << 38) // (c["d"] * c["f"])))
        c["act"] = rng.choice(["silu", "gelu", "gelu_tanh"])
        c["fmt"] = rng.choice(["int8", "e4m3"])
        return c
    c["v"] = _width(rng, 1000, 131072)
    c["t"] = _log(rng, 1, min(8192, (1 << 41) // (c["d"] * c["v"])))
    c["grad"] = rng.choice([True, True, False])
    c["left_out"] = rng.choice([0.0, 0.2, 0.7])
    c["weights"] = rng.choice([False, True])
    c["k"] = _log(rng, 1, 256) if op == "distill" else 0
    c["tau"] = rng.choice([1.0, 2.0, 1.5]) if op == "distill" else 1.0
    return c


# ---------------------------------------------------------------- inputs

def _rows(t, h, pad, dtype):
    """A [t, h] view whose rows lie h + pad apart."""
    return torch.empty((t, h + pad), dtype=dtype, device="cuda")[:, :h]


def _normal(gen, t, h, pad, dtype, scale):
    out = _rows(t, h, pad, dtype)
    out.copy_(torch.randn((t, h), generator=gen, device="cuda").mul_(scale))
    return out


def _act(gen, t, h, pad, dtype):
    """A norm's output: normal, with a few channels that are larger."""
    x = torch.randn((t, h), generator=gen, device="cuda")
    big = torch.rand((h,), generator=gen, device="cuda") < 0.01
    out = _rows(t, h, pad, dtype)
    out.copy_(x * (1.0 + 3.0 * big))
    return out


def _pack(x, fmt):
    """Codes and scale bytes of the checkpoint of x (what the forward left)."""
    y, e = _quantise(x.float(), fmt, x.dtype)
    codes = (y.to(torch.int8).view(torch.uint8) if fmt == "int8"
             else y.to(torch.float8_e4m3fn).view(torch.uint8))
    return codes.contiguous(), (e + 127).to(torch.uint8).contiguous()


def _left_out(gen, t, share):
    """Which tokens carry no loss: runs of them, as prompts are."""
    runs = torch.rand((-(-t // 16),), generator=gen, device="cuda") < share
    return runs.repeat_interleave(16)[:t]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t, d, pad, dt = case["t"], case["d"], case["pad"], TYPES[case["dtype"]]
    s = {"case": dict(case)}
    if case["op"].startswith("ffn"):
        f = case["f"]
        s["w"] = _normal(gen, 2 * f, d, pad, dt, 0.8 / math.sqrt(d))
        if case["op"] != "ffn_grad":
            s["x"] = _act(gen, t, d, pad, dt)
        if case["op"] == "ffn_grad":
            s["x_codes"], s["x_scales"] = _pack(_act(gen, t, d, 0, dt), case["fmt"])
            for name in ("gate", "up"):
                s[name + "_codes"], s[name + "_scales"] = _pack(_act(gen, t, f, 0, dt),
                                                                case["fmt"])
        if case["op"] != "ffn":
            # gradients as loss scaling leaves them in 16 bits
            s["dout"] = _normal(gen, t, f, pad, dt, 0.05)
            if case["acc"]:
                s["dw0"] = _normal(gen, 2 * f, d, 0, dt, 1.0)
        return s
    v, k = case["v"], case["k"]
    s["w"] = _normal(gen, v, d, pad, dt, 2.0 / math.sqrt(d))
    if k:
        # K different ids a token, spread over the vocabulary, largest logit first
        k = min(k, v)
        gap = max(1, v // k)
        steps = torch.randint(1, gap + 1, (t, k), generator=gen, device="cuda")
        ids = (steps.cumsum(1) + torch.randint(0, v, (t, 1), generator=gen, device="cuda")) % v
        drop = torch.rand((t, k), generator=gen, device="cuda").mul_(-3.0)
        s["top"] = (10.0 + drop.cumsum(1) / math.sqrt(k)).contiguous()
        if case["left_out"]:
            held = torch.randint(1, k + 1, (t, 1), generator=gen, device="cuda")
            ids[torch.arange(k, device="cuda")[None, :] >= held] = -1
        first = ids[:, 0].clamp(min=0)
        ids[_left_out(gen, t, case["left_out"])] = -1
        s["ids"] = ids.to(torch.int32).contiguous()
    else:
        first = torch.randint(0, v, (t,), generator=gen, device="cuda")
        s["targets"] = first.masked_fill(_left_out(gen, t, case["left_out"]), -1)
    # a model that has learnt: some tokens' logits stand out at their target
    x = torch.randn((t, d), generator=gen, device="cuda")
    lift = 3.0 * torch.rand((t, 1), generator=gen, device="cuda")
    x += lift * s["w"][first].float()
    s["x"] = _rows(t, d, pad, dt)
    s["x"].copy_(x)
    s["weights"] = (torch.rand((t,), generator=gen, device="cuda").add_(0.5) if case["weights"]
                    else None)
    s["scale"] = 1024.0 / max(1, t)        # the mean over the batch, with loss scaling
    if case["grad"] and case["acc"]:
        s["dw0"] = _normal(gen, v, d, 0, dt, 0.1)
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
    y, e = _quantise(x.to(dtype).float(), fmt, dtype)
    return (_blocks(y) * _pow2(e)[..., None]).reshape(t, -1)[:, :h]


def _unpack(codes, scales, fmt):
    t, h = codes.shape
    y = codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float()
    return (_blocks(y) * _pow2(scales.to(torch.int32) - 127)[..., None]).reshape(t, -1)[:, :h]


def _activation(g, act):
    """(act(g), act'(g))."""
    if act == "silu":
        p = torch.sigmoid(g)
        return g * p, p * (1.0 + g * (1.0 - p))
    if act == "gelu":
        p = 0.5 * torch.erfc(g * -math.sqrt(0.5))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    c = math.sqrt(2.0 / math.pi)
    h = torch.tanh(c * (g + 0.044715 * g * g * g))
    return (0.5 * g * (1.0 + h),
            0.5 * (1.0 + h) + 0.5 * g * (1.0 - h * h) * c * (1.0 + 3.0 * 0.044715 * g * g))


def _ffn_back(s, x, g, u):
    c = s["case"]
    dt = s["dout"].dtype
    do = s["dout"].float()
    a, da = _activation(g, c["act"])
    dgu = torch.cat([do * u * da, do * a], 1)
    dw = dgu.t() @ x
    if c["acc"]:
        dw = dw + s["dw0"].float()
    return {"dx": (dgu @ s["w"].float()).to(dt), "dw": dw.to(dt)}


def _plain(s):
    c = s["case"]
    if c["op"] == "ffn_grad":
        x, g, u = (_unpack(s[n + "_codes"], s[n + "_scales"], c["fmt"])
                   for n in ("x", "gate", "up"))
        return _ffn_back(s, x, g, u)
    x, dt = s["x"].float(), s["x"].dtype
    z = x @ s["w"].float().t()
    if c["op"] in ("ffn", "ffn_step"):
        g, u = z[:, :c["f"]], z[:, c["f"]:]
        out = (_activation(g, c["act"])[0] * u).to(dt)
        if c["op"] == "ffn":
            return out
        return {"out": out, **_ffn_back(s, _through(x, c["fmt"], dt), _through(g, c["fmt"], dt),
                                        _through(u, c["fmt"], dt))}
    tau = c["tau"]
    z = z / tau
    z = z - z.amax(1, keepdim=True)
    p = torch.exp(z)
    total = p.sum(1, keepdim=True)
    ids = s["ids"].long() if c["op"] == "distill" else s["targets"][:, None]
    some = ids >= 0
    at = ids.clamp(min=0)
    if c["op"] == "distill":
        e = (s["top"] / tau).masked_fill(~some, -math.inf)
        e = torch.exp(e - e.amax(1, keepdim=True).clamp(min=-1e30))
        q = e / e.sum(1, keepdim=True).clamp(min=1e-30)
    else:
        q = some.float()
    log_p = z.gather(1, at) - total.log()
    w = some.any(1).float()
    if s["weights"] is not None:
        w = w * s["weights"]
    loss = (q * (torch.log(q.clamp(min=1e-38)) - log_p)).sum(1) * (w * (tau * tau))
    if not c["grad"]:
        return loss
    dz = p.mul_((1.0 / total)).scatter_add_(1, at, -q).mul_((w * (s["scale"] * tau))[:, None])
    dw = dz.t() @ x
    if c["acc"]:
        dw = dw + s["dw0"].float()
    return {"loss": loss, "dx": (dz @ s["w"].float()).to(dt), "dw": dw.to(dt)}


# ---------------------------------------------------------------- the package's calls

def _own(s):
    import zero_sharded_mixed_bucketed_amd as Z

    c = s["case"]
    t, d = c["t"], c["d"]
    dt = s["w"].dtype
    dw = None
    if c["op"] not in ("ffn",) and c.get("grad", True):
        dw = s["dw0"].clone() if c["acc"] else torch.empty(s["w"].shape, dtype=dt, device="cuda")
    if c["op"].startswith("ffn"):
        f = c["f"]
        fmt = Z.CKPT_INT8 if c["fmt"] == "int8" else Z.CKPT_E4M3
        act = {"silu": Z.ACT_SILU, "gelu": Z.ACT_GELU, "gelu_tanh": Z.ACT_GELU_TANH}[c["act"]]
        if c["op"] == "ffn_grad":
            kx, kg, ku = (Z.Ckpt(s[n + "_codes"], s[n + "_scales"], fmt)
                          for n in ("x", "gate", "up"))
            got = {}
        else:
            out = torch.empty((t, f), dtype=dt, device="cuda")
            if c["op"] == "ffn":
                Z.gated_ffn(s["x"], s["w"], out, act)
                return out
            kx, kg, ku = (Z.ckpt_empty(t, h, fmt) for h in (d, f, f))
            Z.ckpt_write(s["x"], kx)
            Z.gated_ffn(s["x"], s["w"], out, act, ckpt_gate=kg, ckpt_up=ku)
            got = {"out": out}
        dx = torch.empty((t, d), dtype=dt, device="cuda")
        Z.gated_ffn_grad(s["dout"], kg, ku, s["w"], act, dx=dx, ckpt_x=kx, dw=dw,
                         accumulate=c["acc"])
        return {**got, "dx": dx, "dw": dw}
    loss = torch.empty(t, dtype=torch.float32, device="cuda")
    dx = torch.empty((t, d), dtype=dt, device="cuda") if c["grad"] else None
    more = {"weights": s["weights"], "scale": s["scale"], "dx": dx, "dw": dw,
            "accumulate": bool(c["grad"] and c["acc"])}
    if c["op"] == "distill":
        Z.distill_loss(s["x"], s["w"], s["ids"], s["top"], loss, temperature=c["tau"], **more)
    else:
        Z.vocab_loss(s["x"], s["w"], s["targets"], loss, **more)
    return {"loss": loss, "dx": dx, "dw": dw} if c["grad"] else loss


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass needs

def work(case):
    t, d, held = case["t"], case["d"], 1.0 + 1.0 / BLOCK
    if case["op"].startswith("ffn"):
        f = case["f"]
        w, product = 4 * f * d, 4 * t * d * f
        forward = {"bytes": 2 * t * d + w + 2 * t * f, "flops": product + 10 * t * f}
        backward = {"bytes": held * t * d + (2 + 2 * held) * t * f + 2 * t * d
                    + w * (3 if case["acc"] else 2), "flops": 2 * product + 20 * t * f}
        if case["op"] == "ffn":
            return forward
        if case["op"] == "ffn_grad":
            return backward
        return {"bytes": forward["bytes"] + backward["bytes"] + held * t * d + 2 * held * t * f,
                "flops": forward["flops"] + backward["flops"]}
    v = case["v"]
    # tokens without a loss need none of it but their zeros
    n = t * (1.0 - case["left_out"])
    lists = 12.0 * t + 8.0 * case["k"] * t
    if not case["grad"]:
        return {"bytes": 2 * n * d + 2 * v * d + lists, "flops": 2 * n * v * d}
    return {"bytes": 2 * n * d + 2 * t * d + v * d * (6 if case["acc"] else 4) + lists,
            "flops": 6 * n * v * d}


# ---------------------------------------------------------------- the definition, 64 bits

def _x_two_to(k):
    """2^k of whole numbers k, exactly: the exponent field of a 64-bit number."""
    return ((k.to(torch.int64) + 1023) << 52).view(torch.float64)


def _x_held(x, fmt, dtype):
    """x (64 bits) as its checkpoint holds it: rounded to the type, then block by block."""
    x = x.to(dtype).double()
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


def _x_act(g, act):
    if act == "silu":
        q = 1 / (1 + torch.exp(-g))
        return q * g, q + g * q * (1 - q)
    if act == "gelu":
        q = (1 + torch.erf(g / math.sqrt(2))) / 2
        return q * g, q + g * torch.exp(-g ** 2 / 2) / math.sqrt(2 * math.pi)
    # tanh(y) = 1 - 2 / (e^(2 y) + 1)
    y = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    q = 1 - 1 / (torch.exp(2 * y) + 1)
    slope = math.sqrt(2 / math.pi) * (1 + 0.134145 * g ** 2)
    return q * g, q + g * 2 * q * (1 - q) * slope


def _x_ffn_back(s, x, g, u):
    c = s["case"]
    do, w = s["dout"].double(), s["w"].double()
    f = c["f"]
    a, slope = _x_act(g, c["act"])
    dg, du = slope * u * do, a * do
    dw = torch.cat([dg.t().contiguous() @ x, du.t().contiguous() @ x], 0)
    return {"dx": dg @ w[:f] + du @ w[f:], "dw": dw + s["dw0"].double() if c["acc"] else dw}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ffn_grad":
        return _x_ffn_back(s, *(_x_codes(s[n + "_codes"], s[n + "_scales"], case["fmt"])
                                for n in ("x", "gate", "up")))
    x, w, dt = s["x"].double(), s["w"].double(), s["x"].dtype
    if case["op"].startswith("ffn"):
        f, fmt = case["f"], case["fmt"]
        g, u = x @ w[:f].t(), x @ w[f:].t()
        out = _x_act(g, case["act"])[0] * u
        if case["op"] == "ffn":
            return out
        return {"out": out, **_x_ffn_back(s, _x_held(x, fmt, dt), _x_held(g, fmt, dt),
                                          _x_held(u, fmt, dt))}
    t, tau = case["t"], case["tau"]
    weight = torch.ones(t, dtype=torch.float64, device="cuda")
    if s["weights"] is not None:
        weight = s["weights"].double()
    if case["op"] == "distill":
        ids = s["ids"].long()
        q = torch.softmax((s["top"].double() / tau).masked_fill(ids < 0, -math.inf), 1)
        q = torch.nan_to_num(q, nan=0.0)               # tokens without entries
    else:
        ids = s["targets"][:, None]
        q = (ids >= 0).double()
    weight = weight * (ids >= 0).any(1)
    spare = torch.where(ids < 0, case["v"], ids)       # absent entries: a column of its own
    loss = torch.empty(t, dtype=torch.float64, device="cuda")
    dx, dw = (torch.empty_like(x), torch.zeros_like(w)) if case["grad"] else (None, None)
    for lo in range(0, t, 2048):                       # 64-bit logits of 2048 tokens at a time
        hi = min(t, lo + 2048)
        z = x[lo:hi] @ w.t() / tau
        log_p = z - torch.logsumexp(z, 1, keepdim=True)
        there = torch.cat([log_p, torch.zeros_like(log_p[:, :1])], 1).gather(1, spare[lo:hi])
        qq = q[lo:hi]
        loss[lo:hi] = weight[lo:hi] * tau ** 2 * (torch.special.xlogy(qq, qq) - qq * there).sum(1)
        if case["grad"]:
            dense = torch.zeros((hi - lo, case["v"] + 1), dtype=torch.float64, device="cuda")
            dense.scatter_add_(1, spare[lo:hi], qq)
            dz = (torch.exp(log_p) - dense[:, :-1]) * (s["scale"] * tau * weight[lo:hi, None])
            dx[lo:hi] = dz @ w
            dw += dz.t().contiguous() @ x[lo:hi]
    if not case["grad"]:
        return loss
    return {"loss": loss, "dx": dx, "dw": dw + s["dw0"].double() if case["acc"] else dw}
