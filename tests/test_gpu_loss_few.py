"""A few tokens with a loss among many rows against the same tokens alone: products cut for
the many rows (whole large tiles, splits by the count, several pieces, operands through
registers) have the same gradients, the rests of their entries among them.

Both sides are within these of the exact values, so of each other twice: the fp32 sums
(layer_util's product), and the gradient by the logits, whose entries' rests are kept in
both (EPS^2), whose other values are rounded once (EPS of p), and whose p is as far off as
its logits' sums.  Without rests on one side dw, in fp32, is EPS of its largest terms off:
a hundred times the bound where p is small."""
import pytest
import torch

import zero_sharded_mixed_bucketed_amd as Z
from act_util import EPS, TORCH, U
from gpu_util import need_gpu
from layer_util import product

pytestmark = pytest.mark.gpu


def _check(got, want, bound, what):
    off = (got.double() - want.double()).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[0], off[bad][0], bound[bad][0])


# dx in 256 x 256 tiles; of more tokens than a piece; odd sizes; in rows of few columns
@pytest.mark.parametrize("rows,d,v", [(8192, 2048, 4104), (27000, 512, 130000),
                                      (3000, 1030, 5001), (5000, 40, 3000)])
@pytest.mark.parametrize("dtype,distil,acc", [("fp16", False, False), ("bf16", True, True),
                                              ("fp16", True, False), ("bf16", False, False)])
@pytest.mark.parametrize("n", [1, 40, 64])
def test_few_tokens_among_many_rows(rows, d, v, dtype, distil, acc, n):
    need_gpu()
    print(flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows + n)
    x = torch.randn((rows, d), generator=gen, device="cuda").to(TORCH[dtype])
    w = (2 * d ** -0.5 * torch.randn((v, d), generator=gen, device="cuda")).to(TORCH[dtype])
    at = torch.randperm(rows, generator=gen, device="cuda")[:n].sort().values
    y = torch.full((rows,), -1, device="cuda")
    y[at] = torch.randint(0, v, (n,), generator=gen, device="cuda")
    weights = torch.rand(rows, generator=gen, device="cuda") + 0.5
    dw0 = torch.randn((v, d), generator=gen, device="cuda") if acc else torch.zeros((v, d), device="cuda")
    scale, got = 0.75, []
    for pick in (torch.arange(rows, device="cuda"), at):
        xs, ys = x[pick], y[pick]
        loss, dx = torch.full((len(pick),), float("nan"), device="cuda"), torch.full_like(xs, 9.0)
        dw = dw0.clone()
        call = dict(weights=weights[pick], scale=scale, dx=dx, dw=dw, accumulate=acc)
        if distil:
            Z.distill_loss(xs, w, ys[:, None], torch.zeros((len(pick), 1), device="cuda"), loss, **call)
        else:
            Z.vocab_loss(xs, w, ys, loss, **call)
        got.append((loss, dx, dw))
    off = y < 0
    assert (got[0][0][off] == 0).all() and (got[0][1][off] == 0).all()

    x64, w64, wt = x[at].double(), w.double(), weights[at].double()[:, None]
    z = x64 @ w64.t()
    dz = (product(d, x64.abs() @ w64.abs().t()) + 2 * U * z.abs()).amax(1, keepdim=True)
    p = torch.softmax(z, 1)
    own = torch.zeros_like(p).scatter_(1, y[at, None], 1.0)
    far = z.amax(1, keepdim=True) - z
    err = wt * (p * (2 * dz + (v / 512 + 80 + 4 * far.clamp(max=90.0)) * U)
                + 2 * U * (p + 24 * own + (p - own).abs()))
    step = torch.where(own > 0, EPS[dtype] ** 2, EPS[dtype])
    tiny = 2.0 ** -25 * 2.0 ** -13 * 1.5                   # fp16's least step, held
    err = err + step * (wt * (p - own).abs() + err) + tiny
    mag = wt * (p - own).abs() + err
    gap = z.abs().amax(1) + torch.log(torch.tensor(float(v))).item() + 1
    loss_err = wt[:, 0] * (2 * dz[:, 0] + (v / 512 + 80) * U + 48 * U * gap)
    _check(got[0][0][at], got[1][0], 2 * loss_err, "loss")
    bound = scale * (err @ w64.abs() + product(2 * v, mag @ w64.abs())) * (1 + 4 * U)
    ref = (scale * ((wt * (p - own)) @ w64)).abs()
    _check(got[0][1][at], got[1][1], 2 * (bound + EPS[dtype] * (ref + bound) + 2.0 ** -25), "dx")
    bound = scale * (err.t().contiguous() @ x64.abs() + product(2 * n, mag.t().contiguous() @ x64.abs()))
    bound = 2 * (bound * (1 + 4 * U) + 2 * U * dw0.double().abs())
    _check(got[0][2], got[1][2], bound, "dw")
    # and what losing the rests on one side would do is seen
    held = 2.0 ** (14 - torch.frexp(weights[at].max()).exponent.item())
    once = ((wt * (p - own)) * held).to(TORCH[dtype]).double() / held
    lost = scale * ((once - wt * (p - own)) * own).t().contiguous() @ x64
    assert (lost.abs() > bound).any()


def test_a_captured_call_follows_the_number_of_tokens():
    """One graph, replayed with none, few, the most that keep rests, one more, and all."""
    need_gpu()
    print(flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    rows, d, v = 200, 72, 900
    x = torch.randn((rows, d), generator=gen, device="cuda").half()
    w = (0.2 * torch.randn((v, d), generator=gen, device="cuda")).half()
    y = torch.randint(0, v, (rows,), generator=gen, device="cuda")
    all_of, loss, dx = y.clone(), torch.empty(rows, device="cuda"), torch.empty_like(x)
    dw = torch.empty((v, d), device="cuda")
    ws = torch.empty(Z.loss_workspace(rows, d, v), dtype=torch.uint8, device="cuda")

    def call():
        Z.vocab_loss(x, w, y, loss, dx=dx, dw=dw, workspace=ws)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for n in (200, 10, 64, 0, 65, 1, 200, 64):
        y.copy_(all_of)
        y[torch.randperm(rows, generator=gen, device="cuda")[n:]] = -1
        call()
        torch.cuda.synchronize()
        want = [t.clone() for t in (loss, dx, dw)]
        for t in (loss, dx, dw, ws):
            t.fill_(99)
        graph.replay()
        _ = torch.randn(1000, device="cuda").sum().item()
        for a, b in zip(want, (loss, dx, dw)):
            assert torch.equal(a, b)
