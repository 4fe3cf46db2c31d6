"""The losses over more tokens than a piece of logits holds, at a width whose dw comes in
whole large tiles without splits: running sums over the pieces are begun, added to and
finished by the product itself, with and without an old dw, against 64-bit results on the
device.  Bounds as in layer_util."""
import os
import re
import subprocess

import pytest
import torch

import zero_sharded_mixed_bucketed_amd as Z
from act_util import EPS, TINY, TORCH, U
from conftest import ROOT
from gpu_util import need_gpu
from layer_util import product

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
T, D, V, PIECE = 27000, 512, 130000, 9216     # three pieces, the last one smaller


def test_sums_over_pieces_are_the_products_own(tmp_path):
    """dw of a piece: 256 x 256 tiles, no splits, and a last row of tiles that is not whole.
    Several pieces: a call of one needs no running sums."""
    assert T * V * 4 > 2 * 6 * 2 ** 30 and V % 256
    need = [Z.loss_workspace(n, D, V, 0, True, True) - Z.loss_workspace(n, D, V, 0, True, False)
            for n in (PIECE, T)]
    assert need[0] < V * D * 4 <= need[1]
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc is not installed")
    exe, csrc = str(tmp_path / "product_plan_check"), os.path.join(
        ROOT, "zero_sharded_mixed_bucketed_amd", "csrc")
    subprocess.run([HIPCC, "--offload-arch=gfx950", "--offload-host-only", "-O1", "-std=c++17",
                    "-I", os.path.join(ROOT, "include"), "-I", csrc, "-x", "hip",
                    os.path.join(ROOT, "tests", "native", "product_plan_check.cpp"),
                    "-Wl,--unresolved-symbols=ignore-all", "-o", exe], check=True,
                   capture_output=True)
    for k in (PIECE, T - 2 * PIECE):
        out = subprocess.run([exe, str(V), str(D), str(k), "1001"], capture_output=True,
                             text=True, check=True).stdout
        assert re.match(r"tile 256 splits 1 most 1 ", out), out


def _rounded(ref, err, dtype):
    return err + EPS[dtype] * (ref.abs() + err) + TINY[dtype] if dtype != "fp32" else err + U * ref.abs()


def _check(got, ref, bound, what):
    off = (got.double() - ref).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[0], off[bad][0], bound[bad][0])


@pytest.mark.gpu
@pytest.mark.parametrize("k,tau", [(0, 1.0), (20, 2.0)])
@pytest.mark.parametrize("dtype,out,acc", [("bf16", "bf16", True), ("fp16", "fp32", True),
                                           ("bf16", "fp32", False), ("fp16", "fp16", False)])
def test_running_sums_of_whole_large_tiles(k, tau, dtype, out, acc):
    need_gpu()
    print(flush=True)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T + k)
    scale = 0.5

    def normal(shape, dt, sigma):
        return (sigma * torch.randn(shape, generator=gen, device="cuda")).to(TORCH[dt])

    x, w = normal((T, D), dtype, 1.0), normal((V, D), dtype, 1.5 * D ** -0.5)
    ids = torch.randint(0, V, (T, max(k, 1)), generator=gen, device="cuda")
    ids[torch.rand(T, generator=gen, device="cuda") < 0.1] = -1
    dw0 = normal((V, D), out, 0.1) if acc else torch.full((V, D), float("nan"), dtype=TORCH[out],
                                                          device="cuda")
    loss, dx, dw = torch.full((T,), float("nan"), device="cuda"), torch.full_like(x, float("nan")), \
        dw0.clone()
    call = dict(scale=scale, dx=dx, dw=dw, accumulate=acc)
    if k:
        top = torch.randn((T, k), generator=gen, device="cuda")
        Z.distill_loss(x, w, ids, top, loss, temperature=tau, **call)
        q = torch.softmax(top.double() / tau, 1)
    else:
        Z.vocab_loss(x, w, ids[:, 0].contiguous(), loss, **call)
        q = torch.ones((T, 1), device="cuda", dtype=torch.float64)

    w64, c = w.double(), scale * tau
    w_abs = w64.abs()
    dw_ref, dw_err = torch.zeros_like(w64), torch.zeros_like(w64)
    on = torch.nonzero(ids[:, 0] >= 0)[:, 0]
    for at in on.split(512):
        x64, qa, ia = x[at].double(), q[at], ids[at]
        z = x64 @ w64.t() / tau
        lse = torch.logsumexp(z, 1, keepdim=True)
        dense = torch.zeros_like(z).scatter_add_(1, ia, qa)
        ref = tau ** 2 * (torch.special.xlogy(qa, qa) - qa * (z - lse).gather(1, ia)).sum(1)
        dz = (product(D, x64.abs() @ w_abs.t()) / tau + 2 * U * z.abs()).amax(1, keepdim=True)
        gap = z.abs().amax(1) + torch.log(torch.tensor(float(V))).item() + 1
        err = (tau ** 2 * (2 * dz[:, 0] + (V / 512 + 80) * U + 16 * U * gap) + 16 * U * ref.abs())
        _check(loss[at], ref, err, "loss")
        p, far = torch.exp(z - lse), z.amax(1, keepdim=True) - z
        d = p - dense
        err = (p * (2 * dz + (V / 512 + 80 + 4 * far.clamp(max=90.0)) * U)
               + 2 * U * (p + 24 * dense + d.abs()))
        err = err + EPS[dtype] * (d.abs() + err) + TINY[dtype] * (2.0 ** -13 if dtype == "fp16" else 1)
        mag = d.abs() + err
        ref = c * (d @ w64)
        bound = c * (err @ w_abs + product(V, mag @ w_abs))
        _check(dx[at], ref, _rounded(ref, bound * (1 + 4 * U), dtype), "dx")
        dw_ref += c * (d.t().contiguous() @ x64)
        # the sums of all tokens, and those of the pieces
        dw_err += c * (err.t().contiguous() @ x64.abs()
                       + product(len(on), mag.t().contiguous() @ x64.abs()))
    off = ids[:, 0] < 0
    assert (loss[off] == 0).all() and (dx[off] == 0).all()
    if acc:
        dw_ref += dw0.double()
    _check(dw, dw_ref, _rounded(dw_ref, dw_err * (1 + 4 * U) + U * dw_ref.abs(), out), "dw")
