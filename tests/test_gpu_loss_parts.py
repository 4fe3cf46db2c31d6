"""The losses over parts of the rows, for less workspace: the parts' losses and dx are the
whole call's, and their dw added up in fp32 its dw, within the same bounds (layer_util)."""
import numpy as np
import pytest
import torch

import zero_sharded_mixed_bucketed_amd as Z
from act_util import TORCH, close, f64
from gpu_util import need_gpu
from layer_util import loss_bounds
from oracle import layer

T, D, V = 700, 136, 3000
PARTS = (0, 256, 300, 556, 700)


def test_parts_need_less_workspace():
    """What a call's workspace is made of: about 4 bytes for each row and word, however much
    else it holds, up to 6 GiB of them; nothing of the kind for cross entropy alone."""
    whole = Z.loss_workspace(8192, 4096, 131072)
    for rows in (256, 1024, 4096):
        part = Z.loss_workspace(rows, 4096, 131072)
        assert rows * 131072 * 4 < part < rows * 131072 * 4.2 + 2 ** 27 and part < whole
        assert Z.loss_workspace(rows, 4096, 131072, 64, False, False) > rows * 131072 * 4
        assert Z.loss_workspace(rows, 4096, 131072, 0, False, False) < rows * 2 ** 15


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("k,tau", [(0, 1.0), (9, 2.0)])
def test_parts_of_the_rows_add_up(dtype, k, tau):
    need_gpu()
    print(flush=True)
    rng = np.random.default_rng(6)
    x, w = (torch.from_numpy(s * rng.standard_normal(n)).to(TORCH[dtype]).cuda()
            for s, n in ((1, (T, D)), (2 * D ** -0.5, (V, D))))
    weights = (rng.random(T) + 0.5) * np.where(np.arange(T) < 300, 1.0, 40.0)
    weights = weights.astype(np.float32).astype(np.float64)
    ids = np.stack([rng.permutation(V)[:max(k, 1)] for _ in range(T)])
    ids[rng.random(T) < 0.3] = -1
    ids[256:300] = -1                                  # a part without a loss
    top, scale = rng.standard_normal((T, max(k, 1))).astype(np.float32), 0.25
    dev = [torch.from_numpy(v).cuda() for v in (ids, top, weights.astype(np.float32))]
    loss, dx = torch.empty(T, device="cuda"), torch.empty_like(x)
    dw = torch.empty((V, D), device="cuda")
    need = Z.loss_workspace(max(np.diff(PARTS)), D, V, k)
    assert need < 0.6 * Z.loss_workspace(T, D, V, k)
    workspace = torch.empty(need, dtype=torch.uint8, device="cuda")
    for lo, hi in zip(PARTS, PARTS[1:]):
        call = dict(weights=dev[2][lo:hi], scale=scale, dx=dx[lo:hi], dw=dw, accumulate=lo > 0,
                    workspace=workspace)
        if k:
            Z.distill_loss(x[lo:hi], w, dev[0][lo:hi], dev[1][lo:hi], loss[lo:hi],
                           temperature=tau, **call)
        else:
            Z.vocab_loss(x[lo:hi], w, dev[0][lo:hi, 0].contiguous(), loss[lo:hi], **call)
    q = None
    if k:
        want = layer.distill_loss(f64(x), f64(w), ids, top.astype(np.float64), tau, weights, scale)
        q, shares = np.zeros((T, V)), layer.shares_of(ids, top.astype(np.float64), tau)
        for r, j in zip(*np.nonzero(ids >= 0)):
            q[r, ids[r, j]] += shares[r, j]
    else:
        want = layer.vocab_loss(f64(x), f64(w), ids[:, 0], weights, scale)
    bounds = loss_bounds(f64(x), f64(w), want[1], want[0], weights, tau, scale, dtype,
                         weights.max(), q)
    close(f64(loss), want[0], bounds[0], "fp32", "loss")
    close(f64(dx), want[2], bounds[1], dtype, "dx")
    close(f64(dw), want[3], bounds[2], "fp32", "dw")
