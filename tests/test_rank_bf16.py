"""A rank's local gradient is fp16: activations in bf16, whose gradients the operators
give in bf16 or fp32, are refused with that reason before anything runs (CPU)."""
import pytest
import torch

import zero_sharded_mixed_bucketed_amd as Z
from zero_sharded_mixed_bucketed_amd import rank as zr

D, F, V = 8, 5, 11


@pytest.mark.parametrize("which", ["gated", "loss", "distill"])
@pytest.mark.parametrize("stage", [1, 2, 3])
def test_bf16_activations_are_refused_with_the_reason(which, stage, monkeypatch):
    ran = []
    for fn in ("gated_ffn_grad", "vocab_loss", "distill_loss"):
        monkeypatch.setattr(zr, fn, lambda *a, **k: ran.append(a))
    st = zr.RankState(1000, 2, 0, stage, device=torch.device("cpu"))
    bucket = None if stage == 1 else torch.zeros(400, dtype=torch.int16)

    def call(dt):
        if which == "gated":
            k = Z.ckpt_empty(3, D, device="cpu")
            st.gated_grad(10, torch.zeros((3, F), dtype=dt), k, k, k,
                          torch.zeros((2 * F, D), dtype=dt), bucket=bucket)
            return
        x, w = torch.zeros((3, D), dtype=dt), torch.zeros((V, D), dtype=dt)
        if which == "loss":
            st.loss_grad(10, x, w, torch.zeros(3), torch.zeros(3), bucket=bucket)
        else:
            st.distill_grad(10, x, w, torch.zeros((3, 2)), torch.zeros((3, 2)), torch.zeros(3),
                            bucket=bucket)

    with pytest.raises(ValueError, match="local gradient is fp16"):
        call(torch.bfloat16)
    assert ran == []
    call(torch.float16)
    assert len(ran) == 1
