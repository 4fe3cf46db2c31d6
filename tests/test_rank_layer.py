"""Where the gradients of a gated block and of the projection onto the vocabulary go in a
rank's local gradient (CPU, no kernel runs)."""
import pytest
import torch

import zero_sharded_mixed_bucketed_amd as Z
from zero_sharded_mixed_bucketed_amd import rank as zr

D, F, V = 8, 5, 11


def _rank(stage, psi=1000):
    return zr.RankState(psi, 2, 0, stage, device=torch.device("cpu"))


def _call(st, monkeypatch, which, lo, **place):
    """The dw, and the other keywords, that the operator gets."""
    got = {}
    fn = {"gated": "gated_ffn_grad", "loss": "vocab_loss", "distill": "distill_loss"}[which]
    monkeypatch.setattr(zr, fn, lambda *a, **k: got.update(k, args=a))
    x, w = torch.zeros((3, D)), torch.zeros((V, D))
    if which == "gated":
        k = Z.ckpt_empty(3, D, device="cpu")
        st.gated_grad(lo, torch.zeros((3, F)), k, k, k, torch.zeros((2 * F, D)), accumulate=True,
                      **place)
        return got, (2 * F, D)
    if which == "loss":
        st.loss_grad(lo, x, w, torch.zeros(3), torch.zeros(3), accumulate=True, **place)
    else:
        st.distill_grad(lo, x, w, torch.zeros((3, 2)), torch.zeros((3, 2)), torch.zeros(3),
                        accumulate=True, **place)
    return got, (V, D)


@pytest.mark.parametrize("which", ["gated", "loss", "distill"])
def test_stage1_writes_to_the_retained_local_gradient(which, monkeypatch):
    st = _rank(1)
    got, shape = _call(st, monkeypatch, which, 100)
    dw = got["dw"]
    assert dw.shape == shape and dw.dtype == torch.float16 and dw.is_contiguous()
    assert dw.data_ptr() == st.local_grad.data_ptr() + 200 and got["accumulate"] is True


@pytest.mark.parametrize("which", ["gated", "loss", "distill"])
@pytest.mark.parametrize("stage", [2, 3])
def test_other_stages_fill_the_bucket_in_hand(which, stage, monkeypatch):
    bucket = torch.zeros(400, dtype=torch.int16)
    got, shape = _call(_rank(stage), monkeypatch, which, 650, bucket=bucket, bucket_offset=600)
    assert got["dw"].shape == shape and got["dw"].data_ptr() == bucket.data_ptr() + 100


@pytest.mark.parametrize("which", ["gated", "loss", "distill"])
@pytest.mark.parametrize("lo", [-1, 599, 950])
def test_places_outside_the_bucket_are_refused(which, lo, monkeypatch):
    with pytest.raises(ValueError):
        _call(_rank(2), monkeypatch, which, lo, bucket=torch.zeros(400, dtype=torch.int16),
              bucket_offset=600)
