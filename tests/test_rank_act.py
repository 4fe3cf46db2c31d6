"""Where a layer's gradients go in a rank's local gradient (CPU, no kernel runs)."""
import pytest
import torch

from zero_sharded_mixed_bucketed_amd import rank as zr


def _rank(stage, psi=1000):
    return zr.RankState(psi, 2, 0, stage, device=torch.device("cpu"))


def test_stage1_slots_are_views_of_the_retained_local_gradient():
    st = _rank(1)
    slot = st.grad_slot(100, 60)
    assert slot.dtype == torch.float16 and slot.numel() == 60
    assert slot.data_ptr() == st.local_grad.data_ptr() + 200
    slot.fill_(1.0)
    assert int((st.local_grad != 0).sum()) == 60


@pytest.mark.parametrize("stage", [2, 3])
def test_other_stages_fill_the_bucket_in_hand(stage):
    st = _rank(stage)
    bucket = torch.zeros(400, dtype=torch.int16)
    slot = st.grad_slot(650, 50, bucket, 600)
    assert slot.data_ptr() == bucket.data_ptr() + 100 and slot.numel() == 50
    with pytest.raises(ValueError):
        st.grad_slot(0, 10)


@pytest.mark.parametrize("args", [(599, 10), (601, 400), (990, 20), (700, -1)])
def test_slots_outside_the_bucket_are_refused(args):
    with pytest.raises(ValueError):
        _rank(2).grad_slot(*args, torch.zeros(400, dtype=torch.int16), 600)


def test_checkpoint_bytes():
    k = _rank(2).checkpoint(64, 256)
    assert k.resident_bytes() == 64 * 256 * 33 // 32


@pytest.mark.parametrize("lo,offset", [(-5, -10), (-1, -1), (3, -2)])
def test_slots_before_the_flat_vector_are_refused(lo, offset):
    """A place or a bucket that begins before flat index 0 is no part of the local
    gradient, wherever it lies in the bucket."""
    with pytest.raises(ValueError):
        _rank(2).grad_slot(lo, 4, torch.zeros(400, dtype=torch.int16), offset)
