"""The gated block's and the losses' host side (no GPU): every bad argument is
rejected before any device call, by the C ABI and by the binding."""
import ctypes
import math

import pytest
import torch

import zero_sharded_mixed_bucketed_amd as Z

P = 0x10000          # an aligned address that is never read
INVAL, RANGE, ALIGN = Z.ZERO_E_INVAL, Z.ZERO_E_RANGE, Z.ZERO_E_ALIGN


def _ckpt(rows, cols, **kw):
    a = Z._CkptArg()
    a.codes, a.scales, a.rows, a.cols = P, P, rows, cols
    a.code_stride, a.scale_stride, a.format = cols, -(-cols // 32), 0
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _set(a, kw):
    for k, v in kw.items():
        setattr(a, k, ctypes.pointer(v) if isinstance(v, Z._CkptArg) else v)
    return a


def _gated(**kw):
    a = Z._GatedFfnArg()
    a.dtype, a.act, a.rows, a.cols, a.width = 0, 0, 4, 70, 40
    a.x, a.x_stride, a.w, a.w_stride, a.out, a.out_stride = P, 70, P, 70, P, 40
    return Z.lib.zero_gated_ffn(ctypes.byref(_set(a, kw)), None)


SIZES = [(dict(cols=0), INVAL), (dict(rows=(1 << 25) + 1), RANGE),
         (dict(cols=(1 << 22) + 1, x_stride=1 << 23, w_stride=1 << 23), RANGE)]
GATED = SIZES + [
    (dict(dtype=2), INVAL), (dict(dtype=-1), INVAL), (dict(act=3), INVAL), (dict(act=-1), INVAL),
    (dict(width=0), INVAL), (dict(width=(1 << 22) + 1, out_stride=1 << 23), RANGE),
    (dict(x=None), INVAL), (dict(w=None), INVAL), (dict(out=None), INVAL),
    (dict(x_stride=69), RANGE), (dict(w_stride=69), RANGE), (dict(out_stride=39), RANGE),
    (dict(x_stride=1 << 60), RANGE), (dict(x=P + 1), ALIGN), (dict(w=P + 1), ALIGN),
    (dict(out=P + 1), ALIGN), (dict(ckpt_gate=_ckpt(4, 39)), RANGE),
    (dict(ckpt_up=_ckpt(5, 40)), RANGE), (dict(ckpt_out=_ckpt(4, 40, format=2)), INVAL),
    (dict(ckpt_out=_ckpt(4, 40, codes=None)), INVAL),
    (dict(ckpt_gate=_ckpt(4, 40), ckpt_up=_ckpt(4, 40, format=1)), INVAL)]


@pytest.mark.parametrize("kw,want", GATED)
def test_bad_gated_blocks(kw, want):
    assert _gated(**kw) == want and Z.last_error() != ""


def test_a_gated_block_without_rows_is_fine():
    assert _gated(rows=0, x=None, w=None, out=None) == Z.ZERO_OK
    assert Z.lib.zero_gated_ffn(None, None) == INVAL


def _gated_grad(**kw):
    a = Z._GatedFfnGradArg()
    a.dtype, a.act, a.rows, a.cols, a.width = 0, 0, 4, 70, 40
    a.dout, a.dout_stride, a.w, a.w_stride, a.dx, a.dx_stride = P, 40, P, 70, P, 70
    a.dw, a.dw_stride, a.workspace, a.workspace_bytes = P, 70, P, 1 << 40
    _set(a, dict(ckpt_gate=_ckpt(4, 40), ckpt_up=_ckpt(4, 40), ckpt_x=_ckpt(4, 70)))
    return Z.lib.zero_gated_ffn_grad(ctypes.byref(_set(a, kw)), None)


NEED = Z.gated_ffn_grad_workspace(4, 70, 40)


@pytest.mark.parametrize("kw,want", [
    (dict(cols=0), INVAL), (dict(rows=(1 << 25) + 1), RANGE), (dict(dtype=2), INVAL),
    (dict(act=3), INVAL), (dict(width=0), INVAL), (dict(dout=None), INVAL), (dict(w=None), INVAL),
    (dict(dx=None, dw=None), INVAL), (dict(dout_stride=39), RANGE), (dict(w_stride=69), RANGE),
    (dict(dx_stride=69), RANGE), (dict(dw_stride=69), RANGE), (dict(dout=P + 1), ALIGN),
    (dict(dx=P + 1), ALIGN), (dict(dw=P + 1), ALIGN), (dict(dw=P + 2, dw_dtype=2), ALIGN),
    (dict(dw_dtype=1), INVAL), (dict(dw_dtype=3), INVAL), (dict(accumulate=2), INVAL),
    (dict(ckpt_gate=None), INVAL), (dict(ckpt_up=None), INVAL), (dict(ckpt_x=None), INVAL),
    (dict(ckpt_x=_ckpt(4, 71)), RANGE), (dict(ckpt_gate=_ckpt(4, 41)), RANGE),
    (dict(ckpt_gate=_ckpt(4, 40, format=1)), INVAL), (dict(workspace=None), INVAL),
    (dict(workspace_bytes=NEED - 1), RANGE), (dict(workspace=P + 8), ALIGN)])
def test_bad_gated_gradients(kw, want):
    assert _gated_grad(**kw) == want and Z.last_error() != ""


def test_gated_gradient_workspace_and_empty_calls():
    assert NEED >= 4 * 80 * 2
    for bad in ((1 << 26, 70, 40), (4, 0, 40), (4, 70, 0), (4, 1 << 23, 40), (4, 70, 1 << 23)):
        assert Z.gated_ffn_grad_workspace(*bad) == 0
    assert _gated_grad(rows=0, accumulate=1, dout=None, w=None, ckpt_gate=None, ckpt_up=None,
                       ckpt_x=None, workspace=None) == Z.ZERO_OK
    assert _gated_grad(rows=0, dw=None, dx=None, dout=None, w=None, ckpt_gate=None, ckpt_up=None,
                       ckpt_x=None) == Z.ZERO_OK
    assert Z.lib.zero_gated_ffn_grad(None, None) == INVAL


def _base(kw):
    a = Z._LossArg()
    a.dtype, a.rows, a.cols, a.vocab, a.scale = 0, 4, 70, 1000, 1.0
    for name in ("x", "w", "dx", "dw"):
        setattr(a, name, P)
        setattr(a, name + "_stride", 70)
    a.loss, a.workspace, a.workspace_bytes = P, P, 1 << 40
    return _set(a, kw)


def _vocab(targets=P, id_bytes=8, **kw):
    return Z.lib.zero_vocab_loss(ctypes.byref(_base(kw)), targets, id_bytes, None)


def _distill(top=None, **kw):
    t = Z._TopLogitsArg(16, P, 16, 4, P, 16, 2, 2.0)
    return Z.lib.zero_distill_loss(ctypes.byref(_base(kw)), ctypes.byref(_set(t, top or {})), None)


LOSS_NEED = Z.loss_workspace(4, 70, 1000)
LOSSES = [
    (dict(dtype=2), INVAL), (dict(cols=0), INVAL), (dict(vocab=0), INVAL),
    (dict(rows=(1 << 25) + 1), RANGE), (dict(vocab=(1 << 24) + 1), RANGE),
    (dict(cols=(1 << 22) + 1, x_stride=1 << 23, w_stride=1 << 23, dx_stride=1 << 23,
          dw_stride=1 << 23), RANGE),
    (dict(x=None), INVAL), (dict(w=None), INVAL), (dict(loss=None), INVAL),
    (dict(scale=math.inf), INVAL), (dict(scale=math.nan), INVAL), (dict(scale=1e39), INVAL),
    (dict(x_stride=69), RANGE), (dict(w_stride=69), RANGE), (dict(dx_stride=69), RANGE),
    (dict(dw_stride=69), RANGE), (dict(x=P + 1), ALIGN), (dict(w=P + 1), ALIGN),
    (dict(dx=P + 1), ALIGN), (dict(dw=P + 1), ALIGN), (dict(dw=P + 2, dw_dtype=2), ALIGN),
    (dict(loss=P + 2), ALIGN), (dict(weights=P + 2), ALIGN), (dict(dw_dtype=1), INVAL),
    (dict(accumulate=-1), INVAL), (dict(workspace=None), INVAL),
    (dict(workspace_bytes=LOSS_NEED - 1), RANGE), (dict(workspace=P + 8), ALIGN)]


@pytest.mark.parametrize("kw,want", LOSSES)
def test_bad_losses(kw, want):
    assert _vocab(**kw) == want and Z.last_error() != ""
    assert _distill(**kw) == want and Z.last_error() != ""


@pytest.mark.parametrize("kw,want", [(dict(targets=None), INVAL), (dict(id_bytes=2), INVAL),
                                     (dict(targets=P + 4), ALIGN)])
def test_bad_targets(kw, want):
    assert _vocab(**kw) == want and Z.last_error() != ""


@pytest.mark.parametrize("top,want", [
    (dict(top=0), INVAL), (dict(top=1025, ids_stride=1025, logits_stride=1025), INVAL),
    (dict(ids=None), INVAL), (dict(logits=None), INVAL), (dict(id_bytes=1), INVAL),
    (dict(ids=P + 2), ALIGN), (dict(ids=P + 4, id_bytes=8), ALIGN), (dict(logits=P + 2), ALIGN),
    (dict(logits=P + 1, logits_dtype=0), ALIGN), (dict(logits_dtype=3), INVAL),
    (dict(ids_stride=15), RANGE), (dict(logits_stride=15), RANGE), (dict(temperature=0.0), INVAL),
    (dict(temperature=-1.0), INVAL), (dict(temperature=math.nan), INVAL),
    (dict(temperature=math.inf), INVAL), (dict(temperature=1e-45), INVAL),
    (dict(temperature=1e30), INVAL)])
def test_bad_top_logits(top, want):
    assert _distill(top) == want and Z.last_error() != ""


def test_loss_workspace_and_empty_calls():
    full = Z.loss_workspace(8192, 4096, 131072)
    no_dw = Z.loss_workspace(8192, 4096, 131072, 0, True, False)
    # the logits and x of a piece, and the running sums of dw, however many tokens
    assert full == no_dw and 2 ** 32 < no_dw < 2 ** 32 + 2 ** 28
    large = Z.loss_workspace(1 << 20, 4096, 131072, 0, True, False)
    assert large < 6 * 2 ** 30 + 2 ** 29             # x, maxima and sums of a piece beside it
    assert Z.loss_workspace(1 << 20, 4096, 131072) - large >= 131072 * 4096 * 4
    # cross entropy alone stores no logits
    assert Z.loss_workspace(8192, 4096, 131072, 0, False, False) < 2 ** 28
    assert Z.loss_workspace(8192, 4096, 131072, 64, False, False) > 2 ** 31
    assert Z.loss_workspace(8192, 4096, 131072, 1025) == 0
    for bad in ((1 << 26, 70, 1000), (4, 0, 1000), (4, 70, 0), (4, 70, 1 << 25)):
        assert Z.loss_workspace(*bad) == 0
    nothing = dict(rows=0, x=None, w=None, dx=None, loss=None, workspace=None)
    assert _vocab(None, dw=None, **nothing) == Z.ZERO_OK
    assert _vocab(None, accumulate=1, **nothing) == Z.ZERO_OK
    assert _distill(dict(ids=None, logits=None), dw=None, **nothing) == Z.ZERO_OK
    assert Z.lib.zero_vocab_loss(None, P, 8, None) == INVAL
    assert Z.lib.zero_distill_loss(ctypes.byref(_base({})), None, None) == INVAL


def test_the_binding_refuses_host_tensors_and_other_shapes():
    x, w = torch.zeros((4, 8), dtype=torch.float16), torch.zeros((6, 8), dtype=torch.float16)
    with pytest.raises(ValueError):
        Z.gated_ffn(x, w, None)
    with pytest.raises(ValueError):
        Z.gated_ffn_grad(x, None, None, w, dx=x)
    with pytest.raises(ValueError):
        Z.vocab_loss(x, w, torch.zeros(4, dtype=torch.int64), torch.zeros(4))
    with pytest.raises(ValueError):
        Z.vocab_loss(x, w, torch.zeros(4), torch.zeros(4))
    with pytest.raises(ValueError):
        Z.distill_loss(x, w, torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2)),
                       torch.zeros(4))
