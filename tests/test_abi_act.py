"""The activation entry points' host side (no GPU): every bad argument is
rejected before any device call, by the C ABI and by the binding."""
import ctypes
import math

import pytest
import torch

import zero_sharded_mixed_bucketed_amd as Z

P = 0x10000          # an aligned address that is never read


def _ckpt(rows=4, cols=70, **kw):
    a = Z._CkptArg()
    a.codes, a.scales, a.rows, a.cols = P, P, rows, cols
    a.code_stride, a.scale_stride, a.format = cols, -(-cols // 32), 0
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def _code(rc):
    assert rc < 0 and Z.last_error() != ""
    return rc


@pytest.mark.parametrize("kw,want", [
    (dict(codes=None), Z.ZERO_E_INVAL), (dict(scales=None), Z.ZERO_E_INVAL),
    (dict(format=2), Z.ZERO_E_INVAL), (dict(format=-1), Z.ZERO_E_INVAL),
    (dict(code_stride=69), Z.ZERO_E_RANGE), (dict(scale_stride=2), Z.ZERO_E_RANGE),
    (dict(code_stride=1 << 59), Z.ZERO_E_RANGE), (dict(rows=1 << 60), Z.ZERO_E_RANGE)])
def test_bad_checkpoints(kw, want):
    k = _ckpt(**kw)
    r = ctypes.byref(k)
    assert _code(Z.lib.zero_ckpt_write(P, 0, 70, r, None)) == want
    assert _code(Z.lib.zero_ckpt_read(r, P, 2, 70, None)) == want
    assert _code(Z.lib.zero_ckpt_weight_grad(r, P, 0, 8, 8, P, 0, 70, 0, P, 1 << 40, None)) == want


@pytest.mark.parametrize("x,dtype,stride,want", [
    (None, 0, 70, Z.ZERO_E_INVAL), (P, 3, 70, Z.ZERO_E_INVAL), (P, -1, 70, Z.ZERO_E_INVAL),
    (P, 0, 69, Z.ZERO_E_RANGE), (P, 0, 1 << 60, Z.ZERO_E_RANGE), (P + 1, 0, 70, Z.ZERO_E_ALIGN)])
def test_bad_matrices(x, dtype, stride, want):
    k = _ckpt()
    assert _code(Z.lib.zero_ckpt_write(x, dtype, stride, ctypes.byref(k), None)) == want
    assert _code(Z.lib.zero_ckpt_read(ctypes.byref(k), x, dtype, stride, None)) == want


def test_write_takes_no_fp32_and_read_needs_its_alignment():
    k = ctypes.byref(_ckpt())
    assert _code(Z.lib.zero_ckpt_write(P, 2, 70, k, None)) == Z.ZERO_E_INVAL
    assert _code(Z.lib.zero_ckpt_read(k, P + 2, 2, 70, None)) == Z.ZERO_E_ALIGN
    assert _code(Z.lib.zero_ckpt_write(P, 0, 70, None, None)) == Z.ZERO_E_INVAL


def test_nothing_to_store_is_fine():
    for rows, cols in ((0, 70), (4, 0), (0, 0)):
        k = ctypes.byref(_ckpt(rows, cols, codes=None, scales=None))
        assert Z.lib.zero_ckpt_write(None, 0, cols, k, None) == Z.ZERO_OK
        assert Z.lib.zero_ckpt_read(k, None, 2, cols, None) == Z.ZERO_OK


def _wg(k=None, dy=P, dtype=0, n=8, dys=8, dw=P, dwt=0, dws=70, acc=0, ws=P, wsb=1 << 40):
    return Z.lib.zero_ckpt_weight_grad(ctypes.byref(k or _ckpt()), dy, dtype, n, dys, dw, dwt,
                                       dws, acc, ws, wsb, None)


@pytest.mark.parametrize("kw,want", [
    (dict(dy=None), Z.ZERO_E_INVAL), (dict(dw=None), Z.ZERO_E_INVAL),
    (dict(dtype=2), Z.ZERO_E_INVAL), (dict(dtype=0, dwt=1), Z.ZERO_E_INVAL),
    (dict(dwt=3), Z.ZERO_E_INVAL), (dict(acc=2), Z.ZERO_E_INVAL), (dict(dys=7), Z.ZERO_E_RANGE),
    (dict(dws=69), Z.ZERO_E_RANGE), (dict(n=(1 << 22) + 1, dys=1 << 23), Z.ZERO_E_RANGE),
    (dict(dy=P + 1), Z.ZERO_E_ALIGN), (dict(dw=P + 2, dwt=2), Z.ZERO_E_ALIGN),
    (dict(dw=P + 1), Z.ZERO_E_ALIGN)])
def test_bad_weight_gradients(kw, want):
    assert _code(_wg(**kw)) == want


def test_weight_gradient_workspace():
    need = Z.ckpt_weight_grad_workspace(16000, 128, 128)
    assert need > 0 and need % (128 * 128 * 4) == 0
    k = _ckpt(16000, 128)
    kw = dict(k=k, n=128, dys=128, dws=128)
    assert _code(_wg(ws=None, **kw)) == Z.ZERO_E_INVAL
    assert _code(_wg(wsb=need - 1, **kw)) == Z.ZERO_E_RANGE
    assert _code(_wg(ws=P + 8, **kw)) == Z.ZERO_E_ALIGN
    assert Z.ckpt_weight_grad_workspace(16, 128, 128) == 0
    assert Z.ckpt_weight_grad_workspace(0, 128, 128) == 0
    assert Z.ckpt_weight_grad_workspace(100, 0, 128) == 0
    assert Z.ckpt_weight_grad_workspace(100, (1 << 22) + 1, 128) == 0


def test_empty_weight_gradients_are_fine():
    assert _wg(n=0, dw=None) == Z.ZERO_OK
    assert _wg(k=_ckpt(4, 0, codes=None), dw=None) == Z.ZERO_OK
    assert _wg(k=_ckpt(0, 70, codes=None), dy=None, acc=1) == Z.ZERO_OK


def _norm(kind=1, eps=1e-5, weight=P, bias=None):
    n = Z._NormArg()
    n.kind, n.eps, n.weight, n.bias = kind, eps, weight, bias
    return n


def _fwd(**kw):
    a = Z._BlockNormArg()
    a.dtype, a.rows, a.cols, a.scale = 0, 4, 70, 1.0
    for name in ("res", "block", "out", "z"):
        setattr(a, name, P)
        setattr(a, name + "_stride", 70)
    a.stats = P
    a.post, a.pre = _norm(), _norm()
    for k, v in kw.items():
        setattr(a, k, ctypes.pointer(v) if isinstance(v, Z._CkptArg) else v)
    return Z.lib.zero_block_norm(ctypes.byref(a), None)


BAD_NORMS = [
    (dict(dtype=2), Z.ZERO_E_INVAL), (dict(cols=0), Z.ZERO_E_INVAL),
    (dict(cols=16385), Z.ZERO_E_RANGE), (dict(rows=1 << 57), Z.ZERO_E_RANGE),
    (dict(scale=math.nan), Z.ZERO_E_INVAL), (dict(scale=1e39), Z.ZERO_E_INVAL),
    (dict(post=_norm(3)), Z.ZERO_E_INVAL), (dict(pre=_norm(-1)), Z.ZERO_E_INVAL),
    (dict(post=_norm(eps=0.0)), Z.ZERO_E_INVAL), (dict(pre=_norm(eps=math.inf)), Z.ZERO_E_INVAL),
    (dict(pre=_norm(eps=1e-60)), Z.ZERO_E_INVAL), (dict(pre=_norm(weight=P + 1)), Z.ZERO_E_ALIGN),
    (dict(post=_norm(bias=P + 1)), Z.ZERO_E_ALIGN), (dict(post=_norm(0)), Z.ZERO_E_INVAL),
    (dict(gate=P + 1), Z.ZERO_E_ALIGN), (dict(gate=P, gate_stride=69), Z.ZERO_E_RANGE),
    (dict(stats=P + 4), Z.ZERO_E_ALIGN), (dict(ckpt_block=_ckpt(5, 70)), Z.ZERO_E_RANGE),
    (dict(ckpt_out=_ckpt(4, 71)), Z.ZERO_E_RANGE)]


@pytest.mark.parametrize("kw,want", BAD_NORMS + [
    (dict(res=None), Z.ZERO_E_INVAL), (dict(block=None), Z.ZERO_E_INVAL),
    (dict(block=None, gate=P, post=_norm(0, weight=None)), Z.ZERO_E_INVAL),
    (dict(block=None, ckpt_block=_ckpt(), post=_norm(0, weight=None)), Z.ZERO_E_INVAL),
    (dict(z=None), Z.ZERO_E_INVAL), (dict(pre=_norm(0, weight=None)), Z.ZERO_E_INVAL),
    (dict(pre=_norm(0, weight=None), z=None, ckpt_z=_ckpt()), Z.ZERO_E_INVAL),
    (dict(pre=_norm(0, weight=None), z=None, out=None, stats=None), Z.ZERO_E_INVAL),
    (dict(res_stride=69), Z.ZERO_E_RANGE), (dict(out=P + 1), Z.ZERO_E_ALIGN),
    (dict(ckpt_z=_ckpt(format=7)), Z.ZERO_E_INVAL)])
def test_bad_block_norms(kw, want):
    assert _code(_fwd(**kw)) == want


def _bwd(**kw):
    a = Z._BlockNormGradArg()
    a.dtype, a.rows, a.cols, a.scale, a.grad_dtype = 0, 4, 70, 1.0, 2
    for name in ("dout", "dz", "dres", "dblock"):
        setattr(a, name, P)
        setattr(a, name + "_stride", 70)
    a.stats, a.dw_pre, a.dw_post = P, P, P
    a.post, a.pre = _norm(), _norm()
    a.ckpt_out = a.ckpt_block = ctypes.pointer(_ckpt())
    a.workspace, a.workspace_bytes = P, 1 << 40
    for k, v in kw.items():
        setattr(a, k, ctypes.pointer(v) if isinstance(v, Z._CkptArg) else v)
    return Z.lib.zero_block_norm_grad(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,want", [c for c in BAD_NORMS if c[0] != dict(post=_norm(0))] + [
    (dict(dz=None), Z.ZERO_E_INVAL), (dict(ckpt_out=None), Z.ZERO_E_INVAL),
    (dict(ckpt_block=None), Z.ZERO_E_INVAL), (dict(stats=None), Z.ZERO_E_INVAL),
    (dict(dgate=P), Z.ZERO_E_INVAL), (dict(grad_dtype=1), Z.ZERO_E_INVAL),
    (dict(accumulate=2), Z.ZERO_E_INVAL), (dict(workspace=None), Z.ZERO_E_INVAL),
    (dict(workspace_bytes=100), Z.ZERO_E_RANGE), (dict(workspace=P + 4), Z.ZERO_E_ALIGN),
    (dict(dw_pre=P + 2), Z.ZERO_E_ALIGN), (dict(dres_stride=69), Z.ZERO_E_RANGE),
    (dict(gate=P, gate_stride=70, dgate=P, dgate_stride=69), Z.ZERO_E_RANGE),
    (dict(pre=_norm(0, weight=None)), Z.ZERO_E_INVAL),
    (dict(post=_norm(0, weight=None)), Z.ZERO_E_INVAL),
    (dict(dres=None, dblock=None, dw_pre=None, dw_post=None), Z.ZERO_E_INVAL)])
def test_bad_block_norm_gradients(kw, want):
    assert _code(_bwd(**kw)) == want


def test_null_arguments():
    assert _code(Z.lib.zero_block_norm(None, None)) == Z.ZERO_E_INVAL
    assert _code(Z.lib.zero_block_norm_grad(None, None)) == Z.ZERO_E_INVAL


def test_norms_without_rows_are_fine():
    assert _fwd(rows=0, res=None, block=P, z=None) == Z.ZERO_OK
    assert _bwd(rows=0, ckpt_out=None, ckpt_block=None, dz=None, accumulate=1) == Z.ZERO_OK
    assert Z.block_norm_grad_workspace(0, 4096) == 0
    assert Z.block_norm_grad_workspace(10, 0) == 0 and Z.block_norm_grad_workspace(10, 16385) == 0
    assert Z.block_norm_grad_workspace(10, 100) >= 10 * 104 * 4


# ---------------------------------------------------------------- the binding

def test_checkpoint_buffers():
    k = Z.ckpt_empty(5, 70, Z.CKPT_INT8, device=torch.device("cpu"))
    assert k.codes.shape == (5, 70) and k.codes.stride(0) == 80 and k.scales.shape == (5, 3)
    assert (k.rows, k.cols) == (5, 70) and k.resident_bytes() == 5 * 73
    part = k.row_range(1, 4)
    assert part.rows == 3 and part.codes.data_ptr() == k.codes.data_ptr() + 80
    with pytest.raises(ValueError):
        Z.ckpt_empty(5, 70, 9, device=torch.device("cpu"))
    u8 = torch.zeros((4, 64), dtype=torch.uint8)
    for codes, scales in ((u8.int(), u8[:, :2]), (u8, u8[:, :3]), (u8.t(), u8[:, :1]),
                          (u8, u8[:3, :2]), (u8[0], u8[0, :2])):
        with pytest.raises(ValueError):
            Z.Ckpt(codes, scales, Z.CKPT_INT8)


def test_host_tensors_are_refused():
    x = torch.zeros((4, 64), dtype=torch.float16)
    k = Z.ckpt_empty(4, 64, Z.CKPT_INT8, device=torch.device("cpu"))
    n = Z.Norm(Z.NORM_RMS, 1e-5)
    for call in (lambda: Z.ckpt_write(x, k), lambda: Z.ckpt_read(k, x),
                 lambda: Z.ckpt_weight_grad(k, x, torch.zeros(64, 64)),
                 lambda: Z.block_norm(x, x, x, x, None, pre=n),
                 lambda: Z.block_norm_grad(x, x, k, k, None, pre=n, dres=x)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        Z.block_norm_grad(None, None, None, None, None)
