"""Python binding of libzero: the per-rank data-parallel hot path of ZeRO
stages 1 and 2 on one MI355X.

Argument marshalling only: every step runs in the HIP kernels of libzero.so
(``csrc/``).  Torch tensors supply device memory and the HIP stream.  The
names follow the C ABI in ``include/zero.h``:

    memory_model(psi, nd, stage)                -> bytes per device
    memory_model_k(psi, nd, stage, k)           -> the same with K bytes of optimizer state
    comm_volume(psi, nd, stage)                 -> Comm (collectives and elements per step)
    shard_geometry(psi, nd, rank)               -> Geom
    bucket_intersect(geom, offset, length)      -> (lo, hi)
    reduce_shard(geom, bucket_offset, bucket_len, slices, grad32, grad16=None)
    adam_scalars(lr, beta1, beta2, eps, step)   -> 7 fp32 scalars
    adam_step_shard(geom, master, m, v, grad, param16, param16_origin,
                    lr, beta1, beta2, eps, step)
    gather_params(psi, nd, lo, length, shards, out)
    launch_occupancy(kernel)                    -> (workgroups per CU, dynamic LDS bytes)

and, for the activations a rank keeps for its backward pass and the local
gradient they give:

    ckpt_empty(rows, cols, fmt)                 -> Ckpt (an 8-bit checkpoint's buffers)
    ckpt_write(x, ckpt)                         fp16/bf16 -> 8 bits
    ckpt_read(ckpt, out)                        8 bits -> fp16/bf16/fp32
    ckpt_weight_grad(ckpt, dy, dw)              a linear layer's weight gradient
    block_norm(res, block, out, z, stats)       the norms around a block, gate, residual scale
    block_norm_grad(dout, dz, ckpt_out, ckpt_block, stats)   their backward

Importing this package fails if libzero.so has not been built: there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libzero.so")

ZERO_OK = 0
ZERO_E_INVAL = -1
ZERO_E_RANGE = -2
ZERO_E_ALIGN = -3
ZERO_E_DEVICE = -4

STAGE_DP, STAGE_OS, STAGE_OS_G, STAGE_OS_G_P = 0, 1, 2, 3

# Symbols that include/zero.h declares.
EXPORTS = ("zero_memory_model", "zero_memory_model_k", "zero_comm_volume",
           "zero_shard_geometry", "zero_bucket_intersect", "zero_row_stride",
           "zero_reduce_shard", "zero_adam_scalars", "zero_adam_step_shard",
           "zero_gather_params", "zero_launch_occupancy", "zero_last_error",
           "zero_ckpt_write", "zero_ckpt_read", "zero_ckpt_weight_grad",
           "zero_ckpt_weight_grad_workspace", "zero_block_norm", "zero_block_norm_grad",
           "zero_block_norm_grad_workspace")

# Kernels of zero_launch_occupancy.
KERNEL_REDUCE_W16, KERNEL_REDUCE_W8, KERNEL_REDUCE_W4, KERNEL_REDUCE_W2 = 0, 1, 2, 3
KERNEL_ADAM_G32, KERNEL_ADAM_G16 = 4, 5

# Formats of an 8-bit checkpoint, and the columns that share a scale byte.
CKPT_INT8, CKPT_E4M3 = 0, 1
CKPT_BLOCK = 32

# Kinds of norm, and the widest row they take.
NORM_NONE, NORM_RMS, NORM_LAYER = 0, 1, 2
NORM_MAX_COLS = 16384


class ZeroError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libzero error {code}: {msg}")
        self.code = code


class Geom(ctypes.Structure):
    _fields_ = [("psi", ctypes.c_uint64), ("nd", ctypes.c_uint32), ("rank", ctypes.c_uint32),
                ("offset", ctypes.c_uint64), ("len", ctypes.c_uint64)]

    def __repr__(self):
        return (f"Geom(psi={self.psi}, nd={self.nd}, rank={self.rank}, offset={self.offset}, "
                f"len={self.len})")


class Comm(ctypes.Structure):
    _fields_ = [("reduce_scatters", ctypes.c_uint32), ("all_gathers", ctypes.c_uint32),
                ("elems", ctypes.c_double), ("elems_sent_per_rank", ctypes.c_double),
                ("bytes_sent_per_rank", ctypes.c_double)]


class Shard(ctypes.Structure):
    _fields_ = [("master", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("grad", ctypes.c_void_p), ("grad_is_fp16", ctypes.c_int),
                ("param16", ctypes.c_void_p), ("param16_origin", ctypes.c_uint64),
                ("param16_len", ctypes.c_uint64)]


class _CkptArg(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("rows", ctypes.c_uint64), ("cols", ctypes.c_uint64),
                ("code_stride", ctypes.c_uint64), ("scale_stride", ctypes.c_uint64),
                ("format", ctypes.c_int)]


class _NormArg(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int), ("eps", ctypes.c_double), ("weight", ctypes.c_void_p),
                ("bias", ctypes.c_void_p)]


class _BlockNormArg(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("rows", ctypes.c_uint64), ("cols", ctypes.c_uint64),
                ("res", ctypes.c_void_p), ("res_stride", ctypes.c_uint64),
                ("block", ctypes.c_void_p), ("block_stride", ctypes.c_uint64),
                ("gate", ctypes.c_void_p), ("gate_stride", ctypes.c_uint64),
                ("scale", ctypes.c_double), ("post", _NormArg), ("pre", _NormArg),
                ("out", ctypes.c_void_p), ("out_stride", ctypes.c_uint64),
                ("z", ctypes.c_void_p), ("z_stride", ctypes.c_uint64),
                ("stats", ctypes.c_void_p), ("ckpt_block", ctypes.POINTER(_CkptArg)),
                ("ckpt_out", ctypes.POINTER(_CkptArg)), ("ckpt_z", ctypes.POINTER(_CkptArg))]


class _BlockNormGradArg(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("rows", ctypes.c_uint64), ("cols", ctypes.c_uint64),
                ("dout", ctypes.c_void_p), ("dout_stride", ctypes.c_uint64),
                ("dz", ctypes.c_void_p), ("dz_stride", ctypes.c_uint64),
                ("ckpt_out", ctypes.POINTER(_CkptArg)),
                ("ckpt_block", ctypes.POINTER(_CkptArg)), ("stats", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("gate_stride", ctypes.c_uint64),
                ("scale", ctypes.c_double), ("post", _NormArg), ("pre", _NormArg),
                ("dres", ctypes.c_void_p), ("dres_stride", ctypes.c_uint64),
                ("dblock", ctypes.c_void_p), ("dblock_stride", ctypes.c_uint64),
                ("dgate", ctypes.c_void_p), ("dgate_stride", ctypes.c_uint64),
                ("dw_pre", ctypes.c_void_p), ("db_pre", ctypes.c_void_p),
                ("dw_post", ctypes.c_void_p), ("db_post", ctypes.c_void_p),
                ("grad_dtype", ctypes.c_int), ("accumulate", ctypes.c_int),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_uint64)]


def hip_runtimes() -> set:
    """Paths of every HIP runtime library mapped into this process."""
    try:
        with open("/proc/self/maps") as f:
            return {line.split()[-1] for line in f if "libamdhip64" in line}
    except OSError:
        return set()


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m zero_sharded_mixed_bucketed_amd._build`")
    # torch ships its own HIP runtime; loading torch first makes libzero's
    # libamdhip64.so.7 dependency resolve to that same, already-mapped runtime.
    # Two runtimes in one process would each own the GPU and hand each other
    # pointers they do not know.
    import torch  # noqa: F401
    lib = ctypes.CDLL(LIB_PATH)
    if len(hip_runtimes()) > 1:
        raise ImportError(f"two HIP runtimes are mapped: {sorted(hip_runtimes())}; "
                          "import torch before any other HIP library")
    u64, u32, vp, ci, dbl = (ctypes.c_uint64, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_int,
                             ctypes.c_double)
    G = ctypes.POINTER(Geom)
    lib.zero_memory_model.argtypes = [u64, u32, ci]
    lib.zero_memory_model.restype = dbl
    lib.zero_memory_model_k.argtypes = [u64, u32, ci, dbl]
    lib.zero_memory_model_k.restype = dbl
    lib.zero_comm_volume.argtypes = [u64, u32, ci, ctypes.POINTER(Comm)]
    lib.zero_comm_volume.restype = ci
    lib.zero_shard_geometry.argtypes = [u64, u32, u32, G]
    lib.zero_shard_geometry.restype = ci
    lib.zero_bucket_intersect.argtypes = [G, u64, u64, ctypes.POINTER(u64), ctypes.POINTER(u64)]
    lib.zero_bucket_intersect.restype = ci
    lib.zero_row_stride.argtypes = [u64, ctypes.POINTER(u64)]
    lib.zero_row_stride.restype = ci
    lib.zero_reduce_shard.argtypes = [G, u64, u64, vp, u64, vp, vp, vp]
    lib.zero_reduce_shard.restype = ci
    lib.zero_adam_scalars.argtypes = [dbl, dbl, dbl, dbl, u64, ctypes.POINTER(ctypes.c_float)]
    lib.zero_adam_scalars.restype = ci
    lib.zero_adam_step_shard.argtypes = [G, ctypes.POINTER(Shard), dbl, dbl, dbl, dbl, u64, vp]
    lib.zero_adam_step_shard.restype = ci
    lib.zero_gather_params.argtypes = [u64, u32, u64, u64, vp, u64, vp, vp]
    lib.zero_gather_params.restype = ci
    lib.zero_launch_occupancy.argtypes = [ci, ctypes.POINTER(ci), ctypes.POINTER(u32)]
    lib.zero_launch_occupancy.restype = ci
    K = ctypes.POINTER(_CkptArg)
    lib.zero_ckpt_write.argtypes = [vp, ci, u64, K, vp]
    lib.zero_ckpt_write.restype = ci
    lib.zero_ckpt_read.argtypes = [K, vp, ci, u64, vp]
    lib.zero_ckpt_read.restype = ci
    lib.zero_ckpt_weight_grad_workspace.argtypes = [u64, u64, u64]
    lib.zero_ckpt_weight_grad_workspace.restype = u64
    lib.zero_ckpt_weight_grad.argtypes = [K, vp, ci, u64, u64, vp, ci, u64, ci, vp, u64, vp]
    lib.zero_ckpt_weight_grad.restype = ci
    lib.zero_block_norm.argtypes = [ctypes.POINTER(_BlockNormArg), vp]
    lib.zero_block_norm.restype = ci
    lib.zero_block_norm_grad_workspace.argtypes = [u64, u64]
    lib.zero_block_norm_grad_workspace.restype = u64
    lib.zero_block_norm_grad.argtypes = [ctypes.POINTER(_BlockNormGradArg), vp]
    lib.zero_block_norm_grad.restype = ci
    lib.zero_last_error.argtypes = []
    lib.zero_last_error.restype = ctypes.c_char_p
    return lib


lib = _load()


def last_error() -> str:
    return lib.zero_last_error().decode()


def _check(rc: int) -> None:
    if rc != ZERO_OK:
        raise ZeroError(rc, last_error())


def memory_model(psi: int, nd: int, stage: int) -> float:
    """Model-state bytes per device for stage 0 (DP), 1, 2 or 3."""
    b = lib.zero_memory_model(psi, nd, stage)
    if b < 0:
        raise ZeroError(ZERO_E_INVAL, last_error())
    return b


def memory_model_k(psi: int, nd: int, stage: int, k: float) -> float:
    """Model-state bytes per device with K bytes of optimizer state per parameter."""
    b = lib.zero_memory_model_k(psi, nd, stage, k)
    if b < 0:
        raise ZeroError(ZERO_E_INVAL, last_error())
    return b


def comm_volume(psi: int, nd: int, stage: int) -> Comm:
    """Per-step communication of one rank for stage 0 (DP), 1, 2 or 3."""
    c = Comm()
    _check(lib.zero_comm_volume(psi, nd, stage, ctypes.byref(c)))
    return c


def shard_geometry(psi: int, nd: int, rank: int) -> Geom:
    g = Geom()
    _check(lib.zero_shard_geometry(psi, nd, rank, ctypes.byref(g)))
    return g


def bucket_intersect(geom: Geom, offset: int, length: int) -> Tuple[int, int]:
    lo, hi = ctypes.c_uint64(), ctypes.c_uint64()
    _check(lib.zero_bucket_intersect(ctypes.byref(geom), offset, length, ctypes.byref(lo),
                                     ctypes.byref(hi)))
    return lo.value, hi.value


def row_stride(length: int) -> int:
    """Advised stride (elements) between the Nd gradient rows of `length` columns."""
    out = ctypes.c_uint64()
    _check(lib.zero_row_stride(length, ctypes.byref(out)))
    return out.value


def adam_scalars(lr: float, beta1: float, beta2: float, eps: float, step: int):
    """(b1, b2, c1, c2, eps, step_size, isb) as fp32 values (Python floats)."""
    out = (ctypes.c_float * 7)()
    _check(lib.zero_adam_scalars(lr, beta1, beta2, eps, step, out))
    return tuple(out)


def launch_occupancy(kernel: int, device=None) -> Tuple[int, int]:
    """(workgroups per CU, dynamic LDS bytes) of a capped kernel's launches on
    `device` (default: the current device)."""
    import torch
    wgs, lds = ctypes.c_int(), ctypes.c_uint32()
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
    with torch.cuda.device(dev):
        _check(lib.zero_launch_occupancy(kernel, ctypes.byref(wgs), ctypes.byref(lds)))
    return wgs.value, lds.value


def _one_device(tensors, stream):
    """The one device every tensor of a call (and the stream, if given) is on."""
    dev = tensors[0].device
    for t in tensors[1:]:
        if t.device != dev:
            raise ValueError(f"tensors of one call are on {dev} and {t.device}")
    if stream is not None and stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    return dev


def _launch(tensors, stream, call) -> None:
    """Runs call(stream_handle) with the tensors' device current: the library
    launches on the current device, on the given stream (default: that
    device's current stream)."""
    import torch
    dev = _one_device([t for t in tensors if t is not None], stream)
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    handle = ctypes.c_void_p(s.cuda_stream)
    if torch.cuda.current_device() == dev.index:
        _check(call(handle))
    else:
        with torch.cuda.device(dev):
            _check(call(handle))


def _dev(t, name, dtypes, numel_at_least=None):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if numel_at_least is not None and t.numel() < numel_at_least:
        raise ValueError(f"{name} holds {t.numel()} elements, needs {numel_at_least}")


def reduce_shard(geom: Geom, bucket_offset: int, bucket_len: int, slices, grad32,
                 grad16=None, stream=None) -> None:
    """The owner's reduce of one bucket (or chunk) into grad32 and/or grad16.

    slices: int16/float16 device tensor [Nd, >= bucket_len] (row stride =
    slices.stride(0)); row k is rank k's local gradient over the bucket.
    grad32: float32 [geom.len] or None; grad16: int16/float16 [geom.len] or
    None (not both None).  An output may alias a row column for column.
    """
    import torch
    f16 = (torch.int16, torch.float16)
    _dev(slices, "slices", f16)
    if slices.dim() != 2 or slices.shape[0] != geom.nd or slices.stride(1) != 1 \
            or slices.shape[1] < bucket_len:
        raise ValueError("slices must be [Nd, >= bucket_len] with unit column stride")
    if grad32 is None and grad16 is None:
        raise ValueError("grad32 and grad16 are both None")
    if grad32 is not None:
        _dev(grad32, "grad32", (torch.float32,), geom.len)
        if not grad32.is_contiguous():
            raise ValueError("grad32 must be contiguous")
    if grad16 is not None:
        _dev(grad16, "grad16", f16, geom.len)
        if not grad16.is_contiguous():
            raise ValueError("grad16 must be contiguous")
    _launch((slices, grad32, grad16), stream, lambda h: lib.zero_reduce_shard(
        ctypes.byref(geom), bucket_offset, bucket_len, slices.data_ptr(), slices.stride(0),
        grad32.data_ptr() if grad32 is not None else None,
        grad16.data_ptr() if grad16 is not None else None, h))


def adam_step_shard(geom: Geom, master, m, v, grad, param16: Optional[object],
                    param16_origin: int, lr: float, beta1: float, beta2: float, eps: float,
                    step: int, stream=None) -> None:
    """One fused Adam step on the shard; writes the fp16 slot of param16.

    master/m/v: float32 [geom.len], updated in place.  grad: float32, or
    int16/float16 fp16 bits, [geom.len].  param16: int16/float16 window of the
    flat fp16 parameter vector starting at flat index param16_origin, or None.
    """
    import torch
    for name, t in (("master", master), ("m", m), ("v", v)):
        _dev(t, name, (torch.float32,), geom.len)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    _dev(grad, "grad", (torch.float32, torch.int16, torch.float16), geom.len)
    if not grad.is_contiguous():
        raise ValueError("grad must be contiguous")
    s = Shard()
    s.master, s.m, s.v = master.data_ptr(), m.data_ptr(), v.data_ptr()
    s.grad = grad.data_ptr()
    s.grad_is_fp16 = 0 if grad.dtype == torch.float32 else 1
    if param16 is not None:
        _dev(param16, "param16", (torch.int16, torch.float16))
        if not param16.is_contiguous():
            raise ValueError("param16 must be contiguous")
        s.param16 = param16.data_ptr()
        s.param16_origin = param16_origin
        s.param16_len = param16.numel()
    _launch((master, m, v, grad, param16), stream, lambda h: lib.zero_adam_step_shard(
        ctypes.byref(geom), ctypes.byref(s), lr, beta1, beta2, eps, step, h))


def gather_params(psi: int, nd: int, lo: int, length: int, shards, out, stream=None) -> None:
    """Stage 3: the fp16 parameters of flat [lo, lo + length) into out, from the
    rank shards (int16/float16 device tensor [Nd, >= S], row k = rank k's
    shard, unit column stride)."""
    import torch
    f16 = (torch.int16, torch.float16)
    _dev(shards, "shards", f16)
    s = -(-psi // nd) if nd > 0 else 0
    if shards.dim() != 2 or shards.shape[0] != nd or shards.stride(1) != 1 \
            or shards.shape[1] < s:
        raise ValueError("shards must be [Nd, >= S] with unit column stride")
    _dev(out, "out", f16, length)
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    _launch((shards, out), stream, lambda h: lib.zero_gather_params(
        psi, nd, lo, length, shards.data_ptr(), shards.stride(0), out.data_ptr(), h))


import torch  # noqa: E402  (after _load, which decides which HIP runtime is mapped)

# ---------------------------------------------------------------------------
# Activations: 8-bit checkpoints, the weight gradient from them, block norms.

_CUDA = torch.device("cuda")    # the current device
_F16_BF16 = (torch.float16, torch.bfloat16)
_FLOATS = (torch.float16, torch.bfloat16, torch.float32)
_CODE = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}


def _matrix(t, name, dtypes, shape=None):
    """(address, row stride) of a device matrix with unit column stride and, if
    given, this shape."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    got = t.shape
    if len(got) != 2:
        raise ValueError(f"{name} must be a matrix with unit column stride")
    if shape is not None and got != shape:
        raise ValueError(f"{name} is {tuple(got)}, expected {tuple(shape)}")
    stride, unit = t.stride()
    if unit != 1 and got[1] > 1:
        raise ValueError(f"{name} must be a matrix with unit column stride")
    return t.data_ptr(), stride if got[0] > 1 else got[1]


def _row(t, name, dtype, cols):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != (cols,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous row of {cols}")
    return t.data_ptr()


def _index(tensors, stream) -> int:
    """The index of the one device that a call's tensors (and stream) are on."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError(f"tensors of one call are on {tensors[0].device} and {t.device}")
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {tensors[0].device}")
    return dev


def _call(dev, stream, call, *args) -> None:
    """call(*args, stream handle) with device `dev` current: on the given stream, or on
    that device's current one."""
    handle = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        rc = call(*args, handle)
    else:
        with torch.cuda.device(dev):
            rc = call(*args, handle)
    if rc != ZERO_OK:
        raise ZeroError(rc, last_error())


class Ckpt:
    """An 8-bit checkpoint's buffers: codes uint8 [rows, cols] and scales uint8
    [rows, ceil(cols / 32)], each with unit column stride, in format CKPT_INT8
    or CKPT_E4M3."""

    def __init__(self, codes, scales, fmt: int):
        if fmt not in (CKPT_INT8, CKPT_E4M3):
            raise ValueError(f"unknown checkpoint format {fmt}")
        for name, t in (("codes", codes), ("scales", scales)):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or t.dim() != 2 \
                    or (t.shape[1] > 1 and t.stride(1) != 1):
                raise ValueError(f"{name} must be a uint8 matrix with unit column stride")
        rows, cols = codes.shape
        if tuple(scales.shape) != (rows, -(-cols // CKPT_BLOCK)):
            raise ValueError(f"scales is {tuple(scales.shape)}, expected "
                             f"{(rows, -(-cols // CKPT_BLOCK))}")
        if codes.device != scales.device:
            raise ValueError(f"codes and scales are on {codes.device} and {scales.device}")
        self.codes, self.scales, self.fmt = codes, scales, fmt

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    @property
    def cols(self) -> int:
        return self.codes.shape[1]

    def tensors(self):
        return self.codes, self.scales

    def resident_bytes(self) -> int:
        """Bytes of codes and scales, without what lies between rows."""
        return self.codes.numel() + self.scales.numel()

    def row_range(self, lo: int, hi: int) -> "Ckpt":
        """The checkpoint of rows [lo, hi), sharing memory: a rank of a group that
        partitions a checkpoint by tokens writes its own range, and a checkpoint
        gathered in rank order is read as one."""
        return Ckpt(self.codes[lo:hi], self.scales[lo:hi], self.fmt)

    def _arg(self):
        codes, scales = self.codes, self.scales
        if not codes.is_cuda or not scales.is_cuda:
            raise ValueError("a checkpoint's codes and scales must be device tensors")
        rows, cols = codes.shape
        return _CkptArg(codes.data_ptr(), scales.data_ptr(), rows, cols,
                        codes.stride(0) if rows > 1 else cols,
                        scales.stride(0) if rows > 1 else scales.shape[1], self.fmt)


def ckpt_empty(rows: int, cols: int, fmt: int = CKPT_INT8, device=None) -> Ckpt:
    """Uninitialised buffers of a checkpoint, code rows on 16 bytes."""
    if fmt not in (CKPT_INT8, CKPT_E4M3):
        raise ValueError(f"unknown checkpoint format {fmt}")
    dev = _CUDA if device is None else device
    k = Ckpt.__new__(Ckpt)
    k.codes = torch.empty_strided((rows, cols), (-(-cols // 16) * 16, 1), dtype=torch.uint8,
                                  device=dev)
    k.scales = torch.empty((rows, -(-cols // CKPT_BLOCK)), dtype=torch.uint8, device=dev)
    k.fmt = fmt
    return k


def _workspace(given, need, dev, stream):
    """(address, bytes, tensor) of a call's workspace: the caller's, or one from the
    caching allocator of the call's stream."""
    if given is not None:
        _dev(given, "workspace", (torch.uint8,), need)
        if not given.is_contiguous():
            raise ValueError("workspace must be contiguous")
        if given.get_device() != dev:
            raise ValueError(f"the workspace is on {given.device}, the tensors on device {dev}")
        return given.data_ptr(), given.numel(), given
    if need == 0:
        return None, 0, None
    if stream is None:
        t = torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", dev))
    else:
        with torch.cuda.stream(stream):
            t = torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", dev))
    return t.data_ptr(), need, t


def ckpt_write(x, ckpt: Ckpt, stream=None) -> None:
    """Stores x (float16/bfloat16 [rows, cols], any row stride) in 8 bits."""
    ptr, stride = _matrix(x, "x", _F16_BF16, ckpt.codes.shape)
    dev = _index((x, ckpt.codes, ckpt.scales), stream)
    _call(dev, stream, lib.zero_ckpt_write, ptr, _CODE[x.dtype], stride,
          ctypes.byref(ckpt._arg()))


def ckpt_read(ckpt: Ckpt, out, stream=None) -> None:
    """Reads the held values into out (float16/bfloat16/float32 [rows, cols])."""
    ptr, stride = _matrix(out, "out", _FLOATS, ckpt.codes.shape)
    dev = _index((out, ckpt.codes, ckpt.scales), stream)
    _call(dev, stream, lib.zero_ckpt_read, ctypes.byref(ckpt._arg()),
          ptr, _CODE[out.dtype], stride)


def ckpt_weight_grad_workspace(rows: int, cols: int, n: int) -> int:
    """Bytes of workspace of ckpt_weight_grad at these sizes (0: none)."""
    return lib.zero_ckpt_weight_grad_workspace(rows, cols, n)


def ckpt_weight_grad(ckpt: Ckpt, dy, dw, accumulate: bool = False, workspace=None,
                     stream=None) -> None:
    """dw (+)= dy^T x of a linear layer y = x W^T, from its input's checkpoint.

    dy: float16/bfloat16 [rows, n]; dw: dy's type or float32 [n, cols], e.g. the
    tensor's place in the flat local gradient.  workspace: uint8 device tensor of
    ckpt_weight_grad_workspace bytes, or None to take it from torch's allocator.
    """
    rows, cols = ckpt.codes.shape
    py, sy = _matrix(dy, "dy", _F16_BF16)
    n = dy.shape[1]
    if dy.shape[0] != rows:
        raise ValueError(f"dy has {dy.shape[0]} rows, the checkpoint {rows}")
    pw, sw = _matrix(dw, "dw", (dy.dtype, torch.float32), (n, cols))
    dev = _index((dy, dw, ckpt.codes, ckpt.scales), stream)
    ws, ws_bytes, held = _workspace(workspace, lib.zero_ckpt_weight_grad_workspace(rows, cols, n),
                                    dev, stream)
    _call(dev, stream, lib.zero_ckpt_weight_grad, ctypes.byref(ckpt._arg()), py,
          _CODE[dy.dtype], n, sy, pw, _CODE[dw.dtype], sw, int(bool(accumulate)), ws, ws_bytes)


class Norm:
    """A norm: kind NORM_RMS or NORM_LAYER (or NORM_NONE), eps, and a row of
    weights and of biases (None: ones, zeros)."""

    def __init__(self, kind: int = NORM_NONE, eps: float = 1e-5, weight=None, bias=None):
        self.kind, self.eps, self.weight, self.bias = kind, eps, weight, bias

    def _arg(self, name, dtype, cols, tensors):
        w, b = self.weight, self.bias
        pw = pb = None
        if w is not None:
            pw = _row(w, name + " weight", dtype, cols)
            tensors.append(w)
        if b is not None:
            pb = _row(b, name + " bias", dtype, cols)
            tensors.append(b)
        return _NormArg(self.kind, self.eps, pw, pb)


_NO_NORM = Norm()


def _gate(gate, dtype, shape, tensors):
    """(address, row stride): a stride of 0 for one row of gates."""
    if gate is None:
        return None, 0
    tensors.append(gate)
    if isinstance(gate, torch.Tensor) and gate.dim() == 1:
        return _row(gate, "gate", dtype, shape[1]), 0
    ptr, stride = _matrix(gate, "gate", (dtype,), shape)
    if stride == 0:
        raise ValueError("gate: give one row for every token as a [cols] tensor")
    return ptr, stride


def _stats(stats, rows, tensors):
    if stats is None:
        return None
    _dev(stats, "stats", (torch.float32,))
    if stats.shape != (rows, 4) or not stats.is_contiguous():
        raise ValueError(f"stats must be a contiguous [{rows}, 4] tensor")
    tensors.append(stats)
    return stats.data_ptr()


def _optional(t, name, dtypes, shape, tensors):
    if t is None:
        return None, 0
    tensors.append(t)
    return _matrix(t, name, dtypes, shape)


def _ckpt(k, tensors):
    if k is None:
        return None
    tensors += (k.codes, k.scales)
    return ctypes.pointer(k._arg())


def block_norm(res, block, out, z, stats, post: Optional[Norm] = None,
               pre: Optional[Norm] = None, gate=None, scale: float = 1.0,
               ckpt_block: Optional[Ckpt] = None, ckpt_out: Optional[Ckpt] = None,
               ckpt_z: Optional[Ckpt] = None, stream=None) -> None:
    """out = res + scale * gate . post(block);  z = pre(out), in one pass.

    res, block, out, z: float16 or bfloat16 [rows, cols] of one type; block None:
    out = res; out or stats None: not written; z None exactly when pre is None.
    gate: None, [cols] (every token) or [rows, cols].  stats: float32 [rows, 4]
    for the backward.  ckpt_*: checkpoints of block, out and z to write too.  out
    may be res and z may be block.
    """
    p_res, s_res = _matrix(res, "res", _F16_BF16)
    shape, dt = res.shape, res.dtype
    rows, cols = shape
    own = (dt,)
    tensors = [res]
    a = _BlockNormArg(
        _CODE[dt], rows, cols, p_res, s_res, *_optional(block, "block", own, shape, tensors),
        *_gate(gate, dt, shape, tensors), scale,
        (post or _NO_NORM)._arg("post", dt, cols, tensors),
        (pre or _NO_NORM)._arg("pre", dt, cols, tensors),
        *_optional(out, "out", own, shape, tensors), *_optional(z, "z", own, shape, tensors),
        _stats(stats, rows, tensors), _ckpt(ckpt_block, tensors), _ckpt(ckpt_out, tensors),
        _ckpt(ckpt_z, tensors))
    _call(_index(tensors, stream), stream, lib.zero_block_norm, ctypes.byref(a))


def block_norm_grad_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace of block_norm_grad's parameter gradients."""
    return lib.zero_block_norm_grad_workspace(rows, cols)


def block_norm_grad(dout, dz, ckpt_out: Optional[Ckpt], ckpt_block: Optional[Ckpt], stats,
                    post: Optional[Norm] = None, pre: Optional[Norm] = None, gate=None,
                    scale: float = 1.0, dres=None, dblock=None, dgate=None, dw_pre=None,
                    db_pre=None, dw_post=None, db_post=None, accumulate: bool = False,
                    workspace=None, stream=None) -> None:
    """The backward of block_norm from the checkpoints of its output and block.

    dout: gradient of out from its other uses, or None; dz: gradient of z.  The
    outputs given are written: dres and dblock [rows, cols]; dgate like the gate;
    dw_* and db_* rows of the norms' weights and biases.  Those rows (and the row
    of a [cols] gate) have one type, the call's or float32, and are added to with
    `accumulate`.  dres may be dout and dblock may be dz.
    """
    first = next((t for t in (dz, dout, dres, dblock) if t is not None), None)
    if first is None:
        raise ValueError("dout, dz, dres and dblock are all None")
    if not isinstance(first, torch.Tensor) or first.dtype not in _F16_BF16 or first.dim() != 2:
        raise ValueError("gradients must be float16 or bfloat16 matrices")
    shape, dt = first.shape, first.dtype
    rows, cols = shape
    own, code = (dt,), _CODE[dt]
    tensors = []
    p_gate, s_gate = _gate(gate, dt, shape, tensors)
    p_dgate, s_dgate, sums = None, 0, {"dw_pre": dw_pre, "db_pre": db_pre, "dw_post": dw_post,
                                       "db_post": db_post}
    if dgate is not None:
        if gate is None:
            raise ValueError("dgate without a gate")
        if s_gate == 0:
            sums["dgate"] = dgate
        else:
            p_dgate, s_dgate = _matrix(dgate, "dgate", own, shape)
            tensors.append(dgate)
    grad_dtype, places = None, {}
    for name, t in sums.items():
        if t is None:
            continue
        if grad_dtype is None:
            grad_dtype = t.dtype
            if grad_dtype != dt and grad_dtype != torch.float32:
                raise ValueError(f"parameter gradients have dtype {grad_dtype}, expected {dt} or "
                                 f"float32")
        places[name] = _row(t, name, grad_dtype, cols)
        tensors.append(t)
    need = lib.zero_block_norm_grad_workspace(rows, cols) if places else 0
    p_out, p_block = _ckpt(ckpt_out, tensors), _ckpt(ckpt_block, tensors)
    p_dout, s_dout = _optional(dout, "dout", own, shape, tensors)
    p_dz, s_dz = _optional(dz, "dz", own, shape, tensors)
    p_stats = _stats(stats, rows, tensors)
    n_post = (post or _NO_NORM)._arg("post", dt, cols, tensors)
    n_pre = (pre or _NO_NORM)._arg("pre", dt, cols, tensors)
    p_dres, s_dres = _optional(dres, "dres", own, shape, tensors)
    p_db, s_db = _optional(dblock, "dblock", own, shape, tensors)
    dev = _index(tensors, stream)
    ws, ws_bytes, held = _workspace(workspace, need, dev, stream)
    a = _BlockNormGradArg(
        code, rows, cols, p_dout, s_dout, p_dz, s_dz, p_out, p_block, p_stats, p_gate, s_gate,
        scale, n_post, n_pre, p_dres, s_dres, p_db, s_db, places.get("dgate", p_dgate), s_dgate,
        places.get("dw_pre"), places.get("db_pre"), places.get("dw_post"), places.get("db_post"),
        2 if grad_dtype == torch.float32 else code, int(bool(accumulate)), ws, ws_bytes)
    _call(dev, stream, lib.zero_block_norm_grad, ctypes.byref(a))
