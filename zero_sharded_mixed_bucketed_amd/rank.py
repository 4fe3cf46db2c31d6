"""One data-parallel rank's model-state buffers for ZeRO stages 1, 2 and 3,
and the steps over them through the C ABI.

What a rank keeps (upskillscore guide "ZeRO: particionar estados do treino
entre GPUs", section "Como funciona", with its 2 Psi / 2 Psi / 12 Psi
accounting; llm-engineer card "ZeRO-2", sections "ZeRO-1's remaining waste"
and "Gradient lifecycle"):

* both stages: the flat fp16 parameter vector [Psi] (the all-gather target;
  the rank writes its slot) and the fp32 master/m/v of its shard [S];
* stage 1 (P_os): its full fp16 local gradient [Psi], kept for the whole
  backward pass; the reduced gradient of the owned slice is written in place
  into that buffer's slot [offset, offset + S) -- 4 Psi + 12 Psi / Nd bytes;
* stage 2 (P_os+g): only a gradient shard [S], fp16 (the guide's accounting,
  2 Psi + 14 Psi / Nd bytes) or fp32; each bucket's local gradient is
  released once its owner has reduced it.
* stage 3 (P_os+g+p; lastdictionary entry "ZeRO"): the parameters are
  partitioned too.  The rank keeps its fp16 parameter shard [S] instead of the
  flat vector (16 Psi / Nd bytes in all).  Each layer's parameters are gathered
  from the rank shards just in time (gather_layer) and released after use.

In backward a rank makes the local gradients that the reduce takes: linear_grad,
norm_grad and gated_grad write the gradients of a layer's tensors to their flat
places in the local gradient (stage 1) or in the bucket that is being filled
(stages 2 and 3), from activations kept in 8 bits (checkpoint; the guide's residual
states); loss_grad and distill_grad begin the backward with the gradient of the
projection onto the vocabulary.  The local gradient is fp16, and so are the
activations of these calls: with bf16 ones the operators themselves give a gradient in
bf16 or fp32, which is not what the reduce reads.

This module allocates with torch and calls the library; no arithmetic of the
path happens here.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import (ACT_SILU, CKPT_INT8, Ckpt, adam_step_shard, block_norm_grad, ckpt_empty,
               ckpt_weight_grad, distill_loss, gated_ffn_grad, gather_params, memory_model,
               reduce_shard, shard_geometry, vocab_loss)

STAGE_OS = 1
STAGE_OS_G = 2
STAGE_OS_G_P = 3


def _fp16(name: str, t) -> None:
    if t.dtype == torch.bfloat16:
        raise ValueError(f"{name} is bf16, and the local gradient is fp16")


class RankState:
    """Device buffers of rank `rank` of `nd` over a `psi`-parameter model.

    grad_dtype is the gradient the reduce writes and Adam reads: "fp16" (the
    pages' accounting) or, for stage 2 only, "fp32".  local_grad (stage 1
    only): an existing contiguous [psi] fp16 buffer to keep as the local
    gradient, e.g. row `rank` of a buffer that holds every rank's local
    gradient when all ranks are simulated on one device.  param_shard (stage 3
    only): likewise, an existing contiguous [S] fp16 buffer to keep as the
    rank's parameter shard.
    """

    def __init__(self, psi: int, nd: int, rank: int, stage: int, grad_dtype: str = "fp16",
                 device: Optional[torch.device] = None, local_grad=None, param_shard=None):
        if stage not in (STAGE_OS, STAGE_OS_G, STAGE_OS_G_P):
            raise ValueError("stage must be 1 (P_os), 2 (P_os+g) or 3 (P_os+g+p)")
        if grad_dtype not in ("fp16", "fp32") or (stage != STAGE_OS_G and grad_dtype != "fp16"):
            raise ValueError("grad_dtype: fp16, or fp32 for stage 2")
        dev = device or torch.device("cuda", torch.cuda.current_device())
        self.stage, self.grad_dtype = stage, grad_dtype
        self.geom = shard_geometry(psi, nd, rank)
        s = self.geom.len
        if stage == STAGE_OS_G_P:
            if param_shard is None:
                param_shard = torch.zeros(s, dtype=torch.int16, device=dev)
            elif (param_shard.dtype not in (torch.int16, torch.float16) or param_shard.dim() != 1
                  or param_shard.numel() != s or not param_shard.is_contiguous()):
                raise ValueError("param_shard must be a contiguous [S] fp16 buffer")
            self.param16 = param_shard                # window origin: the shard's offset
            self.param16_origin = self.geom.offset
        else:
            if param_shard is not None:
                raise ValueError("param_shard is for stage 3")
            self.param16 = torch.zeros(psi, dtype=torch.int16, device=dev)
            self.param16_origin = 0
        self.master = torch.zeros(s, dtype=torch.float32, device=dev)
        self.m = torch.zeros(s, dtype=torch.float32, device=dev)
        self.v = torch.zeros(s, dtype=torch.float32, device=dev)
        lo = self.geom.offset
        if stage == STAGE_OS:
            if local_grad is None:
                local_grad = torch.zeros(psi, dtype=torch.int16, device=dev)
            elif (local_grad.dtype not in (torch.int16, torch.float16) or local_grad.dim() != 1
                  or local_grad.numel() != psi or not local_grad.is_contiguous()):
                raise ValueError("local_grad must be a contiguous [psi] fp16 buffer")
            self.local_grad = local_grad
            self.grad = self.local_grad[lo:lo + s]          # the reduced slice, in place
        else:
            if local_grad is not None:
                raise ValueError("local_grad is for stage 1")
            self.local_grad = None
            dt = torch.int16 if grad_dtype == "fp16" else torch.float32
            self.grad = torch.zeros(s, dtype=dt, device=dev)

    def resident_tensors(self):
        """The buffers this rank keeps across the step (views not counted twice)."""
        ts = [self.param16, self.master, self.m, self.v]
        ts.append(self.local_grad if self.stage == STAGE_OS else self.grad)
        return ts

    def resident_bytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in self.resident_tensors())

    def model_bytes(self) -> float:
        """The guide's per-device bytes for this stage (fp16 gradients)."""
        return memory_model(self.geom.psi, self.geom.nd, self.stage)

    def reduce_bucket(self, bucket_offset: int, bucket_len: int, slices, stream=None) -> None:
        """The owner's reduce of one bucket: slices are the Nd ranks' local
        gradients over [bucket_offset, bucket_offset + bucket_len), one row each.
        In stage 1 row `rank` may be this rank's own local_grad (aliasing it
        column for column is allowed)."""
        if self.grad.dtype == torch.float32:
            reduce_shard(self.geom, bucket_offset, bucket_len, slices, self.grad, None,
                         stream=stream)
        else:
            reduce_shard(self.geom, bucket_offset, bucket_len, slices, None, self.grad,
                         stream=stream)

    def adam_step(self, lr: float, beta1: float, beta2: float, eps: float, step: int,
                  stream=None) -> None:
        adam_step_shard(self.geom, self.master, self.m, self.v, self.grad, self.param16,
                        self.param16_origin, lr, beta1, beta2, eps, step, stream=stream)

    def gather_layer(self, lo: int, length: int, shards, out, stream=None) -> None:
        """Stage 3: the parameters of flat [lo, lo + length) into `out`, from the
        rank shards [Nd, >= S] (row `rank` is this rank's param16 when all ranks
        are simulated on one device)."""
        if self.stage != STAGE_OS_G_P:
            raise ValueError("only stage 3 gathers parameters")
        gather_params(self.geom.psi, self.geom.nd, lo, length, shards, out, stream=stream)

    def checkpoint(self, tokens: int, width: int, fmt: int = CKPT_INT8) -> Ckpt:
        """Buffers for `tokens` activations of `width` columns in 8 bits: 1 + 1/32
        bytes an element (width a multiple of 32) where 16 bits take 2."""
        return ckpt_empty(tokens, width, fmt, device=self.master.device)

    def grad_slot(self, flat_lo: int, count: int, bucket=None, bucket_offset: int = 0):
        """The fp16 elements of flat [flat_lo, flat_lo + count) of the local gradient:
        in stage 1's retained one, or in `bucket`, a contiguous fp16 row that starts
        at flat index bucket_offset."""
        if bucket is None:
            if self.stage != STAGE_OS:
                raise ValueError("stages 2 and 3 keep no local gradient: give the bucket")
            bucket, bucket_offset = self.local_grad, 0
        elif bucket.dtype not in (torch.int16, torch.float16) or bucket.dim() != 1 \
                or not bucket.is_contiguous():
            raise ValueError("bucket must be a contiguous fp16 row")
        lo = flat_lo - bucket_offset
        if count < 0 or bucket_offset < 0 or lo < 0 or lo + count > bucket.numel() \
                or flat_lo + count > self.geom.psi:
            raise ValueError(f"flat [{flat_lo}, +{count}) lies outside the local gradient")
        return bucket[lo:lo + count].view(torch.float16)

    def linear_grad(self, flat_lo: int, ckpt: Ckpt, dy, bucket=None, bucket_offset: int = 0,
                    accumulate: bool = False, workspace=None, stream=None) -> None:
        """The gradient of a linear layer's weight (dy.shape[1] x ckpt.cols, at flat
        index flat_lo) from its input's checkpoint, into the local gradient."""
        n, k = dy.shape[1], ckpt.cols
        dw = self.grad_slot(flat_lo, n * k, bucket, bucket_offset).view(n, k)
        ckpt_weight_grad(ckpt, dy, dw, accumulate=accumulate, workspace=workspace, stream=stream)

    def norm_grad(self, places, dout, dz, ckpt_out, ckpt_block, stats, bucket=None,
                  bucket_offset: int = 0, **call) -> None:
        """block_norm_grad with the parameters' gradients in the local gradient:
        places maps dw_pre, db_pre, dw_post, db_post and dgate (a gate of one row) to
        their flat indices."""
        first = dout if dz is None else dz
        if first is None:
            raise ValueError("dout and dz are both None")
        slots = {name: self.grad_slot(lo, first.shape[1], bucket, bucket_offset)
                 for name, lo in places.items()}
        block_norm_grad(dout, dz, ckpt_out, ckpt_block, stats, **slots, **call)

    def gated_grad(self, flat_lo: int, dout, ckpt_gate: Ckpt, ckpt_up: Ckpt, ckpt_x: Ckpt, w,
                   act: int = ACT_SILU, dx=None, bucket=None, bucket_offset: int = 0,
                   **call) -> None:
        """gated_ffn_grad with the gradient of the block's stacked weight (2 dout.shape[1]
        x ckpt_x.cols, at flat index flat_lo) in the local gradient."""
        _fp16("dout", dout)
        n, k = 2 * dout.shape[1], ckpt_x.cols
        dw = self.grad_slot(flat_lo, n * k, bucket, bucket_offset).view(n, k)
        gated_ffn_grad(dout, ckpt_gate, ckpt_up, w, act, dx=dx, ckpt_x=ckpt_x, dw=dw, **call)

    def loss_grad(self, flat_lo: int, x, w, targets, loss, dx=None, bucket=None,
                  bucket_offset: int = 0, **call) -> None:
        """vocab_loss with the gradient of the projection onto the vocabulary (w's shape,
        at flat index flat_lo) in the local gradient."""
        _fp16("x", x)
        dw = self.grad_slot(flat_lo, w.numel(), bucket, bucket_offset).view(w.shape)
        vocab_loss(x, w, targets, loss, dx=dx, dw=dw, **call)

    def distill_grad(self, flat_lo: int, x, w, ids, logits, loss, dx=None, bucket=None,
                     bucket_offset: int = 0, **call) -> None:
        """distill_loss, likewise."""
        _fp16("x", x)
        dw = self.grad_slot(flat_lo, w.numel(), bucket, bucket_offset).view(w.shape)
        distill_loss(x, w, ids, logits, loss, dx=dx, dw=dw, **call)
