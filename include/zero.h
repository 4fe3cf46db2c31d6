/*
 * zero.h -- C ABI of the per-rank data-parallel hot path of ZeRO stages 1 and 2
 * on one MI355X (gfx950).
 *
 * The method (upskillscore guide "ZeRO: particionar estados do treino entre
 * GPUs", section "Como funciona"; llm-engineer card "ZeRO-2", sections
 * "Gradient lifecycle" and "Why all-gather is still needed"): the flat
 * parameter vector of Psi elements is split into Nd contiguous rank-major
 * partitions.  In backward, each gradient bucket is reduce-scattered as soon as
 * it is ready; the owner of a partition keeps only the reduced gradient of its
 * own slice and releases the rest.  In the optimizer step each rank updates
 * only its partition of the fp32 master weights, momentum and variance (mixed-
 * precision Adam, K = 12 bytes per parameter) and its updated fp16 parameters
 * go to their slot of the flat fp16 parameter vector that the all-gather fills.
 *
 * This library is the one-GPU share of that path: zero_reduce_shard is the
 * owner's side of one bucket's reduce-scatter, with the Nd ranks' local
 * gradients handed over as Nd rows of one device buffer; zero_adam_step_shard is
 * the fused sharded Adam step and the fp16 slot write.  For stage 3, where the
 * parameters are partitioned too, zero_gather_params is the receive side of a
 * layer's parameter all-gather.  No collective runs here.
 *
 * Conventions for every entry point:
 *  - Sizes and offsets are element counts (uint64_t).  Flat indices address
 *    the Psi-long parameter vector in forward layer order.
 *  - Device pointers come from the caller, who owns every buffer; the library
 *    allocates nothing per call and keeps no pointer after it returns.
 *  - Device work is enqueued on `hip_stream` (a hipStream_t; NULL = the null
 *    stream) and the call returns at once; results are valid after the stream
 *    synchronises.  Calls that touch the same buffers must be ordered by the
 *    caller (same stream or events).
 *  - Kernels run on the calling thread's current HIP device; every device
 *    pointer of a call must be memory of that device.
 *  - A negative status is an error.  Arguments are validated before any HIP
 *    call, so a rejected call enqueues nothing and writes nothing.
 *    zero_last_error() returns a message for the calling thread's last error.
 *    Non-finite values in the data are not errors; they propagate per IEEE.
 *  - Several threads may call at once.  The only process-wide state is a cache
 *    of each device's compute-unit count and the dynamic LDS sizes that cap
 *    the streaming kernels' residency (zero_launch_occupancy), resolved under a
 *    lock on first use; the error message is per thread.
 */
#ifndef ZERO_H_
#define ZERO_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define ZERO_OK 0
#define ZERO_E_INVAL (-1)  /* invalid argument: null pointer, Nd = 0, rank >= Nd, bad stage or hyperparameter, geometry mismatch */
#define ZERO_E_RANGE (-2)  /* a range leaves the parameter vector or a buffer (bucket beyond Psi, stride < length, slot outside the fp16 window) */
#define ZERO_E_ALIGN (-3)  /* a device pointer is not aligned to its element size */
#define ZERO_E_DEVICE (-4) /* the HIP runtime reported an error, or the device cannot hold a streaming kernel to its workgroups-per-CU cap (zero_launch_occupancy) */

/* Stages of zero_memory_model. */
#define ZERO_STAGE_DP 0     /* plain data parallelism: full replica */
#define ZERO_STAGE_OS 1     /* P_os: optimizer states partitioned */
#define ZERO_STAGE_OS_G 2   /* P_os+g: optimizer states and gradients partitioned */
#define ZERO_STAGE_OS_G_P 3 /* P_os+g+p: parameters partitioned too */

/* The partition of one data-parallel rank: flat range [offset, offset + len). */
typedef struct zero_geom {
  uint64_t psi;    /* parameters in the model */
  uint32_t nd;     /* data-parallel degree Nd */
  uint32_t rank;   /* this rank, 0 <= rank < nd */
  uint64_t offset; /* first flat index owned */
  uint64_t len;    /* elements owned */
} zero_geom_t;

/*
 * Model-state bytes per device (guide "ZeRO: particionar estados do treino
 * entre GPUs", section "Como funciona"; worked example in section "Na pratica"):
 * with 2 Psi bytes of fp16 parameters, 2 Psi of fp16 gradients and 12 Psi of
 * optimizer state,
 *   stage 0:  16 Psi            stage 2:  2 Psi + 14 Psi / Nd
 *   stage 1:  4 Psi + 12 Psi/Nd  stage 3:  16 Psi / Nd
 * (stage 2 keeps an fp16 gradient shard, the reading that reproduces the
 * guide's 16.6 GB for 7.5B parameters at Nd = 64).  Pure host arithmetic.
 * Returns the byte count (a real number), or a negative value if nd == 0 or
 * the stage is not 0..3.
 */
double zero_memory_model(uint64_t psi, uint32_t nd, int stage);

/*
 * The same accounting with a general optimizer-state multiplier (guide, "Como
 * funciona": K Psi bytes of optimizer state, K = 12 for mixed-precision Adam):
 *   stage 0: (4 + K) Psi          stage 2: 2 Psi + (2 + K) Psi / Nd
 *   stage 1: 4 Psi + K Psi / Nd   stage 3: (4 + K) Psi / Nd
 * zero_memory_model(psi, nd, stage) == zero_memory_model_k(psi, nd, stage, 12).
 * Returns the byte count, or a negative value if nd == 0, the stage is not
 * 0..3, or k is negative or not finite.
 */
double zero_memory_model_k(uint64_t psi, uint32_t nd, int stage, double k);

/* Per-step communication of one data-parallel rank. */
typedef struct zero_comm {
  uint32_t reduce_scatters;    /* gradient reduce-scatters per step */
  uint32_t all_gathers;        /* parameter all-gathers per step */
  double elems;                /* the guide's count: Psi per collective */
  double elems_sent_per_rank;  /* bandwidth-optimal collectives: (Nd - 1) / Nd of Psi each */
  double bytes_sent_per_rank;  /* fp16: 2 bytes per element */
} zero_comm_t;

/*
 * Communication volume per step (guide, "Como funciona": plain DP moves 2 Psi,
 * a reduce-scatter and an all-gather of Psi each; P_os+g keeps 2 Psi; P_os+g+p
 * needs two parameter all-gathers, in forward and backward, plus the gradient
 * reduce-scatter, 3 Psi or 1.5x; lastdictionary entry "ZeRO": stages 1 and 2
 * keep data parallelism's volume).  Fills *out: stages 0-2 one reduce-scatter
 * and one all-gather, stage 3 one reduce-scatter and two all-gathers.  Pure
 * host arithmetic.  Errors: ZERO_E_INVAL for out == NULL, nd == 0 or a stage
 * not 0..3.
 */
int zero_comm_volume(uint64_t psi, uint32_t nd, int stage, zero_comm_t *out);

/*
 * Partition of `rank` (card "ZeRO-2", "Why all-gather is still needed": the
 * all-gather of the rank shards in rank order rebuilds [A, B, C]): shard size
 * S = ceil(psi / nd); rank r owns [min(r S, psi), min((r + 1) S, psi)), so
 * trailing shards may be short or empty.  Fills *out.  Errors: ZERO_E_INVAL
 * for out == NULL, nd == 0, rank >= nd or psi == 0.
 */
int zero_shard_geometry(uint64_t psi, uint32_t nd, uint32_t rank, zero_geom_t *out);

/*
 * Flat range [*lo, *hi) of bucket [bucket_offset, bucket_offset + bucket_len)
 * that the rank owns; *lo == *hi when they do not meet (card "ZeRO-2", the
 * bucket diagram and "Gradient lifecycle": of each bucket reduce-scattered in
 * backward, a rank keeps the part that falls in its own partition).  Errors: ZERO_E_INVAL
 * (null pointer, geometry that zero_shard_geometry would not return),
 * ZERO_E_RANGE (bucket beyond psi).
 */
int zero_bucket_intersect(const zero_geom_t *g, uint64_t bucket_offset, uint64_t bucket_len,
                          uint64_t *lo, uint64_t *hi);

/*
 * Advised row stride, in elements, for the Nd fp16 gradient rows of a bucket
 * (or chunk) of `len` columns that a caller lays out for zero_reduce_shard:
 * len rounded up to a multiple of 64 elements (each row starts on a 128-byte
 * line), plus 1024 elements when that stride is a whole number of MiB.  The
 * reduce reads the Nd rows of a column tile at once, and on MI355X rows a power
 * of two apart read slower: at Nd = 400, rows 4 or 8 MiB apart stream 12-14%
 * slower than the same rows 2 KiB further apart, while on the other strides
 * measured the pad changes nothing beyond run-to-run noise.  Advice only:
 * zero_reduce_shard accepts any slice_stride >= bucket_len.  len == 0 gives 0.
 * Errors: ZERO_E_INVAL (stride NULL), ZERO_E_RANGE (the stride would not fit in
 * 64 bits).
 */
int zero_row_stride(uint64_t len, uint64_t *stride);

/*
 * The owner's reduce of one gradient bucket (guide, "Como funciona": each
 * gradient is reduced only at the process that owns its partition, via
 * reduce-scatter, then released; card "ZeRO-2", "Gradient lifecycle").
 *
 * slices: device, fp16 bit patterns, Nd rows; row k (at slices + k *
 *   slice_stride) is data-parallel rank k's local gradient over the flat range
 *   [bucket_offset, bucket_offset + bucket_len) -- a whole bucket, or any chunk
 *   of one.  Only the columns inside the rank's shard are read.  The buffer must
 *   hold (Nd - 1) * slice_stride + bucket_len elements; slice_stride >=
 *   bucket_len.
 * grad32: device, fp32, the rank's shard-local gradient (g->len elements), or
 *   NULL to keep only the fp16 gradient shard; for every flat i in
 *   bucket-intersect-shard,
 *     grad32[i - g->offset] = RN32(sum_{k = 0..Nd-1} fp32(row_k[i])) * RN32(1/Nd)
 *   with the additions done one at a time in ascending rank order from +0 (each
 *   rounded to fp32) and one fp32 multiply by the correctly rounded 1/Nd.
 *   Elements outside the intersection are not touched.
 * grad16: optional (NULL = none), device, fp16 bit patterns, g->len elements:
 *   the round-to-nearest-even fp16 of the fp32 value above, at the same
 *   elements.  This 2-byte gradient shard is the one the guide's stage-2
 *   accounting keeps (2 Psi + 14 Psi / Nd).  At least one of grad32 and grad16
 *   must be given.
 * Aliasing: an output may share memory with the rows only column for column,
 *   i.e. the output element of flat index i at the address of some row's
 *   element i.  This is how stage 1 (P_os) keeps its reduced shard inside its
 *   own retained full local gradient: grad16 = own_local_grad + g->offset where
 *   row `rank` is own_local_grad + bucket_offset.  Any other overlap is
 *   undefined.
 * The "release" of the rest of the local gradient is the caller freeing
 * `slices` after this call completes on the stream.  An empty intersection is
 * ZERO_OK and enqueues nothing.
 * Nd is at most 2^24 here (the largest Nd for which RN32(1/Nd) is the fp32
 * quotient 1 / fp32(Nd)).
 * Errors: ZERO_E_INVAL (slices NULL, both outputs NULL, bad geometry),
 * ZERO_E_RANGE (bucket beyond psi, slice_stride < bucket_len, size overflow,
 * Nd > 2^24 for a bucket that meets the shard),
 * ZERO_E_ALIGN (slices or grad16 not 2-byte, grad32 not 4-byte aligned),
 * ZERO_E_DEVICE (launch failed, or the launch's residency cap cannot be set on
 * this device).
 */
int zero_reduce_shard(const zero_geom_t *g, uint64_t bucket_offset, uint64_t bucket_len,
                      const uint16_t *slices, uint64_t slice_stride, float *grad32,
                      uint16_t *grad16, void *hip_stream);

/* The rank's optimizer-state shard and its fp16 parameter slot. */
typedef struct zero_shard {
  float *master;           /* device, fp32 master weights, g->len elements, updated in place */
  float *m;                /* device, fp32 first moment, g->len elements, updated in place */
  float *v;                /* device, fp32 second moment, g->len elements, updated in place */
  const void *grad;        /* device, the reduced gradient shard, g->len elements */
  int grad_is_fp16;        /* 0: grad is fp32; 1: grad is fp16 bit patterns */
  uint16_t *param16;       /* device, fp16 window of the flat parameter vector, or NULL (no slot write) */
  uint64_t param16_origin; /* flat index of param16[0] */
  uint64_t param16_len;    /* elements in the window */
} zero_shard_t;

/*
 * Per-step fp32 scalars of the Adam step (Kingma & Ba, Algorithm 1: the
 * bias corrections 1 - beta1^t and 1 - beta2^t of step t; the guide, "Como
 * funciona", names mixed-precision Adam as the optimizer), derived in fp64 and
 * rounded once:
 *   out[0] = b1 = RN32(beta1)          out[1] = b2 = RN32(beta2)
 *   out[2] = c1 = RN32(1 - beta1)      out[3] = c2 = RN32(1 - beta2)
 *   out[4] = e  = RN32(eps)
 *   out[5] = step = RN32(lr / (1 - beta1^t))
 *   out[6] = isb  = RN32(1 / sqrt(1 - beta2^t))
 * (1 - beta and the bias corrections are evaluated in fp64, beta^t with pow).
 * Errors: ZERO_E_INVAL for out == NULL, t == 0, beta outside [0, 1), eps <= 0,
 * or a non-finite lr.
 */
int zero_adam_scalars(double lr, double beta1, double beta2, double eps, uint64_t step,
                      float out[7]);

/*
 * One fused Adam step on the rank's shard (guide, "Como funciona": each process
 * updates only its own partition; lastdictionary entry "ZeRO", usage note: the
 * update itself is plain Adam).  Adam as published by Kingma & Ba (Algorithm 1,
 * bias-corrected, eps outside the square root, step t >= 1, no weight decay),
 * per element j < g->len, in fp32 with every operation rounded once and no
 * fused multiply-add, using the scalars of zero_adam_scalars:
 *   m'  = b1*m + c1*g
 *   v'  = b2*v + c2*(g*g)
 *   den = sqrt(v')*isb + e              (correctly rounded sqrt)
 *   th' = th - step*(m'/den)            (correctly rounded division)
 *   param16[g->offset - param16_origin + j] = fp16_rne(th')
 * Each element of g, master, m, v is read once and master, m, v and the fp16
 * slot are written once (28 bytes per element with an fp16 gradient, 30 with
 * fp32).  Only the slot [g->offset, g->offset + g->len) of the fp16 window is
 * written (card "ZeRO-2", "Why all-gather is still needed": that slot is the
 * rank's contribution to the all-gather of [A, B, C]).
 * Errors: ZERO_E_INVAL (null pointer, bad geometry or hyperparameter),
 * ZERO_E_RANGE (slot outside the fp16 window), ZERO_E_ALIGN (fp32 arrays not
 * 4-byte, fp16 arrays not 2-byte aligned), ZERO_E_DEVICE (launch failed, or the
 * launch's residency cap cannot be set on this device).
 */
int zero_adam_step_shard(const zero_geom_t *g, const zero_shard_t *s, double lr, double beta1,
                         double beta2, double eps, uint64_t step, void *hip_stream);

/*
 * The receive side of one layer's parameter all-gather in stage 3, P_os+g+p
 * (guide, "Como funciona": the parameters are partitioned too and a process
 * that needs another's partition receives it, two parameter all-gathers per
 * step; lastdictionary entry "ZeRO": each layer's parameters are gathered just
 * in time and discarded after use; card "ZeRO-2", "Why all-gather is still
 * needed": the partitions in rank order are the full vector).
 *
 * shards: device, fp16 bit patterns, Nd rows; row k (at shards + k *
 *   shard_stride) is rank k's parameter shard, flat [k S, min((k + 1) S, psi))
 *   with S = ceil(psi / nd) as in zero_shard_geometry; shard_stride >= S.
 * out: device, fp16, len elements: out[j] = the parameter of flat index lo + j.
 *   It must not overlap the shards.
 * Pure data movement (bit-exact).  len == 0 is ZERO_OK and enqueues nothing.
 * Errors: ZERO_E_INVAL (nd == 0, psi == 0, NULL buffer), ZERO_E_RANGE (range
 * beyond psi, shard_stride < S, size overflow), ZERO_E_ALIGN (a buffer not
 * 2-byte aligned), ZERO_E_DEVICE (launch failed).
 */
int zero_gather_params(uint64_t psi, uint32_t nd, uint64_t lo, uint64_t len,
                       const uint16_t *shards, uint64_t shard_stride, uint16_t *out,
                       void *hip_stream);

/* The streaming kernels whose residency the library caps (zero_launch_occupancy). */
#define ZERO_KERNEL_REDUCE_W16 0 /* the reduce with 16-byte row loads (aligned rows) */
#define ZERO_KERNEL_REDUCE_W8 1  /* ... 8-byte row loads */
#define ZERO_KERNEL_REDUCE_W4 2  /* ... 4-byte row loads */
#define ZERO_KERNEL_REDUCE_W2 3  /* ... 2-byte row loads */
#define ZERO_KERNEL_ADAM_G32 4   /* the fused Adam step, fp32 gradient */
#define ZERO_KERNEL_ADAM_G16 5   /* the fused Adam step, fp16 gradient */

/*
 * Launch residency of one capped kernel on the calling thread's current device.
 * No passage defines it: it is a measured property of MI355X.  The reduce and
 * the Adam step stream HBM faster when fewer workgroups share a compute unit
 * (at most 8 for the reduce, 10 for Adam), so every launch asks for dynamic
 * LDS that the kernels never touch.  On the first call that launches on a
 * device, the library resolves, per kernel, the LDS size at which the
 * runtime's occupancy calculator allows exactly that many workgroups per CU,
 * and it refuses to launch (ZERO_E_DEVICE) when no size does.
 * Fills *wgs_per_cu with the workgroups per CU the calculator allows at the
 * resolved size, and *lds_bytes (nullable) with that size.
 * Errors: ZERO_E_INVAL (unknown kernel, wgs_per_cu NULL), ZERO_E_DEVICE (no
 * device, or the cap cannot be reached on it).
 */
int zero_launch_occupancy(int kernel, int *wgs_per_cu, uint32_t *lds_bytes);

/* ------------------------------------------------------------------------
 * Residual states: activations kept for the backward pass in 8 bits, the
 * weight gradient taken from them, the norms around a block, the gated block between
 * them, and the losses over the vocabulary (whose logits are the largest of a step's
 * temporaries).
 *
 * The guide's third class of training memory after optimizer states, gradients
 * and parameters (section "Como funciona": ZeRO-R treats the residual states,
 * activations among them) and what produces the local gradient that
 * zero_reduce_shard takes (card "ZeRO-2", "Gradient lifecycle": a layer's local
 * gradient is made in backward, then reduced).  The entry points below follow
 * the conventions at the top of this file.  16-bit matrices are rows x cols with
 * a row stride in elements (stride >= cols unless there is at most one row);
 * any stride and any base that its element size divides is accepted.  Columns
 * between the rows of a matrix or checkpoint are never written; the weight
 * gradient may read those of its inputs, which reach no result.  Sums are fp32
 * in a fixed order, so equal inputs give equal bits.
 * ------------------------------------------------------------------------ */

/* Element types. */
#define ZERO_F16 0
#define ZERO_BF16 1
#define ZERO_F32 2

/* Formats of an 8-bit checkpoint. */
#define ZERO_CKPT_INT8 0
#define ZERO_CKPT_E4M3 1
#define ZERO_CKPT_BLOCK 32 /* columns that share one scale byte */

/*
 * An 8-bit checkpoint of a rows x cols matrix in device memory: the code of
 * (r, c) is codes[r * code_stride + c], and its value is
 *   value(code) * 2^(b - 127),  b = scales[r * scale_stride + c / 32];
 * b = 255 stands for NaN.  int8 codes are two's complement
 * (-127..127), e4m3 codes are 8-bit floats with 4 exponent and 3 mantissa bits,
 * bias 7, no infinities.  A row has at most 2^31 columns.
 */
typedef struct zero_ckpt {
  uint8_t *codes;
  uint8_t *scales;
  uint64_t rows, cols;
  uint64_t code_stride;  /* bytes between rows of codes, >= cols */
  uint64_t scale_stride; /* bytes between rows of scales, >= ceil(cols / 32) */
  int format;            /* ZERO_CKPT_INT8 or ZERO_CKPT_E4M3 */
} zero_ckpt_t;

/*
 * Stores x (rows x cols of c, fp16 or bf16) as an 8-bit checkpoint.  Per block of
 * 32 columns of a row, with amax its largest magnitude:
 *   int8: 2^e = 2^(floor(log2 amax) - 6), e >= -126;
 *         code = the whole number nearest to x 2^-e (ties to even), held to
 *         +-127; the held value is off by at most 2^(e-1), below 2^e where 127
 *         holds it
 *   e4m3: x is first held to +-1.875 2^E, E = 15 for fp16 and 127 for bf16;
 *         e >= -117 is the least with amax 2^-e <= 448; code = the e4m3 value
 *         nearest to x 2^-e (ties to even)
 * A block with an infinity or NaN is held as NaN throughout, so an overflow stays
 * visible in what is computed from it.  A held value of a finite block is
 * exactly representable in x's type.
 * Errors: ZERO_E_INVAL (NULL, dtype, format), ZERO_E_RANGE (a stride too small, too
 * many columns, size overflow), ZERO_E_ALIGN, ZERO_E_DEVICE (launch failed).
 */
int zero_ckpt_write(const void *x, int dtype, uint64_t x_stride, const zero_ckpt_t *c,
                    void *hip_stream);

/*
 * Reads a checkpoint back into out (fp16, bf16 or fp32), each value rounded to
 * nearest even where the type does not hold it.  Errors as zero_ckpt_write.
 */
int zero_ckpt_read(const zero_ckpt_t *c, void *out, int dtype, uint64_t out_stride,
                   void *hip_stream);

/* Bytes of workspace for zero_ckpt_weight_grad at these sizes (0: none). */
uint64_t zero_ckpt_weight_grad_workspace(uint64_t rows, uint64_t cols, uint64_t n);

/*
 * The weight gradient of a linear layer y = x W^T (W: n x cols) from the 8-bit
 * checkpoint of its input: for every (j, c)
 *   dw[j][c] = sum_{t < rows} dy[t][j] * held(x)[t][c]      (+ dw[j][c] before)
 * with the held values rounded to dy's type (exact for a checkpoint written from
 * that type), exact products, fp32 sums and one rounding to dw's type; with
 * `accumulate` the old value is added in fp32 before it.  rows == 0 gives 0, or
 * leaves dw with `accumulate`.  dw must not overlap the inputs.
 * dy: fp16 or bf16, rows x n.  dw: dy's type or fp32.  workspace: device memory,
 * 16-byte aligned, at least zero_ckpt_weight_grad_workspace bytes, written by the
 * call; calls that may run at the same time need one each.  n and cols are at
 * most 2^22.
 * Errors: ZERO_E_INVAL (NULL, dtype, format, workspace missing), ZERO_E_RANGE (a
 * stride or the workspace too small, n or cols too large, size overflow),
 * ZERO_E_ALIGN, ZERO_E_DEVICE (launch failed).
 */
int zero_ckpt_weight_grad(const zero_ckpt_t *x, const void *dy, int dtype, uint64_t n,
                          uint64_t dy_stride, void *dw, int dw_dtype, uint64_t dw_stride,
                          int accumulate, void *workspace, uint64_t workspace_bytes,
                          void *hip_stream);

/* Norms. */
#define ZERO_NORM_NONE 0  /* the identity */
#define ZERO_NORM_RMS 1   /* x / sqrt(mean x^2 + eps) */
#define ZERO_NORM_LAYER 2 /* (x - mean x) / sqrt(mean (x - mean x)^2 + eps) */
#define ZERO_NORM_MAX_COLS 16384

typedef struct zero_norm {
  int kind;
  double eps;         /* > 0 and finite, unless kind is ZERO_NORM_NONE */
  const void *weight; /* cols elements of the call's type, or NULL (ones) */
  const void *bias;   /* cols elements of the call's type, or NULL (zeros) */
} zero_norm_t;

/* Where a block's output joins the residual stream (zero_block_norm). */
typedef struct zero_block_norm {
  int dtype; /* ZERO_F16 or ZERO_BF16: every matrix and norm parameter */
  uint64_t rows, cols;
  const void *res; /* h */
  uint64_t res_stride;
  const void *block; /* b, or NULL: h' = h */
  uint64_t block_stride;
  const void *gate; /* g, or NULL (ones) */
  uint64_t gate_stride; /* 0: one row of gates for every token */
  double scale;
  zero_norm_t post; /* the norm after the block */
  zero_norm_t pre;  /* the norm before the next block */
  void *out;        /* h', or NULL */
  uint64_t out_stride;
  void *z; /* rows x cols; NULL if and only if pre.kind is ZERO_NORM_NONE */
  uint64_t z_stride;
  float *stats; /* rows x 4 for the backward, 16-byte aligned, or NULL */
  const zero_ckpt_t *ckpt_block; /* each: a checkpoint to write, or NULL */
  const zero_ckpt_t *ckpt_out;
  const zero_ckpt_t *ckpt_z;
} zero_block_norm_t;

/*
 * The norms before and after a block, its gate and its residual scale, in one
 * pass: for each of the rows, in fp32,
 *   o = post(b);  h' = h + scale * (g . o);  z = pre(h')
 * where a norm's value is normalised(x) . weight + bias.  z is computed from h'
 * before its rounding to 16 bits; h' and z are rounded once each.  stats[row] =
 * {mean, 1/deviation} of post's and then of pre's input (mean 0 for RMS; 0 and 1
 * without the norm).  Checkpoints hold b, and h' and z after their rounding, as
 * zero_ckpt_write stores them.  Statistics are fp32: a row whose squares pass its
 * range (bf16 values beyond 1e19) has a deviation of infinity.
 * out may be res and z may be block (same address and stride); other overlaps of
 * an output are undefined.
 * Errors: ZERO_E_INVAL (NULL, dtype, kind, eps, no columns, a gate, post norm or
 * ckpt_block without a block, nothing to write), ZERO_E_RANGE (cols > ZERO_NORM_MAX_COLS, a
 * stride too small, a checkpoint of other sizes, size overflow), ZERO_E_ALIGN,
 * ZERO_E_DEVICE.
 */
int zero_block_norm(const zero_block_norm_t *a, void *hip_stream);

/* The backward of zero_block_norm (zero_block_norm_grad). */
typedef struct zero_block_norm_grad {
  int dtype;
  uint64_t rows, cols;
  const void *dout; /* gradient of h' from its other uses, or NULL (zeros) */
  uint64_t dout_stride;
  const void *dz; /* gradient of z; NULL if and only if pre.kind is ZERO_NORM_NONE */
  uint64_t dz_stride;
  const zero_ckpt_t *ckpt_out;   /* of h'; needed if pre is a norm */
  const zero_ckpt_t *ckpt_block; /* of b; needed if post is a norm or dgate is given; of
                                    ckpt_out's format if both are needed */
  const float *stats;            /* as zero_block_norm left them; needed with a norm */
  const void *gate;
  uint64_t gate_stride;
  double scale;
  zero_norm_t post, pre; /* weights and biases as in the forward */
  void *dres;            /* gradient of h, or NULL */
  uint64_t dres_stride;
  void *dblock; /* gradient of b, or NULL */
  uint64_t dblock_stride;
  void *dgate; /* gradient of g, or NULL: a row of grad_dtype when gate_stride is 0, else rows x
                  cols of dtype */
  uint64_t dgate_stride;
  void *dw_pre, *db_pre, *dw_post, *db_post; /* rows of grad_dtype, or NULL */
  int grad_dtype;                            /* dtype or ZERO_F32 */
  int accumulate; /* add to the parameters' gradients (and a gate row's) instead of setting them */
  void *workspace;
  uint64_t workspace_bytes;
} zero_block_norm_grad_t;

/* Bytes of workspace for the parameters' gradients at these sizes; none is needed
 * when no gradient of a parameter is asked for. */
uint64_t zero_block_norm_grad_workspace(uint64_t rows, uint64_t cols);

/*
 * With x1 = (held(h') - mean1) r1 and x2 = (held(b) - mean2) r2 from the
 * checkpoints and stats, q = dz . w_pre, and [.] for layer norms only:
 *   D = dout + r1 (q - x1 mean(q . x1) - [mean q]);   dres = D
 *   p = scale D . g;  dgate = scale D . (x2 . w_post + b_post);  v = p . w_post
 *   dblock = r2 (v - x2 mean(v . x2) - [mean v])
 *   dw_pre = sum_t dz . x1, db_pre = sum_t dz, dw_post = sum_t p . x2, db_post = sum_t p
 * in fp32, each output rounded once (a norm of kind NONE passes its gradient on).
 * dres may be dout and dblock may be dz (same address and stride); other overlaps
 * of an output are undefined.  Gradients of parameters are summed over the rows
 * in a fixed order through the workspace (16-byte aligned device memory; calls
 * that may run at the same time need one each); rows == 0 gives zeros, or leaves
 * them with `accumulate`.
 * Errors: as zero_block_norm, and ZERO_E_INVAL for a needed input that is NULL, a
 * gradient of a weight or bias of a norm of kind NONE, or no output.
 */
int zero_block_norm_grad(const zero_block_norm_grad_t *a, void *hip_stream);

/* Activations of a gated block. */
#define ZERO_ACT_SILU 0      /* g / (1 + exp(-g)) */
#define ZERO_ACT_GELU 1      /* g (1 + erf(g / sqrt 2)) / 2 */
#define ZERO_ACT_GELU_TANH 2 /* g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2 */

/* A layer's gated feed-forward block up to its last projection (zero_gated_ffn). */
typedef struct zero_gated_ffn {
  int dtype; /* ZERO_F16 or ZERO_BF16: x, w and out */
  int act;
  uint64_t rows, cols, width;
  const void *x; /* rows x cols */
  uint64_t x_stride;
  const void *w; /* 2 width x cols: the gate's rows, then the other projection's */
  uint64_t w_stride;
  void *out; /* rows x width, or NULL */
  uint64_t out_stride;
  const zero_ckpt_t *ckpt_gate; /* each rows x width: a checkpoint to write, or NULL; */
  const zero_ckpt_t *ckpt_up;   /* all of one format */
  const zero_ckpt_t *ckpt_out;
} zero_gated_ffn_t;

/*
 * With w = [wg; wu], for each of the rows:
 *   g = x wg^T;  u = x wu^T;  out = act(g) . u
 * in one kernel: exact products, fp32 sums, out from the sums themselves and rounded
 * once.  The checkpoints hold g, u and out after their rounding to dtype, as
 * zero_ckpt_write stores them: what the backward needs of the block, in 8 bits.  An
 * output must not overlap an input or another output.
 * rows at most 2^25, cols and width at most 2^22, and both > 0.
 * Errors: ZERO_E_INVAL (NULL, dtype, act, format, no columns, nothing to write),
 * ZERO_E_RANGE (sizes, a stride too small, a checkpoint of other sizes, size overflow),
 * ZERO_E_ALIGN, ZERO_E_DEVICE.
 */
int zero_gated_ffn(const zero_gated_ffn_t *a, void *hip_stream);

/* The backward of zero_gated_ffn (zero_gated_ffn_grad). */
typedef struct zero_gated_ffn_grad {
  int dtype;
  int act;
  uint64_t rows, cols, width;
  const void *dout; /* rows x width: gradient of out */
  uint64_t dout_stride;
  const zero_ckpt_t *ckpt_gate; /* as zero_gated_ffn left them, of one format */
  const zero_ckpt_t *ckpt_up;
  const void *w; /* needed for dx */
  uint64_t w_stride;
  void *dx; /* rows x cols, or NULL */
  uint64_t dx_stride;
  const zero_ckpt_t *ckpt_x; /* rows x cols: of x; needed for dw */
  void *dw;                  /* 2 width x cols of dw_dtype, or NULL */
  uint64_t dw_stride;
  int dw_dtype;   /* dtype or ZERO_F32 */
  int accumulate; /* add to dw instead of setting it */
  void *workspace;
  uint64_t workspace_bytes;
} zero_gated_ffn_grad_t;

/* Bytes of workspace of zero_gated_ffn_grad at these sizes (0: sizes it refuses). */
uint64_t zero_gated_ffn_grad_workspace(uint64_t rows, uint64_t cols, uint64_t width);

/*
 * With the held values g and u:
 *   dg = dout . u . act'(g);  du = dout . act(g)     (each rounded to dtype)
 *   dx = dg wg + du wu;  dw = [dg du]^T held(x)      (fp32 sums, one rounding)
 * In fp16, loss scaling has to keep dg and du above 2^-14, or they lose bits.
 * dw is zero_ckpt_weight_grad's of the rounded dg and du.  rows == 0 gives a dw of 0,
 * or leaves it with `accumulate`.  workspace: 16-byte aligned device memory, written
 * by the call; calls that may run at the same time need one each.  An output must not
 * overlap an input or another output.  Sizes as zero_gated_ffn.
 * Errors: as zero_gated_ffn, and ZERO_E_INVAL for a needed input or workspace that is
 * NULL, ZERO_E_RANGE for a workspace too small.
 */
int zero_gated_ffn_grad(const zero_gated_ffn_grad_t *a, void *hip_stream);

/* What a loss over the vocabulary has in common (zero_vocab_loss, zero_distill_loss). */
typedef struct zero_loss {
  int dtype; /* ZERO_F16 or ZERO_BF16: x, w and dx */
  uint64_t rows, cols, vocab;
  const void *x; /* rows x cols: the last hidden states */
  uint64_t x_stride;
  const void *w; /* vocab x cols: the projection onto the vocabulary */
  uint64_t w_stride;
  const float *weights; /* of each row, or NULL (ones) */
  float *loss;          /* of each row */
  double scale;         /* of the gradients: loss scaling, 1 / the number of tokens */
  void *dx;             /* rows x cols, or NULL */
  uint64_t dx_stride;
  void *dw; /* vocab x cols of dw_dtype, or NULL */
  uint64_t dw_stride;
  int dw_dtype;   /* dtype or ZERO_F32 */
  int accumulate; /* add to dw instead of setting it */
  void *workspace;
  uint64_t workspace_bytes;
} zero_loss_t;

/* Bytes of workspace of a loss at these sizes; top: the teacher's entries of a row, 0 for
 * zero_vocab_loss; with_dx, with_dw: whether that gradient is wanted (0: sizes that the
 * losses refuse). */
uint64_t zero_loss_workspace(uint64_t rows, uint64_t cols, uint64_t vocab, uint32_t top,
                             int with_dx, int with_dw);

/*
 * Softmax cross entropy over the vocabulary, from the last hidden states, with its
 * gradients: with z = x w^T (fp32 sums, not rounded),
 *   loss[t] = weights[t] (log(sum over v of exp z[t][v]) - z[t][y]),  y = targets[t]
 *   d[t][v] = weights[t] (softmax(z[t])[v] - (v == y))       (rounded to dtype)
 *   dx = scale d w;  dw = scale d^T x                        (fp32 sums, one rounding)
 * No logits outlive the call, and the loss alone stores none.  For gradients the workspace
 * holds those of a piece of the tokens, 4 bytes each: all tokens' where that is up to about
 * 6 GiB, else 6 GiB (or 256 tokens); besides, a copy of a piece's x and, if there are
 * several pieces, fp32 sums of dw.  For less memory, call with parts of the rows, all but
 * the first with `accumulate` and dw in fp32, which adds them up as a call's own pieces.
 * Of up to 64 rows with a loss, among however many, what the
 * rounding of d leaves out at the targets is kept beside it (16 bits more): a few values
 * hold nearly all of d, and the fewer they are, the further may their roundings be off
 * together.  Before its rounding d
 * is divided by the weights' largest power of two and multiplied by 2^14, which fp16's
 * range asks for, and the products multiplied back.  A weight that is not finite makes
 * its own row's results so, and the dw that it is summed into.
 * A row whose target is negative or whose weight is 0 is left out: its loss and dx are
 * 0, and nothing of it is read into another's result.  A target of vocab or more makes
 * the row's loss NaN and its gradients with it.  targets: id_bytes (4 or 8) wide signed
 * whole numbers.  Sums are in a fixed order.  rows == 0 gives a dw of 0, or leaves it
 * with `accumulate`.  workspace: 16-byte aligned device memory, written by the call;
 * calls that may run at the same time need one each.  An output must not overlap an
 * input or another output.  rows at most 2^25, cols at most 2^22, vocab at most 2^24,
 * both > 0.
 * Errors: ZERO_E_INVAL (NULL, dtype, id_bytes, scale, no columns, workspace missing),
 * ZERO_E_RANGE (sizes, a stride or the workspace too small, size overflow),
 * ZERO_E_ALIGN, ZERO_E_DEVICE.
 */
int zero_vocab_loss(const zero_loss_t *a, const void *targets, int id_bytes, void *hip_stream);

#define ZERO_DISTILL_MAX_TOP 1024

/* A teacher's top logits. */
typedef struct zero_top_logits {
  uint32_t top; /* entries of a row, 1 to ZERO_DISTILL_MAX_TOP */
  const void *ids; /* rows x top signed whole numbers of id_bytes; negative: no entry */
  uint64_t ids_stride;
  int id_bytes; /* 4 or 8 */
  const void *logits; /* rows x top of logits_dtype */
  uint64_t logits_stride;
  int logits_dtype; /* ZERO_F16, ZERO_BF16 or ZERO_F32 */
  double temperature; /* tau > 0 */
} zero_top_logits_t;

/*
 * Distillation from a teacher's top logits s[t][j] of the ids i[t][j], as
 * zero_vocab_loss otherwise: with q[t] = softmax over a row's entries of s[t] / tau and
 * p[t] = softmax over the vocabulary of z[t] / tau,
 *   loss[t] = weights[t] tau^2 sum over j of q[t][j] (log q[t][j] - log p[t][i[t][j]])
 *   d[t][v] = weights[t] (p[t][v] - sum over j with i[t][j] == v of q[t][j])
 *   dx = scale tau d w;  dw = scale tau d^T x
 * Without gradients too, the workspace holds a piece's logits, from which the entries' are
 * read.  A row without entries is left out.  An entry of -infinity has no share; an id that
 * stands in a row twice has both shares.  An id of vocab or more, and logits that give
 * no softmax (NaN, +infinity, -infinity alone), make the row's loss NaN and its
 * gradients with it.
 * Errors: as zero_vocab_loss, and ZERO_E_INVAL for top, temperature or a dtype.
 */
int zero_distill_loss(const zero_loss_t *a, const zero_top_logits_t *t, void *hip_stream);

/* Message of the calling thread's last error ("" if none).  Valid until the
 * thread's next call into the library. */
const char *zero_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* ZERO_H_ */
