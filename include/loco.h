/*
 * loco.h — C ABI of libloco, the GB300 (sm_103a) hot path of LoCo gradient
 * compression.
 *
 * Source of the method: "LoCo: Low-Bit Communication Adaptor for Large-scale
 * Model Training" (Xie, Lin, Toh, Zhou; arXiv 2407.04480), HTML body, §3.1
 * (Eqns 1-3), §3.2 (Eqns 4-7), §3.3 (Eqn 8) and §4 (Adam family, Eqn 9).
 *
 * General conventions (apply to every entry point below):
 *  - Every data pointer is DEVICE memory owned by the caller.  The library
 *    allocates nothing, keeps no state between calls and never synchronises
 *    the stream.  Arrays of per-rank pointers (`codes`, `scales`) are HOST
 *    arrays of device pointers; they are read during the call and copied by
 *    value into the kernel launch, so the caller may free them on return.
 *  - Every call is stream ordered: it validates its arguments on the host,
 *    enqueues its kernel(s) on `stream` (NULL = legacy default stream) and
 *    returns.  On any argument error nothing is launched and nothing is
 *    written.  A failed launch returns LOCO_ERR_CUDA and the CUDA error text
 *    is available from loco_last_error().
 *  - Layouts: flat, contiguous, element i of a bucket of n elements.  Quant
 *    block b covers elements [b*block, min((b+1)*block, n)); nb =
 *    ceil(n / block).  Packed codes of block b start at byte
 *    b*block*bits/8.  4-bit codes are two's-complement nibbles, element 2j of
 *    the block in the low nibble of byte j, element 2j+1 in the high nibble.
 *    8-bit codes are int8.  Padding elements of a ragged last block get code 0.
 *  - Alignment: every buffer of the gradient path (grad, err, err_codes,
 *    err_steps, codes, scales, mean, param, m, v, param_bf16) must be 16-byte aligned
 *    (LOCO_ERR_MISALIGNED otherwise).  The receivers stage each rank's steps
 *    with 16-byte copies, so a rank's scales placed at an offset inside a
 *    larger buffer (an exchange buffer, a shard of a bucket) must start on a
 *    16-byte boundary: a shard of a bucket starting at a multiple of 4 quant
 *    blocks does.
 *  - The calls allocate nothing and never synchronise, so they can be captured
 *    in a CUDA graph.  Step counters, the reset decision and the Adam constants
 *    are computed on the host at call time and become part of the captured
 *    launch: a graph captured at step k replays step k.  The first call of each
 *    configuration (bits, block, W, dtype, ...) on each device queries
 *    occupancy and sets the kernel's shared-memory limit on that device; make
 *    it before capturing.
 *  - Arithmetic is IEEE binary32, round to nearest even, every product and
 *    every sum rounded on its own (no product is fused into a following add);
 *    the exact operation order of each step is stated at the
 *    entry point.  Non-finite inputs are outside the contract: no call reads
 *    or writes out of bounds on them, but the values produced are unspecified.
 */
#ifndef LOCO_H
#define LOCO_H

#include <stdint.h>
#include <stddef.h>

/* The entry points below are the only symbols the library exports; every
 * other symbol (kernels, helpers, the statically linked CUDA runtime) is
 * hidden, so the library can share a process with other CUDA code, including
 * another build of itself. */
#if defined(__GNUC__) || defined(__clang__)
#define LOCO_API __attribute__((visibility("default")))
#else
#define LOCO_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t, declared without the CUDA headers. */
typedef struct CUstream_st* loco_stream_t;

typedef enum {
  LOCO_OK = 0,
  LOCO_ERR_INVALID_ARG = 1,  /* null pointer, n < 0 or n > LOCO_MAX_N, W < 1, step < 1, beta outside [0,1], kappa <= 0, bad scale */
  LOCO_ERR_UNSUPPORTED = 2,  /* bits not in {4,8}, block not in {64,128,256}, W > LOCO_MAX_RANKS, unknown dtype/mode */
  LOCO_ERR_MISALIGNED = 3,   /* a pointer violates the alignment rule above */
  LOCO_ERR_CUDA = 4          /* the kernel launch failed; see loco_last_error() */
} loco_status;

typedef enum { LOCO_F32 = 0, LOCO_BF16 = 1 } loco_dtype;

/* How the quantisation step Delta_b of block b is chosen (the scale s of Eqn 1). */
typedef enum {
  LOCO_SCALE_ABSMAX = 0,  /* Delta_b = A_b / qmax with A_b = max |h_i| over the block's valid elements */
  LOCO_SCALE_FIXED = 1    /* Delta_b = 1/s for every block, s = fixed_scale (the paper's s = 2^19, 2^17; §3.1) */
} loco_scale_mode;

#define LOCO_MAX_RANKS 16

/* Largest bucket a call accepts (2^48 elements, far beyond any device memory);
 * every size the library derives from n then fits in int64_t.  Larger n is
 * LOCO_ERR_INVALID_ARG, and the size helpers below return 0 for it. */
#define LOCO_MAX_N ((int64_t)1 << 48)

/* Sender-side hyper-parameters (§3.1-3.2). */
typedef struct {
  int32_t bits;           /* p of Round_p-bit (Eqn 1): 4 or 8                                    */
  int32_t block;          /* quant block length: 64, 128 or 256 elements                         */
  int32_t scale_mode;     /* loco_scale_mode                                                    */
  float   fixed_scale;    /* s for LOCO_SCALE_FIXED (> 0, finite); ignored for ABSMAX            */
  float   beta;           /* weight of the previous error in the moving average (Eqn 5), [0,1]  */
  float   err_scale_mult; /* kappa = s_e / s (Eqn 7; the paper uses 4 or 6), > 0                 */
  int64_t reset_period;   /* T_c of the periodic reset (Eqn 7; paper 512 or 1024); 0 = never    */
} loco_config;

/* Adam / AdamW hyper-parameters for the fused receiver step (§4, Eqn 9). */
typedef struct {
  float   lr;              /* eta                                                               */
  float   beta1;           /* weight of the previous m: m = beta1*m + (1-beta1)*g               */
  float   beta2;           /* weight of the previous v: v = beta2*v + (1-beta2)*g*g             */
  float   eps;             /* delta                                                             */
  float   weight_decay;    /* decoupled (AdamW) decay; 0 = plain Adam                           */
  int32_t bias_correction; /* 1: bias-corrected step (c1, c2 of loco_adam_step); 0: c1=lr, c2=1  */
  int32_t eps_inside_sqrt; /* 1: 1/sqrt(v+eps) as printed in §4; 0: 1/(sqrt(v)+eps) as in Adam  */
} loco_adam_hparams;

/* nb = ceil(n / block); 0 for n <= 0, n > LOCO_MAX_N or block <= 0. */
LOCO_API int64_t loco_num_blocks(int64_t n, int32_t block);

/* Bytes of packed codes for a bucket of n elements: nb * block * bits / 8; 0 on bad arguments
 * (n <= 0, n > LOCO_MAX_N, bits or block <= 0). */
LOCO_API int64_t loco_code_bytes(int64_t n, int32_t bits, int32_t block);

/*
 * loco_compress — sender side of one LoCo step on one rank's flat gradient bucket.
 * Paper: §3.1 Eqn (2) (compensate), Eqns (1),(3) (low-bit compressor),
 * §3.2 Eqns (4),(5) (moving average of the compression error) and Eqn (7)
 * (error clipping to the 8-bit compressor's range and the periodic reset).
 *
 * Per block b, with qmax = 2^(bits-1)-1, qmin = -2^(bits-1), k = step:
 *   h_i   = f32(g_i) + e_i                                    (Eqn 2)
 *   A_b   = max_i |h_i| over the valid elements
 *   ABSMAX: Delta_b = A_b/qmax, inv_b = qmax/A_b  (both 0 when A_b == 0, or
 *           when qmax/A_b overflows fp32, i.e. A_b < qmax/FLT_MAX)
 *   FIXED:  Delta_b = 1/s,      inv_b = s
 *   q_i   = rint_even(clamp(h_i*inv_b, qmin, qmax))           (Eqns 1, 3)
 *   d_i   = f32(q_i)*Delta_b ;  r_i = h_i - d_i                (Eqn 4)
 *   t_i   = beta*e_i + (1-beta)*r_i                            (Eqn 5; 1-beta formed once in fp32)
 *   De_b  = Delta_b/kappa ; lo = -128*De_b ; hi = 127*De_b
 *   e_i'  = t_i<lo ? lo : (t_i>hi ? hi : t_i)                  (Eqn 7 saturation)
 *   e_i'  = 0 if reset_period > 0 and k % reset_period == 0    (Eqn 7 reset)
 *
 * grad    [n] device, dtype grad_dtype (LOCO_F32 or LOCO_BF16); read only.
 * err     [n] device fp32, in/out: e_{k-1} on entry, e_k on return.  Start a
 *         run with zeros (the paper's e_0 = 0).
 * step    1-based step counter k of this call (>= 1), owned by the caller.
 * codes   [loco_code_bytes(n)] device, out.
 * scales  [nb] device fp32, out: Delta_b (the receiver decodes q*Delta_b).
 * n == 0 is a valid empty call: nothing is launched.
 * grad must not alias err, codes or scales.
 */
LOCO_API loco_status loco_compress(const loco_config* cfg, const void* grad, int32_t grad_dtype,
                          float* err, int64_t n, int64_t step,
                          uint8_t* codes, float* scales, loco_stream_t stream);

/*
 * loco_compress_e8 — loco_compress with the compensation error stored in 8 bits,
 * as the paper keeps it (§3.2 Eqn 7: e_k = compressor(e~_k; s_e, 8) with
 * s_e = kappa*s, decompressed by Eqn 2 before it is added back): one int8 code
 * per element plus one fp32 step per quant block instead of an fp32 error.
 * Codes and scales are bit-identical in format to loco_compress's.
 *
 * Per block b (Delta_b, inv_b, q_i, d_i, r_i as in loco_compress):
 *   e_i    = f32(qe_i) * De_b                        (stored state; zeros to start)
 *   h_i    = f32(g_i) + e_i                           (Eqn 2)
 *   t_i    = beta*e_i + (1-beta)*r_i                  (Eqn 5)
 *   De_b'  = Delta_b/kappa ;  inv_e = kappa*inv_b     (s_e = kappa*s, fp32; 0 if it overflows)
 *   qe_i'  = rint_even(clamp(t_i*inv_e, -128, 127)); 0 on a reset step (Eqn 7)
 * err_codes [n] device int8, in/out (16-byte aligned).
 * err_steps [nb] device fp32, in/out (the De_b; zeros to start).
 * With s_e = 4s..6s the new contribution (1-beta)*r must exceed half a step
 * Delta/(2*kappa) to be stored at all, so beta (weight of the previous error)
 * should be well below 1 with this storage.
 */
LOCO_API loco_status loco_compress_e8(const loco_config* cfg, const void* grad, int32_t grad_dtype,
                             int8_t* err_codes, float* err_steps, int64_t n, int64_t step,
                             uint8_t* codes, float* scales, loco_stream_t stream);

/*
 * loco_decode_reduce — receiver side: decode W ranks' packed buckets and
 * average them in fp32 (§3.3, Eqn 8; the all-to-all variant that never
 * re-compresses a partial sum).
 *
 *   d_{w,i}  = f32(q_{w,i}) * Delta_{w,b}
 *   mean_i   = (((d_{0,i} + d_{1,i}) + d_{2,i}) + ... + d_{W-1,i}) / f32(W)
 *
 * codes[w], scales[w] (host array of W device pointers) hold rank w's output
 * of loco_compress with the same bits/block.  Only cfg->bits and cfg->block
 * are read.  mean [n] device fp32, out; it must not alias any input.
 * 1 <= W <= LOCO_MAX_RANKS.
 */
LOCO_API loco_status loco_decode_reduce(const loco_config* cfg, const uint8_t* const* codes,
                               const float* const* scales, int32_t W, int64_t n,
                               float* mean, loco_stream_t stream);

/*
 * loco_adam_step — loco_decode_reduce fused with one Adam(W) update of the
 * rank's parameters (§4, Eqn 9: the optimizer consumes the averaged low-bit
 * gradient g~ of Eqn 8).  g~_i is formed exactly as in loco_decode_reduce and
 * is never written to memory.  Per element, in this order (Kingma & Ba's Adam
 * with decoupled weight decay; the bias corrections of their Algorithm 1,
 * m_hat = m/(1 - beta1^t) and v_hat = v/(1 - beta2^t), are folded into the
 * step size and the denominator, as torch.optim.AdamW arranges them, except
 * that 1/sqrt(1 - beta2^t) is a rounded factor rather than a divisor; the same
 * update in exact arithmetic, a different rounding in fp32):
 *   p   = p - (lr*wd)*p
 *   m   = beta1*m + (1-beta1)*g~
 *   v   = beta2*v + (1-beta2)*(g~*g~)
 *   den = sqrt(v)*c2 + eps        c2 = 1/sqrt(1 - beta2^t)
 *        (eps_inside_sqrt: den = sqrt(v*c2 + eps), c2 = 1/(1 - beta2^t))
 *   p   = p - c1*(m/den)          c1 = lr/(1 - beta1^t)
 * lr*wd, 1-beta1 and 1-beta2 are formed once in fp32; c1 and c2 once in
 * double from the fp32 hyper-parameters, rounded to fp32 (c1 = lr, c2 = 1
 * without bias correction).  The paper's own convention (beta on the new
 * term, no bias correction, 1/sqrt(v+delta)) is beta1 = 1-0.1,
 * beta2 = 1-beta2_paper, bias_correction = 0, eps_inside_sqrt = 1.
 * param, m, v [n] device fp32, in/out.  t = 1-based optimizer step.
 */
LOCO_API loco_status loco_adam_step(const loco_config* cfg, const uint8_t* const* codes,
                           const float* const* scales, int32_t W, int64_t n,
                           float* param, float* m, float* v,
                           const loco_adam_hparams* hp, int64_t t, loco_stream_t stream);

/*
 * loco_adam_step_bf16 — loco_adam_step that also writes the updated parameters
 * rounded to bf16 (nearest, halves to even) into param_bf16 [n] (device,
 * 16-byte aligned, out): the 16-bit parameter copy a sharded data-parallel job
 * all-gathers after the update (the 16-bit parameters of the Table I memory
 * and communication comparison, §4).  Everything else as loco_adam_step.
 */
LOCO_API loco_status loco_adam_step_bf16(const loco_config* cfg, const uint8_t* const* codes,
                                const float* const* scales, int32_t W, int64_t n,
                                float* param, float* m, float* v, uint16_t* param_bf16,
                                const loco_adam_hparams* hp, int64_t t, loco_stream_t stream);

/*
 * loco_sgd_step — loco_decode_reduce fused with one LoCo-SGD step (§4: the
 * SGD iterate theta_{k+1} = theta_k - eta * g~_k with g~ from Eqn 8):
 *   p = p - lr*g~          (one fp32 product, one fp32 subtraction)
 * g~ is formed exactly as in loco_decode_reduce and never written to memory.
 * param [n] device fp32, in/out.  param_bf16 [n] device, out, or NULL: when
 * given it receives the updated parameters rounded to bf16 (nearest even).
 */
LOCO_API loco_status loco_sgd_step(const loco_config* cfg, const uint8_t* const* codes,
                          const float* const* scales, int32_t W, int64_t n,
                          float* param, uint16_t* param_bf16, float lr, loco_stream_t stream);

/*
 * loco_shard_range — shard j of W of a bucket for the sharded receiver of
 * §3.3 (the all-to-all variant around Eqn 8): every rank compresses its whole
 * bucket, sends the low-bit codes and steps of shard j to rank j, and rank j
 * decodes and averages the W slices it receives (loco_decode_reduce, or a
 * fused optimizer step, on the shard's n_j = hi - lo elements) and updates its
 * part of the parameters.
 *
 * The bucket is cut into units of U = 4*block elements (so every shard starts
 * on a quant-block boundary and its codes and steps start 16-byte aligned in
 * the rank's buffers); with nu = ceil(n / U), shard j holds units
 * [j*base + min(j, rem), (j+1)*base + min(j+1, rem)) where base = nu / W and
 * rem = nu % W, clipped to n.  Shards are contiguous, in rank order, cover
 * [0, n) exactly, and differ in length by at most one unit; when nu < W the
 * last W - nu shards are empty (lo == hi).  Shard j's codes are bytes
 * [lo*bits/8, lo*bits/8 + loco_code_bytes(hi - lo)) of a rank's codes and its
 * steps are floats [lo/block, lo/block + ceil((hi - lo)/block)) of its scales.
 *
 * lo, hi (host, out): element range of shard j.  Errors: NULL lo or hi,
 * n < 0 or n > LOCO_MAX_N, W < 1, j outside [0, W) -> LOCO_ERR_INVALID_ARG;
 * block not in {64, 128, 256} or W > LOCO_MAX_RANKS -> LOCO_ERR_UNSUPPORTED.
 * Host only: no CUDA call.
 */
LOCO_API loco_status loco_shard_range(int64_t n, int32_t block, int32_t W, int32_t j, int64_t* lo, int64_t* hi);

/* ==========================================================================
 * Layers in front of the gradient bucket: normalisation, linear layers and the
 * 8-bit activation checkpoints their backward passes read.
 *
 * Matrices are row major: element (i, j) of a matrix p is p[i*ld + j], ld >=
 * cols counted in elements, the columns of a row contiguous.  A matrix or
 * vector needs only its element type's alignment (a slice of a flat bucket or
 * a view of a wider matrix is fine); 16-byte aligned bases with ld a multiple
 * of 8 (bf16) or 4 (fp32) elements take the wide loads.  codes and workspace
 * must be 16-byte aligned.  rows and cols are at most LOCO_MAX_DIM.
 * Outputs must not overlap any other buffer, with one exception: the output of
 * an entry point that takes a residual may be the residual itself (same
 * pointer, ld and type).  Column ranges of one wider matrix do not overlap.
 * Statuses are those above: a null, short or overlapping buffer, a size or ld
 * out of range is LOCO_ERR_INVALID_ARG, an unknown dtype, activation or kind
 * LOCO_ERR_UNSUPPORTED, a misaligned pointer LOCO_ERR_MISALIGNED.
 * Arithmetic is binary32 (sums, statistics and accumulators included); an
 * output is rounded once, to its own type.  Activations use the hardware's 2^x
 * and 1/x: with u = 2^-24 their relative error is at most (10 + 1.5 |v|) u for
 * SiLU, (26 + 1.13 v^2) u for GELU and (10 + 6 |g|) u for its tanh form, g = 2
 * sqrt(2/pi) (v + 0.044715 v^3), in the lower tails too; a slope's is at most
 * twice that, relative to the sum of its two terms' magnitudes.  An activation
 * or slope below 2^-100 in magnitude may come out as 0.  NaN and infinities propagate as
 * the formulas have it: an output that reads none is not touched by them.
 * Results do not change from run to run.
 * ========================================================================== */

#define LOCO_MAX_DIM ((int64_t)0x7fffffff)

/* Values of a checkpoint that share one step. */
#define LOCO_CKPT_BLOCK 32

typedef enum {
  LOCO_ACT_NONE = 0,      /* v                                                               */
  LOCO_ACT_RELU = 1,      /* max(v, 0)                                                       */
  LOCO_ACT_GELU = 2,      /* v * (1 + erf(v / sqrt 2)) / 2                                    */
  LOCO_ACT_GELU_TANH = 3, /* v * (1 + tanh(sqrt(2/pi) * (v + 0.044715 v^3))) / 2              */
  LOCO_ACT_SILU = 4       /* v / (1 + exp(-v))                                               */
} loco_act;

typedef enum {
  LOCO_NORM_LAYER = 0, /* rows less their mean, over the root of their variance + eps */
  LOCO_NORM_RMS = 1    /* rows over the root of their mean square + eps; no mean is taken */
} loco_norm_kind;

typedef struct {
  int32_t kind;        /* loco_norm_kind                                              */
  float   eps;         /* added to the variance; finite, >= 0                         */
  int32_t x_dtype;     /* loco_dtype of x, dx and the residual gradient               */
  int32_t y_dtype;     /* loco_dtype of y and dy                                      */
  int32_t param_dtype; /* loco_dtype of gamma and beta                                */
  int32_t grad_dtype;  /* loco_dtype of dgamma and dbeta                              */
} loco_norm_config;

typedef struct {
  int32_t act;         /* loco_act                                                    */
  int32_t out_dtype;   /* loco_dtype of the outputs (y; dx; dw and db) and the residual */
  int32_t param_dtype; /* loco_dtype of bias (forward), gamma and beta (weight gradient) */
} loco_linear_config;

/*
 * 8-bit activation checkpoint of a matrix [rows, cols]: every row is cut into
 * blocks of LOCO_CKPT_BLOCK = 32 values (nb = ceil(cols/32)); with A the
 * block's largest magnitude,
 *   e = max(floor(log2 A) - 6, -126)          (-126 for A = 0)
 *   c = rint_even(v * 2^-e) clamped to [-127, 127]
 * codes  [rows, nb*32] int8, contiguous; the padding of a ragged block is 0
 * scales [rows, nb] uint8, contiguous: e + 127; 255 marks a block that held
 *        a NaN or an infinity (codes 0), which reads back as NaN
 * The step 2^e is a power of two, so c * 2^e is exact in bf16 (and fp32): a
 * tensor-core product over restored values rounds none of its operands, and a
 * bf16 value is off by at most half a step (an fp32 value within the last
 * step below 2^(e+7) by less than one).
 */

/* Bytes of codes (rows * nb * 32) and of scales (rows * nb); 0 for rows or cols outside [1, LOCO_MAX_DIM]. */
LOCO_API int64_t loco_ckpt_code_bytes(int64_t rows, int64_t cols);
LOCO_API int64_t loco_ckpt_scale_bytes(int64_t rows, int64_t cols);

/* x [rows, cols] (x_dtype, row pitch ldx) -> codes, scales.  rows == 0 or cols == 0 is an empty call. */
LOCO_API loco_status loco_ckpt_encode(const void* x, int32_t x_dtype, int64_t ldx, int64_t rows, int64_t cols,
                             int8_t* codes, uint8_t* scales, loco_stream_t stream);

/*
 * out = act(c * 2^e * gamma_j + beta_j), [rows, cols] of out_dtype, row pitch
 * ldo.  gamma, beta [cols] of param_dtype, each may be NULL (1 and 0): a norm's
 * output from its checkpoint.  LOCO_ACT_NONE without them restores the values.
 */
LOCO_API loco_status loco_ckpt_decode(const int8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                             int32_t act, const void* gamma, const void* beta, int32_t param_dtype,
                             void* out, int32_t out_dtype, int64_t ldo, loco_stream_t stream);

/*
 * loco_norm_forward — per row i of x [rows, cols]:
 *   LAYER: m = mean_j x_j, r = 1/sqrt(mean_j (x_j - m)^2 + eps)
 *   RMS:   m = 0,          r = 1/sqrt(mean_j x_j^2 + eps)
 *   xhat_j = (x_j - m) * r ;  y_j = xhat_j * gamma_j + beta_j
 * gamma, beta [cols], each may be NULL.  mean, rstd [rows] fp32, out, each may
 * be NULL (a RMS norm's mean is not written).  codes/scales: checkpoint of
 * xhat, out, both or neither.  cols >= 1; rows == 0 is an empty call.
 */
LOCO_API loco_status loco_norm_forward(const loco_norm_config* cfg, const void* x, int64_t ldx, int64_t rows,
                              int64_t cols, const void* gamma, const void* beta, void* y, int64_t ldy,
                              float* mean, float* rstd, int8_t* codes, uint8_t* scales, loco_stream_t stream);

/* Bytes of workspace loco_norm_backward needs for dgamma/dbeta; 0 for sizes out of range. */
LOCO_API int64_t loco_norm_workspace_bytes(int64_t rows, int64_t cols);

/*
 * loco_norm_backward — gradients of loco_norm_forward for dy [rows, cols] (y_dtype):
 *   g_j = dy_j * gamma_j
 *   dx_j = r * (g_j - [LAYER: mean_k g_k] - xhat_j * mean_k(g_k * xhat_k)) + residual_j
 *   dgamma_j = sum_i dy_ij * xhat_ij ;  dbeta_j = sum_i dy_ij
 * xhat comes from x (with mean and rstd as the forward pass wrote them; mean is
 * not read for RMS) or, where x is NULL, from the checkpoint codes/scales.
 * residual [rows, cols] of x_dtype (the gradient that reached x past the
 * norm) may be NULL, and may be dx itself.  dgamma, dbeta [cols] of grad_dtype,
 * each may be NULL; workspace (ws_bytes >= loco_norm_workspace_bytes) may be
 * NULL when both are.  rows == 0 writes zeros to dgamma and dbeta.
 */
LOCO_API loco_status loco_norm_backward(const loco_norm_config* cfg, const void* dy, int64_t lddy, const void* x,
                               int64_t ldx, const int8_t* codes, const uint8_t* scales, const float* mean,
                               const float* rstd, int64_t rows, int64_t cols, const void* gamma,
                               const void* residual, int64_t ldr, void* dx, int64_t lddx, void* dgamma,
                               void* dbeta, void* workspace, int64_t ws_bytes, loco_stream_t stream);

/*
 * loco_linear_align — copies a bf16 matrix src [rows, cols] to rows that start
 * on 16-byte boundaries: dst 16-byte aligned, ldd a multiple of 8.  The columns
 * from cols to the next multiple of 8 are written as zeros (dst holds them in
 * its last row too).  The entry points below take operands with any pitch, but
 * the tensor memory accelerator only reads aligned rows: in large
 * products a copy costs less than reading operands as they lie (T = 4095, N =
 * 4097, K = 4099: 438 us as they lie, 136 us with both copied).  rows == 0 or
 * cols == 0 is an empty call.
 */
LOCO_API loco_status loco_linear_align(const void* src, int64_t lds, int64_t rows, int64_t cols, void* dst,
                                       int64_t ldd, loco_stream_t stream);

/*
 * Whether two matrices of elements of bytes_a and bytes_b (1 to 16) bytes may
 * share a byte: 1 or 0, by the rule of the entry points (of different pitches
 * and several rows each, whether their ranges of memory meet; else exactly).
 * An entry point that is given a copy of an operand cannot see what the
 * operand itself overlaps: this can.  A NULL or empty matrix overlaps none;
 * sizes that no entry point takes give 1.
 */
LOCO_API int32_t loco_matrices_overlap(const void* a, int64_t lda, int64_t rows_a, int64_t cols_a, int32_t bytes_a,
                                       const void* b, int64_t ldb, int64_t rows_b, int64_t cols_b, int32_t bytes_b);

/*
 * loco_linear_forward — z = x w^T + bias ;  y = act(z) + residual.
 * x [T, K] and w [N, K] bf16, products exact and accumulated in fp32 (but for a
 * few rows by the tensor cores, which cut a partial sum rather than round it: up
 * to 2.2 units of 2^-24 of the sum of the terms' magnitudes measured at K =
 * 4096, 3.6 at 11008); bias [N]
 * of param_dtype or NULL; residual [T, N] and y [T, N] of out_dtype, residual
 * may be NULL or y itself.  codes/scales: checkpoint of z [T, N], out, both or
 * neither.  T == 0 or N == 0 is an empty call; K == 0 gives z = bias.
 */
LOCO_API loco_status loco_linear_forward(const loco_linear_config* cfg, const void* x, int64_t ldx, const void* w,
                                int64_t ldw, const void* bias, const void* residual, int64_t ldr, int64_t T,
                                int64_t N, int64_t K, void* y, int64_t ldy, int8_t* codes, uint8_t* scales,
                                loco_stream_t stream);

/*
 * loco_linear_backward_input — dx = (dy w) * act'(z) + residual.
 * dy [T, N] and w [N, K] bf16; z [T, K], the pre-activation of the layer that
 * produced x, from its checkpoint codes/scales (ignored for LOCO_ACT_NONE):
 * then dx is that layer's dz.  residual and dx [T, K] of out_dtype, residual
 * may be NULL or dx itself.  T == 0 or K == 0 is an empty call.
 */
LOCO_API loco_status loco_linear_backward_input(const loco_linear_config* cfg, const void* dy, int64_t lddy,
                                       const void* w, int64_t ldw, const int8_t* codes, const uint8_t* scales,
                                       const void* residual, int64_t ldr, int64_t T, int64_t N, int64_t K,
                                       void* dx, int64_t lddx, loco_stream_t stream);

/* Bytes of workspace loco_linear_backward_weight needs where beta is given; 0 for N out of range. */
LOCO_API int64_t loco_linear_workspace_bytes(int64_t N);

/*
 * loco_linear_backward_weight — dw = dy^T x ;  db_n = sum_t dy_tn.
 * dy [T, N] bf16; x [T, K] bf16 or, where x is NULL, v * gamma_k + beta_k of
 * the values v a checkpoint codes/scales of [T, K] stands for (a norm's output
 * from the checkpoint of its normalised rows; gamma, beta [K] of param_dtype,
 * each may be NULL, ignored with x), formed as
 *   dw_nk = gamma_k * (sum_t dy_tn v_tk) + beta_k * db_n.
 * dw [N, K] and db [N] of out_dtype; db may be NULL.  cfg->act is not read.
 * workspace (ws_bytes >= loco_linear_workspace_bytes(N)) may be NULL without
 * beta, and with x.  T == 0 writes zeros, whatever x, gamma and beta are; it
 * reads none of them and needs no workspace.
 */
LOCO_API loco_status loco_linear_backward_weight(const loco_linear_config* cfg, const void* dy, int64_t lddy,
                                        const void* x, int64_t ldx, const int8_t* codes, const uint8_t* scales,
                                        const void* gamma, const void* beta, int64_t T, int64_t N, int64_t K,
                                        void* dw, int64_t lddw, void* db, void* workspace, int64_t ws_bytes,
                                        loco_stream_t stream);

/*
 * Waits inside the linear-layer kernels (a tile's copies, a tile's products)
 * end after two seconds and 20 microseconds per 64 of the summed dimension at
 * most; a kernel that gave one up counts it.  What it had not finished of its
 * output is then not written, or, where several CTAs add up parts of a sum, NaN
 * (and the checkpoint's scales 255).  This reads the count of the current device
 * since the library was loaded into *count (host).  It synchronises with the
 * device: for diagnosis, not for the training loop.
 */
LOCO_API loco_status loco_linear_timeouts(int64_t* count);

/* Static text for a status code. */
LOCO_API const char* loco_status_string(loco_status s);

/* Text of the last LOCO_ERR_CUDA (or argument error) raised on the calling
 * host thread; "" if none.  Thread local; valid until the next call. */
LOCO_API const char* loco_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* LOCO_H */
