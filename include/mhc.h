/*
 * mhc.h: C ABI of the GB300 (sm_103a) mHC layer boundary, n_hc = 4.
 *
 * The boundary between layer l and l+1 of a manifold-constrained
 * hyper-connection stack, per token (X_{l+1} = B_l X_l + C_l F_l(A_l X_l),
 * "The Hyper Connection Preprocessing GPU Kernel Study", section "why this
 * kernel is called pre"):
 *   post  (residual update): residual'[s] = bf16(post[s]*x + sum_j comb[j][s]*residual[j])
 *   pre   (coefficients and layer input of the next layer): sum of squares of
 *         the flattened 4H residual -> rstd; 24 mixes = TF32(fn) . residual;
 *         pre = sigmoid(..)+eps, post = 2 sigmoid(..), comb = Sinkhorn(softmax(..));
 *         layer_input = bf16(bf16(sum_j pre[j]*residual[j]) * rstd_li * norm_w).
 * The fused entry point does both in one pass over the residual; its shifted
 * form collapses with the previous boundary's pre ("vllm.models.deepseek_v41
 * .nvidia.ops.mhc_boundary", mhc_shifted_post_pre_boundary).
 *
 * Conventions for every entry point below.
 *   - Tensors are plain, contiguous, row-major buffers. "bf16" buffers hold
 *     bfloat16 bit patterns as uint16_t. Unless stated otherwise a pointer is a
 *     DEVICE pointer on the current CUDA device, owned by the caller; the
 *     library never frees or retains it past the call.
 *   - Every pointer must be 16-byte aligned (MHC_ERR_ALIGN otherwise).
 *   - tokens T >= 0 (T == 0 is a no-op returning MHC_OK); hidden H must be a
 *     multiple of 32 in [32, 65536] (MHC_ERR_UNSUPPORTED otherwise).
 *   - stream is a cudaStream_t passed as void* (NULL = legacy default stream).
 *     Work is enqueued asynchronously; argument errors are returned before
 *     anything is enqueued. A launch failure returns MHC_ERR_CUDA.
 *   - No entry point allocates device memory. Scratch space, where needed, is
 *     the caller's `workspace` (see mhc_workspace_bytes).
 *   - Device-side waits are bounded: a kernel whose wait runs out records
 *     MHC_ERR_DEVICE_TIMEOUT in a per-device status word and returns early;
 *     read it with mhc_get_device_status().
 *   - Outputs must not overlap inputs or each other, except that
 *     residual_out may be exactly the residual buffer (in-place update).
 *     Partial overlap returns MHC_ERR_ALIAS.
 *   - Entry points are thread-safe; results are deterministic run to run
 *     for a given (T, H) (fixed reduction order).
 */
#ifndef MHC_H
#define MHC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MHC_OK = 0,
    MHC_ERR_NULL = 1,           /* a required pointer is NULL */
    MHC_ERR_ALIGN = 2,          /* a pointer is not 16-byte aligned */
    MHC_ERR_SHAPE = 3,          /* negative T, bad params (sinkhorn_iters < 1) */
    MHC_ERR_UNSUPPORTED = 4,    /* H outside the supported set, or not an sm_103 device */
    MHC_ERR_ALIAS = 5,          /* an output overlaps an input or another output */
    MHC_ERR_CUDA = 6,           /* a CUDA runtime/driver call failed */
    MHC_ERR_DEVICE_TIMEOUT = 7, /* a device-side bounded wait ran out */
    MHC_ERR_WORKSPACE = 8       /* workspace NULL or smaller than mhc_workspace_bytes */
} mhc_status;

/* Scalar parameters of a boundary ("mhc_boundary" page, mhc_shifted_post_pre_boundary
 * arguments hc_norm_eps, hc_pre_eps, hc_post_scale, sinkhorn_eps,
 * num_sinkhorn_iters, norm_eps). */
typedef struct {
    float hc_norm_eps;   /* eps inside rstd = rsqrt(ssq / (4H) + hc_norm_eps) */
    float hc_pre_eps;    /* pre = sigmoid(.) + hc_pre_eps */
    float hc_post_mult;  /* post = sigmoid(.) * hc_post_mult (2 in DeepSeek) */
    float sinkhorn_eps;  /* softmax floor and Sinkhorn denominator eps */
    float norm_eps;      /* eps of the layer RMSNorm of the collapse (over H) */
    int sinkhorn_iters;  /* >= 1: one column step, then iters-1 (row, column) steps */
    int batch_invariant; /* nonzero: every output of a token is bitwise the same
                          * whatever the batch it comes in (its size, its
                          * position): the hidden-slice plan then depends on
                          * the hidden size only and every reduction runs in
                          * one fixed order. The pages have no counterpart.
                          * Costs latency on small batches (fewer slices). */
} mhc_params;

/* Element types. norm_w of the boundary is F32 or BF16 (the DeepSeek boundary
 * kernel reads bf16 weights; fp32 is the common checkpoint dtype); F16 is for
 * the gated residual block below. */
typedef enum { MHC_F32 = 0, MHC_BF16 = 1, MHC_F16 = 2 } mhc_dtype;

/* ---------------------------------------------------------------------- */
/* Weight preparation ("mhc_boundary" page, prepare_boundary_weight).       */

/* Bytes of the prepared mixer for hidden H: 48 rows x 4H bf16 = 384*H. */
size_t mhc_weight_bytes(int hidden);

/*
 * fn: [24, 4H] fp32, rows 0-3 pre, 4-7 post, 8-23 comb (row-major 4x4),
 *     column s*H + h multiplies stream s, hidden h of the residual.
 * weight: output, mhc_weight_bytes(H) bytes, 16-byte aligned.
 *
 * Each weight w is rounded to TF32 (round half away from zero on the bit
 * pattern: r = (bits(w) + 0x1000) & ~0x1FFF) and split into two bf16 parts,
 * hi = bf16_rne(r) and lo = bf16_rne(r - hi), with hi + lo == r exactly, so
 * BF16 tensor-core products reproduce TF32 products exactly. Layout (uint16
 * units): stacked row r in [0, 48) holds hi of mix r (r < 24) or lo of mix
 * r - 24; for hidden chunk c in [0, H/32), stream s and element e in [0, 32)
 * the value for column k = s*H + 32c + e is at
 *     ((c*4 + s)*48 + r)*32 + 8*((e/8) ^ ((r/2) % 4)) + (e % 8),
 * i.e. per (chunk, stream) a 48 x 64-byte tile, K-major, in the 64-byte
 * swizzled order the tensor cores read from shared memory.
 * This layout deliberately departs from the page's prepared weight, which
 * gathers the same hi/lo parts into register fragments of the warp-level
 * m16n8k16 MMA ([16 slices, k16 steps, 3 m16 tiles, 32 lanes, 4] int32):
 * here the 5th-generation tensor cores read both operands from shared
 * memory, so each (chunk, stream) tile lands there with one bulk copy,
 * already in the swizzled order their descriptors expect. The rounding and
 * the split are the page's, value for value.
 * Inputs must be finite (NaN payloads are not preserved by the rounding).
 */
mhc_status mhc_prepare_weight(const float *fn, int hidden, void *weight, void *stream);

/* ---------------------------------------------------------------------- */
/* Residual update alone ("mhc_boundary" page, residual_update).            */

/*
 * x: [T, H] bf16 layer output; residual: [T, 4, H] bf16; post: [T, 4] fp32;
 * comb: [T, 4, 4] fp32 where comb[t][j][s] carries stream j into stream s.
 * residual_out: [T, 4, H] bf16 (may be == residual).
 *   residual_out[t][s][h] = bf16_rne(chain), chain = post[s]*x[h], then
 *   fma(comb[j][s], residual[j][h], chain) for j = 0..3, every operand and
 *   result of the chain flushed to zero when subnormal.
 */
mhc_status mhc_post(const uint16_t *x, const uint16_t *residual, const float *post,
                    const float *comb, uint16_t *residual_out, int64_t tokens,
                    int hidden, void *stream);

/* ---------------------------------------------------------------------- */
/* Pre and fused boundary.                                                  */

/* Bytes of caller-provided device scratch for mhc_pre / mhc_boundary_fused
 * at (T, H): per-token partial mixes and sums of squares of every hidden
 * slice, and the publication flags. 0 when T == 0. It needs no
 * initialisation. Calls may be captured into a CUDA graph (they allocate
 * nothing and never synchronise). A call whose blocks wait on one another
 * (every shifted call, and the unshifted calls of at most 128 tokens whose
 * streaming kernel forms the coefficients) marks its progress with a flag
 * value; captured, it takes the value from a cell in the workspace and
 * advances the cell itself, so each replay has its own value and replays
 * may run with new contents in the same buffers (no extra kernel). Calls
 * that share a workspace must not overlap in time. The cell sits at the
 * start of the workspace whatever the call's shape, so calls of different
 * shapes, eager or captured, may share one workspace sized for the largest. */
size_t mhc_workspace_bytes(int64_t tokens, int hidden);

/*
 * Unshifted pre ("The Hyper Connection Preprocessing GPU Kernel Study",
 * mhc_pre_big_fuse with the in-kernel square sum; mixes computed in-kernel).
 * residual: [T, 4, H] bf16. weight: from mhc_prepare_weight(fn, H).
 * scale: [3] fp32 (pre, post, comb). base: [24] fp32 (rows of fn).
 * norm_w: [H] of norm_dtype, or NULL to write the raw collapse.
 * Outputs: layer_input [T, H] bf16, pre_out [T, 4], post_out [T, 4],
 * comb_out [T, 4, 4] fp32.
 *   ssq = sum over the 4H values of residual^2, rstd = rsqrt(ssq/(4H) + hc_norm_eps)
 *   mix[n] = sum_k TF32(fn[n][k]) * residual_flat[k]        (fp32 accumulate)
 *   pre[i] = sigmoid(fma(mix[i]*rstd, scale[0], base[i])) + hc_pre_eps
 *   post[i] = sigmoid(fma(mix[4+i]*rstd, scale[1], base[4+i])) * hc_post_mult
 *   comb = Sinkhorn of row softmax of fma(mix[8+4i+k]*rstd, scale[2], base[8+4i+k])
 *          (entries fma(e, 1/sum e, sinkhorn_eps)), sigmoid(v) = 1/min(1+exp(-v), 2^126)
 *   li[h] = bf16(fma chain of pre[j]*residual[j][h]), rstd_li = rsqrt(sum li^2 / H + norm_eps)
 *   layer_input[h] = bf16((li[h]*rstd_li) * norm_w[h])   (li itself when norm_w == NULL)
 * workspace: device scratch of at least mhc_workspace_bytes(T, H) bytes.
 */
mhc_status mhc_pre(const uint16_t *residual, const void *weight, const float *scale,
                   const float *base, const void *norm_w, mhc_dtype norm_dtype,
                   const mhc_params *params, int64_t tokens, int hidden,
                   uint16_t *layer_input, float *pre_out, float *post_out,
                   float *comb_out, void *workspace, size_t workspace_bytes,
                   void *stream);

/*
 * Fused post + pre boundary ("mhc_boundary" page, mhc_shifted_post_pre_boundary
 * and MhcBoundaryKernel): the residual update of mhc_post, then the pre of
 * mhc_pre computed on the UPDATED residual.
 * pre_lag: [T, 4] fp32 pre of the previous boundary (shifted form: the layer
 * input collapses the updated residual with pre_lag, all in one pass over
 * the residual), or NULL (unshifted form: it collapses with this boundary's
 * own pre_out, which re-reads the updated residual).
 * Other arguments as in mhc_post and mhc_pre. residual_out may be == residual.
 * Limits of the shifted form: its blocks wait on one another within one
 * launch, so every hidden slice of a 128-token tile must be resident at
 * once, and an item's collapse must fit its tensor-memory buffer. H / 32
 * must therefore have a divisor d <= 8 with H / (32 d) <= 152 (slices of d
 * chunks of 32, at most one per streaming multiprocessor of a GB300): every
 * multiple of 256 up to 38912 qualifies (7168: 28 slices of 256), H = 65536
 * or 32 * 157 does not. Other H return MHC_ERR_UNSUPPORTED before anything
 * is enqueued. The unshifted form has no such limit.
 */
mhc_status mhc_boundary_fused(const uint16_t *x, const uint16_t *residual,
                              const float *post, const float *comb,
                              const float *pre_lag, const void *weight,
                              const float *scale, const float *base,
                              const void *norm_w, mhc_dtype norm_dtype,
                              const mhc_params *params, int64_t tokens, int hidden,
                              uint16_t *residual_out, uint16_t *layer_input,
                              float *pre_out, float *post_out, float *comb_out,
                              void *workspace, size_t workspace_bytes, void *stream);

/*
 * Unshifted pre from split-K mixes ("The Hyper Connection Preprocessing GPU
 * Kernel Study", the pure path: "square sum and RMSNorm" path 1 and
 * "explaining split-K"): a previous GEMM split the 4H-long contraction of the
 * flattened residual with fn into n_splits parts and left
 *   dot_mix [n_splits, T, 24] fp32   partial mixes (no TF32 rounding implied),
 *   sqrsum  [n_splits, T]     fp32   partial sums of squares of the residual.
 * mix = sum of the splits, ssq = sum of the splits (each in split order, in
 * fp32); rstd = rsqrt(ssq / 4H + hc_norm_eps); pre / post / comb as in
 * mhc_pre; layer_input = the collapse of residual [T, 4, H] with this pre,
 * RMS-normed with norm_w (or the raw collapse when norm_w is NULL).
 * n_splits in [1, 64] (the page's kernel takes 1, 2, 4, 8 or 16), else
 * MHC_ERR_SHAPE. No workspace. Outputs as in mhc_pre; none may alias an
 * input. Enqueued on `stream`: one kernel for up to 1024 tokens (the collapse
 * overlapping the coefficients), else two (coefficients, then the collapse);
 * always two when params->batch_invariant is set.
 */
mhc_status mhc_pre_split_k(const uint16_t *residual, const float *dot_mix, const float *sqrsum,
                           int n_splits, const float *scale, const float *base,
                           const void *norm_w, mhc_dtype norm_dtype, const mhc_params *params,
                           int64_t tokens, int hidden, uint16_t *layer_input, float *pre_out,
                           float *post_out, float *comb_out, void *stream);

/* ---------------------------------------------------------------------- */
/* Allocation-free variant. The pages this library follows have no          */
/* counterpart of this entry point.                                         */

/*
 * mhc_boundary_fused without a workspace, for callers that cannot allocate
 * device memory: code running where cudaMalloc is not permitted or not
 * wanted, such as a serving engine whose memory planner owns every device
 * allocation, or a latency-critical loop that cannot afford the implicit
 * device synchronisation of cudaMalloc/cudaFree. Arguments and results are
 * those of mhc_boundary_fused.
 *
 * Scratch: a fixed 4 MiB array in the library's own device memory, which
 * every GPU that loads the library keeps until the process exits. A call
 * whose mhc_workspace_bytes(tokens, hidden) exceeds 4 MiB returns
 * MHC_ERR_WORKSPACE without enqueuing anything (every decode batch of up to
 * 128 tokens at hidden up to 8192 fits).
 * Set-up: the first call on a device, with that device current, looks up
 * the array's device address; make that first call before any stream
 * capture. Sharing: every call on a device uses the same array and leaves
 * its contents behind; calls that can overlap on the GPU (unordered streams,
 * concurrent host threads) race on it and must be serialised by the caller.
 * No entry needs to start at zero: each call writes every entry it reads.
 * The call allocates nothing (no cudaMalloc, cudaFree or allocating library
 * routine).
 */
mhc_status mhc_boundary_fused_noalloc(const uint16_t *x, const uint16_t *residual,
                                      const float *post, const float *comb,
                                      const float *pre_lag, const void *weight,
                                      const float *scale, const float *base,
                                      const void *norm_w, mhc_dtype norm_dtype,
                                      const mhc_params *params, int64_t tokens, int hidden,
                                      uint16_t *residual_out, uint16_t *layer_input,
                                      float *pre_out, float *post_out, float *comb_out,
                                      void *stream);

/* ---------------------------------------------------------------------- */
/* Gated residual block with a norm on either side (one residual stream),   */
/* its backward pass, and activation checkpoints in 8 bits. The pages have  */
/* no counterpart of these entry points.                                    */

/*
 * Per token, between one block of a network (whose output is y) and the next
 * (whose input is h):
 *   n  = y * rstd_post * (w_post + weight_offset),  rstd_post = 1 / sqrt(mean(y^2) + eps_post)
 *   residual_out = scale * residual + act(gate) * n
 *   h  = residual_out * rstd_pre * (w_pre + weight_offset),
 *        rstd_pre = 1 / sqrt(mean(residual_out^2) + eps_pre)
 * post_norm == 0 leaves the first line out (n = y, rstd_post = 1, and w_post
 * must be NULL). A NULL weight means a weight_offset + w of 1.
 * All arithmetic is fp32; h comes from the unrounded residual_out, and each
 * output is rounded once.
 *
 * Unlike the boundary's, these entry points take any hidden in [1, 65536],
 * and rows that lie `stride` elements apart (>= 0; the elements of a row are
 * contiguous); a pointer needs its element type's alignment only. Fastest are
 * rows on boundaries of 8 elements (pointers and strides, hidden a multiple of
 * 8). Rows off 16-byte boundaries are read in whole blocks of 16 bytes: up to
 * 15 bytes before and after a row are read too (and left alone), which any
 * device allocation that begins and ends on such a boundary holds.
 */
typedef enum {
    MHC_GATE_NONE = 0,      /* act(gate) = 1 */
    MHC_GATE_CHANNEL = 1,   /* gate [H] */
    MHC_GATE_TOKEN = 2,     /* gate [T], gate_stride apart */
    MHC_GATE_FULL = 3       /* gate [T, H], rows gate_stride apart */
} mhc_gate_form;

typedef enum { MHC_ACT_NONE = 0, MHC_ACT_SIGMOID = 1, MHC_ACT_TANH = 2 } mhc_gate_act;

typedef enum {
    MHC_SCALE_NONE = 0,     /* scale = 1 */
    MHC_SCALE_ONE = 1,      /* scale [1] */
    MHC_SCALE_CHANNEL = 2   /* scale [H] */
} mhc_scale_form;

typedef struct {
    int64_t tokens;               /* T >= 0 */
    int hidden;                   /* H in [1, 65536] */
    mhc_dtype dtype;              /* y, h, their gradients */
    mhc_dtype residual_dtype;     /* residual, residual_out, their gradients: dtype or F32 */
    const void *w_post;           /* [H] or NULL */
    const void *w_pre;            /* [H] or NULL */
    mhc_dtype w_post_dtype, w_pre_dtype;
    const void *gate;             /* by gate_form; NULL with MHC_GATE_NONE */
    mhc_dtype gate_dtype;         /* dtype or F32 */
    mhc_gate_form gate_form;
    mhc_gate_act gate_act;
    int64_t gate_stride;          /* elements; TOKEN and FULL */
    const float *res_scale;       /* by scale_form; NULL with MHC_SCALE_NONE */
    mhc_scale_form scale_form;
    float eps_post, eps_pre;      /* >= 0 */
    float weight_offset;          /* added to w_post and w_pre (1 where weights are kept as w - 1) */
    int post_norm;
} mhc_block;

/*
 * An activation checkpoint: rows in groups of 32 values (the last one of a row
 * may be shorter), one scale byte a group. With m the group's largest
 * magnitude and Q the format's largest value (448 for E4M3, 127 for INT8),
 * k is the least integer, at least -126, with m <= Q * 2^k; the scale byte is
 * k + 127 and a value x is held as x * 2^-k rounded to nearest, ties to even.
 * Scaling by 2^-k is exact, so a code is off by that one rounding and is
 * bitwise the same whatever path wrote it. A group with an infinity or a NaN
 * has the scale byte 255 and codes 0, and reads back as NaN throughout.
 */
typedef enum { MHC_CKPT_E4M3 = 1, MHC_CKPT_INT8 = 2 } mhc_ckpt_format;

typedef struct {
    uint8_t *codes;    /* [T, H] contiguous */
    uint8_t *scales;   /* [T, ceil(H / 32)] contiguous */
} mhc_ckpt;

/*
 * The block boundary above. y, residual: inputs. residual_out [T, H] of
 * residual_dtype (may be exactly the residual buffer when residual_stride is
 * H or there is one token) and h [T, H] of dtype: outputs, contiguous. rstd: [T, 2] fp32 (rstd_post,
 * rstd_pre), what the backward pass needs beside y and residual, or NULL.
 * ckpt_y, ckpt_residual, ckpt_h: each NULL or a checkpoint to write of the
 * inputs y and residual and of the rounded h, in the same pass.
 */
mhc_status mhc_block_norm(const mhc_block *block, const void *y, int64_t y_stride,
                          const void *residual, int64_t residual_stride, void *residual_out,
                          void *h, float *rstd, mhc_ckpt_format format, const mhc_ckpt *ckpt_y,
                          const mhc_ckpt *ckpt_residual, const mhc_ckpt *ckpt_h, void *stream);

/* Bytes of device scratch of mhc_block_norm_backward: the partial sums over
 * tokens of the weights' gradients. 0 when T == 0. Needs no initialisation. It lies
 * on a 16-byte boundary; only from a 32-byte one on does the call go by runs of 8
 * elements, else by single ones. */
size_t mhc_block_norm_backward_workspace_bytes(int64_t tokens, int hidden);

/*
 * Backward pass of mhc_block_norm. d_residual_out [T, H] of residual_dtype (or
 * NULL: zero) and d_h [T, H] of dtype: the outputs' gradients. y and residual:
 * the inputs, or NULL with ckpt_y / ckpt_residual given: then their
 * checkpointed values are used. rstd as mhc_block_norm wrote it;
 * residual_out is formed anew from y and residual. With ro the unrounded
 * residual_out and n, g = act(gate) as above:
 *   D          = d_residual_out + rstd_pre*d_h*w2 - ro*rstd_pre^3*mean(d_h*w2*ro)
 *   d_residual = scale * D                 d_res_scale = sum residual * D
 *   d_y        = rstd_post*g*D*w1 - y*rstd_post^3*mean(g*D*w1*y)   (post_norm 0: g*D)
 *   d_w_post   = sum_t g*D*y*rstd_post     d_w_pre = sum_t d_h*ro*rstd_pre
 *   d_gate     = act'(gate) * n * D, summed over what the gate is shared by
 * Outputs: d_y [T, H] of dtype, d_residual [T, H] of residual_dtype (may be
 * exactly the d_residual_out buffer when its stride is H or T is 1), both contiguous;
 * d_w_post, d_w_pre [H] fp32; d_gate [H] fp32 (CHANNEL), [T] fp32 (TOKEN) or
 * [T, H] of gate_dtype (FULL); d_res_scale [1] or [H] fp32. Any of the last
 * four may be NULL where it is not wanted, and must be where there is no such
 * input. Sums over tokens run in an order fixed by the call's sizes, types, forms
 * and alignment: results are the same run to run. The sum of a single scale's
 * gradient is held in 48 bits. T == 0 writes zeros to the sums.
 */
mhc_status mhc_block_norm_backward(const mhc_block *block, const void *d_residual_out,
                                   int64_t d_residual_out_stride, const void *d_h,
                                   int64_t d_h_stride, const void *y, int64_t y_stride,
                                   const void *residual, int64_t residual_stride,
                                   mhc_ckpt_format format, const mhc_ckpt *ckpt_y,
                                   const mhc_ckpt *ckpt_residual, const float *rstd, void *d_y,
                                   void *d_residual, float *d_w_post, float *d_w_pre,
                                   void *d_gate, float *d_res_scale, void *workspace,
                                   size_t workspace_bytes, void *stream);

/* x [T, H] of dtype, rows `stride` elements apart -> out. */
mhc_status mhc_ckpt_pack(const void *x, int64_t stride, mhc_dtype dtype, int64_t tokens,
                         int hidden, mhc_ckpt_format format, const mhc_ckpt *out, void *stream);

/*
 * What the checkpoint stands for -> x [T, H] of dtype, contiguous. F32 holds
 * every value exactly but 2^128, which the largest values of F32 and BF16 may
 * round to and which reads as infinity; BF16 the same and all but those below
 * 2^-126 (rounded). F16 rounds, and gives the largest finite value (65504) of
 * either sign for what lies past it: finite values of any type read back finite.
 */
mhc_status mhc_ckpt_unpack(const mhc_ckpt *ckpt, mhc_ckpt_format format, int64_t tokens,
                           int hidden, mhc_dtype dtype, void *x, void *stream);

/* Bytes of device scratch of mhc_ckpt_linear_dw: x in 16 bits, the sums of
 * tokens that are split, scales of x's columns, and, unless `aligned` (d_out is on a
 * 16-byte boundary and its stride, at least n, a multiple of 16 bytes), d_out's
 * rows on such boundaries. 0 when T == 0 or
 * the call would be refused for its sizes. Needs no initialisation. */
size_t mhc_ckpt_linear_dw_workspace_bytes(int64_t tokens, int n, int k, int aligned);

/*
 * Weight gradient of a projection out = x W^T whose input was checkpointed:
 *   d_w[i][j] = sum_t d_out[t][i] * x[t][j]      (accumulate: added to d_w)
 * d_out: [T, n] of dtype (BF16 or F16), rows d_out_stride elements apart.
 * x: a checkpoint [T, k]; its values are exact in bf16, but 2^128 is infinite.
 * With an F16 d_out they go to fp16 without a power of two that the values of a
 * group of 32 columns share over up to 1024 tokens, and that their sums get back:
 * with 2^K the largest of their scales, nothing overflows, and a value is off by
 * at most 2^(K - 32) (E4M3) or 2^(K - 34) (INT8); those whose own scale is within
 * 2^22 or 2^33 of it are exact. d_w: [n, k] contiguous, of d_w_dtype (any); products
 * and sums are fp32, rounded once; the order of the sums is fixed by the
 * sizes. T < 2^31 - 64; n, k in [1, 65536]. T == 0 writes zeros (accumulate:
 * leaves d_w as it is).
 */
mhc_status mhc_ckpt_linear_dw(const void *d_out, int64_t d_out_stride, mhc_dtype dtype,
                              const mhc_ckpt *x, mhc_ckpt_format format, int64_t tokens, int n,
                              int k, void *d_w, mhc_dtype d_w_dtype, int accumulate,
                              void *workspace, size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------- */
/*
 * The layers on either side of a boundary: layer norm, the projection with its
 * epilogue, their gradients, and the orthogonalised update of a weight.
 * Matrices are rows `stride` elements apart (>= 0) on any boundary of their
 * type; outputs are contiguous. Sums are fp32 and rounded once; their order is
 * fixed by the call's sizes, types and alignment. tokens < 2^31 - 1024, other
 * sizes in [1, 65536]; workspaces lie on a 16-byte boundary and need no
 * initialisation.
 */
typedef enum {
    MHC_LINEAR_NONE = 0,
    MHC_LINEAR_RELU = 1,
    MHC_LINEAR_RELU2 = 2,       /* relu squared */
    MHC_LINEAR_SILU = 3,        /* z / (1 + exp(-z)) */
    MHC_LINEAR_GELU = 4,        /* z * Phi(z), by erfc */
    MHC_LINEAR_GELU_TANH = 5    /* 0.5 z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) */
} mhc_linear_act;

/* Whether `rows` rows of 16-bit elements lie as the tensor cores' loads want
 * them: on 16-byte boundaries, the stride a multiple of 8 and at least n (one
 * row: any stride). Others are copied into the workspace first. */
int mhc_linear_rows_aligned(const void *p, int64_t stride, int64_t rows, int n);

/* Bytes of device scratch of mhc_linear, mhc_linear_dx and mhc_linear_dw: sums
 * of a split product, and copies of operands that are not aligned as above. 0 when T == 0 or the call would be refused for its sizes. */
size_t mhc_linear_workspace_bytes(int64_t tokens, int n, int k, int x_aligned, int w_aligned);
size_t mhc_linear_dx_workspace_bytes(int64_t tokens, int n, int k, int d_out_aligned, int w_aligned);
size_t mhc_linear_dw_workspace_bytes(int64_t tokens, int n, int k, int d_out_aligned, int x_aligned);

/*
 * A projection with its epilogue:
 *   z = x w^T + bias,   out = act(z) + residual
 * x [T, k] and w [n, k] of dtype (BF16 or F16); bias [n] of bias_dtype (dtype
 * or F32) or NULL; residual [T, n] of out_dtype or NULL; out [T, n] of
 * out_dtype (dtype or F32), which may be exactly the residual buffer when its
 * stride is n or T is 1; z_out [T, n] of dtype, what the backward pass of act
 * needs, or NULL (out is formed from the unrounded z). Up to 64 tokens the
 * weights are streamed once through all SMs.
 */
mhc_status mhc_linear(const void *x, int64_t x_stride, const void *w, int64_t w_stride, mhc_dtype dtype,
                      int64_t tokens, int n, int k, const void *bias, mhc_dtype bias_dtype,
                      const void *residual, int64_t residual_stride, mhc_linear_act act, void *out,
                      mhc_dtype out_dtype, void *z_out, void *workspace, size_t workspace_bytes,
                      void *stream);

/*
 * The gradient of its input, through the activation of the layer below:
 *   d_x = (d_out w) * act'(z)
 * d_out [T, n], w [n, k], z [T, k] of dtype; z NULL with MHC_LINEAR_NONE: the
 * product alone. d_x [T, k] of d_x_dtype (dtype or F32). relu'(0) = 0.
 */
mhc_status mhc_linear_dx(const void *d_out, int64_t d_out_stride, const void *w, int64_t w_stride,
                         mhc_dtype dtype, int64_t tokens, int n, int k, const void *z, int64_t z_stride,
                         mhc_linear_act act, void *d_x, mhc_dtype d_x_dtype, void *workspace,
                         size_t workspace_bytes, void *stream);

/*
 * The gradients of its weight and bias:
 *   d_w = d_out^T x,   d_bias = sum over tokens of d_out
 * d_out [T, n] and x [T, k] of dtype; d_w [n, k] of d_w_dtype (any); d_bias [n]
 * fp32 or NULL. accumulate: both are added to what is there. T == 0 writes zeros
 * (accumulate: leaves them).
 */
mhc_status mhc_linear_dw(const void *d_out, int64_t d_out_stride, const void *x, int64_t x_stride,
                         mhc_dtype dtype, int64_t tokens, int n, int k, void *d_w, mhc_dtype d_w_dtype,
                         float *d_bias, int accumulate, void *workspace, size_t workspace_bytes,
                         void *stream);

/*
 * Layer norm of each row, with mean and variance over its H values:
 *   out = (x - mean) * rstd * w + b,   rstd = 1 / sqrt(mean((x - mean)^2) + eps)
 * x [T, H] of dtype (any); w, b [H] of w_dtype, b_dtype (any), each or NULL
 * (1 and 0); out [T, H] of out_dtype: dtype, or any 16-bit type beside an F32
 * x. stats [T, 2] fp32 (mean, rstd), what the backward pass needs, or NULL.
 */
mhc_status mhc_layer_norm(const void *x, int64_t x_stride, mhc_dtype dtype, int64_t tokens, int hidden,
                          const void *w, mhc_dtype w_dtype, const void *b, mhc_dtype b_dtype, float eps,
                          void *out, mhc_dtype out_dtype, float *stats, void *stream);

/* Bytes of device scratch of mhc_layer_norm_backward: partial sums over tokens. */
size_t mhc_layer_norm_backward_workspace_bytes(int64_t tokens, int hidden);

/*
 * Its backward pass. With h = (x - mean) * rstd and e = d_out * w:
 *   d_x = rstd * (e - mean(e) - h * mean(e * h)) + d_residual
 *   d_w = sum over tokens of d_out * h,   d_b = sum over tokens of d_out
 * d_out [T, H] of out_dtype as above; x, stats as in the forward call; d_residual [T, H]
 * of dtype: the gradient that reaches x past the norm, or NULL; d_x [T, H] of dtype, which
 * may be exactly the d_residual buffer when its stride is H or T is 1; d_w, d_b [H] fp32, each or
 * NULL. T == 0 writes zeros to the sums.
 */
mhc_status mhc_layer_norm_backward(const void *d_out, int64_t d_out_stride, mhc_dtype out_dtype,
                                   const void *x, int64_t x_stride, mhc_dtype dtype, const float *stats,
                                   int64_t tokens, int hidden, const void *w, mhc_dtype w_dtype,
                                   const void *d_residual, int64_t d_residual_stride, void *d_x,
                                   float *d_w, float *d_b, void *workspace, size_t workspace_bytes,
                                   void *stream);

/* Bytes of device scratch of mhc_orthogonalize. */
size_t mhc_orthogonalize_workspace_bytes(int batch, int m, int n);

/*
 * The orthogonalised update of `batch` weights [m, n], batch_stride elements
 * apart, by Newton-Schulz products:
 *   X = G / (|G| + eps)  (the Frobenius norm),  then `steps` times
 *   A = X X^T,  X <- (a I + b A + c A A) X
 * G of dtype (any); out [batch, m, n] of out_dtype (BF16 or F16: matrices are
 * held in 22 bits between the products, which is what a 16-bit result takes).
 * steps in [1, 100]; |a| < 16, |b|, |c| <= 1000. Elements of A, of the
 * polynomial and of X past 16 overflow to infinity. A G of zeros gives zeros. batch in [0, 65535].
 */
mhc_status mhc_orthogonalize(const void *g, int64_t row_stride, int64_t batch_stride, mhc_dtype dtype,
                             int batch, int m, int n, int steps, float a, float b, float c, float eps,
                             void *out, mhc_dtype out_dtype, void *workspace, size_t workspace_bytes,
                             void *stream);

/* ---------------------------------------------------------------------- */
/* Status and diagnostics.                                                  */

/* Synchronises `stream`, then reads and clears the current device's status
 * word. Returns MHC_OK, MHC_ERR_DEVICE_TIMEOUT (a kernel's bounded wait ran
 * out since the last read) or MHC_ERR_CUDA. */
mhc_status mhc_get_device_status(void *stream);

/* Extra detail of the last timeout read by mhc_get_device_status: the wait
 * site id (0 if none). */
int mhc_last_timeout_site(void);

/* Human-readable name of a status. Static storage; never NULL. */
const char *mhc_status_string(mhc_status status);

/* Limit of every device-side wait, in nanoseconds (default 1e9 = 1 s).
 * Applies to launches enqueued after the call. ns == 0 restores the default. */
void mhc_set_wait_timeout_ns(uint64_t ns);

/* Test hook for the bounded-wait machinery: launches one CTA that waits on a
 * shared-memory barrier nothing ever arrives at, under the current limit,
 * so that the wait runs out and the kernel returns. Enqueued on `stream`;
 * read the outcome with mhc_get_device_status(). */
mhc_status mhc_debug_unarmed_wait(void *stream);

/* Benchmark hook: the next mhc_pre / mhc_boundary_fused call made by this
 * host thread records `event` (a cudaEvent_t passed as void*) on its stream
 * right after its streaming kernel and before its finishing kernel (the
 * unshifted forms), so that the two kernels can be timed apart with events;
 * a shifted call is the streaming kernel alone, and the event follows it.
 * Consumed by that call; NULL clears a pending event. */
void mhc_debug_record_between(void *event);

/* Test hook for the coefficients' reciprocal (the "mhc_boundary" page's rcp:
 * hardware approximation plus one Newton-Raphson step): compares it with the
 * correctly rounded fp32 reciprocal for the bit patterns first_bits ..
 * first_bits + count - 1 (no wrap past 0xFFFFFFFF, else MHC_ERR_SHAPE).
 * result: device pointer to two u64, 8-byte aligned, set by the caller to
 * {0, ~0} beforehand; result[0] += the number of differing patterns,
 * result[1] = min(its value, the smallest differing pattern). Enqueued on
 * `stream`. The pages have no counterpart. */
mhc_status mhc_debug_rcp_check(uint32_t first_bits, uint64_t count, unsigned long long *result,
                               void *stream);

/* Test hook for the two forms of the coefficients: from reduced values
 * values [tokens][25] fp32 (24 mixes, then the 4H sum of squares), forms
 * pre / post / comb once with one thread per token and once with 16 lanes
 * per token (the form a single-wave shifted call uses), into out_thread and
 * out_lanes [tokens][24] fp32 (pre 4, post 4, comb 16). The two must be
 * bitwise equal. scale [3], base [24] and params as in mhc_pre; device
 * pointers, 16-byte aligned; outputs must not overlap the inputs or each
 * other. Enqueued on `stream`. The pages have no counterpart. */
mhc_status mhc_debug_coef_check(const float *values, const float *scale, const float *base,
                                const mhc_params *params, int hidden, int64_t tokens,
                                float *out_thread, float *out_lanes, void *stream);

/* Slice plan chosen for (T, H): writes the number of hidden slices and the
 * slice width. For tests and the benchmark's byte accounting. */
mhc_status mhc_plan(int64_t tokens, int hidden, int *n_slices, int *slice_width);

/* Whether a shifted mhc_boundary_fused call of (T, H) on the current device
 * runs on one thread-block cluster ("mhc_boundary" page, MhcBoundaryKernel:
 * the hidden slices of one token tile in one cluster, exchanging partial
 * mixes and sums of squares through distributed shared memory): *ctas = the
 * cluster size (the number of hidden slices), or 0 when the call takes the
 * slice-parallel streaming kernel. A call can take a cluster when it has 1 to
 * 64 tokens, params->batch_invariant is 0, its H / 32 chunks split into at
 * most 16 slices of at most 32 chunks and such a cluster can be resident on
 * the device; by default it does so where that is the faster path (a slice
 * of one chunk; of two chunks for up to 32 tokens; of up to four chunks for
 * up to 16 tokens: hidden sizes up to 2048; at hidden 7168 the slice-parallel
 * kernel, which spreads the work over 112 CTAs instead of 16, is faster).
 * Cluster calls need no workspace contents (a workspace is
 * still passed and checked); after the call its bytes 256 .. 256 + 112 T
 * hold each token's 24 mixes and 4H sum of squares as 28 fp32 (the last
 * three zero). Queries the device once per shape. */
mhc_status mhc_plan_cluster(int64_t tokens, int hidden, int *ctas);

/* Benchmark hook: enable = 0 launches the boundary kernels as plain stream
 * kernels; nonzero (the default) as programmatic dependents of the previous
 * kernel on the stream, whose set-up (barriers, tensor memory, descriptor and
 * weight-tile prefetches into L2) overlaps that kernel's end while every
 * read of global memory waits for its completion ("mhc_boundary" page,
 * griddepcontrol around the kernel's prologue). Process-wide. */
void mhc_debug_set_pdl(int enable);

/* Test hook for the dependent launch: a kernel that lets the next kernel on
 * `stream` start at once, waits delay_ns (at most 1,000,000, else
 * MHC_ERR_SHAPE) and then copies n bf16 values from src to dst (device
 * pointers, 16-byte aligned, not overlapping). The pages have no
 * counterpart. */
mhc_status mhc_debug_delayed_copy(const uint16_t *src, uint16_t *dst, int64_t n,
                                  uint32_t delay_ns, void *stream);

/* Test and benchmark hook for the shifted form's decode path, process-wide:
 * 0 (the default) as described at mhc_plan_cluster; 1 every later call takes
 * the slice-parallel streaming kernel; 2 every call that can take a cluster
 * does. Other values act as 0. */
void mhc_debug_set_decode_path(int path);

/* Benchmark hook: the number of kernels this library has launched in the
 * process so far (every entry point that launches, counted when the launch
 * succeeded; thread-safe, process-wide, never reset). The difference across
 * a timed region is the number of the library's kernels in it. */
uint64_t mhc_debug_launch_count(void);

#ifdef __cplusplus
}
#endif
#endif /* MHC_H */
