// Internal declarations of the gated residual block, its backward pass and
// the 8-bit checkpoints. Not part of the C ABI; the enums' values are mhc.h's.
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "mhc.h"

namespace mhc {

// What the entry points share (mhc_api.cu). Both return an mhc_status.
// Whether the current device runs this library; its SM count and status word.
int require_device(int *sms, unsigned int **status);
int note_launch(cudaError_t e);       // of one kernel launch; counts it when it went out
bool pdl_enabled();                   // launch as programmatic dependents
unsigned long long wait_timeout_ns();
// cuTensorMapEncodeTiled for a 2D row-major tensor of 16-bit elements: `inner`
// of them a row, rows `pitch_bytes` apart, boxes of 64 x box_rows in the
// 128-byte swizzle.
bool encode_rows16(CUtensorMap *m, bool bf16, const void *ptr, unsigned long long inner,
                   unsigned long long rows, unsigned long long pitch_bytes, unsigned int box_rows);

constexpr int kCkptGroup = 32;                      // values that share a scale byte
constexpr int kBlockMaxHidden = 65536;
inline long long ckpt_groups(int H) { return (H + kCkptGroup - 1) / kCkptGroup; }

// What both directions read of a block (mhc_block, resolved).
struct BlockForm {
    long long T;
    int H;
    const void *w_post, *w_pre;
    int w_post_dtype, w_pre_dtype;
    const void *gate;
    int gate_dtype, gate_form, gate_act;
    long long gate_stride;
    const float *res_scale;
    int scale_form;
    float eps_post, eps_pre, weight_offset;
    int post_norm;
    float inv_h;                                    // 1 / H
};

struct Ckpt {
    uint8_t *codes;                                 // NULL: none
    uint8_t *scales;
};

struct BlockFwdArgs {
    BlockForm f;
    const void *y, *residual;
    long long y_stride, r_stride;
    void *residual_out, *h;
    float *rstd;                                    // [T][2] or NULL
    int format;                                     // of every checkpoint
    Ckpt ck_y, ck_r, ck_h;
};

// Sums over tokens, one set per CTA of the row kernel: sums[p][0] for d_w_post
// (and a channel gate), sums[p][1] for d_w_pre, sums[p][2] for a channel
// scale, each [H]; scale_sums[p][2] for a single scale, in two floats.
constexpr int kBackSums = 3;
struct BlockBwdArgs {
    BlockForm f;
    const void *d_ro, *d_h, *y, *residual;          // y / residual NULL: from the checkpoint
    long long d_ro_stride, d_h_stride, y_stride, r_stride;
    int format;
    Ckpt ck_y, ck_r;
    const float *rstd;
    void *d_y, *d_r;
    void *d_gate;                                   // written here for TOKEN and FULL
    float *sums, *scale_sums;
};

struct BlockSumArgs {
    BlockForm f;
    const float *sums, *scale_sums;
    int parts;                                      // CTAs of the row kernel; 0: write zeros
    float *d_w_post, *d_w_pre, *d_gate, *d_res_scale;   // each or NULL; d_gate for CHANNEL only
};

// CTAs of the backward row kernel at most: its sums' sets in the workspace.
constexpr int kBackMaxParts = 304;

cudaError_t launch_block_fwd(const BlockFwdArgs &a, int dtype, int r_dtype, int sms, bool pdl,
                             cudaStream_t s);
// *parts: the sets of sums it leaves
cudaError_t launch_block_bwd(const BlockBwdArgs &a, int dtype, int r_dtype, int sms, bool pdl,
                             int *parts, cudaStream_t s);
cudaError_t launch_block_sums(const BlockSumArgs &a, bool pdl, cudaStream_t s);

struct CkptArgs {
    const void *x;                                  // pack: in
    void *out;                                      // unpack: out
    long long stride;                               // of x or out, in elements
    long long T;
    int H;
    Ckpt c;
};
cudaError_t launch_ckpt_pack(const CkptArgs &a, int dtype, int format, int sms, bool pdl, cudaStream_t s);
cudaError_t launch_ckpt_unpack(const CkptArgs &a, int dtype, int format, int sms, bool pdl, cudaStream_t s);

struct DwArgs {
    const void *d_out;
    long long d_out_stride;
    int dtype;                                      // MHC_BF16 or MHC_F16
    Ckpt x;
    int format;
    long long T;
    int n, k;
    void *d_w;
    int d_w_dtype, accumulate;
    void *workspace;
};
// Whether the rows of d_out lie apart and on 16-byte boundaries (else they are copied there first).
bool dw_rows_aligned(const void *d_out, long long stride, long long T, int n);
size_t dw_workspace(long long T, int n, int k, bool d_aligned);
// An mhc_status: several launches, each counted.
int launch_dw(const DwArgs &a, bool d_aligned, int sms, unsigned int *status, bool pdl, cudaStream_t s);

}  // namespace mhc
