// Internal declarations of the products with an epilogue, their gradients, layer norm and the
// orthogonalised update. Not part of the C ABI; the enums' values are mhc.h's.
#pragma once
#include "block_internal.h"

namespace mhc {

// cuTensorMapEncodeTiled for `batch` row-major matrices of 16-bit elements: rows of `inner` elements
// `pitch_bytes` apart, matrices `batch_bytes`; boxes of 64 x box_rows in the 128-byte swizzle.
bool encode_matrices16(CUtensorMap *m, bool bf16, const void *ptr, unsigned long long inner, unsigned long long rows,
                       unsigned long long batch, unsigned long long pitch_bytes, unsigned long long batch_bytes,
                       unsigned int box_rows);

// One operand of a product: element (row, k) is at p[row * pitch + k], or with `turned` at p[k * pitch + row].
struct Operand {
    const void *p;
    long long pitch;                                // in elements, a multiple of 8; p on 16 bytes
    bool turned;
};

// What is done to the sums before they are stored.
enum Epilogue : int {
    EPI_SUMS,       // out = acc, or added to out; of the splits: fp32 sums
    EPI_LINEAR,     // z = acc + bias, out = act(z) + residual
    EPI_SLOPE       // out = acc * act'(z)
};
struct EpilogueArgs {
    void *out;                                      // [m][n], contiguous
    int out_dtype, accumulate;
    const void *bias;                               // [n] or NULL
    int bias_dtype;
    const void *residual;                           // rows or NULL
    long long residual_stride;
    int residual_dtype;
    void *z;                                        // LINEAR: [m][n] contiguous, to write, or NULL; SLOPE: rows to read
    long long z_stride;
    int z_dtype;
    int act;
    int wide;                                       // every row that is written lies on the boundaries of runs of 8
    int extra_runs, bias_runs;                      // and of residual or of z that is read, and the bias
};
struct Product {
    long long m;
    int n;
    long long k;
    bool bf16;                                      // the operands' type, else fp16
    bool exact;                                     // sums in short pieces, for an fp32 result
    Operand a, b;                                   // [m][k], [n][k]
    Epilogue kind;
    EpilogueArgs epi;
    float *parts;                                   // of split sums, product_parts_bytes()
    float *row_sums;                                // EPI_SUMS, a turned: [m], to take the sums over k of a's rows, or NULL
    int add_row_sums;
};
size_t product_parts_bytes(long long m, int n, long long k);
// Whether the sums over k of a's rows come cheaper beside the products than from launch_column_sums().
bool product_sums_rows(long long m, int n, long long k);
// An mhc_status: one launch, or two where the summed axis is split.
int launch_product(const Product &p, int sms, unsigned int *status, bool pdl, cudaStream_t s);

// Up to kFewTokens rows of a: the same product by a kernel that is bound by reading b once.
constexpr int kFewTokens = 64;
int launch_few_tokens(const Product &p, int sms, unsigned int *status, bool pdl, cudaStream_t s);

// 16-bit rows to rows `pitch` apart, on 16-byte boundaries; two such jobs, either with no rows.
struct CopyJob {
    const void *src;
    long long stride, rows;
    int n;
    void *dst;
    long long pitch;
};
cudaError_t launch_copy_rows16(const CopyJob &a, const CopyJob &b, int sms, bool pdl, cudaStream_t s);
// Sums over rows of a 16-bit [rows][n]: out[n] fp32 (accumulate: added); the copies beside it.
int launch_column_sums(const void *x, long long stride, int dtype, long long rows, int n, float *out, int accumulate, const CopyJob &a,
                       const CopyJob &b, int sms, bool pdl, cudaStream_t s);

struct LayerNormArgs {
    long long T;
    int H;
    const void *x, *w, *b;
    long long x_stride;
    int x_dtype, w_dtype, b_dtype, out_dtype;
    float eps, inv_h;
    void *out;
    float *stats;                                   // [T][2]: mean, rstd; or NULL
    int out_runs;                                   // out's rows lie on the boundaries of runs of 8
};
cudaError_t launch_layer_norm(const LayerNormArgs &a, int sms, unsigned int *status, bool pdl, cudaStream_t s);

struct LayerNormBackArgs {
    long long T;
    int H;
    const void *d_out, *x, *d_residual, *w;
    long long d_stride, x_stride, r_stride;
    int d_dtype, x_dtype, w_dtype;
    const float *stats;
    float inv_h;
    void *d_x;
    float *d_w, *d_b;                               // each or NULL
    float *sums;                                    // layer_norm_sums_bytes()
    int out_runs;                                   // d_x's rows lie on the boundaries of runs of 8
};
size_t layer_norm_sums_bytes(long long T, int H);
int launch_layer_norm_back(const LayerNormBackArgs &a, unsigned int *status, bool pdl, cudaStream_t s);

struct OrthogonalArgs {
    const void *g;
    int dtype;
    long long row_stride, batch_stride;
    int batch, m, n, steps;
    float a, b, c, eps;
    void *out;
    int out_dtype;
    void *workspace;
};
size_t orthogonal_workspace(int batch, int m, int n);
int launch_orthogonal(const OrthogonalArgs &a, int sms, unsigned int *status, bool pdl, cudaStream_t s);

}  // namespace mhc
