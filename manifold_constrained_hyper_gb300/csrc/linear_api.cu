// Host side of the products with an epilogue, their gradients, layer norm and the orthogonalised update
// (include/mhc.h): argument validation and dispatch.
#include <cmath>

#include "api_common.h"
#include "linear_internal.h"
#include "orthogonal.h"

using namespace mhc;

namespace {

constexpr int64_t kMostTokens = (int64_t(1) << 31) - 1024;

bool width_ok(int w) { return w >= 1 && w <= kBlockMaxHidden; }
bool half_ok(mhc_dtype d) { return d == MHC_BF16 || d == MHC_F16; }
bool act_ok(mhc_linear_act a) { return a >= MHC_LINEAR_NONE && a <= MHC_LINEAR_GELU_TANH; }
bool sizes_ok(int64_t T, int n, int k) { return T > 0 && T < kMostTokens && width_ok(n) && width_ok(k); }
size_t up256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }
long long pitch16(long long w) { return (w + 7) / 8 * 8; }
size_t copy_bytes(int64_t rows, int w, bool aligned) { return aligned ? 0 : up256(static_cast<size_t>(rows) * pitch16(w) * 2); }
bool on_runs(const void *p, mhc_dtype d) { return aligned(p, d == MHC_F32 ? 32 : 16); }

// Operand `o` from rows that lie as they do, or from a copy of them at *at, which moves on past it.
void operand(Operand *o, CopyJob *job, const void *p, int64_t stride, int64_t rows, int w, bool turned, uint8_t **at) {
    *o = {p, rows == 1 ? pitch16(w) : stride, turned};
    *job = {};
    if (mhc_linear_rows_aligned(p, stride, rows, w)) return;
    *o = {*at, pitch16(w), turned};
    *job = {p, stride, rows, w, *at, pitch16(w)};
    *at += copy_bytes(rows, w, false);
}
int copy(const CopyJob (&jobs)[2], int sms, bool pdl, cudaStream_t s) {
    if (!jobs[0].rows && !jobs[1].rows) return MHC_OK;
    return note_launch(launch_copy_rows16(jobs[0], jobs[1], sms, pdl, s));
}

// mhc_linear and mhc_linear_dx: x [T, k], w [n, k] or, turned, [k, n], into out [T, n].
size_t forward_bytes(int64_t T, int n, int k, bool x_aligned, bool w_aligned, bool turned) {
    if (!sizes_ok(T, n, k)) return 0;
    return copy_bytes(T, k, x_aligned) + (turned ? copy_bytes(k, n, w_aligned) : copy_bytes(n, k, w_aligned)) +
           (T > kFewTokens ? product_parts_bytes(T, n, k) : 0);
}
struct Forward {
    const void *x, *w;
    int64_t x_stride, w_stride;
    mhc_dtype dtype;
    int64_t T;
    int n, k;
    bool turned;
    Epilogue kind;
    EpilogueArgs e;
    void *workspace;
};
mhc_status forward(const Forward &f, void *stream) {
    int sms = 0;
    unsigned int *status = nullptr;
    if (int r = require_device(&sms, &status)) return static_cast<mhc_status>(r);
    const bool pdl = pdl_enabled();
    cudaStream_t const s = static_cast<cudaStream_t>(stream);
    uint8_t *at = static_cast<uint8_t *>(f.workspace);
    Product p = {};
    CopyJob jobs[2];
    operand(&p.a, &jobs[0], f.x, f.x_stride, f.T, f.k, false, &at);
    operand(&p.b, &jobs[1], f.w, f.w_stride, f.turned ? f.k : f.n, f.turned ? f.n : f.k, f.turned, &at);
    if (int r = copy(jobs, sms, pdl, s)) return static_cast<mhc_status>(r);
    p.m = f.T;
    p.n = f.n;
    p.k = f.k;
    p.bf16 = f.dtype == MHC_BF16;
    p.exact = f.e.out_dtype == MHC_F32;
    p.kind = f.kind;
    p.epi = f.e;
    if (f.T <= kFewTokens) return static_cast<mhc_status>(launch_few_tokens(p, sms, status, pdl, s));
    p.parts = product_parts_bytes(f.T, f.n, f.k) ? reinterpret_cast<float *>(at) : nullptr;
    return static_cast<mhc_status>(launch_product(p, sms, status, pdl, s));
}

}  // namespace

extern "C" {

int mhc_linear_rows_aligned(const void *p, int64_t stride, int64_t rows, int n) { return dw_rows_aligned(p, stride, rows, n); }

size_t mhc_linear_workspace_bytes(int64_t tokens, int n, int k, int x_aligned, int w_aligned) {
    return forward_bytes(tokens, n, k, x_aligned != 0, w_aligned != 0, false);
}
size_t mhc_linear_dx_workspace_bytes(int64_t tokens, int n, int k, int d_out_aligned, int w_aligned) {
    return forward_bytes(tokens, k, n, d_out_aligned != 0, w_aligned != 0, true);
}
size_t mhc_linear_dw_workspace_bytes(int64_t tokens, int n, int k, int d_out_aligned, int x_aligned) {
    if (!sizes_ok(tokens, n, k)) return 0;
    return copy_bytes(tokens, n, d_out_aligned != 0) + copy_bytes(tokens, k, x_aligned != 0) +
           product_parts_bytes(n, k, tokens);
}

mhc_status mhc_linear(const void *x, int64_t x_stride, const void *w, int64_t w_stride, mhc_dtype dtype, int64_t tokens,
                      int n, int k, const void *bias, mhc_dtype bias_dtype, const void *residual, int64_t residual_stride,
                      mhc_linear_act act, void *out, mhc_dtype out_dtype, void *z_out, void *workspace,
                      size_t workspace_bytes, void *stream) {
    if (tokens < 0 || x_stride < 0 || w_stride < 0 || residual_stride < 0 || !act_ok(act)) return MHC_ERR_SHAPE;
    if (!width_ok(n) || !width_ok(k) || tokens >= kMostTokens) return MHC_ERR_UNSUPPORTED;
    if (!half_ok(dtype) || (out_dtype != dtype && out_dtype != MHC_F32)) return MHC_ERR_UNSUPPORTED;
    if (bias && bias_dtype != dtype && bias_dtype != MHC_F32) return MHC_ERR_UNSUPPORTED;
    if (tokens == 0) return MHC_OK;
    if (!x || !w || !out) return MHC_ERR_NULL;
    if (!aligned(x, 2) || !aligned(w, 2) || !aligned(z_out, 2) || !aligned(out, size_of(out_dtype)) ||
        !aligned(residual, size_of(out_dtype)) || (bias && !aligned(bias, size_of(bias_dtype))) || !aligned(workspace, 16))
        return MHC_ERR_ALIGN;
    const size_t need = mhc_linear_workspace_bytes(tokens, n, k, mhc_linear_rows_aligned(x, x_stride, tokens, k),
                                                   mhc_linear_rows_aligned(w, w_stride, n, k));
    if (need && !workspace) return MHC_ERR_NULL;
    if (workspace_bytes < need) return MHC_ERR_WORKSPACE;
    Span ins[4] = {};
    if (!rows_span(x, x_stride, tokens, k, 2, &ins[0]) || !rows_span(w, w_stride, n, k, 2, &ins[1])) return MHC_ERR_SHAPE;
    if (bias) ins[2] = {bias, n * size_of(bias_dtype)};
    if (residual && !rows_span(residual, residual_stride, tokens, n, size_of(out_dtype), &ins[3])) return MHC_ERR_SHAPE;
    const Span outs[] = {{out, static_cast<size_t>(tokens) * n * size_of(out_dtype)},
                         {z_out, z_out ? static_cast<size_t>(tokens) * n * 2 : 0},
                         {workspace, need}};
    if (aliased(outs, 3, ins, 4, 0, 3)) return MHC_ERR_ALIAS;
    Forward f = {x, w, x_stride, w_stride, dtype, tokens, n, k, false, EPI_LINEAR, {}, workspace};
    f.e.out = out;
    f.e.out_dtype = out_dtype;
    f.e.bias = bias;
    f.e.bias_dtype = bias_dtype;
    f.e.residual = residual;
    f.e.residual_stride = tokens == 1 ? n : residual_stride;
    f.e.residual_dtype = out_dtype;
    f.e.z = z_out;
    f.e.z_dtype = dtype;
    f.e.act = act;
    f.e.wide = n % 8 == 0 && on_runs(out, out_dtype) && on_runs(z_out, dtype);
    f.e.extra_runs = on_runs(residual, out_dtype) && f.e.residual_stride % 8 == 0;
    f.e.bias_runs = !bias || on_runs(bias, bias_dtype);
    return forward(f, stream);
}

mhc_status mhc_linear_dx(const void *d_out, int64_t d_out_stride, const void *w, int64_t w_stride, mhc_dtype dtype,
                         int64_t tokens, int n, int k, const void *z, int64_t z_stride, mhc_linear_act act, void *d_x,
                         mhc_dtype d_x_dtype, void *workspace, size_t workspace_bytes, void *stream) {
    if (tokens < 0 || d_out_stride < 0 || w_stride < 0 || z_stride < 0 || !act_ok(act)) return MHC_ERR_SHAPE;
    if (!width_ok(n) || !width_ok(k) || tokens >= kMostTokens) return MHC_ERR_UNSUPPORTED;
    if (!half_ok(dtype) || (d_x_dtype != dtype && d_x_dtype != MHC_F32)) return MHC_ERR_UNSUPPORTED;
    if (tokens == 0) return MHC_OK;
    if (!d_out || !w || !d_x || (act != MHC_LINEAR_NONE && !z)) return MHC_ERR_NULL;
    if (!aligned(d_out, 2) || !aligned(w, 2) || !aligned(z, 2) || !aligned(d_x, size_of(d_x_dtype)) || !aligned(workspace, 16))
        return MHC_ERR_ALIGN;
    const size_t need = mhc_linear_dx_workspace_bytes(tokens, n, k, mhc_linear_rows_aligned(d_out, d_out_stride, tokens, n),
                                                      mhc_linear_rows_aligned(w, w_stride, n, k));
    if (need && !workspace) return MHC_ERR_NULL;
    if (workspace_bytes < need) return MHC_ERR_WORKSPACE;
    Span ins[3] = {};
    if (!rows_span(d_out, d_out_stride, tokens, n, 2, &ins[0]) || !rows_span(w, w_stride, n, k, 2, &ins[1])) return MHC_ERR_SHAPE;
    if (act != MHC_LINEAR_NONE && !rows_span(z, z_stride, tokens, k, 2, &ins[2])) return MHC_ERR_SHAPE;
    const Span outs[] = {{d_x, static_cast<size_t>(tokens) * k * size_of(d_x_dtype)}, {workspace, need}};
    if (aliased(outs, 2, ins, 3, -1, -1)) return MHC_ERR_ALIAS;
    const bool slope = act != MHC_LINEAR_NONE;
    Forward f = {d_out, w, d_out_stride, w_stride, dtype, tokens, k, n, true, slope ? EPI_SLOPE : EPI_LINEAR, {}, workspace};
    f.e.out = d_x;
    f.e.out_dtype = d_x_dtype;
    if (slope) {
        f.e.z = const_cast<void *>(z);
        f.e.z_dtype = dtype;
        f.e.z_stride = tokens == 1 ? k : z_stride;
        f.e.act = act;
    }
    f.e.wide = k % 8 == 0 && on_runs(d_x, d_x_dtype);
    f.e.extra_runs = !slope || (on_runs(z, dtype) && f.e.z_stride % 8 == 0);
    f.e.bias_runs = 1;
    return forward(f, stream);
}

mhc_status mhc_linear_dw(const void *d_out, int64_t d_out_stride, const void *x, int64_t x_stride, mhc_dtype dtype,
                         int64_t tokens, int n, int k, void *d_w, mhc_dtype d_w_dtype, float *d_bias, int accumulate,
                         void *workspace, size_t workspace_bytes, void *stream) {
    if (tokens < 0 || d_out_stride < 0 || x_stride < 0 || !dtype_ok(d_w_dtype)) return MHC_ERR_SHAPE;
    if (!width_ok(n) || !width_ok(k) || tokens >= kMostTokens || !half_ok(dtype)) return MHC_ERR_UNSUPPORTED;
    if (!d_w || (tokens > 0 && (!d_out || !x))) return MHC_ERR_NULL;
    if (!aligned(d_out, 2) || !aligned(x, 2) || !aligned(d_w, size_of(d_w_dtype)) || !aligned(d_bias, 4) || !aligned(workspace, 16))
        return MHC_ERR_ALIGN;
    const bool da = mhc_linear_rows_aligned(d_out, d_out_stride, tokens, n), xa = mhc_linear_rows_aligned(x, x_stride, tokens, k);
    const size_t need = mhc_linear_dw_workspace_bytes(tokens, n, k, da, xa);
    if (need && !workspace) return MHC_ERR_NULL;
    if (workspace_bytes < need) return MHC_ERR_WORKSPACE;
    Span ins[2] = {};
    if (tokens > 0 && (!rows_span(d_out, d_out_stride, tokens, n, 2, &ins[0]) || !rows_span(x, x_stride, tokens, k, 2, &ins[1])))
        return MHC_ERR_SHAPE;
    const Span outs[] = {{d_w, static_cast<size_t>(n) * k * size_of(d_w_dtype)},
                         {d_bias, d_bias ? static_cast<size_t>(n) * 4 : 0},
                         {workspace, need}};
    if (aliased(outs, 3, ins, 2, -1, -1)) return MHC_ERR_ALIAS;
    if (tokens == 0 && accumulate) return MHC_OK;
    int sms = 0;
    unsigned int *status = nullptr;
    if (int r = require_device(&sms, &status)) return static_cast<mhc_status>(r);
    const bool pdl = pdl_enabled();
    cudaStream_t const s = static_cast<cudaStream_t>(stream);
    uint8_t *at = static_cast<uint8_t *>(workspace);
    Product p = {};
    p.m = n;
    p.n = k;
    p.k = tokens;
    p.bf16 = dtype == MHC_BF16;
    p.exact = d_w_dtype == MHC_F32;
    p.kind = EPI_SUMS;
    p.epi.out = d_w;
    p.epi.out_dtype = d_w_dtype;
    p.epi.accumulate = accumulate != 0;
    p.epi.wide = k % 8 == 0 && on_runs(d_w, d_w_dtype);
    p.epi.extra_runs = p.epi.bias_runs = 1;
    CopyJob jobs[2] = {};
    if (tokens > 0) {
        operand(&p.a, &jobs[0], d_out, d_out_stride, tokens, n, true, &at);
        operand(&p.b, &jobs[1], x, x_stride, tokens, k, true, &at);
    }
    // the bias's sums go beside the products, or else the copies beside them
    const bool beside = d_bias && tokens > 0 && product_sums_rows(n, k, tokens);
    if (beside) {
        p.row_sums = d_bias;
        p.add_row_sums = accumulate != 0;
    }
    if (int r = d_bias && !beside ? launch_column_sums(d_out, tokens == 1 ? n : d_out_stride, dtype, tokens, n, d_bias, accumulate, jobs[0], jobs[1], sms, pdl, s)
                       : copy(jobs, sms, pdl, s))
        return static_cast<mhc_status>(r);
    p.parts = product_parts_bytes(n, k, tokens) ? reinterpret_cast<float *>(at) : nullptr;
    return static_cast<mhc_status>(launch_product(p, sms, status, pdl, s));
}

mhc_status mhc_layer_norm(const void *x, int64_t x_stride, mhc_dtype dtype, int64_t tokens, int hidden, const void *w,
                          mhc_dtype w_dtype, const void *b, mhc_dtype b_dtype, float eps, void *out, mhc_dtype out_dtype,
                          float *stats, void *stream) {
    if (tokens < 0 || x_stride < 0 || !(eps >= 0.f) || std::isinf(eps) || !dtype_ok(dtype) || !dtype_ok(out_dtype) ||
        (w && !dtype_ok(w_dtype)) || (b && !dtype_ok(b_dtype)))
        return MHC_ERR_SHAPE;
    if (!width_ok(hidden) || tokens >= kMostTokens || (out_dtype != dtype && dtype != MHC_F32)) return MHC_ERR_UNSUPPORTED;
    if (tokens == 0) return MHC_OK;
    if (!x || !out) return MHC_ERR_NULL;
    if (!aligned(x, size_of(dtype)) || !aligned(out, size_of(out_dtype)) || !aligned(stats, 4) ||
        (w && !aligned(w, size_of(w_dtype))) || (b && !aligned(b, size_of(b_dtype))))
        return MHC_ERR_ALIGN;
    Span ins[3] = {};
    if (!rows_span(x, x_stride, tokens, hidden, size_of(dtype), &ins[0])) return MHC_ERR_SHAPE;
    if (w) ins[1] = {w, hidden * size_of(w_dtype)};
    if (b) ins[2] = {b, hidden * size_of(b_dtype)};
    const Span outs[] = {{out, static_cast<size_t>(tokens) * hidden * size_of(out_dtype)},
                         {stats, stats ? static_cast<size_t>(tokens) * 8 : 0}};
    if (aliased(outs, 2, ins, 3, -1, -1)) return MHC_ERR_ALIAS;
    int sms = 0;
    unsigned int *status = nullptr;
    if (int r = require_device(&sms, &status)) return static_cast<mhc_status>(r);
    const LayerNormArgs a = {tokens, hidden, x, w, b, tokens == 1 ? hidden : x_stride, dtype, w_dtype, b_dtype, out_dtype, eps,
                             1.f / static_cast<float>(hidden), out, stats, hidden % 8 == 0 && on_runs(out, out_dtype)};
    return static_cast<mhc_status>(note_launch(launch_layer_norm(a, sms, status, pdl_enabled(), static_cast<cudaStream_t>(stream))));
}

size_t mhc_layer_norm_backward_workspace_bytes(int64_t tokens, int hidden) {
    return tokens > 0 && tokens < kMostTokens && width_ok(hidden) ? layer_norm_sums_bytes(tokens, hidden) : 0;
}

mhc_status mhc_layer_norm_backward(const void *d_out, int64_t d_out_stride, mhc_dtype out_dtype, const void *x, int64_t x_stride,
                                   mhc_dtype dtype, const float *stats, int64_t tokens, int hidden, const void *w,
                                   mhc_dtype w_dtype, const void *d_residual, int64_t d_residual_stride, void *d_x, float *d_w,
                                   float *d_b, void *workspace, size_t workspace_bytes, void *stream) {
    if (tokens < 0 || d_out_stride < 0 || x_stride < 0 || d_residual_stride < 0 || !dtype_ok(dtype) || !dtype_ok(out_dtype) ||
        (w && !dtype_ok(w_dtype)))
        return MHC_ERR_SHAPE;
    if (!width_ok(hidden) || tokens >= kMostTokens || (out_dtype != dtype && dtype != MHC_F32)) return MHC_ERR_UNSUPPORTED;
    if (tokens > 0 && (!d_out || !x || !stats || !d_x)) return MHC_ERR_NULL;
    if (!aligned(d_out, size_of(out_dtype)) || !aligned(x, size_of(dtype)) || !aligned(d_residual, size_of(dtype)) ||
        !aligned(d_x, size_of(dtype)) || !aligned(stats, 4) || !aligned(d_w, 4) || !aligned(d_b, 4) ||
        (w && !aligned(w, size_of(w_dtype))) || !aligned(workspace, 16))
        return MHC_ERR_ALIGN;
    const size_t need = d_w || d_b ? mhc_layer_norm_backward_workspace_bytes(tokens, hidden) : 0;
    if (need && !workspace) return MHC_ERR_NULL;
    if (workspace_bytes < need) return MHC_ERR_WORKSPACE;
    Span ins[5] = {};
    if (tokens > 0) {
        if (!rows_span(d_out, d_out_stride, tokens, hidden, size_of(out_dtype), &ins[0]) ||
            !rows_span(x, x_stride, tokens, hidden, size_of(dtype), &ins[1]) ||
            (d_residual && !rows_span(d_residual, d_residual_stride, tokens, hidden, size_of(dtype), &ins[2])))
            return MHC_ERR_SHAPE;
        ins[3] = {stats, static_cast<size_t>(tokens) * 8};
        if (w) ins[4] = {w, hidden * size_of(w_dtype)};
    }
    const Span outs[] = {{d_x, static_cast<size_t>(tokens) * hidden * size_of(dtype)},
                         {d_w, d_w ? static_cast<size_t>(hidden) * 4 : 0},
                         {d_b, d_b ? static_cast<size_t>(hidden) * 4 : 0},
                         {workspace, need}};
    if (aliased(outs, 4, ins, 5, 0, 2)) return MHC_ERR_ALIAS;
    int sms = 0;
    unsigned int *status = nullptr;
    if (int r = require_device(&sms, &status)) return static_cast<mhc_status>(r);
    const bool one = tokens == 1;
    const LayerNormBackArgs a = {tokens, hidden, d_out, x, d_residual, w, one ? hidden : d_out_stride, one ? hidden : x_stride,
                                 one ? hidden : d_residual_stride, out_dtype, dtype, w_dtype, stats,
                                 1.f / static_cast<float>(hidden), d_x, d_w, d_b, static_cast<float *>(workspace),
                                 hidden % 8 == 0 && on_runs(d_x, dtype)};
    return static_cast<mhc_status>(launch_layer_norm_back(a, status, pdl_enabled(), static_cast<cudaStream_t>(stream)));
}

size_t mhc_orthogonalize_workspace_bytes(int batch, int m, int n) {
    return batch > 0 && batch <= 65535 && width_ok(m) && width_ok(n) ? orthogonal_workspace(batch, m, n) : 0;
}

mhc_status mhc_orthogonalize(const void *g, int64_t row_stride, int64_t batch_stride, mhc_dtype dtype, int batch, int m, int n,
                             int steps, float a, float b, float c, float eps, void *out, mhc_dtype out_dtype, void *workspace,
                             size_t workspace_bytes, void *stream) {
    if (batch < 0 || row_stride < 0 || batch_stride < 0 || !dtype_ok(dtype) || steps < 1 || steps > 100 || !(eps >= 0.f) ||
        std::isinf(eps) || !(std::fabs(a) < kNsMostUnit) || !(std::fabs(b) <= 1000.f) || !(std::fabs(c) <= 1000.f))
        return MHC_ERR_SHAPE;
    if (!width_ok(m) || !width_ok(n) || batch > 65535 || !half_ok(out_dtype)) return MHC_ERR_UNSUPPORTED;
    if (batch == 0) return MHC_OK;
    const size_t need = mhc_orthogonalize_workspace_bytes(batch, m, n);
    if (!g || !out || (need && !workspace)) return MHC_ERR_NULL;
    if (!aligned(g, size_of(dtype)) || !aligned(out, 2) || !aligned(workspace, 16)) return MHC_ERR_ALIGN;
    if (workspace_bytes < need) return MHC_ERR_WORKSPACE;
    Span in;
    if (batch_stride > (int64_t(1) << 45) || !rows_span(g, row_stride, m, n, size_of(dtype), &in)) return MHC_ERR_SHAPE;
    in.n += static_cast<size_t>(batch - 1) * batch_stride * size_of(dtype);
    const Span outs[] = {{out, static_cast<size_t>(batch) * m * n * 2}, {workspace, need}};
    if (aliased(outs, 2, &in, 1, -1, -1)) return MHC_ERR_ALIAS;
    int sms = 0;
    unsigned int *status = nullptr;
    if (int r = require_device(&sms, &status)) return static_cast<mhc_status>(r);
    const OrthogonalArgs o = {g, dtype, m == 1 ? pitch16(n) : row_stride, batch == 1 ? 0 : batch_stride, batch, m, n, steps,
                              a, b, c, eps, out, out_dtype, workspace};
    return static_cast<mhc_status>(launch_orthogonal(o, sms, status, pdl_enabled(), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
