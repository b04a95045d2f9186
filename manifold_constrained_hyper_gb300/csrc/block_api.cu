// Host side of the gated residual block's, the checkpoints' and the weight
// gradient's entry points (include/mhc.h): argument validation and dispatch.
#include <cmath>

#include "api_common.h"
#include "block_internal.h"
#include "mhc.h"
#include "mhc_internal.h"

using namespace mhc;

namespace {

bool format_ok(mhc_ckpt_format f) { return f == MHC_CKPT_E4M3 || f == MHC_CKPT_INT8; }
Span codes_span(const mhc_ckpt *c, int64_t T, int H) {
    return {c ? c->codes : nullptr, c ? static_cast<size_t>(T) * H : 0};
}
Span scales_span(const mhc_ckpt *c, int64_t T, int H) {
    return {c ? c->scales : nullptr, c ? static_cast<size_t>(T) * ckpt_groups(H) : 0};
}
Ckpt ckpt_of(const mhc_ckpt *c) { return c ? Ckpt{c->codes, c->scales} : Ckpt{nullptr, nullptr}; }

mhc_status check_block(const mhc_block *b, BlockForm *f) {
    if (!b) return MHC_ERR_NULL;
    if (b->tokens < 0) return MHC_ERR_SHAPE;
    if (b->hidden < 1 || b->hidden > kBlockMaxHidden) return MHC_ERR_UNSUPPORTED;
    if (!size_fits(b->tokens, b->hidden)) return MHC_ERR_SHAPE;
    if (!dtype_ok(b->dtype) || (b->residual_dtype != b->dtype && b->residual_dtype != MHC_F32))
        return MHC_ERR_SHAPE;
    if ((b->w_post && !dtype_ok(b->w_post_dtype)) || (b->w_pre && !dtype_ok(b->w_pre_dtype)))
        return MHC_ERR_SHAPE;
    if (b->gate_form < MHC_GATE_NONE || b->gate_form > MHC_GATE_FULL || b->gate_act < MHC_ACT_NONE ||
        b->gate_act > MHC_ACT_TANH || b->scale_form < MHC_SCALE_NONE || b->scale_form > MHC_SCALE_CHANNEL)
        return MHC_ERR_SHAPE;
    // a NaN fails these too
    if (!(b->eps_post >= 0.f) || !(b->eps_pre >= 0.f) || !std::isfinite(b->weight_offset)) return MHC_ERR_SHAPE;
    if (!b->post_norm && b->w_post) return MHC_ERR_SHAPE;
    if (b->gate_form == MHC_GATE_NONE) {
        if (b->gate || b->gate_act != MHC_ACT_NONE) return MHC_ERR_SHAPE;
    } else {
        if (b->gate_dtype != b->dtype && b->gate_dtype != MHC_F32) return MHC_ERR_SHAPE;
        if (b->gate_form != MHC_GATE_CHANNEL && b->gate_stride < 0) return MHC_ERR_SHAPE;
    }
    if (b->scale_form == MHC_SCALE_NONE && b->res_scale) return MHC_ERR_SHAPE;
    if (b->tokens > 0) {
        if (b->gate_form != MHC_GATE_NONE && !b->gate) return MHC_ERR_NULL;
        if (b->scale_form != MHC_SCALE_NONE && !b->res_scale) return MHC_ERR_NULL;
    }
    if (!aligned(b->w_post, b->w_post ? size_of(b->w_post_dtype) : 1) ||
        !aligned(b->w_pre, b->w_pre ? size_of(b->w_pre_dtype) : 1) ||
        !aligned(b->gate, b->gate ? size_of(b->gate_dtype) : 1) || !aligned(b->res_scale, 4))
        return MHC_ERR_ALIGN;
    f->T = b->tokens;
    f->H = b->hidden;
    f->w_post = b->w_post;
    f->w_pre = b->w_pre;
    f->w_post_dtype = b->w_post_dtype;
    f->w_pre_dtype = b->w_pre_dtype;
    f->gate = b->gate;
    f->gate_dtype = b->gate_dtype;
    f->gate_form = b->gate_form;
    f->gate_act = b->gate_act;
    f->gate_stride = b->gate_stride;
    f->res_scale = b->res_scale;
    f->scale_form = b->scale_form;
    f->eps_post = b->eps_post;
    f->eps_pre = b->eps_pre;
    f->weight_offset = b->weight_offset;
    f->post_norm = b->post_norm != 0;
    f->inv_h = 1.f / static_cast<float>(b->hidden);
    return MHC_OK;
}

// The ranges of what both directions read of the block.
bool form_spans(const mhc_block *b, Span out[4]) {
    const size_t H = static_cast<size_t>(b->hidden);
    out[0] = {b->w_post, b->w_post ? H * size_of(b->w_post_dtype) : 0};
    out[1] = {b->w_pre, b->w_pre ? H * size_of(b->w_pre_dtype) : 0};
    out[2] = {b->res_scale, b->scale_form == MHC_SCALE_CHANNEL ? H * 4 : b->scale_form == MHC_SCALE_ONE ? 4 : 0};
    out[3] = {nullptr, 0};
    const size_t e = b->gate ? size_of(b->gate_dtype) : 0;
    if (b->gate_form == MHC_GATE_CHANNEL) out[3] = {b->gate, H * e};
    if (b->gate_form == MHC_GATE_TOKEN) return rows_span(b->gate, b->gate_stride, b->tokens, 1, e, &out[3]);
    if (b->gate_form == MHC_GATE_FULL) return rows_span(b->gate, b->gate_stride, b->tokens, b->hidden, e, &out[3]);
    return true;
}

// Tokens of a weight gradient at most: what a box's 32-bit row coordinate reaches.
constexpr int64_t kDwMaxTokens = (int64_t(1) << 31) - 64;

bool ckpt_ok(const mhc_ckpt *c) { return c->codes && c->scales; }

}  // namespace

extern "C" {

mhc_status mhc_block_norm(const mhc_block *block, const void *y, int64_t y_stride, const void *residual,
                          int64_t residual_stride, void *residual_out, void *h, float *rstd,
                          mhc_ckpt_format format, const mhc_ckpt *ckpt_y, const mhc_ckpt *ckpt_residual,
                          const mhc_ckpt *ckpt_h, void *stream) {
    BlockFwdArgs a = {};
    if (mhc_status s = check_block(block, &a.f)) return s;
    const mhc_ckpt *const cks[] = {ckpt_y, ckpt_residual, ckpt_h};
    for (const mhc_ckpt *c : cks)
        if (c && !format_ok(format)) return MHC_ERR_SHAPE;
    if (y_stride < 0 || residual_stride < 0) return MHC_ERR_SHAPE;
    const int64_t T = block->tokens;
    const int H = block->hidden;
    if (T == 0) return MHC_OK;
    if (!y || !residual || !residual_out || !h) return MHC_ERR_NULL;
    for (const mhc_ckpt *c : cks)
        if (c && !ckpt_ok(c)) return MHC_ERR_NULL;
    const size_t e = size_of(block->dtype), re = size_of(block->residual_dtype);
    if (!aligned(y, e) || !aligned(h, e) || !aligned(residual, re) || !aligned(residual_out, re) ||
        !aligned(rstd, 4))
        return MHC_ERR_ALIGN;
    Span ins[6];
    if (!rows_span(y, y_stride, T, H, e, &ins[0]) || !rows_span(residual, residual_stride, T, H, re, &ins[1]) ||
        !form_spans(block, ins + 2))
        return MHC_ERR_SHAPE;
    const size_t n = static_cast<size_t>(T) * H;
    const Span outs[] = {{residual_out, n * re}, {h, n * e}, {rstd, rstd ? static_cast<size_t>(T) * 8 : 0},
                         codes_span(ckpt_y, T, H), scales_span(ckpt_y, T, H),
                         codes_span(ckpt_residual, T, H), scales_span(ckpt_residual, T, H),
                         codes_span(ckpt_h, T, H), scales_span(ckpt_h, T, H)};
    // one row has no stride
    if (aliased(outs, 9, ins, 6, T == 1 || residual_stride == H ? 0 : -1, 1)) return MHC_ERR_ALIAS;
    int sms = 0;
    if (int s = require_device(&sms, nullptr)) return static_cast<mhc_status>(s);
    a.y = y;
    a.residual = residual;
    a.y_stride = y_stride;
    a.r_stride = residual_stride;
    a.residual_out = residual_out;
    a.h = h;
    a.rstd = rstd;
    a.format = format;
    a.ck_y = ckpt_of(ckpt_y);
    a.ck_r = ckpt_of(ckpt_residual);
    a.ck_h = ckpt_of(ckpt_h);
    return static_cast<mhc_status>(note_launch(launch_block_fwd(
        a, block->dtype, block->residual_dtype, sms, pdl_enabled(), static_cast<cudaStream_t>(stream))));
}

size_t mhc_block_norm_backward_workspace_bytes(int64_t tokens, int hidden) {
    if (tokens <= 0 || hidden < 1 || hidden > kBlockMaxHidden) return 0;
    const size_t parts = static_cast<size_t>(tokens < kBackMaxParts ? tokens : kBackMaxParts);
    return (parts * kBackSums * static_cast<size_t>(hidden) + 2 * parts) * sizeof(float);
}

mhc_status mhc_block_norm_backward(const mhc_block *block, const void *d_residual_out,
                                   int64_t d_residual_out_stride, const void *d_h, int64_t d_h_stride,
                                   const void *y, int64_t y_stride, const void *residual,
                                   int64_t residual_stride, mhc_ckpt_format format, const mhc_ckpt *ckpt_y,
                                   const mhc_ckpt *ckpt_residual, const float *rstd, void *d_y,
                                   void *d_residual, float *d_w_post, float *d_w_pre, void *d_gate,
                                   float *d_res_scale, void *workspace, size_t workspace_bytes,
                                   void *stream) {
    BlockBwdArgs a = {};
    if (mhc_status s = check_block(block, &a.f)) return s;
    if ((ckpt_y || ckpt_residual) && !format_ok(format)) return MHC_ERR_SHAPE;
    if (d_residual_out_stride < 0 || d_h_stride < 0 || y_stride < 0 || residual_stride < 0) return MHC_ERR_SHAPE;
    // either the values or their checkpoint
    if ((y && ckpt_y) || (residual && ckpt_residual)) return MHC_ERR_SHAPE;
    // no gradient of an input that is not there
    if ((d_w_post && !block->w_post) || (d_w_pre && !block->w_pre) ||
        (d_gate && block->gate_form == MHC_GATE_NONE) || (d_res_scale && block->scale_form == MHC_SCALE_NONE))
        return MHC_ERR_SHAPE;
    const int64_t T = block->tokens;
    const int H = block->hidden;
    const size_t e = size_of(block->dtype), re = size_of(block->residual_dtype);
    const bool full = block->gate_form == MHC_GATE_FULL;
    const size_t ge = full ? size_of(block->gate_dtype) : 4;
    if (!aligned(d_y, e) || !aligned(d_h, e) || !aligned(y, e) || !aligned(d_residual_out, re) ||
        !aligned(d_residual, re) || !aligned(residual, re) || !aligned(rstd, 4) || !aligned(d_w_post, 4) ||
        !aligned(d_w_pre, 4) || !aligned(d_gate, ge) || !aligned(d_res_scale, 4) || !aligned(workspace, 16))
        return MHC_ERR_ALIGN;
    const size_t n = static_cast<size_t>(T) * H;
    const size_t need = mhc_block_norm_backward_workspace_bytes(T, H);
    if (T > 0) {
        if (!d_h || (!y && !ckpt_y) || (!residual && !ckpt_residual) || !rstd || !d_y || !d_residual || !workspace)
            return MHC_ERR_NULL;
        if ((ckpt_y && !ckpt_ok(ckpt_y)) || (ckpt_residual && !ckpt_ok(ckpt_residual))) return MHC_ERR_NULL;
        if (workspace_bytes < need) return MHC_ERR_WORKSPACE;
        Span ins[13] = {};
        if ((d_residual_out && !rows_span(d_residual_out, d_residual_out_stride, T, H, re, &ins[0])) ||
            !rows_span(d_h, d_h_stride, T, H, e, &ins[1]) ||
            (y && !rows_span(y, y_stride, T, H, e, &ins[2])) ||
            (residual && !rows_span(residual, residual_stride, T, H, re, &ins[3])) || !form_spans(block, ins + 4))
            return MHC_ERR_SHAPE;
        ins[8] = codes_span(ckpt_y, T, H);
        ins[9] = scales_span(ckpt_y, T, H);
        ins[10] = codes_span(ckpt_residual, T, H);
        ins[11] = scales_span(ckpt_residual, T, H);
        ins[12] = {rstd, static_cast<size_t>(T) * 8};
        const size_t nh = static_cast<size_t>(H) * 4;
        const size_t ng = block->gate_form == MHC_GATE_CHANNEL ? nh : full ? n * ge : static_cast<size_t>(T) * 4;
        const Span outs[] = {{d_residual, n * re}, {d_y, n * e}, {d_w_post, d_w_post ? nh : 0},
                             {d_w_pre, d_w_pre ? nh : 0}, {d_gate, d_gate ? ng : 0},
                             {d_res_scale, d_res_scale ? (block->scale_form == MHC_SCALE_CHANNEL ? nh : 4) : 0},
                             {workspace, need}};
        if (aliased(outs, 7, ins, 13, T == 1 || d_residual_out_stride == H ? 0 : -1, 0)) return MHC_ERR_ALIAS;
    }
    int sms = 0;
    if (int s = require_device(&sms, nullptr)) return static_cast<mhc_status>(s);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int parts = 0;
    float *sums = static_cast<float *>(workspace);
    if (T > 0) {
        const size_t most = static_cast<size_t>(T < kBackMaxParts ? T : kBackMaxParts);
        a.d_ro = d_residual_out;
        a.d_h = d_h;
        a.y = y;
        a.residual = residual;
        a.d_ro_stride = d_residual_out_stride;
        a.d_h_stride = d_h_stride;
        a.y_stride = y_stride;
        a.r_stride = residual_stride;
        a.format = format;
        a.ck_y = ckpt_of(ckpt_y);
        a.ck_r = ckpt_of(ckpt_residual);
        a.rstd = rstd;
        a.d_y = d_y;
        a.d_r = d_residual;
        a.d_gate = block->gate_form == MHC_GATE_CHANNEL ? nullptr : d_gate;
        a.sums = sums;
        a.scale_sums = sums + most * kBackSums * static_cast<size_t>(H);
        if (int s = note_launch(launch_block_bwd(a, block->dtype, block->residual_dtype, sms, pdl_enabled(),
                                                 &parts, st)))
            return static_cast<mhc_status>(s);
    }
    BlockSumArgs b = {};
    b.f = a.f;
    if (T == 0) {
        // zeros, whatever the weights and the gate hold: neither is read (a gate may be missing here)
        b.f.gate_form = MHC_GATE_NONE;
        b.f.gate = nullptr;
        b.f.w_post = nullptr;
    }
    b.sums = a.sums;
    b.scale_sums = a.scale_sums;
    b.parts = parts;
    b.d_w_post = d_w_post;
    b.d_w_pre = d_w_pre;
    b.d_gate = block->gate_form == MHC_GATE_CHANNEL ? static_cast<float *>(d_gate) : nullptr;
    b.d_res_scale = d_res_scale;
    if (!b.d_w_post && !b.d_w_pre && !b.d_gate && !b.d_res_scale) return MHC_OK;
    return static_cast<mhc_status>(note_launch(launch_block_sums(b, pdl_enabled(), st)));
}

mhc_status mhc_ckpt_pack(const void *x, int64_t stride, mhc_dtype dtype, int64_t tokens, int hidden,
                         mhc_ckpt_format format, const mhc_ckpt *out, void *stream) {
    if (tokens < 0 || stride < 0 || !dtype_ok(dtype) || !format_ok(format)) return MHC_ERR_SHAPE;
    if (hidden < 1 || hidden > kBlockMaxHidden) return MHC_ERR_UNSUPPORTED;
    if (!size_fits(tokens, hidden)) return MHC_ERR_SHAPE;
    if (tokens == 0) return MHC_OK;
    if (!x || !out || !ckpt_ok(out)) return MHC_ERR_NULL;
    if (!aligned(x, size_of(dtype))) return MHC_ERR_ALIGN;
    Span in;
    if (!rows_span(x, stride, tokens, hidden, size_of(dtype), &in)) return MHC_ERR_SHAPE;
    const Span outs[] = {codes_span(out, tokens, hidden), scales_span(out, tokens, hidden)};
    if (aliased(outs, 2, &in, 1, -1, -1)) return MHC_ERR_ALIAS;
    int sms = 0;
    if (int s = require_device(&sms, nullptr)) return static_cast<mhc_status>(s);
    const CkptArgs a = {x, nullptr, stride, tokens, hidden, ckpt_of(out)};
    return static_cast<mhc_status>(note_launch(
        launch_ckpt_pack(a, dtype, format, sms, pdl_enabled(), static_cast<cudaStream_t>(stream))));
}

mhc_status mhc_ckpt_unpack(const mhc_ckpt *ckpt, mhc_ckpt_format format, int64_t tokens, int hidden,
                           mhc_dtype dtype, void *x, void *stream) {
    if (tokens < 0 || !dtype_ok(dtype) || !format_ok(format)) return MHC_ERR_SHAPE;
    if (hidden < 1 || hidden > kBlockMaxHidden) return MHC_ERR_UNSUPPORTED;
    if (!size_fits(tokens, hidden)) return MHC_ERR_SHAPE;
    if (tokens == 0) return MHC_OK;
    if (!x || !ckpt || !ckpt_ok(ckpt)) return MHC_ERR_NULL;
    if (!aligned(x, size_of(dtype))) return MHC_ERR_ALIGN;
    const Span ins[] = {codes_span(ckpt, tokens, hidden), scales_span(ckpt, tokens, hidden)};
    const Span out = {x, static_cast<size_t>(tokens) * hidden * size_of(dtype)};
    if (aliased(&out, 1, ins, 2, -1, -1)) return MHC_ERR_ALIAS;
    int sms = 0;
    if (int s = require_device(&sms, nullptr)) return static_cast<mhc_status>(s);
    const CkptArgs a = {nullptr, x, hidden, tokens, hidden, ckpt_of(ckpt)};
    return static_cast<mhc_status>(note_launch(
        launch_ckpt_unpack(a, dtype, format, sms, pdl_enabled(), static_cast<cudaStream_t>(stream))));
}

size_t mhc_ckpt_linear_dw_workspace_bytes(int64_t tokens, int n, int k, int aligned) {
    if (tokens <= 0 || n < 1 || n > kBlockMaxHidden || k < 1 || k > kBlockMaxHidden || tokens > kDwMaxTokens)
        return 0;
    return dw_workspace(tokens, n, k, aligned != 0);
}

mhc_status mhc_ckpt_linear_dw(const void *d_out, int64_t d_out_stride, mhc_dtype dtype, const mhc_ckpt *x,
                              mhc_ckpt_format format, int64_t tokens, int n, int k, void *d_w,
                              mhc_dtype d_w_dtype, int accumulate, void *workspace, size_t workspace_bytes,
                              void *stream) {
    if (tokens < 0 || d_out_stride < 0 || !dtype_ok(d_w_dtype) || !format_ok(format)) return MHC_ERR_SHAPE;
    if (n < 1 || n > kBlockMaxHidden || k < 1 || k > kBlockMaxHidden) return MHC_ERR_UNSUPPORTED;
    if (dtype != MHC_BF16 && dtype != MHC_F16) return MHC_ERR_UNSUPPORTED;
    if (tokens > kDwMaxTokens) return MHC_ERR_UNSUPPORTED;
    if (!d_w) return MHC_ERR_NULL;
    if (tokens > 0 && (!d_out || !x || !ckpt_ok(x))) return MHC_ERR_NULL;
    if (!aligned(d_out, 2) || !aligned(d_w, size_of(d_w_dtype)) || !aligned(workspace, 16)) return MHC_ERR_ALIGN;
    const bool rows16 = dw_rows_aligned(d_out, d_out_stride, tokens, n);
    const size_t need = mhc_ckpt_linear_dw_workspace_bytes(tokens, n, k, rows16);
    if (need && !workspace) return MHC_ERR_NULL;
    if (workspace_bytes < need) return MHC_ERR_WORKSPACE;
    Span ins[3] = {};
    if (tokens > 0) {
        if (!rows_span(d_out, d_out_stride, tokens, n, 2, &ins[0])) return MHC_ERR_SHAPE;
        ins[1] = codes_span(x, tokens, k);
        ins[2] = scales_span(x, tokens, k);
    }
    const Span outs[] = {{d_w, static_cast<size_t>(n) * k * size_of(d_w_dtype)}, {workspace, need}};
    if (aliased(outs, 2, ins, 3, -1, -1)) return MHC_ERR_ALIAS;
    if (tokens == 0 && accumulate) return MHC_OK;
    int sms = 0;
    unsigned int *status = nullptr;
    if (int s = require_device(&sms, &status)) return static_cast<mhc_status>(s);
    DwArgs a = {};
    a.d_out = d_out;
    a.d_out_stride = d_out_stride;
    a.dtype = dtype;
    a.x = ckpt_of(x);
    a.format = format;
    a.T = tokens;
    a.n = n;
    a.k = k;
    a.d_w = d_w;
    a.d_w_dtype = d_w_dtype;
    a.accumulate = accumulate != 0;
    a.workspace = workspace;
    return static_cast<mhc_status>(
        launch_dw(a, rows16, sms, status, pdl_enabled(), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
