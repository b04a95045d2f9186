// The gated residual block and its backward pass for rows too wide for
// registers (above 8192 columns; backward also the widest rows on any boundary of which
// two do not fit shared memory): one CTA per row, a warp per group
// of 32 columns, each pass over the row reading it again (from L1 or L2 after
// the first). Any stride and alignment.
#include "block_common.cuh"

namespace mhc {
namespace {

__device__ __forceinline__ float gate_at(const BlockForm &f, long long t, int i, float token) {
    if (f.gate_form == MHC_GATE_CHANNEL) return gate_value(load_any(f.gate, f.gate_dtype, i), f.gate_act);
    if (f.gate_form == MHC_GATE_FULL)
        return gate_value(load_any(f.gate, f.gate_dtype, t * f.gate_stride + i), f.gate_act);
    return token;
}
__device__ __forceinline__ float token_gate(const BlockForm &f, long long t) {
    return f.gate_form == MHC_GATE_TOKEN
               ? gate_value(load_any(f.gate, f.gate_dtype, t * f.gate_stride), f.gate_act) : 1.f;
}
__device__ __forceinline__ float scale_at(const BlockForm &f, int i) {
    if (f.scale_form == MHC_SCALE_NONE) return 1.f;
    return f.res_scale[f.scale_form == MHC_SCALE_ONE ? 0 : i];
}

template <class TY, class TR>
__global__ void block_fwd_loop_kernel(const BlockFwdArgs a) {
    __shared__ float red[2][32];
    griddep_wait();
    const BlockForm &f = a.f;
    const int H = f.H, groups = (H + 31) / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int which = 0;      // the area of the next block_sum
    for (long long t = blockIdx.x; t < f.T; t += gridDim.x) {
        const TY *y = static_cast<const TY *>(a.y) + t * a.y_stride;
        const TR *r = static_cast<const TR *>(a.residual) + t * a.r_stride;
        float s[1] = {0.f};
        float rstd1 = 1.f;
        if (f.post_norm) {
            for (int i = threadIdx.x; i < H; i += blockDim.x) {
                const float v = to_f32(y[i]);
                s[0] = fmaf(v, v, s[0]);
            }
            block_sum(s, red[which]);
            which ^= 1;
            rstd1 = __frsqrt_rn(fmaf(s[0], f.inv_h, f.eps_post));
        }
        const float token = token_gate(f, t);
        auto out_at = [&](int i) {
            const float n = to_f32(y[i]) * rstd1 * weight_at(f.w_post, f.w_post_dtype, f.weight_offset, i);
            return fmaf(scale_at(f, i), to_f32(r[i]), gate_at(f, t, i, token) * n);
        };
        s[0] = 0.f;
        for (int i = threadIdx.x; i < H; i += blockDim.x) {
            const float v = out_at(i);
            s[0] = fmaf(v, v, s[0]);
        }
        block_sum(s, red[which]);
        which ^= 1;
        const float rstd2 = __frsqrt_rn(fmaf(s[0], f.inv_h, f.eps_pre));
        for (int g = warp; g < groups; g += warps) {
            const int i = g * 32 + lane;
            const bool in = i < H;
            float ro = 0.f, h = 0.f, yv = 0.f, rv = 0.f;
            if (in) {
                yv = to_f32(y[i]);
                rv = to_f32(r[i]);
                ro = out_at(i);
                const TY hv = from_f32<TY>(ro * rstd2 * weight_at(f.w_pre, f.w_pre_dtype, f.weight_offset, i));
                h = to_f32(hv);
                static_cast<TR *>(a.residual_out)[t * H + i] = from_f32<TR>(ro);
                static_cast<TY *>(a.h)[t * H + i] = hv;
            }
            if (a.ck_y.codes) ckpt_store_lane(a.ck_y, a.format, t, H, groups, g, lane, yv);
            if (a.ck_r.codes) ckpt_store_lane(a.ck_r, a.format, t, H, groups, g, lane, rv);
            if (a.ck_h.codes) ckpt_store_lane(a.ck_h, a.format, t, H, groups, g, lane, h);
        }
        if (a.rstd && threadIdx.x == 0) {
            a.rstd[2 * t] = rstd1;
            a.rstd[2 * t + 1] = rstd2;
        }
    }
}

template <class TY, class TR>
__global__ void block_bwd_loop_kernel(const BlockBwdArgs a) {
    __shared__ float red[2][3 * 32];
    griddep_wait();
    const BlockForm &f = a.f;
    const int H = f.H, groups = (H + 31) / 32;
    float *sums = a.sums + static_cast<long long>(blockIdx.x) * kBackSums * H;
    float scale_sum = 0.f;
    bool first = true;
    int which = 0;
    for (long long t = blockIdx.x; t < f.T; t += gridDim.x, first = false, which ^= 1) {
        const float rstd1 = f.post_norm ? a.rstd[2 * t] : 1.f, rstd2 = a.rstd[2 * t + 1];
        const float token = token_gate(f, t);
        const float gate_all = f.gate_form == MHC_GATE_TOKEN ? token : 1.f;
        auto slope_at = [&](float z) {
            float g, slope;
            gate_both(z, f.gate_act, &g, &slope);
            return slope;
        };
        struct Elem { float y, r, df, dh, w1, w2, a, g, z, u, n, ro; };
        auto load = [&](int i) {
            Elem e;
            e.y = a.y ? to_f32(static_cast<const TY *>(a.y)[t * a.y_stride + i])
                      : ckpt_load(a.ck_y, a.format, t, H, groups, i);
            e.r = a.residual ? to_f32(static_cast<const TR *>(a.residual)[t * a.r_stride + i])
                             : ckpt_load(a.ck_r, a.format, t, H, groups, i);
            e.df = a.d_ro ? to_f32(static_cast<const TR *>(a.d_ro)[t * a.d_ro_stride + i]) : 0.f;
            e.dh = to_f32(static_cast<const TY *>(a.d_h)[t * a.d_h_stride + i]);
            e.w1 = weight_at(f.w_post, f.w_post_dtype, f.weight_offset, i);
            e.w2 = weight_at(f.w_pre, f.w_pre_dtype, f.weight_offset, i);
            e.a = scale_at(f, i);
            e.z = f.gate_form == MHC_GATE_FULL ? load_any(f.gate, f.gate_dtype, t * f.gate_stride + i) : 0.f;
            e.g = gate_at(f, t, i, token);
            e.u = e.y * rstd1;
            e.n = e.u * e.w1;
            e.ro = fmaf(e.a, e.r, e.g * e.n);
            return e;
        };
        // c2 = sum d_h w2 ro; with D = (d_ro + rstd2 d_h w2) - q ro, the sum of
        // w1 g D y splits into two that need no q. A token's gate is taken out
        // of them: its own gradient wants the sum without it.
        float s[3] = {0.f, 0.f, 0.f};
        for (int i = threadIdx.x; i < H; i += blockDim.x) {
            const Elem e = load(i);
            const float dv = e.dh * e.w2;
            const float gy = (f.gate_form == MHC_GATE_TOKEN ? 1.f : e.g) * e.w1 * e.y;
            s[0] = fmaf(dv, e.ro, s[0]);
            s[1] = fmaf(gy, fmaf(rstd2, dv, e.df), s[1]);
            s[2] = fmaf(gy, e.ro, s[2]);
        }
        block_sum(s, red[which]);
        const float q = rstd2 * (rstd2 * (rstd2 * (s[0] * f.inv_h)));
        const float c1 = fmaf(-q, s[2], s[1]);
        const float p = f.post_norm ? rstd1 * (rstd1 * (rstd1 * (gate_all * c1 * f.inv_h))) : 0.f;
        for (int i = threadIdx.x; i < H; i += blockDim.x) {
            const Elem e = load(i);
            const float D = fmaf(-q, e.ro, fmaf(rstd2, e.dh * e.w2, e.df));
            static_cast<TR *>(a.d_r)[t * H + i] = from_f32<TR>(e.a * D);
            static_cast<TY *>(a.d_y)[t * H + i] =
                from_f32<TY>(fmaf(-p, e.y, rstd1 * (e.g * D * e.w1)));
            const float s0 = (f.gate_form == MHC_GATE_CHANNEL ? 1.f : e.g) * D * e.u;
            const float s1 = e.dh * e.ro * rstd2, s2 = e.r * D;
            sums[i] = first ? s0 : sums[i] + s0;
            sums[H + i] = first ? s1 : sums[H + i] + s1;
            if (f.scale_form == MHC_SCALE_CHANNEL) sums[2 * H + i] = first ? s2 : sums[2 * H + i] + s2;
            else scale_sum += s2;
            if (f.gate_form == MHC_GATE_FULL && a.d_gate)
                store_any(a.d_gate, f.gate_dtype, t * H + i, slope_at(e.z) * e.n * D);
        }
        if (f.gate_form == MHC_GATE_TOKEN && a.d_gate && threadIdx.x == 0) {
            const float z = load_any(f.gate, f.gate_dtype, t * f.gate_stride);
            static_cast<float *>(a.d_gate)[t] = slope_at(z) * rstd1 * c1;
        }
    }
    float s[1] = {scale_sum};
    __syncthreads();
    block_sum(s, red[0]);
    if (threadIdx.x == 0) a.scale_sums[blockIdx.x] = s[0];
}

unsigned loop_threads(int H) { return H <= 256 ? 64 : H <= 2048 ? 256 : 512; }

template <class TY, class TR>
cudaError_t fwd_loop(const BlockFwdArgs &a, int sms, bool pdl, cudaStream_t s) {
    const long long cap = static_cast<long long>(sms) * 8;
    return launch_block_kernel(block_fwd_loop_kernel<TY, TR>, static_cast<unsigned>(a.f.T < cap ? a.f.T : cap),
                               loop_threads(a.f.H), 0, pdl, s, a);
}
template <class TY, class TR>
cudaError_t bwd_loop(const BlockBwdArgs &a, bool pdl, int *parts, cudaStream_t s) {
    *parts = static_cast<int>(a.f.T < kBackMaxParts ? a.f.T : kBackMaxParts);
    return launch_block_kernel(block_bwd_loop_kernel<TY, TR>, *parts, loop_threads(a.f.H), 0, pdl, s, a);
}

}  // namespace

cudaError_t launch_block_fwd_loop(const BlockFwdArgs &a, int dtype, int r_dtype, int sms, bool pdl,
                                  cudaStream_t s) {
    if (dtype == MHC_F32) return fwd_loop<float, float>(a, sms, pdl, s);
    if (dtype == MHC_BF16)
        return r_dtype == MHC_F32 ? fwd_loop<__nv_bfloat16, float>(a, sms, pdl, s)
                                  : fwd_loop<__nv_bfloat16, __nv_bfloat16>(a, sms, pdl, s);
    return r_dtype == MHC_F32 ? fwd_loop<__half, float>(a, sms, pdl, s)
                              : fwd_loop<__half, __half>(a, sms, pdl, s);
}

cudaError_t launch_block_bwd_loop(const BlockBwdArgs &a, int dtype, int r_dtype, bool pdl,
                                  int *parts, cudaStream_t s) {
    if (dtype == MHC_F32) return bwd_loop<float, float>(a, pdl, parts, s);
    if (dtype == MHC_BF16)
        return r_dtype == MHC_F32 ? bwd_loop<__nv_bfloat16, float>(a, pdl, parts, s)
                                  : bwd_loop<__nv_bfloat16, __nv_bfloat16>(a, pdl, parts, s);
    return r_dtype == MHC_F32 ? bwd_loop<__half, float>(a, pdl, parts, s)
                              : bwd_loop<__half, __half>(a, pdl, parts, s);
}

}  // namespace mhc
