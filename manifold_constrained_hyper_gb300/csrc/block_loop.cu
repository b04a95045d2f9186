// The gated residual block and its backward pass for rows too wide for
// registers (above 8192 columns; backward also the widest rows on any boundary of which
// two do not fit shared memory): one CTA per row, N columns a thread at a time,
// each pass over the row reading it again (from L1 or L2 after the first). N is 8 for
// rows on boundaries of 8 elements, else 1. Bound by L2: every row reads the parameters
// again in each pass (fp32 ones are four to eight times a 16-bit row's own bytes). Measured,
// bf16, channel gate and scale: 2048 x 8200 111 us forward and 202 backward, 8201 wide 133 and
// 437 (2048 x 8192 by the row kernels: 28 and 48).
#include "block_rows.cuh"

namespace mhc {
namespace {

// N columns from i on: of a row of a known type, of one known at run time.
template <int N, class T>
__device__ __forceinline__ void get(const T *row, int i, float (&v)[N]) {
    if constexpr (N == 8) {
        const Run r = load8(row + i);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = run_at(r, e);
    } else {
        v[0] = to_f32(row[i]);
    }
}
template <int N>
__device__ __forceinline__ void get_any(const void *row, int dtype, long long i, float (&v)[N]) {
    if (dtype == MHC_F32) get<N>(static_cast<const float *>(row) + i, 0, v);
    else if (dtype == MHC_BF16) get<N>(static_cast<const __nv_bfloat16 *>(row) + i, 0, v);
    else get<N>(static_cast<const __half *>(row) + i, 0, v);
}
template <int N, class T>
__device__ __forceinline__ void put(T *row, int i, const float (&v)[N]) {
    if constexpr (N == 8) store8(row + i, run_of(v));
    else row[i] = from_f32<T>(v[0]);
}
template <int N>
__device__ __forceinline__ void fill(float x, float (&v)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = x;
}
template <int N>
__device__ __forceinline__ void get_weight(const void *w, int dtype, float offset, int i, float (&v)[N]) {
    fill(1.f, v);
    if (!w) return;
    get_any(w, dtype, i, v);
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] += offset;
}
template <int N>
__device__ __forceinline__ void get_scale(const BlockForm &f, int i, float (&v)[N]) {
    if (f.scale_form == MHC_SCALE_CHANNEL) get<N>(f.res_scale, i, v);
    else fill(f.scale_form == MHC_SCALE_ONE ? *f.res_scale : 1.f, v);
}
// The gate before its function (a token's is one value: not here).
template <int N>
__device__ __forceinline__ void get_gate(const BlockForm &f, long long t, int i, float (&v)[N]) {
    if (f.gate_form == MHC_GATE_CHANNEL) get_any(f.gate, f.gate_dtype, i, v);
    else if (f.gate_form == MHC_GATE_FULL) get_any(f.gate, f.gate_dtype, t * f.gate_stride + i, v);
}
template <int N>
__device__ __forceinline__ void get_held(const Ckpt &c, int format, long long t, int H, int groups, int i, float (&v)[N]) {
    if constexpr (N == 8) {
        const Run r = ckpt_values8(*reinterpret_cast<const uint2 *>(c.codes + t * H + i), c.scales[t * groups + i / 32], format);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = run_at(r, e);
    } else {
        v[0] = ckpt_load(c, format, t, H, groups, i);
    }
}
// Whole warps, of neighbouring columns; past the row's end zeros.
template <int N>
__device__ __forceinline__ void put_held(const Ckpt &c, int format, long long t, int H, int groups, int i, const float (&v)[N]) {
    if constexpr (N == 8) {
        const Run r = run_of(v);
        const uint32_t byte = format == MHC_CKPT_E4M3 ? ckpt_byte_quad<MHC_CKPT_E4M3>(r) : ckpt_byte_quad<MHC_CKPT_INT8>(r);
        if (i >= H) return;
        *reinterpret_cast<uint2 *>(c.codes + t * H + i) =
            format == MHC_CKPT_E4M3 ? ckpt_codes8<MHC_CKPT_E4M3>(r, byte) : ckpt_codes8<MHC_CKPT_INT8>(r, byte);
        if ((threadIdx.x & 3) == 0) c.scales[t * groups + i / 32] = static_cast<uint8_t>(byte);
    } else if (i / 32 < groups) {
        ckpt_store_lane(c, format, t, H, groups, i / 32, threadIdx.x & 31, v[0]);
    }
}
__device__ __forceinline__ float token_gate(const BlockForm &f, long long t) {
    return f.gate_form == MHC_GATE_TOKEN
               ? gate_value(load_any(f.gate, f.gate_dtype, t * f.gate_stride), f.gate_act) : 1.f;
}

template <class TY, class TR, int N>
__global__ void __launch_bounds__(512) block_fwd_loop_kernel(const BlockFwdArgs a) {
    __shared__ float red[2][32];
    griddep_wait();
    const BlockForm &f = a.f;
    const int H = f.H, groups = (H + 31) / 32, step = blockDim.x * N;
    const bool gated = f.gate_form == MHC_GATE_CHANNEL || f.gate_form == MHC_GATE_FULL;
    int which = 0;      // the area of the next block_sum
    for (long long t = blockIdx.x; t < f.T; t += gridDim.x) {
        const TY *const y_row = static_cast<const TY *>(a.y) + t * a.y_stride;
        const TR *const r_row = static_cast<const TR *>(a.residual) + t * a.r_stride;
        float s[1] = {0.f};
        float rstd1 = 1.f;
        if (f.post_norm) {
            for (int i = threadIdx.x * N; i < H; i += step) {
                float y[N];
                get<N>(y_row, i, y);
#pragma unroll
                for (int e = 0; e < N; ++e) s[0] = fmaf(y[e], y[e], s[0]);
            }
            block_sum(s, red[which]);
            which ^= 1;
            rstd1 = __frsqrt_rn(fmaf(s[0], f.inv_h, f.eps_post));
        }
        const float token = token_gate(f, t);
        auto load = [&](int i, float (&y)[N], float (&r)[N], float (&ro)[N]) {
            float w[N], g[N], sc[N];
            get<N>(y_row, i, y);
            get<N>(r_row, i, r);
            get_weight(f.w_post, f.w_post_dtype, f.weight_offset, i, w);
            get_scale(f, i, sc);
            if (gated) get_gate(f, t, i, g);
#pragma unroll
            for (int e = 0; e < N; ++e)
                ro[e] = fmaf(sc[e], r[e], (gated ? gate_value(g[e], f.gate_act) : token) * (y[e] * rstd1 * w[e]));
        };
        s[0] = 0.f;
        for (int i = threadIdx.x * N; i < H; i += step) {
            float y[N], r[N], ro[N];
            load(i, y, r, ro);
#pragma unroll
            for (int e = 0; e < N; ++e) s[0] = fmaf(ro[e], ro[e], s[0]);
        }
        block_sum(s, red[which]);
        which ^= 1;
        const float rstd2 = __frsqrt_rn(fmaf(s[0], f.inv_h, f.eps_pre));
        for (int i0 = 0; i0 < H; i0 += step) {          // whole warps: checkpoints are written by groups of lanes
            const int i = i0 + threadIdx.x * N;
            float y[N], r[N], ro[N], h[N];
            fill(0.f, y);
            fill(0.f, r);
            fill(0.f, h);
            if (i < H) {
                load(i, y, r, ro);
                get_weight(f.w_pre, f.w_pre_dtype, f.weight_offset, i, h);
#pragma unroll
                for (int e = 0; e < N; ++e) h[e] = to_f32(from_f32<TY>(ro[e] * rstd2 * h[e]));     // as it is stored
                put(static_cast<TR *>(a.residual_out) + t * H, i, ro);
                put(static_cast<TY *>(a.h) + t * H, i, h);
            }
            if (a.ck_y.codes) put_held(a.ck_y, a.format, t, H, groups, i, y);
            if (a.ck_r.codes) put_held(a.ck_r, a.format, t, H, groups, i, r);
            if (a.ck_h.codes) put_held(a.ck_h, a.format, t, H, groups, i, h);
        }
        if (a.rstd && threadIdx.x == 0) {
            a.rstd[2 * t] = rstd1;
            a.rstd[2 * t + 1] = rstd2;
        }
    }
}

template <class TY, class TR, int N>
__global__ void __launch_bounds__(512) block_bwd_loop_kernel(const BlockBwdArgs a) {
    __shared__ float red[2][3 * 32];
    griddep_wait();
    const BlockForm &f = a.f;
    const int H = f.H, groups = (H + 31) / 32, step = blockDim.x * N;
    const bool gated = f.gate_form == MHC_GATE_CHANNEL || f.gate_form == MHC_GATE_FULL;
    float *const sums = a.sums + static_cast<long long>(blockIdx.x) * kBackSums * H;
    LongSum scale_sum;
    bool first = true;
    int which = 0;
    for (long long t = blockIdx.x; t < f.T; t += gridDim.x, first = false, which ^= 1) {
        const float rstd1 = f.post_norm ? a.rstd[2 * t] : 1.f, rstd2 = a.rstd[2 * t + 1];
        const float token = token_gate(f, t);
        struct Cols { float y[N], r[N], df[N], dh[N], w1[N], w2[N], sc[N], z[N]; };
        auto load = [&](int i, Cols &c) {
            if (a.y) get<N>(static_cast<const TY *>(a.y) + t * a.y_stride, i, c.y);
            else get_held(a.ck_y, a.format, t, H, groups, i, c.y);
            if (a.residual) get<N>(static_cast<const TR *>(a.residual) + t * a.r_stride, i, c.r);
            else get_held(a.ck_r, a.format, t, H, groups, i, c.r);
            fill(0.f, c.df);
            if (a.d_ro) get<N>(static_cast<const TR *>(a.d_ro) + t * a.d_ro_stride, i, c.df);
            get<N>(static_cast<const TY *>(a.d_h) + t * a.d_h_stride, i, c.dh);
            get_weight(f.w_post, f.w_post_dtype, f.weight_offset, i, c.w1);
            get_weight(f.w_pre, f.w_pre_dtype, f.weight_offset, i, c.w2);
            get_scale(f, i, c.sc);
            if (gated) get_gate(f, t, i, c.z);
        };
        // c2 = sum d_h w2 ro; with D = (d_ro + rstd2 d_h w2) - q ro, the sum of
        // w1 g D y splits into two that need no q. A token's gate is taken out
        // of them: its own gradient wants the sum without it.
        float s[3] = {0.f, 0.f, 0.f};
        for (int i = threadIdx.x * N; i < H; i += step) {
            Cols c;
            load(i, c);
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const float gy = (gated ? gate_value(c.z[e], f.gate_act) : 1.f) * c.w1[e] * c.y[e];
                const float ro = fmaf(c.sc[e], c.r[e], token * rstd1 * gy), dv = c.dh[e] * c.w2[e];
                s[0] = fmaf(dv, ro, s[0]);
                s[1] = fmaf(gy, fmaf(rstd2, dv, c.df[e]), s[1]);
                s[2] = fmaf(gy, ro, s[2]);
            }
        }
        block_sum(s, red[which]);
        float row_scale = 0.f;
        const float q = rstd2 * (rstd2 * (rstd2 * (s[0] * f.inv_h)));
        const float c1 = fmaf(-q, s[2], s[1]);
        const float p = f.post_norm ? rstd1 * (rstd1 * (rstd1 * (token * c1 * f.inv_h))) : 0.f;
        for (int i = threadIdx.x * N; i < H; i += step) {
            Cols c;
            load(i, c);
            float dr[N], dy[N], s0[N], s1[N], s2[N], dz[N];
#pragma unroll
            for (int e = 0; e < N; ++e) {
                float g = token, slope = 0.f;
                if (gated) gate_both(c.z[e], f.gate_act, &g, &slope);
                const float u = c.y[e] * rstd1, n = u * c.w1[e], ro = fmaf(c.sc[e], c.r[e], g * n);
                const float D = fmaf(-q, ro, fmaf(rstd2, c.dh[e] * c.w2[e], c.df[e]));
                dr[e] = c.sc[e] * D;
                dy[e] = fmaf(-p, c.y[e], rstd1 * (g * D * c.w1[e]));
                s0[e] = (f.gate_form == MHC_GATE_CHANNEL ? 1.f : g) * D * u;
                s1[e] = c.dh[e] * ro * rstd2;
                s2[e] = c.r[e] * D;
                dz[e] = slope * n * D;
            }
            put(static_cast<TR *>(a.d_r) + t * H, i, dr);
            put(static_cast<TY *>(a.d_y) + t * H, i, dy);
            if (f.gate_form == MHC_GATE_FULL && a.d_gate) {
                if (f.gate_dtype == MHC_F32) put(static_cast<float *>(a.d_gate) + t * H, i, dz);
                else put(static_cast<TY *>(a.d_gate) + t * H, i, dz);
            }
            auto add = [&](float *to, const float (&v)[N]) {
                float w[N];
                fill(0.f, w);
                if (!first) get<N>(to, i, w);
#pragma unroll
                for (int e = 0; e < N; ++e) w[e] += v[e];
                put(to, i, w);
            };
            add(sums, s0);
            add(sums + H, s1);
            if (f.scale_form == MHC_SCALE_CHANNEL) {
                add(sums + 2 * static_cast<long long>(H), s2);
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) row_scale += s2[e];
            }
        }
        if (f.gate_form == MHC_GATE_TOKEN && a.d_gate && threadIdx.x == 0) {
            float g, slope;
            gate_both(load_any(f.gate, f.gate_dtype, t * f.gate_stride), f.gate_act, &g, &slope);
            static_cast<float *>(a.d_gate)[t] = slope * rstd1 * c1;
        }
        scale_sum.add(row_scale);
    }
    __syncthreads();
    block_long_sum(scale_sum, red[0]);
    if (threadIdx.x == 0) {
        a.scale_sums[2 * blockIdx.x] = scale_sum.hi;
        a.scale_sums[2 * blockIdx.x + 1] = scale_sum.lo;
    }
}

bool codes_fit(const Ckpt &c) { return (reinterpret_cast<uintptr_t>(c.codes) & 7u) == 0; }
template <class TY, class TR>
cudaError_t fwd_loop(const BlockFwdArgs &a, int sms, bool pdl, cudaStream_t s) {
    const BlockForm &f = a.f;
    const bool vec = f.H % 8 == 0 && rows_of_runs(a.residual_out, f.H, sizeof(TR), f.T) && rows_of_runs(a.h, f.H, sizeof(TY), f.T) &&
                     params_of_runs(f) && rows_of_runs(a.y, a.y_stride, sizeof(TY), f.T) &&
                     rows_of_runs(a.residual, a.r_stride, sizeof(TR), f.T) &&
                     (f.gate_form != MHC_GATE_FULL || rows_of_runs(f.gate, f.gate_stride, elem_bytes(f.gate_dtype), f.T)) &&
                     codes_fit(a.ck_y) && codes_fit(a.ck_r) && codes_fit(a.ck_h);
    const long long cap = static_cast<long long>(sms) * 8;
    return launch_block_kernel(vec ? block_fwd_loop_kernel<TY, TR, 8> : block_fwd_loop_kernel<TY, TR, 1>,
                               static_cast<unsigned>(f.T < cap ? f.T : cap), 512, 0, pdl, s, a);
}
template <class TY, class TR>
cudaError_t bwd_loop(const BlockBwdArgs &a, bool pdl, int *parts, cudaStream_t s) {
    const BlockForm &f = a.f;
    const bool full = f.gate_form == MHC_GATE_FULL;
    const bool vec = f.H % 8 == 0 && codes_fit(a.ck_y) && codes_fit(a.ck_r) && rows_of_runs(a.d_y, f.H, sizeof(TY), f.T) &&
                     rows_of_runs(a.d_r, f.H, sizeof(TR), f.T) && rows_of_runs(a.sums, f.H, 4, f.T) && params_of_runs(f) &&
                     (!full || !a.d_gate || rows_of_runs(a.d_gate, f.H, elem_bytes(f.gate_dtype), f.T)) &&
                     (!a.y || rows_of_runs(a.y, a.y_stride, sizeof(TY), f.T)) &&
                     (!a.residual || rows_of_runs(a.residual, a.r_stride, sizeof(TR), f.T)) &&
                     (!a.d_ro || rows_of_runs(a.d_ro, a.d_ro_stride, sizeof(TR), f.T)) &&
                     rows_of_runs(a.d_h, a.d_h_stride, sizeof(TY), f.T) &&
                     (!full || rows_of_runs(f.gate, f.gate_stride, elem_bytes(f.gate_dtype), f.T));
    *parts = static_cast<int>(f.T < kBackMaxParts ? f.T : kBackMaxParts);
    return launch_block_kernel(vec ? block_bwd_loop_kernel<TY, TR, 8> : block_bwd_loop_kernel<TY, TR, 1>, *parts, 512, 0, pdl,
                               s, a);
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
