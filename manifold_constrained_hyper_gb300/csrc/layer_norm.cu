// Layer norm, out = (x - mean) * rstd * w + b, bound by memory: each row is read once, into registers,
// where the mean comes first and then the sum of the centred squares (no cancellation for rows far off zero).
#include "layer_norm.cuh"

namespace mhc {
namespace {

// A group of `warps` warps a row, R runs of 8 columns a thread.
template <class TX, class TO, int R, bool RUNS>
__global__ void __launch_bounds__(kLnThreads) ln_rows_kernel(const LayerNormArgs a, int warps) {
    __shared__ float red[16][2 * 16];
    const int lane = threadIdx.x & 31, groups = blockDim.x / (32 * warps), group = threadIdx.x / (32 * warps);
    const int mine = threadIdx.x - group * 32 * warps, warp = mine >> 5;
    int turn = 0;
    griddep_wait();
    for (long long t = static_cast<long long>(blockIdx.x) * groups + group; t < a.T; t += static_cast<long long>(gridDim.x) * groups) {
        const TX *const x = static_cast<const TX *>(a.x) + t * a.x_stride;
        TO *const out = static_cast<TO *>(a.out) + t * a.H;
        Run v[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * warps * 32 + mine) * 8;
            v[r] = run_splat(0.f);
            if (c < a.H) v[r] = ln_load<RUNS>(x, c, a.H);
        }
        float s[1] = {0.f};
#pragma unroll
        for (int r = 0; r < R; ++r) s[0] += run_sum(v[r]);
        group_sums(s, warps, warp, lane, group + 1, red[group], &turn);
        const float mean = s[0] * a.inv_h;
        s[0] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * warps * 32 + mine) * 8;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[r].p[q] = add2(v[r].p[q], splat2(-mean));
            if (c >= a.H) continue;
            const Run m = RUNS ? v[r] : ln_masked(v[r], c, a.H);
            uint64_t q2 = mul2(m.p[0], m.p[0]);
#pragma unroll
            for (int q = 1; q < 4; ++q) q2 = fma2(m.p[q], m.p[q], q2);
            s[0] += f2_lo(q2) + f2_hi(q2);
        }
        group_sums(s, warps, warp, lane, group + 1, red[group], &turn);
        const float rstd = 1.f / sqrtf(s[0] * a.inv_h + a.eps);
        if (a.stats && mine == 0) {
            a.stats[2 * t] = mean;
            a.stats[2 * t + 1] = rstd;
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * warps * 32 + mine) * 8;
            if (c >= a.H) continue;
            const Run w = ln_param<RUNS>(a.w, a.w_dtype, c, a.H, 1.f), b = ln_param<RUNS>(a.b, a.b_dtype, c, a.H, 0.f);
            Run o;
#pragma unroll
            for (int q = 0; q < 4; ++q) o.p[q] = fma2(mul2(v[r].p[q], splat2(rstd)), w.p[q], b.p[q]);
            ln_store<RUNS>(out, c, a.H, o);
        }
    }
}

// Rows too wide to be held: a CTA a row, which is read three times (twice from L2).
template <class TX, class TO>
__global__ void __launch_bounds__(kLnThreads) ln_loop_kernel(const LayerNormArgs a) {
    __shared__ float red[2 * 16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kLnThreads / 32;
    int turn = 0;
    griddep_wait();
    for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
        const TX *const x = static_cast<const TX *>(a.x) + t * a.x_stride;
        TO *const out = static_cast<TO *>(a.out) + t * a.H;
        float s[1] = {0.f};
        for (int c = threadIdx.x * 8; c < a.H; c += kLnThreads * 8) s[0] += run_sum(load8_any(x, c, a.H));
        group_sums(s, warps, warp, lane, 1, red, &turn);
        const float mean = s[0] * a.inv_h;
        s[0] = 0.f;
        for (int c = threadIdx.x * 8; c < a.H; c += kLnThreads * 8) {
            Run v = load8_any(x, c, a.H);
#pragma unroll
            for (int q = 0; q < 4; ++q) v.p[q] = add2(v.p[q], splat2(-mean));
            v = ln_masked(v, c, a.H);
#pragma unroll
            for (int q = 0; q < 4; ++q) v.p[q] = mul2(v.p[q], v.p[q]);
            s[0] += run_sum(v);
        }
        group_sums(s, warps, warp, lane, 1, red, &turn);
        const float rstd = 1.f / sqrtf(s[0] * a.inv_h + a.eps);
        if (a.stats && threadIdx.x == 0) {
            a.stats[2 * t] = mean;
            a.stats[2 * t + 1] = rstd;
        }
        for (int c = threadIdx.x * 8; c < a.H; c += kLnThreads * 8) {
            Run v = load8_any(x, c, a.H);
            const Run w = ln_param<false>(a.w, a.w_dtype, c, a.H, 1.f), b = ln_param<false>(a.b, a.b_dtype, c, a.H, 0.f);
#pragma unroll
            for (int q = 0; q < 4; ++q) v.p[q] = fma2(mul2(add2(v.p[q], splat2(-mean)), splat2(rstd)), w.p[q], b.p[q]);
            ln_store<false>(out, c, a.H, v);
        }
    }
}

bool on_runs(const void *p, int dtype) { return (reinterpret_cast<uintptr_t>(p) & (dtype == MHC_F32 ? 31u : 15u)) == 0; }

template <class TX, class TO>
cudaError_t launch_types(const LayerNormArgs &a, int sms, bool pdl, cudaStream_t s) {
    if (a.H > kLnMaxHeld)
        return launch_block_kernel(ln_loop_kernel<TX, TO>, static_cast<unsigned>(a.T < 4 * sms ? a.T : 4 * sms), kLnThreads, 0, pdl, s, a);
    const bool runs = a.H % 8 == 0 && a.x_stride % 8 == 0 && on_runs(a.x, a.x_dtype) && on_runs(a.out, a.out_dtype) &&
                      on_runs(a.w, a.w_dtype) && on_runs(a.b, a.b_dtype);
    const int need = (a.H + 255) / 256;             // warps of one run a lane
    const int R = need <= 1 ? 1 : need <= 2 ? 2 : 4, warps = (need + R - 1) / R, groups = kLnThreads / (32 * warps);
    const long long blocks = (a.T + groups - 1) / groups, cap = 4LL * sms;
    auto pick = [&](auto r) {
        constexpr int N = decltype(r)::value;
        return runs ? ln_rows_kernel<TX, TO, N, true> : ln_rows_kernel<TX, TO, N, false>;
    };
    auto *const kern = R == 1   ? pick(std::integral_constant<int, 1>())
                       : R == 2 ? pick(std::integral_constant<int, 2>())
                                : pick(std::integral_constant<int, 4>());
    return launch_block_kernel(kern, static_cast<unsigned>(blocks < cap ? blocks : cap), 32 * warps * groups, 0, pdl, s, a, warps);
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormArgs &a, int sms, bool pdl, cudaStream_t s) {
    if (a.x_dtype == MHC_BF16) return launch_types<__nv_bfloat16, __nv_bfloat16>(a, sms, pdl, s);
    if (a.x_dtype == MHC_F16) return launch_types<__half, __half>(a, sms, pdl, s);
    if (a.out_dtype == MHC_BF16) return launch_types<float, __nv_bfloat16>(a, sms, pdl, s);
    if (a.out_dtype == MHC_F16) return launch_types<float, __half>(a, sms, pdl, s);
    return launch_types<float, float>(a, sms, pdl, s);
}

}  // namespace mhc
