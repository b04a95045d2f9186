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

// The same for many rows on the boundaries of runs: rows to come staged in shared memory, where the
// parameters lie too.
constexpr int kRingThreads = 768;
template <class TX, class TO, int R>
__global__ void __launch_bounds__(kRingThreads) ln_ring_kernel(const LayerNormArgs a, const __grid_constant__ LnRing ring, int warps) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[8][2 * 16];
    __shared__ int abort_flag;
    const int lane = threadIdx.x & 31, groups = blockDim.x / (32 * warps), group = threadIdx.x / (32 * warps);
    const int mine = threadIdx.x - group * 32 * warps, warp = mine >> 5;
    const bool affine = a.w || a.b;
    float *const par = reinterpret_cast<float *>(smem + 256);
    const int par_bytes = affine ? (8 * a.H + 127) / 128 * 128 : 0, stages_at = 256 + par_bytes + group * ring.stages * ring.stage_bytes;
    const LnStages rows{ring, smem_addr(smem) + group * ring.stages * 8, smem_addr(smem) + stages_at, smem + stages_at, &abort_flag};
    int turn = 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < groups * ring.stages; ++s) mbar_init(smem_addr(smem) + 8 * s, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    griddep_wait();
    const long long first = static_cast<long long>(blockIdx.x) * groups + group, step = static_cast<long long>(gridDim.x) * groups;
    auto order = [&](int k) {
        const long long t = first + k * step;
        if (t < a.T) rows.order(k, {static_cast<const TX *>(a.x) + t * a.x_stride, nullptr, nullptr});
    };
    if (mine == 0)
        for (int k = 0; k < ring.stages; ++k) order(k);
    if (affine) {
        for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
            par[c] = a.w ? load_any(a.w, a.w_dtype, c) : 1.f;
            par[a.H + c] = a.b ? load_any(a.b, a.b_dtype, c) : 0.f;
        }
    }
    __syncthreads();
    int k = 0;
    for (long long t = first; t < a.T; t += step, ++k) {
        rows.wait(k);
        const TX *const x = reinterpret_cast<const TX *>(rows.row(k, 0));
        Run v[R];
        float s[1] = {0.f};
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * warps * 32 + mine) * 8;
            v[r] = run_splat(0.f);
            if (c < a.H) v[r] = load8_shared(x + c);
            s[0] += run_sum(v[r]);
        }
        group_sums(s, warps, warp, lane, group + 1, red[group], &turn);
        if (mine == 0) order(k + ring.stages);      // every thread of the group has the row
        const float mean = s[0] * a.inv_h;
        s[0] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * warps * 32 + mine) * 8;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[r].p[q] = add2(v[r].p[q], splat2(-mean));
            if (c >= a.H) continue;
            uint64_t q2 = mul2(v[r].p[0], v[r].p[0]);
#pragma unroll
            for (int q = 1; q < 4; ++q) q2 = fma2(v[r].p[q], v[r].p[q], q2);
            s[0] += f2_lo(q2) + f2_hi(q2);
        }
        group_sums(s, warps, warp, lane, group + 1, red[group], &turn);
        const float rstd = 1.f / sqrtf(s[0] * a.inv_h + a.eps);
        if (a.stats && mine == 0) {
            a.stats[2 * t] = mean;
            a.stats[2 * t + 1] = rstd;
        }
        TO *const out = static_cast<TO *>(a.out) + t * a.H;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * warps * 32 + mine) * 8;
            if (c >= a.H) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[r].p[q] = mul2(v[r].p[q], splat2(rstd));
            if (affine) {
                const Run w = load8_shared(par + c), b = load8_shared(par + a.H + c);
#pragma unroll
                for (int q = 0; q < 4; ++q) v[r].p[q] = fma2(v[r].p[q], w.p[q], b.p[q]);
            }
            store8(out + c, v[r]);
        }
    }
    if (abort_flag && mine == 0) {
        const long long left = first < a.T ? (a.T - first + step - 1) / step : 0;
        rows.drain(static_cast<int>(left));
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

constexpr int kRingSmem = 220 * 1024;

// Many rows on the boundaries of runs: a CTA an SM, as many groups as 768 threads give, as many stages as
// shared memory holds, at most 4 a group.
template <class TX, class TO>
cudaError_t launch_ring(const LayerNormArgs &a, int sms, unsigned int *status, bool pdl, cudaStream_t s) {
    const int need = (a.H + 255) / 256, R = need <= 6 ? 2 : 4, warps = (need + R - 1) / R;
    int groups = kRingThreads / (32 * warps);
    if (groups > 8) groups = 8;
    LnRing ring = {};
    ring.row_bytes[0] = ring.stage_bytes = a.H * static_cast<int>(sizeof(TX));
    ring.stage_bytes = (ring.stage_bytes + 127) / 128 * 128;
    const int par = a.w || a.b ? (8 * a.H + 127) / 128 * 128 : 0;
    ring.stages = (kRingSmem - 256 - par) / (groups * ring.stage_bytes);
    if (ring.stages > 4) ring.stages = 4;
    ring.status = status;
    ring.timeout_ns = wait_timeout_ns();
    const int smem = 256 + par + groups * ring.stages * ring.stage_bytes;
    auto *const kern = R == 2 ? ln_ring_kernel<TX, TO, 2> : ln_ring_kernel<TX, TO, 4>;
    static std::atomic<uint64_t> done[2];
    if (cudaError_t e = ln_allow_smem(reinterpret_cast<const void *>(kern), kRingSmem, &done[R == 2])) return e;
    const long long blocks = (a.T + groups - 1) / groups;
    return launch_block_kernel(kern, static_cast<unsigned>(blocks < sms ? blocks : sms), 32 * warps * groups, smem, pdl, s, a, ring, warps);
}

template <class TX, class TO>
cudaError_t launch_types(const LayerNormArgs &a, int sms, unsigned int *status, bool pdl, cudaStream_t s) {
    if (a.H > kLnMaxHeld)
        return launch_block_kernel(ln_loop_kernel<TX, TO>, static_cast<unsigned>(a.T < 4 * sms ? a.T : 4 * sms), kLnThreads, 0, pdl, s, a);
    const bool runs = a.H % 8 == 0 && a.x_stride % 8 == 0 && on_runs(a.x, a.x_dtype) && on_runs(a.out, a.out_dtype) &&
                      on_runs(a.w, a.w_dtype) && on_runs(a.b, a.b_dtype);
    if (runs && a.H > 512 && a.T >= 8LL * sms) return launch_ring<TX, TO>(a, sms, status, pdl, s);
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

cudaError_t launch_layer_norm(const LayerNormArgs &a, int sms, unsigned int *status, bool pdl, cudaStream_t s) {
    if (a.x_dtype == MHC_BF16) return launch_types<__nv_bfloat16, __nv_bfloat16>(a, sms, status, pdl, s);
    if (a.x_dtype == MHC_F16) return launch_types<__half, __half>(a, sms, status, pdl, s);
    if (a.out_dtype == MHC_BF16) return launch_types<float, __nv_bfloat16>(a, sms, status, pdl, s);
    if (a.out_dtype == MHC_F16) return launch_types<float, __half>(a, sms, status, pdl, s);
    return launch_types<float, float>(a, sms, status, pdl, s);
}

}  // namespace mhc
