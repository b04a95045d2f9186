// Layer norm, out = (x - mean) * rstd * w + b, bound by memory: each row is read once, into registers,
// where the mean comes first and then the sum of the centred squares (no cancellation for rows far off zero).
// 8192 x 7168 fp32 to bf16: 58.4 us, 0.89 of the copy rate (without rows to come 81); bf16 51.7, where the two sums of
// a row, one after the other, bound it; 1 x 7168 3.4. Rows above 8192 columns: 8192 x 8200 bf16 179, 0.22.
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
            ln_store<RUNS>(out, c, a.H, o, a.out_runs);
        }
    }
}

// The same for many rows: rows to come staged in shared memory, where the parameters lie too.
template <class TX, class TO, int R, bool RUNS>
__global__ void __launch_bounds__(kLnRingThreads) ln_ring_kernel(const LayerNormArgs a, const __grid_constant__ LnRing ring, int warps) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[kLnRingGroups][2 * 16];
    __shared__ int abort_flag;
    const int lane = threadIdx.x & 31, groups = (blockDim.x - 32) / (32 * warps), group = threadIdx.x / (32 * warps);
    const int mine = threadIdx.x - group * 32 * warps, warp = mine >> 5;
    const bool affine = a.w || a.b, filler = threadIdx.x >= blockDim.x - 32;
    float *const par = reinterpret_cast<float *>(smem + kLnRingBars);
    const int Hp = (a.H + 7) / 8 * 8, par_bytes = affine ? (8 * Hp + 127) / 128 * 128 : 0;
    const int which = filler ? lane : group, places_at = kLnRingBars + par_bytes + which * ring.stages * ring.place[kLnArrays];
    LnPlace place = {smem_addr(smem) + which * ring.stages * 16, smem_addr(smem) + places_at, 0, 0};
    if (threadIdx.x == 0) {
        ln_bars_init(smem_addr(smem), groups * ring.stages, warps);
        abort_flag = 0;
    }
    __syncthreads();
    griddep_wait();
    const long long first = static_cast<long long>(blockIdx.x) * groups + which, step = static_cast<long long>(gridDim.x) * groups;
    if (filler) {
        ln_fill(ring, place, lane < groups, first < a.T ? static_cast<int>((a.T - first + step - 1) / step) : 0, &abort_flag,
                [&](int k, const void *(&src)[kLnArrays]) {
                    src[0] = static_cast<const TX *>(a.x) + (first + k * step) * a.x_stride;
                    src[1] = src[2] = nullptr;
                });
        return;
    }
    if (affine) {
        ln_stage_param(par, a.w, a.w_dtype, a.H, Hp, 1.f, 32 * warps * groups);
        ln_stage_param(par + Hp, a.b, a.b_dtype, a.H, Hp, 0.f, 32 * warps * groups);
        named_barrier_sync(kLnAllBarrier, 32 * warps * groups);
    }
    int turn = 0;
    for (long long t = first; t < a.T; t += step, place.next(ring)) {
        mbar_wait(place.full(), place.turn, &abort_flag, ring.timeout_ns, ring.status, SITE_LN_ROW);
        const uint8_t *const x = smem + places_at + place.at * ring.place[kLnArrays];
        const TX *const from = static_cast<const TX *>(a.x) + t * a.x_stride;
        Run v[R];
        float s[1] = {0.f};
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * warps * 32 + mine) * 8;
            v[r] = run_splat(0.f);
            if (c < a.H) v[r] = ln_staged<RUNS>(x, ln_skew(from), c, a.H, from);
            s[0] += run_sum(v[r]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(place.empty());      // the row is in registers
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
        TO *const out = static_cast<TO *>(a.out) + t * a.H;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * warps * 32 + mine) * 8;
            if (c >= a.H) continue;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[r].p[q] = mul2(v[r].p[q], splat2(rstd));
            if (affine) {
                const Run w = load8_shared(par + c), b = load8_shared(par + Hp + c);
#pragma unroll
                for (int q = 0; q < 4; ++q) v[r].p[q] = fma2(v[r].p[q], w.p[q], b.p[q]);
            }
            ln_store<RUNS>(out, c, a.H, v[r], a.out_runs);
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
            ln_store<false>(out, c, a.H, v, a.out_runs);
        }
    }
}

bool on_runs(const void *p, int dtype) { return (reinterpret_cast<uintptr_t>(p) & (dtype == MHC_F32 ? 31u : 15u)) == 0; }

template <class TX, class TO>
cudaError_t launch_ring(const LayerNormArgs &a, bool runs, int sms, unsigned int *status, bool pdl, cudaStream_t s) {
    LnRing ring = {};
    ring.row_bytes[0] = a.H * static_cast<int>(sizeof(TX));
    ln_places(ring.row_bytes, ring.place);
    const LnRingShape p = ln_ring_shape(a.H, ring.place[kLnArrays], runs, a.w || a.b);
    ring.stages = p.stages;
    ring.status = status;
    ring.timeout_ns = wait_timeout_ns();
    auto *const kern = p.R == 2 ? (runs ? ln_ring_kernel<TX, TO, 2, true> : ln_ring_kernel<TX, TO, 2, false>)
                              : ln_ring_kernel<TX, TO, 4, true>;
    static std::atomic<uint64_t> done[4];
    if (cudaError_t e = ln_allow_smem(reinterpret_cast<const void *>(kern), kLnRingSmem, &done[2 * (p.R == 2) + runs])) return e;
    const long long blocks = (a.T + p.groups - 1) / p.groups;
    return launch_block_kernel(kern, static_cast<unsigned>(blocks < sms ? blocks : sms), 32 * (p.warps * p.groups + 1), p.smem, pdl, s, a, ring, p.warps);
}

template <class TX, class TO>
cudaError_t launch_types(const LayerNormArgs &a, int sms, unsigned int *status, bool pdl, cudaStream_t s) {
    if (a.H > kLnMaxHeld)
        return launch_block_kernel(ln_loop_kernel<TX, TO>, static_cast<unsigned>(a.T < 4 * sms ? a.T : 4 * sms), kLnThreads, 0, pdl, s, a);
    const bool runs = a.H % 8 == 0 && a.x_stride % 8 == 0 && on_runs(a.x, a.x_dtype) && on_runs(a.out, a.out_dtype) &&
                      on_runs(a.w, a.w_dtype) && on_runs(a.b, a.b_dtype);
    // Staged where a row takes several warps and there are several rows a group. Measured among rows that L2 does not hold, staged against
    // from memory: 8192 x 7168 fp32 58 us against 83 (bf16 53 against 52), 8192 x 4096 bf16 32 against 43, 8192 x 1024 11.5 against 12.4; with
    // 2432 rows 22 against 30 (7168 fp32), 21 against 18 (7168 bf16), 13.4 against 14.7 (4096 bf16), 5.7 against 4.3 (1024 bf16); with 608 rows
    // always slower (4096 bf16 5.9 against 5.0). Up to 512 columns a row is one warp's work: 8192 x 512 7.9 against 5.4.
    if (a.H > 512 && a.T >= 8LL * sms) return launch_ring<TX, TO>(a, runs, sms, status, pdl, s);
    const LnRows p = ln_rows(a.H);
    const long long blocks = (a.T + p.groups - 1) / p.groups, cap = 4LL * sms;
    auto pick = [&](auto r) {
        constexpr int N = decltype(r)::value;
        return runs ? ln_rows_kernel<TX, TO, N, true> : ln_rows_kernel<TX, TO, N, false>;
    };
    auto *const kern = p.R == 1   ? pick(std::integral_constant<int, 1>())
                       : p.R == 2 ? pick(std::integral_constant<int, 2>())
                                  : pick(std::integral_constant<int, 4>());
    return launch_block_kernel(kern, static_cast<unsigned>(blocks < cap ? blocks : cap), 32 * p.warps * p.groups, 0, pdl, s, a, p.warps);
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
