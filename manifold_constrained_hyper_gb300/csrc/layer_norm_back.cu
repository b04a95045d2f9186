// Layer norm's backward pass. With h = (x - mean) * rstd and e = d_out * w:
//   d_x = rstd * (e - mean(e) - h * mean(e * h)) + d_residual,   d_w = sum_t d_out * h,   d_b = sum_t d_out.
// One pass over the rows: the two row sums in one reduction, the sums over tokens in registers, a set for
// each group of warps; a CTA's groups meet in shared memory, and the CTAs' sets are added by a second
// kernel in their order. 4096 x 4096 bf16 with d_residual: 30.7 us, 0.65 of the copy rate, bound by a row's chain with two
// groups an SM; 8192 x 7168 fp32 with a bf16 d_out 97, 0.90, and with
// d_residual, whose bytes are a third of all, 129, 0.94; 2047 x 1102 fp32 13.0. Rows above 8192 columns are far from it: 8192 x 8200 bf16 824.
#include "layer_norm.cuh"
#include "mhc_internal.h"

namespace mhc {
namespace {

constexpr int kR = kLnBackRuns;

// The groups' sums over tokens to the CTA's set, or, where it is the only CTA, to the outputs, in the groups' order, through
// meet [groups][2][Hp].
template <int R>
__device__ __forceinline__ void meet_sums(float *meet, const LayerNormBackArgs &a, const Run (&dw)[R], const Run (&db)[R], int groups, int group,
                                          int warps, int mine) {
    const int H = a.H, Hp = (H + 7) / 8 * 8;
    float *const set = a.sums + static_cast<long long>(blockIdx.x) * 2 * H;
    float *const to_w = gridDim.x == 1 ? a.d_w : set, *const to_b = gridDim.x == 1 ? a.d_b : set + H;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int c = (r * warps * 32 + mine) * 8;
        if (c >= H) continue;
        float *const to = meet + static_cast<long long>(group) * 2 * Hp + c;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            *reinterpret_cast<uint64_t *>(to + 2 * q) = dw[r].p[q];
            *reinterpret_cast<uint64_t *>(to + Hp + 2 * q) = db[r].p[q];
        }
    }
    const int threads = 32 * warps * groups;
    named_barrier_sync(kLnAllBarrier, threads);
    for (int c = threadIdx.x; c < 2 * Hp; c += threads) {
        const int col = c < Hp ? c : c - Hp;
        if (col >= H) continue;
        float v = meet[c];
        for (int g = 1; g < groups; ++g) v += meet[static_cast<long long>(g) * 2 * Hp + c];
        float *const out = c < Hp ? to_w : to_b;
        if (out) out[col] = v;
    }
}

template <class TX, class TD, int R, bool RUNS>
__global__ void __launch_bounds__(kLnThreads) ln_back_rows_kernel(const LayerNormBackArgs a, int warps) {
    extern __shared__ float sums[];                 // [groups][2][H]
    __shared__ float red[16][2 * 16 * 2];
    const int lane = threadIdx.x & 31, groups = blockDim.x / (32 * warps), group = threadIdx.x / (32 * warps);
    const int mine = threadIdx.x - group * 32 * warps, warp = mine >> 5;
    const bool want = a.d_w || a.d_b;
    int turn = 0;
    Run dw[R], db[R];
#pragma unroll
    for (int r = 0; r < R; ++r) dw[r] = db[r] = run_splat(0.f);
    griddep_wait();
    for (long long t = static_cast<long long>(blockIdx.x) * groups + group; t < a.T; t += static_cast<long long>(gridDim.x) * groups) {
        const TX *const x = static_cast<const TX *>(a.x) + t * a.x_stride;
        const TD *const d = static_cast<const TD *>(a.d_out) + t * a.d_stride;
        const float mean = a.stats[2 * t], rstd = a.stats[2 * t + 1];
        Run h[R], e[R];
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * warps * 32 + mine) * 8;
            h[r] = e[r] = run_splat(0.f);
            if (c >= a.H) continue;
            h[r] = ln_load<RUNS>(x, c, a.H);
            e[r] = ln_load<RUNS>(d, c, a.H);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * warps * 32 + mine) * 8;
            if (c >= a.H) continue;
            const Run w = ln_param<RUNS>(a.w, a.w_dtype, c, a.H, 1.f);
            uint64_t s1 = 0ull, s2 = 0ull;
#pragma unroll
            for (int q = 0; q < 4; ++q) h[r].p[q] = mul2(add2(h[r].p[q], splat2(-mean)), splat2(rstd));
            if (!RUNS) h[r] = ln_masked(h[r], c, a.H);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                dw[r].p[q] = fma2(e[r].p[q], h[r].p[q], dw[r].p[q]);
                db[r].p[q] = add2(db[r].p[q], e[r].p[q]);
                e[r].p[q] = mul2(e[r].p[q], w.p[q]);
                s1 = add2(s1, e[r].p[q]);
                s2 = fma2(e[r].p[q], h[r].p[q], s2);
            }
            s[0] += f2_lo(s1) + f2_hi(s1);
            s[1] += f2_lo(s2) + f2_hi(s2);
        }
        group_sums(s, warps, warp, lane, group + 1, red[group], &turn);
        const float m1 = -s[0] * a.inv_h, m2 = -s[1] * a.inv_h;
        TX *const out = static_cast<TX *>(a.d_x) + t * a.H;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * warps * 32 + mine) * 8;
            if (c >= a.H) continue;
            Run add = run_splat(0.f);
            if (a.d_residual) add = ln_load<RUNS>(static_cast<const TX *>(a.d_residual) + t * a.r_stride, c, a.H);
            Run o;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                o.p[q] = fma2(fma2(h[r].p[q], splat2(m2), add2(e[r].p[q], splat2(m1))), splat2(rstd), add.p[q]);
            ln_store<RUNS>(out, c, a.H, o, a.out_runs);
        }
    }
    if (!want) return;
    meet_sums<R>(sums, a, dw, db, groups, group, warps, mine);
}

// The same for many rows: rows to come staged in shared memory, where the
// weight lies too.
// SELF: a group is 8 or 16 warps, and with one more warp there would be room for one group less, or for 96
// registers a thread: its first thread orders its rows itself (8192 x 4096 bf16: 57 us, with a warp for it and one
// group 62, with 96 registers 67; 8192 x 7168, where there is one group anyway, 99 us by its first thread and 83 by a warp).
template <class TX, class TD, int R, bool RUNS, bool SELF>
__global__ void __launch_bounds__(kLnThreads) ln_back_ring_kernel(const LayerNormBackArgs a, const __grid_constant__ LnRing ring, int warps) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[16][2 * 16 * 2];
    __shared__ int abort_flag;
    const int lane = threadIdx.x & 31, groups = (blockDim.x - (SELF ? 0 : 32)) / (32 * warps), group = threadIdx.x / (32 * warps);
    const int mine = threadIdx.x - group * 32 * warps, warp = mine >> 5, threads = 32 * warps * groups;
    const bool filler = !SELF && threadIdx.x >= threads;
    float *const par = reinterpret_cast<float *>(smem + kLnBackRingBars);
    const int Hp = (a.H + 7) / 8 * 8, par_bytes = (4 * Hp + 127) / 128 * 128;
    const int which = filler ? lane : group, places_at = kLnBackRingBars + par_bytes + which * ring.stages * ring.place[kLnArrays];
    LnPlace place = {smem_addr(smem) + which * ring.stages * 16, smem_addr(smem) + places_at, 0, 0};
    if (threadIdx.x == 0) {
        ln_bars_init(smem_addr(smem), groups * ring.stages, warps);
        abort_flag = 0;
    }
    __syncthreads();
    griddep_wait();
    const long long first = static_cast<long long>(blockIdx.x) * groups + which, step = static_cast<long long>(gridDim.x) * groups;
    auto sources = [&](long long t, const void *(&src)[kLnArrays]) {
        src[0] = static_cast<const TX *>(a.x) + t * a.x_stride;
        src[1] = static_cast<const TD *>(a.d_out) + t * a.d_stride;
        src[2] = a.d_residual ? static_cast<const TX *>(a.d_residual) + t * a.r_stride : nullptr;
    };
    if (filler) {
        ln_fill(ring, place, lane < groups, first < a.T ? static_cast<int>((a.T - first + step - 1) / step) : 0, &abort_flag,
                [&](int k, const void *(&src)[kLnArrays]) { sources(first + k * step, src); });
        return;
    }
    // SELF: the next place to fill and its row
    LnPlace fill = place;
    long long next = first;
    auto order = [&] {
        if (next >= a.T) return;
        const void *src[kLnArrays];
        sources(next, src);
        ln_order(ring, fill, src, policy_evict_first());
        fill.next(ring);
        next += step;
    };
    if (SELF && mine == 0)
        for (int k = 0; k < ring.stages; ++k) order();
    ln_stage_param(par, a.w, a.w_dtype, a.H, Hp, 1.f, threads);
    Run dw[R], db[R];
#pragma unroll
    for (int r = 0; r < R; ++r) dw[r] = db[r] = run_splat(0.f);
    named_barrier_sync(kLnAllBarrier, threads);
    int turn = 0;
    float next_mean = first < a.T ? a.stats[2 * first] : 0.f, next_rstd = first < a.T ? a.stats[2 * first + 1] : 0.f;
    for (long long t = first; t < a.T; t += step, place.next(ring)) {
        const float mean = next_mean, rstd = next_rstd;
        if (t + step < a.T) {
            next_mean = a.stats[2 * (t + step)];
            next_rstd = a.stats[2 * (t + step) + 1];
        }
        mbar_wait(place.full(), place.turn, &abort_flag, ring.timeout_ns, ring.status, SITE_LN_ROW);
        const TX *const x = static_cast<const TX *>(a.x) + t * a.x_stride;
        const TD *const d = static_cast<const TD *>(a.d_out) + t * a.d_stride;
        const uint8_t *const staged = smem + places_at + place.at * ring.place[kLnArrays];
        Run h[R], e[R];
        float s[2] = {0.f, 0.f};
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * warps * 32 + mine) * 8;
            h[r] = e[r] = run_splat(0.f);
            if (c >= a.H) continue;
            h[r] = ln_staged<RUNS>(staged, ln_skew(x), c, a.H, x);
            e[r] = ln_staged<RUNS>(staged + ring.place[1], ln_skew(d), c, a.H, d);
            const Run w = load8_shared(par + c);
            uint64_t s1 = 0ull, s2 = 0ull;
#pragma unroll
            for (int q = 0; q < 4; ++q) h[r].p[q] = mul2(add2(h[r].p[q], splat2(-mean)), splat2(rstd));
            if (!RUNS) h[r] = ln_masked(h[r], c, a.H);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                dw[r].p[q] = fma2(e[r].p[q], h[r].p[q], dw[r].p[q]);
                db[r].p[q] = add2(db[r].p[q], e[r].p[q]);
                e[r].p[q] = mul2(e[r].p[q], w.p[q]);
                s1 = add2(s1, e[r].p[q]);
                s2 = fma2(e[r].p[q], h[r].p[q], s2);
            }
            s[0] += f2_lo(s1) + f2_hi(s1);
            s[1] += f2_lo(s2) + f2_hi(s2);
        }
        if (!SELF && !a.d_residual) {
            __syncwarp();
            if (lane == 0) mbar_arrive(place.empty());      // the row is in registers
        }
        group_sums(s, warps, warp, lane, group + 1, red[group], &turn);
        // SELF: every thread of the group has the row; with d_residual, which is read below, it has done with the one before
        if (SELF && mine == 0 && (!a.d_residual || t > first)) order();
        const float m1 = -s[0] * a.inv_h, m2 = -s[1] * a.inv_h;
        TX *const out = static_cast<TX *>(a.d_x) + t * a.H;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int c = (r * warps * 32 + mine) * 8;
            if (c >= a.H) continue;
            Run o, add = run_splat(0.f);
            if (a.d_residual) {
                const TX *const g = static_cast<const TX *>(a.d_residual) + t * a.r_stride;
                add = ln_staged<RUNS>(staged + ring.place[2], ln_skew(g), c, a.H, g);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
                o.p[q] = fma2(fma2(h[r].p[q], splat2(m2), add2(e[r].p[q], splat2(m1))), splat2(rstd), add.p[q]);
            ln_store<RUNS>(out, c, a.H, o, a.out_runs);
        }
        if (!SELF && a.d_residual) {
            __syncwarp();
            if (lane == 0) mbar_arrive(place.empty());
        }
    }
    if (SELF && mine == 0 && *reinterpret_cast<volatile int *>(&abort_flag))
        ln_drain(ring, fill, first < a.T ? static_cast<int>((next - first) / step) : 0);
    if (!a.d_w && !a.d_b) return;
    // the groups' sums meet in the stages, which hold nothing on its way any more, and each thread adds some columns
    named_barrier_sync(kLnAllBarrier, threads);
    meet_sums<R>(reinterpret_cast<float *>(smem + kLnBackRingBars + par_bytes), a, dw, db, groups, group, warps, mine);
}

// Rows too wide to be held: a CTA a row, read twice; its sums over tokens in its set, each column its thread's.
template <class TX, class TD>
__global__ void __launch_bounds__(kLnThreads) ln_back_loop_kernel(const LayerNormBackArgs a) {
    __shared__ float red[2 * 16 * 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = kLnThreads / 32;
    const bool want = a.d_w || a.d_b;
    float *const set = a.sums + static_cast<long long>(blockIdx.x) * 2 * a.H;
    int turn = 0;
    griddep_wait();
    for (long long t = blockIdx.x; t < a.T; t += gridDim.x) {
        const TX *const x = static_cast<const TX *>(a.x) + t * a.x_stride;
        const TD *const d = static_cast<const TD *>(a.d_out) + t * a.d_stride;
        const float mean = a.stats[2 * t], rstd = a.stats[2 * t + 1];
        const bool first = t == blockIdx.x;
        auto load = [&](int c, Run *h, Run *e) {
            *h = load8_any(x, c, a.H);
            *e = load8_any(d, c, a.H);
#pragma unroll
            for (int q = 0; q < 4; ++q) h->p[q] = mul2(add2(h->p[q], splat2(-mean)), splat2(rstd));
            *h = ln_masked(*h, c, a.H);
        };
        float s[2] = {0.f, 0.f};
        for (int c = threadIdx.x * 8; c < a.H; c += kLnThreads * 8) {
            Run h, e;
            load(c, &h, &e);
            if (want)
                for (int k = 0; k < 8 && c + k < a.H; ++k) {
                    const float w = run_at(e, k) * run_at(h, k), b = run_at(e, k);
                    set[c + k] = first ? w : set[c + k] + w;
                    set[a.H + c + k] = first ? b : set[a.H + c + k] + b;
                }
            const Run w = ln_param<false>(a.w, a.w_dtype, c, a.H, 1.f);
            Run p;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                e.p[q] = mul2(e.p[q], w.p[q]);
                p.p[q] = mul2(e.p[q], h.p[q]);
            }
            s[0] += run_sum(e);
            s[1] += run_sum(p);
        }
        group_sums(s, warps, warp, lane, 1, red, &turn);
        const float m1 = -s[0] * a.inv_h, m2 = -s[1] * a.inv_h;
        TX *const out = static_cast<TX *>(a.d_x) + t * a.H;
        for (int c = threadIdx.x * 8; c < a.H; c += kLnThreads * 8) {
            Run h, e;
            load(c, &h, &e);
            const Run w = ln_param<false>(a.w, a.w_dtype, c, a.H, 1.f);
            Run add = run_splat(0.f), o;
            if (a.d_residual) add = load8_any(static_cast<const TX *>(a.d_residual) + t * a.r_stride, c, a.H);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                o.p[q] = fma2(fma2(h.p[q], splat2(m2), fma2(e.p[q], w.p[q], splat2(m1))), splat2(rstd), add.p[q]);
            ln_store<false>(out, c, a.H, o, a.out_runs);
        }
    }
}

// The sets in their order (none: zeros); a CTA 32 columns of one of the two sums, its 8 warps shares of the sets.
__global__ void __launch_bounds__(256) ln_back_join_kernel(const float *sums, int parts, int H, float *d_w, float *d_b) {
    __shared__ float red[8][33];
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, which = blockIdx.y, c = blockIdx.x * 32 + lane;
    float *const out = which ? d_b : d_w;
    if (!out) return;
    float v = 0.f;
    if (c < H)
#pragma unroll 8
        for (int p = warp; p < parts; p += 8) v += sums[(static_cast<long long>(p) * 2 + which) * H + c];
    red[warp][lane] = v;
    __syncthreads();
    if (warp || c >= H) return;
    v = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v += red[k][lane];
    out[c] = v;
}

bool on_runs(const void *p, int dtype) { return (reinterpret_cast<uintptr_t>(p) & (dtype == MHC_F32 ? 31u : 15u)) == 0; }

template <class TX, class TD>
cudaError_t launch_types(const LayerNormBackArgs &a, unsigned int *status, bool pdl, cudaStream_t s) {
    const LnBack p = ln_back(a.T, a.H, kGridCap);
    if (a.H > kLnMaxHeld)
        return launch_block_kernel(ln_back_loop_kernel<TX, TD>, static_cast<unsigned>(p.parts), kLnThreads, 0, pdl, s, a);
    const bool runs = a.H % 8 == 0 && a.x_stride % 8 == 0 && a.d_stride % 8 == 0 && on_runs(a.x, a.x_dtype) &&
                      on_runs(a.d_out, a.d_dtype) && on_runs(a.d_x, a.x_dtype) && on_runs(a.w, a.w_dtype) &&
                      (!a.d_residual || (a.r_stride % 8 == 0 && on_runs(a.d_residual, a.x_dtype)));
    if (p.ring) {
        LnRing ring = {};
        ring.row_bytes[0] = a.H * static_cast<int>(sizeof(TX));
        ring.row_bytes[1] = a.H * static_cast<int>(sizeof(TD));
        ring.row_bytes[2] = a.d_residual ? ring.row_bytes[0] : 0;
        ln_places(ring.row_bytes, ring.place);
        const LnBackRing q = ln_back_ring(p, a.H, ring.place[kLnArrays], a.d_residual);
        ring.stages = q.stages;
        ring.status = status;
        ring.timeout_ns = wait_timeout_ns();
        const bool self = p.self;
        auto *const kern = self ? (runs ? ln_back_ring_kernel<TX, TD, kR, true, true> : ln_back_ring_kernel<TX, TD, kR, false, true>)
                                : (runs ? ln_back_ring_kernel<TX, TD, kR, true, false> : ln_back_ring_kernel<TX, TD, kR, false, false>);
        if (ring.stages) {
            static std::atomic<uint64_t> done[4];
            if (cudaError_t e = ln_allow_smem(reinterpret_cast<const void *>(kern), kLnBackRingSmem, &done[2 * self + runs])) return e;
            return launch_block_kernel(kern, static_cast<unsigned>(p.parts), 32 * (p.warps * p.groups + !self), q.smem, pdl, s, a, ring, p.warps);
        }
    }
    auto *const kern = p.R == 1 ? (runs ? ln_back_rows_kernel<TX, TD, 1, true> : ln_back_rows_kernel<TX, TD, 1, false>)
                                : (runs ? ln_back_rows_kernel<TX, TD, kR, true> : ln_back_rows_kernel<TX, TD, kR, false>);
    static std::atomic<uint64_t> done[4];
    if (cudaError_t e = ln_allow_smem(reinterpret_cast<const void *>(kern), kLnBackMeetSmem, &done[2 * (p.R == 1) + runs])) return e;
    return launch_block_kernel(kern, static_cast<unsigned>(p.parts), 32 * p.warps * p.groups, a.d_w || a.d_b ? ln_back_meet(p, a.H) : 0, pdl, s, a, p.warps);
}

}  // namespace

size_t layer_norm_sums_bytes(long long T, int H) {
    const int parts = T > 0 ? ln_back(T, H, kGridCap).parts : 0;
    return parts > 1 || H > kLnMaxHeld ? static_cast<size_t>(parts) * 2 * H * 4 : 0;
}

int launch_layer_norm_back(const LayerNormBackArgs &a, unsigned int *status, bool pdl, cudaStream_t s) {
    int parts = 0;
    if (a.T > 0) {
        cudaError_t e;
        if (a.x_dtype == MHC_BF16) e = launch_types<__nv_bfloat16, __nv_bfloat16>(a, status, pdl, s);
        else if (a.x_dtype == MHC_F16) e = launch_types<__half, __half>(a, status, pdl, s);
        else if (a.d_dtype == MHC_BF16) e = launch_types<float, __nv_bfloat16>(a, status, pdl, s);
        else if (a.d_dtype == MHC_F16) e = launch_types<float, __half>(a, status, pdl, s);
        else e = launch_types<float, float>(a, status, pdl, s);
        if (int r = note_launch(e)) return r;
        parts = ln_back(a.T, a.H, kGridCap).parts;
        if (parts == 1 && a.H <= kLnMaxHeld) return MHC_OK;     // the row kernel wrote the sums
    }
    if (!a.d_w && !a.d_b) return MHC_OK;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.H + 31) / 32, 2);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return note_launch(cudaLaunchKernelEx(&cfg, ln_back_join_kernel, static_cast<const float *>(a.sums), parts, a.H, a.d_w, a.d_b));
}

}  // namespace mhc
