// Backward pass of the gated residual block for rows of up to 8192 columns.
//
// With D the gradient that reaches residual_out, the row needs two sums that
// follow one another: mean(d_h w2 ro) for D, then mean(g D w1 y) for d_y. D is
// linear in the first, so the second splits into two sums that need no D, and
// one reduction of three sums serves the row.
//
// Bound by memory: 12 bytes a column with 16-bit types. A CTA's groups of warps
// have a row each in flight, 16 columns a thread; the rows to come are staged in
// shared memory by bulk copies. What every row needs again, both weights, the
// scale and the sums over tokens (d_w_post, d_w_pre, d_res_scale), lies in
// tensor memory, 16 columns of each array for a thread, and so do a full gate's
// values and slopes between the two passes over a row: in registers they
// would not leave room for the row, and in shared memory not for the rows to
// come. The sums leave it once, and a second kernel adds the CTAs' in their order.
//
// A single scale's gradient, one sum over all tokens and columns, is held in two floats from a thread's
// part of a row on (LongSum): its terms may all but cancel.
//
// Measured, bf16, channel gate and scale, with the second kernel: 8192 x 7168 136 us, 5.2 TB/s of the
// bytes that it must move (0.77 of a copy's rate), from int8 checkpoints 161; strided by 7171 elements
// 163, 7169 wide 198 (single elements); 512 x 7168 19.4 us, 4.2 of it the second kernel.
#pragma once
#include <type_traits>

#include "block_rows.cuh"

namespace mhc {

cudaError_t launch_block_bwd_loop(const BlockBwdArgs &a, int dtype, int r_dtype, bool pdl, int *parts, cudaStream_t s);

namespace {

constexpr int kBwdRuns = 2;
constexpr int kBwdStages = 32;
constexpr int kBwdGroups = 15;                      // named barriers 1 .. 15
constexpr int kBwdThreads = 512;
constexpr size_t kBwdSmem = 216 * 1024;             // dynamic; the group sums take 6 KB beside it
constexpr int kBwdArrays = 8;                       // in tensor memory: 16 warps, four to a quadrant of lanes
constexpr int kBwdTmemCols = 512;
static_assert(4 * kBwdArrays * kBwdRuns * 8 <= kBwdTmemCols, "four warps' arrays fit a quadrant's columns");
enum BwdSite : int { SITE_BWD_ROW = 75 };
enum BwdArray : int { T_W1, T_W2, T_SCALE, T_DW1, T_DW2, T_DSCALE, T_Y, T_R, T_GATE, T_SLOPE };

// The place of an array among a thread's eight. y and the residual go there in
// the first pass over a row, unpacked, and come back in the second, but where a
// full gate's two arrays and a channel scale's leave no room for them.
template <bool FULL, bool SCALED>
__device__ constexpr int bwd_cell(int array) {
    if (array == T_GATE) return SCALED ? 6 : 2;
    if (array == T_SLOPE) return SCALED ? 7 : 5;
    return array;
}

struct BwdRing {
    int groups;                                     // of a CTA, blockDim.x / groups threads each
    int stages;
    // bytes of a row's place in a stage, 0 where there is none: y, residual (or their
    // codes), d_ro, d_h, gate, the scale bytes of y and residual
    uint32_t place[7], stage_bytes;
    unsigned int *status;
    unsigned long long timeout_ns;
};

// FULL, SCALED, HELD: whether a call may have a full gate, a channel scale,
// checkpoints in the place of y or residual.
template <class TY, class TR, int MODE, bool FULL, bool SCALED, bool HELD>
__global__ void __launch_bounds__(kBwdThreads, 1) block_bwd_kernel(const BlockBwdArgs a, const BwdRing ring) {
    constexpr int RUNS = kBwdRuns, MAXW = kBwdThreads / 32;
    constexpr bool STAGED = MODE != ROWS_VEC;
    constexpr bool KEPT = !(FULL && SCALED);        // y and the residual between the passes
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) float red[kBwdGroups][2][3 * MAXW];
    __shared__ __align__(8) uint64_t bars[kBwdStages];
    __shared__ volatile int armed[kBwdStages];      // the filling each stage is in
    __shared__ float scale_red[64];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const BlockForm &f = a.f;
    const int H = f.H, groups = (H + 31) / 32;
    Place at;
    at.H = H;
    at.threads = blockDim.x / ring.groups;
    const int grp = threadIdx.x / at.threads, tid = threadIdx.x - grp * at.threads;
    at.thread = tid;
    const int warp = tid >> 5, warps = at.threads >> 5;
    const bool full_gate = FULL && f.gate_form == MHC_GATE_FULL, scaled = SCALED && f.scale_form == MHC_SCALE_CHANNEL;
    const bool token_gate = f.gate_form == MHC_GATE_TOKEN;
    const uint32_t ge = f.gate_dtype == MHC_F32 ? 4 : 2;
    const bool y_held = HELD && !a.y, r_held = HELD && !a.residual;
    const uint32_t bar = smem_addr(bars);

    if (threadIdx.x < 32) {
        tmem_alloc(smem_addr(&tmem_slot), kBwdTmemCols);
        tmem_relinquish();
    }
    for (int i = threadIdx.x; i < ring.groups * 2 * 3 * MAXW; i += blockDim.x) (&red[0][0][0])[i] = 0.f;
    if (STAGED && threadIdx.x < ring.stages) {          // 32 at most: the first warp, a lane a stage
        mbar_init(bar + 8 * threadIdx.x, 1);
        armed[threadIdx.x] = -1;
        abort_flag = 0;
        fence_mbar_init();
    }
    if (STAGED)
        for (int s = threadIdx.x; s < ring.stages; s += blockDim.x) {
            uint8_t *place = smem + s * ring.stage_bytes;
#pragma unroll
            for (int k = 0; k < 5; ++k) {
                zero_place_end(place, ring.place[k], MODE != ROWS_RING);
                place += ring.place[k];
            }
        }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // this thread's arrays: its warp's quadrant of lanes, the warp's share of the columns
    const uint32_t tmem0 = tmem_slot, cta_warp = threadIdx.x >> 5;
    const uint32_t tmem = tmem0 + ((cta_warp & 3) << 21) + (cta_warp >> 2) * (kBwdArrays * RUNS * 8);
    auto cell = [&](int array, int j) { return tmem + (bwd_cell<FULL, SCALED>(array) * RUNS + j) * 8; };
    griddep_wait();
    // The CTA's rows are blockIdx.x + k gridDim.x, k = 0, 1, ...: group k mod
    // groups takes row k, from stage k mod stages.
    const long long row0 = blockIdx.x + static_cast<long long>(grp) * gridDim.x;
    const long long row_step = static_cast<long long>(gridDim.x) * ring.groups;
    // where a row's parts begin in global memory, and their bytes
    struct Source {
        const void *p[7];
        uint32_t bytes[7];
    };
    auto source = [&](long long t) {
        Source c = {};
        c.p[0] = y_held ? static_cast<const void *>(a.ck_y.codes + t * H) : static_cast<const TY *>(a.y) + t * a.y_stride;
        c.bytes[0] = H * (y_held ? 1 : sizeof(TY));
        c.p[1] = r_held ? static_cast<const void *>(a.ck_r.codes + t * H)
                        : static_cast<const TR *>(a.residual) + t * a.r_stride;
        c.bytes[1] = H * (r_held ? 1 : sizeof(TR));
        c.p[2] = static_cast<const TR *>(a.d_ro) + t * a.d_ro_stride;
        c.bytes[2] = a.d_ro ? H * sizeof(TR) : 0;
        c.p[3] = static_cast<const TY *>(a.d_h) + t * a.d_h_stride;
        c.bytes[3] = H * sizeof(TY);
        c.p[4] = static_cast<const uint8_t *>(f.gate) + t * f.gate_stride * ge;
        c.bytes[4] = full_gate ? H * ge : 0;
        c.p[5] = a.ck_y.scales + t * groups;
        c.bytes[5] = y_held ? groups : 0;
        c.p[6] = a.ck_r.scales + t * groups;
        c.bytes[6] = r_held ? groups : 0;
        return c;
    };
    constexpr int PARTS = HELD ? 7 : FULL ? 5 : 4;
    auto fetch = [&](long long t, int s, int filling) {     // one thread a stage
        const uint32_t b = bar + 8 * s;
        uint32_t dst = smem_addr(smem) + s * ring.stage_bytes, total = 0;
        const uint64_t pol = policy_evict_first();
        const Source c = source(t);
#pragma unroll
        for (int k = 0; k < PARTS; ++k)
            if (c.bytes[k]) total += skewed_bytes(c.p[k], c.bytes[k]);
        stage_arm(&armed[s], filling, b, total);
#pragma unroll
        for (int k = 0; k < PARTS; ++k) {
            if (c.bytes[k]) bulk_load_row(dst, c.p[k], c.bytes[k], b, pol);
            dst += ring.place[k];
        }
    };
    if (STAGED && threadIdx.x < ring.stages) {
        const long long t = blockIdx.x + static_cast<long long>(threadIdx.x) * gridDim.x;
        if (t < f.T) fetch(t, threadIdx.x, 0);
    }
    __syncwarp();
    // w1 = (w_post + offset) * act of a channel gate, w2 = w_pre + offset, a channel scale; the sums
#pragma unroll
    for (int j = 0; j < RUNS; ++j) {
        const RowParams p = load_row_params<MODE>(f, at, j);
        __syncwarp();
        tmem_run_store(cell(T_W1, j), p.w1);
        tmem_run_store(cell(T_W2, j), p.w2);
        if (SCALED) tmem_run_store(cell(T_SCALE, j), p.sc);
        tmem_run_store(cell(T_DW1, j), run_splat(0.f));
        tmem_run_store(cell(T_DW2, j), run_splat(0.f));
        if (SCALED) tmem_run_store(cell(T_DSCALE, j), run_splat(0.f));
    }
    tmem_st_wait();
    const uint64_t scale = splat2(f.scale_form == MHC_SCALE_ONE ? *f.res_scale : 1.f);
    LongSum scale_sum;

    // What a row needs beside its columns, fetched a row ahead and left as it
    // was loaded: arithmetic on it here would wait for it.
    struct Ahead {
        float rstd1, rstd2;
        uint32_t token;                             // bits of its gate
    };
    auto ahead = [&](long long t) {
        Ahead n = {};
        if (t >= f.T) return n;
        n.rstd1 = a.rstd[2 * t];
        n.rstd2 = a.rstd[2 * t + 1];
        if (token_gate)
            n.token = f.gate_dtype == MHC_F32 ? static_cast<const uint32_t *>(f.gate)[t * f.gate_stride]
                                              : static_cast<const uint16_t *>(f.gate)[t * f.gate_stride];
        return n;
    };
    auto token_of = [&](uint32_t bits) {
        if (f.gate_dtype == MHC_F32) return __uint_as_float(bits);
        if (f.gate_dtype == MHC_BF16) return __uint_as_float(bits << 16);
        return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
    };

    // A wait that runs out is recorded, and the rows left go by with what the
    // stages hold: no later wait takes long, and nothing more is fetched.
    int which = 0, s = grp, filling = 0;
    bool ok = true;
    Ahead next = ahead(row0);
    for (long long t = row0; t < f.T; t += row_step) {
        // the columns' addresses are formed anew for each row: kept across rows, those of every
        // tensor would take the registers that hold the row
        if (MODE == ROWS_ANY) asm volatile("" : "+r"(at.thread));
        const Ahead now = next;
        next = ahead(t + row_step);
        const float rstd1 = f.post_norm ? now.rstd1 : 1.f, rstd2 = now.rstd2;
        float token = 1.f, token_slope = 0.f;
        if (token_gate) gate_both(token_of(now.token), f.gate_act, &token, &token_slope);
        const uint8_t *st[7];
        st[0] = smem + s * ring.stage_bytes;
#pragma unroll
        for (int k = 1; k < PARTS; ++k) st[k] = st[k - 1] + ring.place[k - 1];
        if (STAGED) {
            ok = stage_wait(&armed[s], filling, bar + 8 * s, &abort_flag, ring.timeout_ns, ring.status, SITE_BWD_ROW) && ok;
            __syncwarp();
        }

        // a run of y, the residual, the gradients, the full gate, from the stage or from memory
        auto row_run = [&](int k, const auto *row, int j) {
            using T = typename std::remove_cv<typename std::remove_reference<decltype(*row)>::type>::type;
            if constexpr (MODE == ROWS_RING) return staged_run(reinterpret_cast<const T *>(st[k]), at, j);
            else if constexpr (MODE == ROWS_VEC) return load_run(row, at, j);
            else if constexpr (MODE == ROWS_SKEW) return staged_skewed<T>(st[k], skew16(row), at, j);
            else return staged_single(reinterpret_cast<const T *>(st[k] + skew16(row)), at, j);
        };
        auto held = [&](const Ckpt &c, int k, int k_scales, int j) {
            const uint8_t *const codes = c.codes + t * H, *const scales = c.scales + t * groups;
            const uint8_t *const byte_at = STAGED ? st[k_scales] + skew16(scales) : scales;
            if constexpr (MODE != ROWS_ANY) {
                const int i = run_read_col(at, j);
                uint2 w = *reinterpret_cast<const uint2 *>((STAGED ? st[k] + skew16(codes) : codes) + i);
                if (!run_in<MODE>(at, j)) w = make_uint2(0u, 0u);
                return ckpt_values8(w, byte_at[i / 32], a.format);
            } else {
                const int col = run_col<MODE>(at, j);
                const uint8_t *const code_at = st[k] + skew16(codes);
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int i = min(col + e * at.threads, H - 1);
                    const float x = (a.format == MHC_CKPT_E4M3 ? ckpt_value<MHC_CKPT_E4M3>(code_at[i])
                                                      : ckpt_value<MHC_CKPT_INT8>(code_at[i])) *
                           ckpt_unit(byte_at[i / 32]);
                    v[e] = col + e * at.threads < H ? x : 0.f;
                }
                return run_of(v);
            }
        };
        auto load_y = [&](int j) {
            if (y_held) return held(a.ck_y, 0, 5, j);
            return row_run(0, static_cast<const TY *>(a.y) + t * a.y_stride, j);
        };
        auto load_r = [&](int j) {
            if (r_held) return held(a.ck_r, 1, 6, j);
            return row_run(1, static_cast<const TR *>(a.residual) + t * a.r_stride, j);
        };
        auto load_df = [&](int j) { return row_run(2, static_cast<const TR *>(a.d_ro) + t * a.d_ro_stride, j); };
        auto load_dh = [&](int j) { return row_run(3, static_cast<const TY *>(a.d_h) + t * a.d_h_stride, j); };
        auto load_z = [&](int j) {
            return f.gate_dtype == MHC_F32 ? row_run(4, static_cast<const float *>(f.gate) + t * f.gate_stride, j)
                                           : row_run(4, static_cast<const TY *>(f.gate) + t * f.gate_stride, j);
        };

        const uint64_t r2 = splat2(rstd2), tr2 = splat2(token * rstd1);
        uint64_t s0 = 0, s1 = 0, s2 = 0;
        Run ev[RUNS];                               // d_ro + rstd_pre d_h w2
#pragma unroll
        for (int j = 0; j < RUNS; ++j) {
            LoadingRun w1_in, w2_in, sc_in, sum2_in;
            __syncwarp();
            tmem_run_load(cell(T_W1, j), w1_in);
            if (SCALED) tmem_run_load(cell(T_SCALE, j), sc_in);
            tmem_run_load(cell(T_W2, j), w2_in);
            tmem_run_load(cell(T_DW2, j), sum2_in);
            Run y = load_y(j), ro = load_r(j);
            if (KEPT) {
                __syncwarp();
                tmem_run_store(cell(T_Y, j), y);
                tmem_run_store(cell(T_R, j), ro);
            }
            if (full_gate) {
                Run z = load_z(j), slope;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float g0, g1, h0, h1;
                    gate_both(f2_lo(z.p[i]), f.gate_act, &g0, &h0);
                    gate_both(f2_hi(z.p[i]), f.gate_act, &g1, &h1);
                    z.p[i] = f2_pack(g0, g1);
                    slope.p[i] = f2_pack(h0, h1);
                    y.p[i] = mul2(y.p[i], z.p[i]);
                }
                __syncwarp();
                tmem_run_store(cell(T_GATE, j), z);
                tmem_run_store(cell(T_SLOPE, j), slope);
            }
            const Run dh = load_dh(j);
            ev[j] = run_splat(0.f);
            if (a.d_ro) ev[j] = load_df(j);
            __syncwarp();
            const Run w1 = tmem_run_wait(w1_in), w2 = tmem_run_wait(w2_in);
            Run sum2 = tmem_run_wait(sum2_in), sc;
            if (SCALED) sc = tmem_run_wait(sc_in);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y.p[i] = mul2(y.p[i], w1.p[i]);                            // g w1 y, without a token's gate
                ro.p[i] = fma2(y.p[i], tr2, mul2(SCALED ? sc.p[i] : scale, ro.p[i]));
                sum2.p[i] = fma2(mul2(dh.p[i], r2), ro.p[i], sum2.p[i]);
                const uint64_t dv = mul2(dh.p[i], w2.p[i]);
                ev[j].p[i] = fma2(r2, dv, ev[j].p[i]);
                if (MODE != ROWS_VEC || run_in<MODE>(at, j)) {
                    s0 = fma2(dv, ro.p[i], s0);
                    s1 = fma2(y.p[i], ev[j].p[i], s1);
                    s2 = fma2(y.p[i], ro.p[i], s2);
                }
            }
            if (MODE == ROWS_VEC) __syncwarp();
            tmem_run_store(cell(T_DW2, j), sum2);
        }
        float sum[3] = {f2_lo(s0) + f2_hi(s0), f2_lo(s1) + f2_hi(s1), f2_lo(s2) + f2_hi(s2)};
        group_sum<3, MAXW>(sum, red[grp][which], 1 + grp, warp, warps);
        which ^= 1;
        // The row's stage is free when every thread of the group has read it: past the first pass where y and
        // the residual are kept, else past the second. Then the group's next row: `groups` stages
        // on, their number more than that.
        auto release = [&] {
            if (warps == 1) __syncwarp();
            const long long refill = t + static_cast<long long>(ring.stages) * gridDim.x;
            if (tid == 0 && refill < f.T && ok) fetch(refill, s, 1 + filling);
            __syncwarp();
            s += ring.groups;
            if (s >= ring.stages) {
                s -= ring.stages;
                ++filling;
            }
        };
        if (STAGED && KEPT) release();
        const float q = rstd2 * (rstd2 * (rstd2 * (sum[0] * f.inv_h)));
        const float c1 = fmaf(-q, sum[2], sum[1]);
        const float p = f.post_norm ? rstd1 * (rstd1 * (rstd1 * (token * c1 * f.inv_h))) : 0.f;
        const uint64_t q2 = splat2(-q), p2 = splat2(-p);
        uint64_t scale2 = 0;                        // a single scale's terms of this row
        tmem_st_wait();
#pragma unroll
        for (int j = 0; j < RUNS; ++j) {
            LoadingRun w1_in, sc_in, sum1_in, sums_in, y_in, r_in;
            tmem_run_load(cell(T_W1, j), w1_in);
            tmem_run_load(cell(T_DW1, j), sum1_in);
            if (SCALED) {
                tmem_run_load(cell(T_SCALE, j), sc_in);
                tmem_run_load(cell(T_DSCALE, j), sums_in);
            }
            Run y, r, sc, sums;
            if (KEPT) {
                tmem_run_load(cell(T_Y, j), y_in);
                tmem_run_load(cell(T_R, j), r_in);
            } else {
                y = load_y(j);
                r = load_r(j);
                __syncwarp();
            }
            const Run w1 = tmem_run_wait(w1_in);
            Run sum1 = tmem_run_wait(sum1_in);
            if (KEPT) {
                y = tmem_run_wait(y_in);
                r = tmem_run_wait(r_in);
            }
            if (SCALED) {
                sc = tmem_run_wait(sc_in);
                sums = tmem_run_wait(sums_in);
            }
            if (full_gate) {
                LoadingRun gate_in, slope_in;
                tmem_run_load(cell(T_GATE, j), gate_in);
                tmem_run_load(cell(T_SLOPE, j), slope_in);
                const Run gate = tmem_run_wait(gate_in);
                Run z = tmem_run_wait(slope_in);    // the slope, then d_gate
                const uint64_t u1 = splat2(rstd1);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t g = gate.p[i], u = mul2(y.p[i], u1), wu = mul2(w1.p[i], u);
                    const uint64_t ro = fma2(g, wu, mul2(SCALED ? sc.p[i] : scale, r.p[i])), D = fma2(q2, ro, ev[j].p[i]);
                    const uint64_t gD = mul2(g, D);
                    sum1.p[i] = fma2(gD, u, sum1.p[i]);
                    z.p[i] = mul2(z.p[i], mul2(wu, D));                                     // d_gate
                    y.p[i] = fma2(p2, y.p[i], mul2(u1, mul2(w1.p[i], gD)));                 // d_y
                    ev[j].p[i] = D;
                }
                if (a.d_gate) {
                    if (f.gate_dtype == MHC_F32) store_run<MODE>(static_cast<float *>(a.d_gate) + t * H, at, j, z);
                    else store_run<MODE>(static_cast<TY *>(a.d_gate) + t * H, at, j, z);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t ro = fma2(mul2(y.p[i], w1.p[i]), tr2, mul2(SCALED ? sc.p[i] : scale, r.p[i]));
                    const uint64_t D = fma2(q2, ro, ev[j].p[i]), trD = mul2(tr2, D);
                    sum1.p[i] = fma2(trD, y.p[i], sum1.p[i]);
                    y.p[i] = fma2(p2, y.p[i], mul2(w1.p[i], trD));
                    ev[j].p[i] = D;
                }
            }
            store_run<MODE>(static_cast<TY *>(a.d_y) + t * H, at, j, y);
            if (!SCALED && run_col<MODE>(at, j) < H) {
                const Run d = MODE == ROWS_ANY ? run_within<MODE>(ev[j], at, j) : ev[j];
#pragma unroll
                for (int i = 0; i < 4; ++i) scale2 = fma2(r.p[i], d.p[i], scale2);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (SCALED) sums.p[i] = fma2(r.p[i], ev[j].p[i], sums.p[i]);
                ev[j].p[i] = mul2(SCALED ? sc.p[i] : scale, ev[j].p[i]);
            }
            store_run<MODE>(static_cast<TR *>(a.d_r) + t * H, at, j, ev[j]);
            __syncwarp();
            tmem_run_store(cell(T_DW1, j), sum1);
            if (SCALED) tmem_run_store(cell(T_DSCALE, j), sums);
        }
        if (!SCALED) scale_sum.add(f2_lo(scale2) + f2_hi(scale2));
        tmem_st_wait();
        if (STAGED && !KEPT) {
            if (warps > 1) named_barrier_sync(1 + grp, at.threads);
            release();
        }
        if (token_gate && a.d_gate && tid == 0) static_cast<float *>(a.d_gate)[t] = token_slope * rstd1 * c1;
    }
    if (STAGED && !ok && tid == 0) {
        // copies that may still be in flight, before the CTA's memory goes: each
        // stage's last, in either parity
        int gave_up = 0;
        for (int k = 0; k < 2 * ring.stages; ++k)
            mbar_wait(bar + 8 * (k >> 1), k & 1, &gave_up, ring.timeout_ns, ring.status, SITE_BWD_ROW);
    }

    // The groups' sums, through the place of the stages, each column's then in the groups'
    // order; an array's halves go round the groups. One group's straight out.
    __syncthreads();
    float *const out = a.sums + static_cast<long long>(blockIdx.x) * kBackSums * H;
    const int arrays = scaled ? 3 : 2, column = at.threads * RUNS * 8;
#pragma unroll
    for (int k = 0; k < (SCALED ? 3 : 2); ++k) {
        if (k >= arrays) break;
#pragma unroll
        for (int j = 0; j < RUNS; ++j) {
            LoadingRun acc_in;
            __syncwarp();
            tmem_run_load(cell(T_DW1 + k, j), acc_in);
            const Run acc = tmem_run_wait(acc_in);
            if (ring.groups == 1) store_run<MODE>(out + static_cast<long long>(k) * H, at, j, acc);
            else keep_run(reinterpret_cast<float *>(smem) + (k * ring.groups + grp) * column, at, j, acc);
        }
    }
    if (ring.groups > 1) {
        __syncthreads();
        for (int i = grp; i < arrays * RUNS; i += ring.groups) {
            const int k = i / RUNS, j = i - k * RUNS;
            const float *const kept = reinterpret_cast<const float *>(smem) + k * ring.groups * column;
            Run acc = kept_run(kept, at, j);
            for (int g = 1; g < ring.groups; ++g) {
                const Run more = kept_run(kept + g * column, at, j);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc.p[e] = add2(acc.p[e], more.p[e]);
            }
            store_run<MODE>(out + static_cast<long long>(k) * H, at, j, acc);
        }
    }
    if (SCALED && f.scale_form == MHC_SCALE_ONE) {
        // a single scale in the general form: its columns' sums
#pragma unroll
        for (int j = 0; j < RUNS; ++j) {
            LoadingRun acc_in;
            __syncwarp();
            tmem_run_load(cell(T_DSCALE, j), acc_in);
            const Run acc = run_within<MODE>(tmem_run_wait(acc_in), at, j);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                scale_sum.add(f2_lo(acc.p[i]));
                scale_sum.add(f2_hi(acc.p[i]));
            }
        }
    }
    block_long_sum(scale_sum, scale_red);
    if (threadIdx.x == 0) {
        a.scale_sums[2 * blockIdx.x] = scale_sum.hi;
        a.scale_sums[2 * blockIdx.x + 1] = scale_sum.lo;
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x < 32) {
        tc_fence_after();
        tmem_dealloc(tmem0, kBwdTmemCols);
    }
}

template <class TY, class TR, int MODE, bool FULL, bool SCALED, bool HELD>
cudaError_t bwd_launch(const BlockBwdArgs &a, const BwdRing &ring, unsigned grid, int threads, size_t smem, bool pdl,
                       cudaStream_t s) {
    static SmemGrant grant;
    auto kern = block_bwd_kernel<TY, TR, MODE, FULL, SCALED, HELD>;
    if (cudaError_t e = grant_smem(kern, grant, smem, kBwdSmem)) return e;
    return launch_block_kernel(kern, grid, threads * ring.groups, smem, pdl, s, a, ring);
}

template <class TY, class TR>
cudaError_t block_bwd(const BlockBwdArgs &a, int dtype, int r_dtype, int sms, bool pdl, int *parts, cudaStream_t s) {
    const BlockForm &f = a.f;
    const int H = f.H;
    if (H > 8192) return launch_block_bwd_loop(a, dtype, r_dtype, pdl, parts, s);
    const bool full = f.gate_form == MHC_GATE_FULL, scaled = f.scale_form == MHC_SCALE_CHANNEL;
    const bool held = !a.y || !a.residual;
    // what is written, the weights and the codes allow runs of 8; the inputs too
    auto codes_fit = [&](const Ckpt &c) { return (reinterpret_cast<uintptr_t>(c.codes) & 7u) == 0; };
    const bool out_vec = H % 8 == 0 && (a.y || codes_fit(a.ck_y)) && (a.residual || codes_fit(a.ck_r)) &&
                         rows_of_runs(a.d_y, H, sizeof(TY), f.T) && rows_of_runs(a.d_r, H, sizeof(TR), f.T) &&
                         rows_of_runs(a.sums, H, 4, f.T) && params_of_runs(f) &&
                         (!full || !a.d_gate || rows_of_runs(a.d_gate, H, elem_bytes(f.gate_dtype), f.T));
    const bool vec = out_vec && (!a.y || rows_of_runs(a.y, a.y_stride, sizeof(TY), f.T)) &&
                     (!a.residual || rows_of_runs(a.residual, a.r_stride, sizeof(TR), f.T)) &&
                     (!a.d_ro || rows_of_runs(a.d_ro, a.d_ro_stride, sizeof(TR), f.T)) &&
                     rows_of_runs(a.d_h, a.d_h_stride, sizeof(TY), f.T) &&
                     (!full || rows_of_runs(f.gate, f.gate_stride, elem_bytes(f.gate_dtype), f.T));
    BwdRing ring = {};
    const int threads = row_threads(H, kBwdRuns);
    // as many groups as fit, but no more than give every SM a row
    long long groups = kBwdThreads / threads;
    const long long rows = (f.T + sms - 1) / sms;
    if (groups > kBwdGroups) groups = kBwdGroups;
    ring.groups = static_cast<int>(rows < groups ? rows : groups);
    // where the groups' sums meet at the end
    auto sums = [&] { return ring.groups == 1 ? 0 : static_cast<size_t>(3) * ring.groups * threads * kBwdRuns * 32; };
    const unsigned grid = static_cast<unsigned>(f.T < sms ? f.T : sms);
    *parts = static_cast<int>(grid);
    const int scale_bytes = static_cast<int>(ckpt_groups(H));
    ring.place[0] = row_place(H, a.y ? sizeof(TY) : 1, !vec || !a.y);
    ring.place[1] = row_place(H, a.residual ? sizeof(TR) : 1, !vec || !a.residual);
    ring.place[2] = a.d_ro ? row_place(H, sizeof(TR), !vec) : 0;
    ring.place[3] = row_place(H, sizeof(TY), !vec);
    ring.place[4] = full ? row_place(H, elem_bytes(f.gate_dtype), !vec) : 0;
    ring.place[5] = a.y ? 0 : row_place(scale_bytes, 1, true);
    ring.place[6] = a.residual ? 0 : row_place(scale_bytes, 1, true);
    for (uint32_t b : ring.place) ring.stage_bytes += b;
    long long stages = static_cast<long long>(kBwdSmem / ring.stage_bytes);
    if (stages > kBwdStages) stages = kBwdStages;
    if (stages > rows) stages = rows;
    // two stages at least, or all of the rows; else (the widest types above 5000 columns and more) from memory
    if (stages < 2 && stages < rows) {
        if (!vec) return launch_block_bwd_loop(a, dtype, r_dtype, pdl, parts, s);
        return bwd_launch<TY, TR, ROWS_VEC, true, true, true>(a, ring, grid, threads, sums(), pdl, s);
    }
    // a stage for each group and one to fill meanwhile, or all of the rows
    if (ring.groups >= stages) ring.groups = static_cast<int>(stages == rows ? stages : stages - 1);
    ring.stages = static_cast<int>(stages);
    size_t smem = static_cast<size_t>(ring.stage_bytes) * ring.stages;
    if (smem < sums()) smem = sums();
    int n = 0;
    if (require_device(&n, &ring.status)) return cudaErrorUnknown;
    ring.timeout_ns = wait_timeout_ns();
    if (!vec) {
        if (held || (full && scaled))
            return out_vec ? bwd_launch<TY, TR, ROWS_SKEW, true, true, true>(a, ring, grid, threads, smem, pdl, s)
                           : bwd_launch<TY, TR, ROWS_ANY, true, true, true>(a, ring, grid, threads, smem, pdl, s);
        if (full)
            return out_vec ? bwd_launch<TY, TR, ROWS_SKEW, true, false, false>(a, ring, grid, threads, smem, pdl, s)
                           : bwd_launch<TY, TR, ROWS_ANY, true, false, false>(a, ring, grid, threads, smem, pdl, s);
        return out_vec ? bwd_launch<TY, TR, ROWS_SKEW, false, true, false>(a, ring, grid, threads, smem, pdl, s)
                       : bwd_launch<TY, TR, ROWS_ANY, false, true, false>(a, ring, grid, threads, smem, pdl, s);
    }
    if (full)
        return scaled || held ? bwd_launch<TY, TR, ROWS_RING, true, true, true>(a, ring, grid, threads, smem, pdl, s)
                              : bwd_launch<TY, TR, ROWS_RING, true, false, false>(a, ring, grid, threads, smem, pdl, s);
    if (held)
        return scaled ? bwd_launch<TY, TR, ROWS_RING, false, true, true>(a, ring, grid, threads, smem, pdl, s)
                      : bwd_launch<TY, TR, ROWS_RING, false, false, true>(a, ring, grid, threads, smem, pdl, s);
    return scaled ? bwd_launch<TY, TR, ROWS_RING, false, true, false>(a, ring, grid, threads, smem, pdl, s)
                  : bwd_launch<TY, TR, ROWS_RING, false, false, false>(a, ring, grid, threads, smem, pdl, s);
}

}  // namespace
}  // namespace mhc
