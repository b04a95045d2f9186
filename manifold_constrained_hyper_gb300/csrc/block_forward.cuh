// The gated residual block's boundary for rows of up to 8192 columns: a group
// of warps holds a row in registers, so that y, residual and a full gate are
// read once and both norms' sums run over registers; what every row needs (both
// weights with their offset and a channel gate, a channel scale) lies in
// shared memory.
//
// Bound by memory: 8 bytes a column with 16-bit types (10 with a full gate),
// which leaves the issue slots some 40 instructions a column at full rate; so
// the arithmetic is on packed pairs and a thread holds 32 columns, over which
// a row's fixed costs (two sums, a wait, addresses) spread. A row's two sums
// follow one another: a CTA's groups have a row each in flight, and the rows
// to come are staged in shared memory by bulk copies meanwhile, a stage
// refilled as soon as its row is in registers. With 16 columns a thread
// 8192 x 7168 takes 2 to 10 % longer.
//
// Measured, bf16: 8192 x 7168 with a full sigmoid gate 99.6 us, 5.9 TB/s of the bytes that it
// must move (0.88 of a copy's rate), with a channel gate and scale 80 to 84; strided by
// 7171 elements 100 to 112, 7169 wide 158 (single elements: bound by instructions); one row of 7168 4.7 us.
#pragma once
#include <type_traits>

#include "block_rows.cuh"

namespace mhc {

cudaError_t launch_block_fwd_loop(const BlockFwdArgs &a, int dtype, int r_dtype, int sms, bool pdl, cudaStream_t s);

namespace {

constexpr int kFwdStages = 32;
// Columns up to which rows go by registers alone (8192 rows: of 256 columns 5.8 us, staged 11.8; of 512
// 10.2 and 12.6; of 1024 17.7 and 14.7).
constexpr int kFwdNarrow = 512;
constexpr int kFwdGroups = 15;                      // named barriers 1 .. 15
constexpr size_t kFwdSmem = 224 * 1024;             // dynamic
enum FwdSite : int { SITE_FWD_ROW = 70 };

struct FwdRing {
    int groups;                                     // of a CTA, blockDim.x / groups threads each
    int stages;
    uint32_t y_place, r_place, g_place;             // bytes of a row's place in a stage; g_place 0: no full gate
    uint32_t row_bytes;                             // of its copies, in ROWS_RING
    unsigned int *status;
    unsigned long long timeout_ns;
};

// FULL, SCALED, CKPT: whether a call may have a full gate, a channel scale,
// checkpoints. RUNS of 8 columns a thread: 4, and 2 of rows on any boundary or most with checkpoints, in blocks of up to 512
// threads of 128 registers; 1, up to 1024 threads of 64, for a few rows or narrow ones.
template <class TY, class TR, int MODE, int RUNS, bool FULL, bool SCALED, bool CKPT>
__global__ void __launch_bounds__(RUNS == 1 ? 1024 : 512, 1) block_fwd_kernel(const BlockFwdArgs a, const FwdRing ring) {
    constexpr int MAXW = 32 / RUNS, GROUPS = RUNS == 1 ? 32 : kFwdGroups;
    constexpr bool STAGED = MODE != ROWS_VEC;
    // past the row's end its last run again, left out of the sums, instead of zeros: from global memory, and
    // where the zeros' place takes registers that are not there (8192 x 7168 with int8 checkpoints: spills, 10 us)
    constexpr bool GUARD = MODE == ROWS_VEC || (CKPT && RUNS == 4);
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) float red[GROUPS][2][MAXW];
    __shared__ __align__(8) uint64_t bars[kFwdStages];
    __shared__ volatile int armed[kFwdStages];      // the filling each stage is in
    __shared__ int abort_flag;
    const BlockForm &f = a.f;
    Place at;
    at.H = f.H;
    at.threads = blockDim.x / ring.groups;
    const int grp = threadIdx.x / at.threads;
    at.thread = threadIdx.x - grp * at.threads;
    const int warp = at.thread >> 5, warps = at.threads >> 5;
    const bool full_gate = FULL && f.gate_form == MHC_GATE_FULL;
    const uint32_t stage_bytes = ring.y_place + ring.r_place + ring.g_place;
    const uint32_t ge = f.gate_dtype == MHC_F32 ? 4 : 2;
    const uint32_t y_bytes = f.H * sizeof(TY), r_bytes = f.H * sizeof(TR), g_bytes = f.H * ge;    // of a row
    // (w_post + offset) * act of a channel gate; w_pre + offset; a channel scale; then the stages
    float *const w1_kept = reinterpret_cast<float *>(smem), *const w2_kept = w1_kept + 8 * RUNS * at.threads,
          *const sc_kept = w2_kept + 8 * RUNS * at.threads;
    const uint32_t stage0 = (SCALED ? 3 : 2) * 32 * RUNS * at.threads;
    const uint32_t bar = smem_addr(bars);

    for (int i = threadIdx.x; i < ring.groups * 2 * MAXW; i += blockDim.x) (&red[0][0][0])[i] = 0.f;
    // The stages are set up, and filled for the first time, by a lane of the first warp each; with
    // checkpoints and 32 columns a thread by one thread: there the registers are short (spills:
    // 8192 x 7168 with int8 checkpoints 116 us, 159).
    constexpr bool LANES = !(CKPT && RUNS == 4);
    const int first_stage = LANES ? threadIdx.x : 0, stage_step = LANES ? 32 : 1;
    if (STAGED && threadIdx.x < (LANES ? 32 : 1)) {
        for (int s = first_stage; s < ring.stages; s += stage_step) {
            mbar_init(bar + 8 * s, 1);
            armed[s] = -1;
        }
        abort_flag = 0;
        fence_mbar_init();
    }
    if (STAGED && !GUARD)
        for (int s = threadIdx.x; s < ring.stages; s += blockDim.x) {
            uint8_t *const place = smem + stage0 + s * stage_bytes;
            zero_place_end(place, ring.y_place, MODE != ROWS_RING);
            zero_place_end(place + ring.y_place, ring.r_place, MODE != ROWS_RING);
            zero_place_end(place + ring.y_place + ring.r_place, ring.g_place, MODE != ROWS_RING);
        }
    __syncthreads();
    griddep_wait();
    // The CTA's rows are blockIdx.x + k gridDim.x, k = 0, 1, ...: group k mod
    // groups takes row k, from stage k mod stages.
    auto fetch = [&](long long t, int s, int filling) {     // one thread a stage
        const uint32_t b = bar + 8 * s, dst = smem_addr(smem) + stage0 + s * stage_bytes;
        const uint64_t pol = policy_evict_first();
        const TY *const y = static_cast<const TY *>(a.y) + t * a.y_stride;
        const TR *const r = static_cast<const TR *>(a.residual) + t * a.r_stride;
        const uint8_t *const g = static_cast<const uint8_t *>(f.gate) + t * f.gate_stride * ge;
        if (MODE == ROWS_RING) {
            stage_arm(&armed[s], filling, b, ring.row_bytes);
            bulk_load(dst, y, y_bytes, b, pol);
            bulk_load(dst + ring.y_place, r, r_bytes, b, pol);
            if (FULL && ring.g_place) bulk_load(dst + ring.y_place + ring.r_place, g, g_bytes, b, pol);
        } else {
            stage_arm(&armed[s], filling, b, skewed_bytes(y, y_bytes) + skewed_bytes(r, r_bytes) +
                                                 (FULL && ring.g_place ? skewed_bytes(g, g_bytes) : 0));
            bulk_load_row(dst, y, y_bytes, b, pol);
            bulk_load_row(dst + ring.y_place, r, r_bytes, b, pol);
            if (FULL && ring.g_place) bulk_load_row(dst + ring.y_place + ring.r_place, g, g_bytes, b, pol);
        }
    };
    if (STAGED && threadIdx.x < (LANES ? 32 : 1))
        for (int s = first_stage; s < ring.stages; s += stage_step) {
            const long long t = blockIdx.x + static_cast<long long>(s) * gridDim.x;
            if (t < f.T) fetch(t, s, 0);
        }
    if (grp == 0) {
#pragma unroll
        for (int j = 0; j < RUNS; ++j) {
            const RowParams p = load_row_params<MODE>(f, at, j);
            keep_run(w1_kept, at, j, p.w1);
            keep_run(w2_kept, at, j, p.w2);
            if (SCALED) keep_run(sc_kept, at, j, p.sc);
        }
    }
    if (ring.groups > 1) __syncthreads();           // one group: each thread reads what it wrote
    const uint64_t scale = splat2(f.scale_form == MHC_SCALE_ONE ? *f.res_scale : 1.f);

    // A wait that runs out is recorded, and the rows left go by with what the
    // stages hold: no later wait takes long, and nothing more is fetched.
    int which = 0, s = grp, filling = 0;
    bool ok = true;
    const long long row_step = static_cast<long long>(gridDim.x) * ring.groups;
    for (long long t = blockIdx.x + static_cast<long long>(grp) * gridDim.x; t < f.T; t += row_step) {
        // the columns' addresses are formed anew for each row: kept across rows, those of every
        // tensor would take the registers that hold the row
        if (MODE == ROWS_ANY) asm volatile("" : "+r"(at.thread));
        const uint8_t *const st = smem + stage0 + s * stage_bytes;
        if (STAGED)
            ok = stage_wait(&armed[s], filling, bar + 8 * s, &abort_flag, ring.timeout_ns, ring.status, SITE_FWD_ROW) && ok;
        const TY *const y_row = static_cast<const TY *>(a.y) + t * a.y_stride;
        const TR *const r_row = static_cast<const TR *>(a.residual) + t * a.r_stride;
        const uint8_t *const g_row = static_cast<const uint8_t *>(f.gate) + t * f.gate_stride * ge;
        auto load_y = [&](int j) {
            if constexpr (MODE == ROWS_RING) return staged_run<GUARD>(reinterpret_cast<const TY *>(st), at, j);
            else if constexpr (MODE == ROWS_VEC) return load_run(y_row, at, j);
            else if constexpr (MODE == ROWS_SKEW) return staged_skewed<TY>(st, skew16(y_row), at, j);
            else return staged_single(reinterpret_cast<const TY *>(st + skew16(y_row)), at, j);
        };
        auto load_r = [&](int j) {
            const uint8_t *const row = st + ring.y_place;
            if constexpr (MODE == ROWS_RING) return staged_run<GUARD>(reinterpret_cast<const TR *>(row), at, j);
            else if constexpr (MODE == ROWS_VEC) return load_run(r_row, at, j);
            else if constexpr (MODE == ROWS_SKEW) return staged_skewed<TR>(row, skew16(r_row), at, j);
            else return staged_single(reinterpret_cast<const TR *>(row + skew16(r_row)), at, j);
        };
        auto load_z = [&](int j) {
            const uint8_t *const row = st + ring.y_place + ring.r_place;
            if constexpr (MODE == ROWS_RING) return staged_run_any(row, f.gate_dtype, at, j);
            else if constexpr (MODE == ROWS_VEC) return load_run_any(g_row, f.gate_dtype, at, j);
            else if constexpr (MODE == ROWS_SKEW)
                return f.gate_dtype == MHC_F32 ? staged_skewed<float>(row, skew16(g_row), at, j)
                                               : staged_skewed<TY>(row, skew16(g_row), at, j);
            else return f.gate_dtype == MHC_F32
                            ? staged_single(reinterpret_cast<const float *>(row + skew16(g_row)), at, j)
                            : staged_single(reinterpret_cast<const TY *>(row + skew16(g_row)), at, j);
        };
        Run y[RUNS], v[RUNS];
        uint64_t s2 = 0;
#pragma unroll
        for (int j = 0; j < RUNS; ++j) {
            y[j] = load_y(j);
            v[j] = load_r(j);
        }
#pragma unroll
        for (int j = 0; j < RUNS; ++j) {
            if (!GUARD || run_in<MODE>(at, j)) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s2 = fma2(y[j].p[i], y[j].p[i], s2);
            }
            if (CKPT && a.ck_y.codes) store_ckpt<MODE>(a.ck_y, a.format, t, at, j, y[j]);
            if (CKPT && a.ck_r.codes) store_ckpt<MODE>(a.ck_r, a.format, t, at, j, v[j]);
            if (full_gate) {
                Run g = load_z(j);
                run_gate(g, f.gate_act);
#pragma unroll
                for (int i = 0; i < 4; ++i) y[j].p[i] = mul2(y[j].p[i], g.p[i]);
            }
            const Run w = kept_run(w1_kept, at, j);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[j].p[i] = mul2(y[j].p[i], w.p[i]);
            if constexpr (SCALED) {
                const Run sc = kept_run(sc_kept, at, j);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[j].p[i] = mul2(v[j].p[i], sc.p[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[j].p[i] = mul2(v[j].p[i], scale);
            }
        }
        float rstd1 = 1.f, sum[1];
        if (f.post_norm) {
            sum[0] = f2_lo(s2) + f2_hi(s2);
            group_sum<1, MAXW>(sum, red[grp][which], 1 + grp, warp, warps);
            which ^= 1;
            rstd1 = __frsqrt_rn(fmaf(sum[0], f.inv_h, f.eps_post));
        } else if (STAGED && warps > 1) {
            named_barrier_sync(1 + grp, at.threads);
        }
        if (STAGED) {
            // the row is in registers: its stage is free
            if (warps == 1) __syncwarp();
            const long long next = t + static_cast<long long>(ring.stages) * gridDim.x;
            if (at.thread == 0 && next < f.T && ok) fetch(next, s, filling + 1);
            // the group's next row: `groups` stages on, their number more than that
            s += ring.groups;
            if (s >= ring.stages) {
                s -= ring.stages;
                ++filling;
            }
        }
        float tr = rstd1;
        if (f.gate_form == MHC_GATE_TOKEN)
            tr *= gate_value(load_any(f.gate, f.gate_dtype, t * f.gate_stride), f.gate_act);
        const uint64_t tr2 = splat2(tr);
        s2 = 0;
#pragma unroll
        for (int j = 0; j < RUNS; ++j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j].p[i] = fma2(y[j].p[i], tr2, v[j].p[i]);
            if (!GUARD || run_in<MODE>(at, j)) {
#pragma unroll
                for (int i = 0; i < 4; ++i) s2 = fma2(v[j].p[i], v[j].p[i], s2);
            }
            store_run<MODE>(static_cast<TR *>(a.residual_out) + t * f.H, at, j, v[j]);
        }
        sum[0] = f2_lo(s2) + f2_hi(s2);
        group_sum<1, MAXW>(sum, red[grp][which], 1 + grp, warp, warps);
        which ^= 1;
        const float rstd2 = __frsqrt_rn(fmaf(sum[0], f.inv_h, f.eps_pre));
        const uint64_t r2 = splat2(rstd2);
#pragma unroll
        for (int j = 0; j < RUNS; ++j) {
            const Run w = kept_run(w2_kept, at, j);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[j].p[i] = mul2(mul2(v[j].p[i], r2), w.p[i]);
            store_run<MODE>(static_cast<TY *>(a.h) + t * f.H, at, j, v[j]);
            if (CKPT && a.ck_h.codes) {
                // of h as it is stored
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[j].p[i] = f2_pack(to_f32(from_f32<TY>(f2_lo(v[j].p[i]))), to_f32(from_f32<TY>(f2_hi(v[j].p[i]))));
                store_ckpt<MODE>(a.ck_h, a.format, t, at, j, v[j]);
            }
        }
        if (a.rstd && at.thread == 0) {
            a.rstd[2 * t] = rstd1;
            a.rstd[2 * t + 1] = rstd2;
        }
    }
    if (STAGED && !ok && at.thread == 0) {
        // copies that may still be in flight, before the CTA's memory goes: each
        // stage's last, in either parity
        int gave_up = 0;
        for (int k = 0; k < 2 * ring.stages; ++k)
            mbar_wait(bar + 8 * (k >> 1), k & 1, &gave_up, ring.timeout_ns, ring.status, SITE_FWD_ROW);
    }
}

template <class TY, class TR, int MODE, int RUNS, bool FULL, bool SCALED, bool CKPT>
cudaError_t fwd_launch(const BlockFwdArgs &a, const FwdRing &ring, unsigned grid, int threads, size_t smem, bool pdl,
                       cudaStream_t s) {
    static SmemGrant grant;
    auto kern = block_fwd_kernel<TY, TR, MODE, RUNS, FULL, SCALED, CKPT>;
    // with one run a thread: the kept columns of 1024 threads
    if (cudaError_t e = grant_smem(kern, grant, smem, RUNS == 1 ? 96 * 1024 : kFwdSmem)) return e;
    return launch_block_kernel(kern, grid, threads * ring.groups, smem, pdl, s, a, ring);
}

template <class TY, class TR>
cudaError_t block_fwd(const BlockFwdArgs &a, int dtype, int r_dtype, int sms, bool pdl, cudaStream_t s) {
    const BlockForm &f = a.f;
    if (f.H > 8192) return launch_block_fwd_loop(a, dtype, r_dtype, sms, pdl, s);
    const bool full = f.gate_form == MHC_GATE_FULL, scaled = f.scale_form == MHC_SCALE_CHANNEL;
    const Ckpt cks[] = {a.ck_y, a.ck_r, a.ck_h};
    // what is written and the weights allow runs of 8; the inputs too
    bool out_vec = f.H % 8 == 0 && rows_of_runs(a.residual_out, f.H, sizeof(TR), f.T) &&
                   rows_of_runs(a.h, f.H, sizeof(TY), f.T) && params_of_runs(f);
    bool ckpt = false;
    for (const Ckpt &c : cks) {
        out_vec = out_vec && (reinterpret_cast<uintptr_t>(c.codes) & 7u) == 0;
        ckpt = ckpt || c.codes;
    }
    const bool vec = out_vec && rows_of_runs(a.y, a.y_stride, sizeof(TY), f.T) &&
                     rows_of_runs(a.residual, a.r_stride, sizeof(TR), f.T) &&
                     (!full || rows_of_runs(f.gate, f.gate_stride, elem_bytes(f.gate_dtype), f.T));
    FwdRing ring = {};
    ring.groups = 1;
    const long long rows = (f.T + sms - 1) / sms;
    // one row a CTA at most: nothing to stage ahead (1 x 7168 4.5 us, staged 5.4; 64 x 2048 2.9 and 5.2)
    if (vec && (rows == 1 || f.H <= kFwdNarrow)) {
        // a thread for each run of a row; a row's warp needs no barrier
        const int threads = row_threads(f.H, 1);
        long long groups = 1024 / threads;
        if (threads > 32 && groups > kFwdGroups) groups = kFwdGroups;
        ring.groups = static_cast<int>(rows < groups ? rows : groups);
        return fwd_launch<TY, TR, ROWS_VEC, 1, true, true, true>(a, ring, static_cast<unsigned>(f.T < sms ? f.T : sms),
                                                                 threads, 3 * 32 * threads, pdl, s);
    }
    // as many groups as fit, but no more than give every SM a row
    // 32 columns a thread; with checkpoints 16, since their registers would spill (a step, forward and backward,
    // of 4096 x 4096 with an fp32 residual and e4m3 checkpoints 98.9 us, with 32 columns 109.7; with a
    // full gate 144 and 173), but where nothing does (bf16 alone) and 16 would leave one row a CTA in
    // flight (8192 x 7168 with int8 checkpoints: 275 us, with 16 columns 283).
    constexpr bool kWideCkpt = std::is_same<TR, __nv_bfloat16>::value;
    const bool wide_ckpt = kWideCkpt && !full && f.H > 4096;
    const int runs = vec && (!ckpt || wide_ckpt) ? 4 : 2, threads = row_threads(f.H, runs);
    long long groups = 512 / threads;
    if (groups > kFwdGroups) groups = kFwdGroups;
    ring.groups = static_cast<int>(rows < groups ? rows : groups);
    const unsigned grid = static_cast<unsigned>(f.T < sms ? f.T : sms);
    const size_t kept = static_cast<size_t>(vec && !full && !scaled ? 2 : 3) * 32 * runs * threads;
    ring.y_place = row_place(f.H, sizeof(TY), !vec);
    ring.r_place = row_place(f.H, sizeof(TR), !vec);
    ring.g_place = full ? row_place(f.H, elem_bytes(f.gate_dtype), !vec) : 0;
    ring.row_bytes = static_cast<uint32_t>(f.H) * (sizeof(TY) + sizeof(TR) + (full ? elem_bytes(f.gate_dtype) : 0));
    // a stage for each group and one to fill meanwhile, or all of the rows; with the widest types (96 KB a
    // row of 8192) one stage and one group
    const size_t bytes = ring.y_place + ring.r_place + ring.g_place;
    long long stages = static_cast<long long>((kFwdSmem - kept) / bytes);
    if (stages > kFwdStages) stages = kFwdStages;
    if (stages > rows) stages = rows;
    if (ring.groups >= stages) ring.groups = static_cast<int>(stages == rows || stages == 1 ? stages : stages - 1);
    ring.stages = static_cast<int>(stages);
    const size_t smem = kept + bytes * ring.stages;
    int n = 0;
    if (require_device(&n, &ring.status)) return cudaErrorUnknown;
    ring.timeout_ns = wait_timeout_ns();
    if (!out_vec)
        return ckpt ? fwd_launch<TY, TR, ROWS_ANY, 2, true, true, true>(a, ring, grid, threads, smem, pdl, s)
                    : fwd_launch<TY, TR, ROWS_ANY, 2, true, true, false>(a, ring, grid, threads, smem, pdl, s);
    if (!vec)
        return ckpt ? fwd_launch<TY, TR, ROWS_SKEW, 2, true, true, true>(a, ring, grid, threads, smem, pdl, s)
                    : fwd_launch<TY, TR, ROWS_SKEW, 2, true, true, false>(a, ring, grid, threads, smem, pdl, s);
    if (ckpt && runs == 2) {
        if (full) return fwd_launch<TY, TR, ROWS_RING, 2, true, true, true>(a, ring, grid, threads, smem, pdl, s);
        return scaled ? fwd_launch<TY, TR, ROWS_RING, 2, false, true, true>(a, ring, grid, threads, smem, pdl, s)
                      : fwd_launch<TY, TR, ROWS_RING, 2, false, false, true>(a, ring, grid, threads, smem, pdl, s);
    }
    if constexpr (kWideCkpt) {
        if (ckpt)
            return scaled ? fwd_launch<TY, TR, ROWS_RING, 4, false, true, true>(a, ring, grid, threads, smem, pdl, s)
                          : fwd_launch<TY, TR, ROWS_RING, 4, false, false, true>(a, ring, grid, threads, smem, pdl, s);
    }
    if (full) return fwd_launch<TY, TR, ROWS_RING, 4, true, true, false>(a, ring, grid, threads, smem, pdl, s);
    return scaled ? fwd_launch<TY, TR, ROWS_RING, 4, false, true, false>(a, ring, grid, threads, smem, pdl, s)
                  : fwd_launch<TY, TR, ROWS_RING, 4, false, false, false>(a, ring, grid, threads, smem, pdl, s);
}

}  // namespace
}  // namespace mhc
