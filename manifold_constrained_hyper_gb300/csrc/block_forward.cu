// The gated residual block's boundary for rows of up to 16384 columns: a CTA
// holds a row in registers (16 columns a thread), so that y, residual and a
// full gate are read once and both norms' sums run over registers.
//
// Bound by memory: 8 bytes a column with 16-bit types (10 with a full gate).
// A row's two sums follow one another, so a CTA alone would leave memory idle
// for most of a row's time: persistent CTAs have the rows to come staged in
// shared memory by bulk copies, refilled as soon as a row is in registers.
#include "block_rows.cuh"

namespace mhc {

cudaError_t launch_block_fwd_loop(const BlockFwdArgs &a, int dtype, int r_dtype, int sms, bool pdl, cudaStream_t s);

namespace {

constexpr int kMaxStages = 4;
constexpr size_t kSmemMost = 224 * 1024;            // dynamic, of an SM
enum FwdSite : int { SITE_FWD_ROW = 70 };

struct FwdRing {
    int stages;
    uint32_t y_bytes, r_bytes, g_bytes;             // of a row; g_bytes 0: no full gate
    unsigned int *status;
    unsigned long long timeout_ns;
};

template <int FMT, int VEC>
__device__ __forceinline__ void store_ckpt(const Ckpt &c, long long t, int H, int groups, int col, bool in,
                                           const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        const uint32_t byte = ckpt_byte_quad<FMT>(v, 0xffffffffu);
        if (!in) return;
        *reinterpret_cast<uint2 *>(c.codes + t * H + col) = ckpt_codes8<FMT>(v, byte);
        if ((threadIdx.x & 3) == 0) c.scales[t * groups + col / 32] = static_cast<uint8_t>(byte);
    } else {
        uint32_t byte;
        const uint32_t code = ckpt_encode_lane<FMT>(v[0], &byte);
        if (in) c.codes[t * H + col] = static_cast<uint8_t>(code);
        if (in && (threadIdx.x & 31) == 0) c.scales[t * groups + col / 32] = static_cast<uint8_t>(byte);
    }
}
template <int VEC>
__device__ __forceinline__ void store_ckpt(const Ckpt &c, int format, long long t, int H, int groups, int col,
                                           bool in, const float (&v)[VEC]) {
    if (format == MHC_CKPT_E4M3) store_ckpt<MHC_CKPT_E4M3, VEC>(c, t, H, groups, col, in, v);
    else store_ckpt<MHC_CKPT_INT8, VEC>(c, t, H, groups, col, in, v);
}

template <class TY, class TR, int MODE, int COLS>
__global__ void __launch_bounds__(1024, 1) block_fwd_kernel(const BlockFwdArgs a, const FwdRing ring) {
    constexpr int VEC = Runs<MODE, COLS>::kVec, RUNS = Runs<MODE, COLS>::kRuns;
    extern __shared__ __align__(128) uint8_t stage[];
    __shared__ float red[2][32];
    __shared__ __align__(8) uint64_t bars[kMaxStages];
    __shared__ int abort_flag;
    const BlockForm &f = a.f;
    const int H = f.H, groups = (H + 31) / 32, threads = blockDim.x;
    const int warp = threadIdx.x >> 5, warps = threads >> 5;
    const bool full_gate = f.gate_form == MHC_GATE_FULL;
    const uint32_t stage_bytes = ring.y_bytes + ring.r_bytes + ring.g_bytes;
    const size_t ge = f.gate_dtype == MHC_F32 ? 4 : 2;

    if (MODE == ROWS_RING && threadIdx.x == 0) {
        for (int s = 0; s < ring.stages; ++s) mbar_init(smem_addr(&bars[s]), 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    griddep_wait();
    auto fetch = [&](long long t, int s) {          // one thread
        const uint32_t bar = smem_addr(&bars[s]), dst = smem_addr(stage) + s * stage_bytes;
        const uint64_t pol = policy_evict_first();
        mbar_arrive_expect_tx(bar, stage_bytes);
        bulk_load(dst, static_cast<const TY *>(a.y) + t * a.y_stride, ring.y_bytes, bar, pol);
        bulk_load(dst + ring.y_bytes, static_cast<const TR *>(a.residual) + t * a.r_stride, ring.r_bytes, bar, pol);
        if (ring.g_bytes)
            bulk_load(dst + ring.y_bytes + ring.r_bytes,
                      static_cast<const uint8_t *>(f.gate) + t * f.gate_stride * ge, ring.g_bytes, bar, pol);
    };
    if (MODE == ROWS_RING) {
        if (threadIdx.x == 0)
            for (int s = 0; s < ring.stages; ++s) {
                const long long t = blockIdx.x + static_cast<long long>(s) * gridDim.x;
                if (t < f.T) fetch(t, s);
            }
        __syncthreads();
    }

    int col[RUNS];
    bool in[RUNS];
    float w1[RUNS][VEC];                            // (w_post + offset) * act of a channel gate
#pragma unroll
    for (int j = 0; j < RUNS; ++j) {
        col[j] = (j * threads + static_cast<int>(threadIdx.x)) * VEC;
        in[j] = col[j] < H;
#pragma unroll
        for (int e = 0; e < VEC; ++e) w1[j][e] = 0.f;
        if (!in[j]) continue;
        load_weights<VEC>(f.w_post, f.w_post_dtype, f.weight_offset, col[j], w1[j]);
        if (f.gate_form == MHC_GATE_CHANNEL) {
            float g[VEC];
            load_params<VEC>(f.gate, f.gate_dtype, col[j], g);
            gate_values<VEC>(g, f.gate_act);
#pragma unroll
            for (int e = 0; e < VEC; ++e) w1[j][e] *= g[e];
        }
    }

    // A wait that runs out is recorded, and the rows left go by with what the
    // stages hold: no later wait takes long, and nothing more is fetched.
    int which = 0, s = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (long long t = blockIdx.x; t < f.T; t += gridDim.x) {
        const uint8_t *const st = stage + s * stage_bytes;
        if (MODE == ROWS_RING) {
            ok = mbar_wait(smem_addr(&bars[s]), phase, &abort_flag, ring.timeout_ns, ring.status, SITE_FWD_ROW) && ok;
        }
        float token = 1.f;
        if (f.gate_form == MHC_GATE_TOKEN)
            token = gate_value(load_any(f.gate, f.gate_dtype, t * f.gate_stride), f.gate_act);
        float y[RUNS][VEC], v[RUNS][VEC], sum[1] = {0.f};
#pragma unroll
        for (int j = 0; j < RUNS; ++j) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) y[j][e] = v[j][e] = 0.f;
            if (in[j]) {
                if (MODE == ROWS_RING) {
                    load_run<VEC>(reinterpret_cast<const TY *>(st) + col[j], y[j]);
                    load_run<VEC>(reinterpret_cast<const TR *>(st + ring.y_bytes) + col[j], v[j]);
                } else {
                    load_run<VEC>(static_cast<const TY *>(a.y) + t * a.y_stride + col[j], y[j]);
                    load_run<VEC>(static_cast<const TR *>(a.residual) + t * a.r_stride + col[j], v[j]);
                }
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) sum[0] = fmaf(y[j][e], y[j][e], sum[0]);
            if (a.ck_y.codes) store_ckpt<VEC>(a.ck_y, a.format, t, H, groups, col[j], in[j], y[j]);
            if (a.ck_r.codes) store_ckpt<VEC>(a.ck_r, a.format, t, H, groups, col[j], in[j], v[j]);
        }
        // the residual's scale, and a full gate, before the first sum: the stage is free after it
#pragma unroll
        for (int j = 0; j < RUNS; ++j) {
            if (!in[j]) continue;
            if (f.scale_form != MHC_SCALE_NONE) {
                float sc[VEC];
                load_scale<VEC>(f, col[j], sc);
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[j][e] *= sc[e];
            }
            float g[VEC];
            if (full_gate) {
                const void *const row = MODE == ROWS_RING
                    ? static_cast<const void *>(st + ring.y_bytes + ring.r_bytes)
                    : static_cast<const uint8_t *>(f.gate) + t * f.gate_stride * ge;
                load_params<VEC>(row, f.gate_dtype, col[j], g);
                gate_values<VEC>(g, f.gate_act);
            }
#pragma unroll
            for (int e = 0; e < VEC; ++e) y[j][e] *= w1[j][e] * (full_gate ? g[e] : token);
        }
        float rstd1 = 1.f;
        if (f.post_norm) {
            group_sum<1>(sum, red[which], 1, warp, warps);
            which ^= 1;
            rstd1 = __frsqrt_rn(fmaf(sum[0], f.inv_h, f.eps_post));
        } else if (MODE == ROWS_RING) {
            __syncthreads();
        }
        if (MODE == ROWS_RING) {
            if (warps == 1) __syncwarp();
            const long long next = t + static_cast<long long>(ring.stages) * gridDim.x;
            if (threadIdx.x == 0 && next < f.T && ok) fetch(next, s);
            if (++s == ring.stages) {
                s = 0;
                phase ^= 1;
            }
        }
        sum[0] = 0.f;
#pragma unroll
        for (int j = 0; j < RUNS; ++j) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                v[j][e] = fmaf(y[j][e], rstd1, v[j][e]);
                sum[0] = fmaf(v[j][e], v[j][e], sum[0]);
            }
            if (in[j]) store_run<VEC>(static_cast<TR *>(a.residual_out) + t * H + col[j], v[j]);
        }
        group_sum<1>(sum, red[which], 1, warp, warps);
        which ^= 1;
        const float rstd2 = __frsqrt_rn(fmaf(sum[0], f.inv_h, f.eps_pre));
#pragma unroll
        for (int j = 0; j < RUNS; ++j) {
            float w2[VEC];
            if (in[j]) {
                load_weights<VEC>(f.w_pre, f.w_pre_dtype, f.weight_offset, col[j], w2);
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[j][e] *= rstd2 * w2[e];
                store_run<VEC>(static_cast<TY *>(a.h) + t * H + col[j], v[j]);
            }
            if (a.ck_h.codes) {
                // of h as it is stored
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[j][e] = to_f32(from_f32<TY>(v[j][e]));
                store_ckpt<VEC>(a.ck_h, a.format, t, H, groups, col[j], in[j], v[j]);
            }
        }
        if (a.rstd && threadIdx.x == 0) {
            a.rstd[2 * t] = rstd1;
            a.rstd[2 * t + 1] = rstd2;
        }
    }
    if (MODE == ROWS_RING && !ok && threadIdx.x == 0) {
        // copies that may still be in flight, before the CTA's memory goes
        int gave_up = 0;
        for (int k = 0; k < ring.stages; ++k)
            mbar_wait(smem_addr(&bars[k]), k < s ? phase ^ 1 : phase, &gave_up, ring.timeout_ns, ring.status, SITE_FWD_ROW);
    }
}

template <class TY, class TR, int MODE, int COLS>
cudaError_t fwd_rows_by(const BlockFwdArgs &a, int sms, bool pdl, cudaStream_t s) {
    static SmemGrant grant;
    const BlockForm &f = a.f;
    const int threads = row_threads(f.H, COLS);
    // 64 registers a thread: 1024 threads of an SM
    int per_sm = 1024 / threads < 32 ? 1024 / threads : 32;
    FwdRing ring = {};
    size_t smem = 0;
    if (MODE == ROWS_RING) {
        ring.y_bytes = f.H * sizeof(TY);
        ring.r_bytes = f.H * sizeof(TR);
        ring.g_bytes = f.gate_form == MHC_GATE_FULL ? f.H * elem_bytes(f.gate_dtype) : 0;
        const size_t bytes = ring.y_bytes + ring.r_bytes + ring.g_bytes, most = kSmemMost;
        while (per_sm > 1 && most / per_sm < 2 * bytes + 1536) --per_sm;
        long long stages = static_cast<long long>((most / per_sm - 1536) / bytes);
        ring.stages = static_cast<int>(stages < 1 ? 1 : stages > kMaxStages ? kMaxStages : stages);
        smem = ring.stages * bytes;
        unsigned int *status = nullptr;
        int n = 0;
        if (require_device(&n, &status)) return cudaErrorUnknown;
        ring.status = status;
        ring.timeout_ns = wait_timeout_ns();
        if (cudaError_t e = grant_smem(block_fwd_kernel<TY, TR, MODE, COLS>, grant, smem, kSmemMost)) return e;
    }
    const long long cap = static_cast<long long>(sms) * per_sm;
    return launch_block_kernel(block_fwd_kernel<TY, TR, MODE, COLS>, static_cast<unsigned>(f.T < cap ? f.T : cap), threads,
                               smem, pdl, s, a, ring);
}

template <class TY, class TR, int MODE>
cudaError_t fwd_rows(const BlockFwdArgs &a, int sms, bool pdl, cudaStream_t s) {
    return a.f.H <= 8 * 1024 ? fwd_rows_by<TY, TR, MODE, 8>(a, sms, pdl, s) : fwd_rows_by<TY, TR, MODE, 16>(a, sms, pdl, s);
}

template <class TY, class TR>
cudaError_t fwd(const BlockFwdArgs &a, int dtype, int r_dtype, int sms, bool pdl, cudaStream_t s) {
    const BlockForm &f = a.f;
    if (f.H > 16 * 1024) return launch_block_fwd_loop(a, dtype, r_dtype, sms, pdl, s);
    const Ckpt cks[] = {a.ck_y, a.ck_r, a.ck_h};
    bool vec = f.H % 8 == 0 && rows16(a.y, a.y_stride, f.H, sizeof(TY), f.T) &&
               rows16(a.residual, a.r_stride, f.H, sizeof(TR), f.T) &&
               rows16(a.residual_out, f.H, f.H, sizeof(TR), f.T) && rows16(a.h, f.H, f.H, sizeof(TY), f.T) &&
               params16(f) &&
               (f.gate_form != MHC_GATE_FULL || rows16(f.gate, f.gate_stride, f.H, elem_bytes(f.gate_dtype), f.T));
    for (const Ckpt &c : cks) vec = vec && (reinterpret_cast<uintptr_t>(c.codes) & 7u) == 0;
    if (!vec) return fwd_rows<TY, TR, ROWS_ANY>(a, sms, pdl, s);
    // a row a CTA: nothing to fetch ahead
    if (f.T <= sms) return fwd_rows<TY, TR, ROWS_VEC>(a, sms, pdl, s);
    return fwd_rows<TY, TR, ROWS_RING>(a, sms, pdl, s);
}

}  // namespace

cudaError_t launch_block_fwd(const BlockFwdArgs &a, int dtype, int r_dtype, int sms, bool pdl, cudaStream_t s) {
    if (dtype == MHC_F32) return fwd<float, float>(a, dtype, r_dtype, sms, pdl, s);
    if (dtype == MHC_BF16)
        return r_dtype == MHC_F32 ? fwd<__nv_bfloat16, float>(a, dtype, r_dtype, sms, pdl, s)
                                  : fwd<__nv_bfloat16, __nv_bfloat16>(a, dtype, r_dtype, sms, pdl, s);
    return r_dtype == MHC_F32 ? fwd<__half, float>(a, dtype, r_dtype, sms, pdl, s)
                              : fwd<__half, __half>(a, dtype, r_dtype, sms, pdl, s);
}

}  // namespace mhc
