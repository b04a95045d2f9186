// Backward pass of the gated residual block for rows of up to 8192 columns.
//
// With D the gradient that reaches residual_out, the row needs two sums that
// follow one another: mean(d_h w2 ro) for D, then mean(g D w1 y) for d_y. D is
// linear in the first, so the second splits into two sums that need no D, and
// one reduction of three sums serves the row.
//
// Bound by memory: 12 bytes a column with 16-bit types. A thread holds 16
// columns and their sums over tokens (d_w_post, d_w_pre, d_res_scale) in
// registers for all the rows that its group of warps passes over; the rows
// to come are staged in shared memory by bulk copies. One CTA an SM, with as
// many groups as fit 16 warps; the sums leave it once, and a second kernel
// adds the CTAs' in their order.
#include "block_rows.cuh"

namespace mhc {

cudaError_t launch_block_bwd_loop(const BlockBwdArgs &a, int dtype, int r_dtype, bool pdl, int *parts, cudaStream_t s);

namespace {

constexpr int kCols = 16;
constexpr int kMaxStages = 4;
constexpr int kMaxGroups = 16;
constexpr int kMaxThreads = 512;
constexpr size_t kSmemMost = 216 * 1024;            // dynamic; the group sums take 6 KB beside it
enum BwdSite : int { SITE_BWD_ROW = 75 };

struct BwdRing {
    int groups;                                     // of a CTA, blockDim.x / groups threads each
    int stages;
    uint32_t bytes[5], stage_bytes;                 // y, residual (or their codes), d_ro, d_h, gate: of a row
    unsigned int *status;
    unsigned long long timeout_ns;
};

// act(z) and act'(z) together. The sigmoid from e = exp(-|z|): s = 1 / (1 + e) or e / (1 + e), s' = e / (1 + e)^2.
__device__ __forceinline__ void gate_both(float z, int act, float *g, float *slope) {
    *g = z;
    *slope = 1.f;
    if (act == MHC_ACT_SIGMOID) {
        const float e = expf(-fabsf(z)), s = 1.f / (1.f + e);
        *g = z >= 0.f ? s : e * s;
        *slope = e * s * s;
        if (z != z) *g = z;
    } else if (act == MHC_ACT_TANH) {
        *g = tanhf(z);
        const float e = expf(-2.f * fabsf(z)), s = 1.f / (1.f + e);
        *slope = 4.f * e * s * s;
    }
}

template <class TY, class TR, int MODE>
__global__ void __launch_bounds__(kMaxThreads, 1) block_bwd_kernel(const BlockBwdArgs a, const BwdRing ring) {
    constexpr int VEC = Runs<MODE, kCols>::kVec, RUNS = Runs<MODE, kCols>::kRuns;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ float red[kMaxGroups / 2][2][3 * 32];
    __shared__ __align__(8) uint64_t bars[kMaxGroups * kMaxStages];
    __shared__ float scale_red[32];
    __shared__ int abort_flag;
    const BlockForm &f = a.f;
    const int H = f.H, groups = (H + 31) / 32;
    const int threads = blockDim.x / ring.groups;
    const int grp = threadIdx.x / threads, tid = threadIdx.x - grp * threads;
    const int warp = tid >> 5, warps = threads >> 5;
    const bool full_gate = f.gate_form == MHC_GATE_FULL, token_gate = f.gate_form == MHC_GATE_TOKEN;
    const size_t ge = f.gate_dtype == MHC_F32 ? 4 : 2;
    // (w_post + offset) * act of a channel gate, for every column
    float *const gw = reinterpret_cast<float *>(smem);
    uint8_t *const stages = smem + (static_cast<size_t>(H) * 4 + 127) / 128 * 128 +
                            static_cast<size_t>(grp) * ring.stages * ring.stage_bytes;
    uint64_t *const bar = bars + grp * kMaxStages;

    if (MODE == ROWS_RING && threadIdx.x == 0) {
        for (int s = 0; s < kMaxGroups * kMaxStages; ++s) mbar_init(smem_addr(&bars[s]), 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    __syncthreads();
    griddep_wait();
    const long long row0 = static_cast<long long>(blockIdx.x) * ring.groups + grp;
    const long long row_step = static_cast<long long>(gridDim.x) * ring.groups;
    auto fetch = [&](long long t, int s) {          // one thread of the group
        const uint32_t b = smem_addr(&bar[s]);
        uint32_t dst = smem_addr(stages) + s * ring.stage_bytes;
        const uint64_t pol = policy_evict_first();
        mbar_arrive_expect_tx(b, ring.stage_bytes);
        bulk_load(dst, a.y ? static_cast<const void *>(static_cast<const TY *>(a.y) + t * a.y_stride)
                           : a.ck_y.codes + t * H, ring.bytes[0], b, pol);
        dst += ring.bytes[0];
        bulk_load(dst, a.residual ? static_cast<const void *>(static_cast<const TR *>(a.residual) + t * a.r_stride)
                                  : a.ck_r.codes + t * H, ring.bytes[1], b, pol);
        dst += ring.bytes[1];
        if (ring.bytes[2])
            bulk_load(dst, static_cast<const TR *>(a.d_ro) + t * a.d_ro_stride, ring.bytes[2], b, pol);
        dst += ring.bytes[2];
        bulk_load(dst, static_cast<const TY *>(a.d_h) + t * a.d_h_stride, ring.bytes[3], b, pol);
        dst += ring.bytes[3];
        if (ring.bytes[4])
            bulk_load(dst, static_cast<const uint8_t *>(f.gate) + t * f.gate_stride * ge, ring.bytes[4], b, pol);
    };
    if (MODE == ROWS_RING && tid == 0)
        for (int s = 0; s < ring.stages; ++s)
            if (row0 + s * row_step < f.T) fetch(row0 + s * row_step, s);
    for (int c = threadIdx.x; c < H; c += blockDim.x) {
        float w = weight_at(f.w_post, f.w_post_dtype, f.weight_offset, c);
        if (f.gate_form == MHC_GATE_CHANNEL) w *= gate_value(load_any(f.gate, f.gate_dtype, c), f.gate_act);
        gw[c] = w;
    }
    __syncthreads();

    int col[RUNS];
    bool in[RUNS];
    float acc0[RUNS][VEC], acc1[RUNS][VEC], acc2[RUNS][VEC], scale_sum = 0.f;
#pragma unroll
    for (int j = 0; j < RUNS; ++j) {
        col[j] = (j * threads + tid) * VEC;
        in[j] = col[j] < H;
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc0[j][e] = acc1[j][e] = acc2[j][e] = 0.f;
    }

    // What a row needs beside its columns, fetched a row ahead.
    struct Ahead {
        float rstd1, rstd2, token_z;
        uint8_t by[RUNS], br[RUNS];
    };
    auto ahead = [&](long long t) {
        Ahead n;
        n.rstd1 = n.rstd2 = n.token_z = 0.f;
        if (t >= f.T) return n;
        n.rstd1 = a.rstd[2 * t];
        n.rstd2 = a.rstd[2 * t + 1];
        if (token_gate) n.token_z = load_any(f.gate, f.gate_dtype, t * f.gate_stride);
#pragma unroll
        for (int j = 0; j < RUNS; ++j) {
            n.by[j] = n.br[j] = 0;
            if (in[j] && !a.y) n.by[j] = a.ck_y.scales[t * groups + col[j] / 32];
            if (in[j] && !a.residual) n.br[j] = a.ck_r.scales[t * groups + col[j] / 32];
        }
        return n;
    };

    int which = 0, s = 0, last = -1;
    uint32_t phase = 0;
    bool ok = true;
    Ahead next = ahead(row0);
    for (long long t = row0; t < f.T; t += row_step) {
        const Ahead now = next;
        next = ahead(t + row_step);
        const float rstd1 = f.post_norm ? now.rstd1 : 1.f, rstd2 = now.rstd2;
        float token = 1.f, token_slope = 0.f;
        if (token_gate) gate_both(now.token_z, f.gate_act, &token, &token_slope);
        const uint8_t *const st = stages + static_cast<size_t>(s) * ring.stage_bytes;
        const uint8_t *const st_r = st + ring.bytes[0], *const st_f = st_r + ring.bytes[1],
                      *const st_h = st_f + ring.bytes[2], *const st_g = st_h + ring.bytes[3];
        if (MODE == ROWS_RING)
            ok = mbar_wait(smem_addr(&bar[s]), phase, &abort_flag, ring.timeout_ns, ring.status, SITE_BWD_ROW) && ok;

        // a run's y, residual and full gate, from the stage or from memory
        auto held = [&](const Ckpt &c, const uint8_t *staged, uint32_t byte, int j, float (&v)[VEC]) {
            if constexpr (VEC == 8) {
                const uint8_t *const p = MODE == ROWS_RING ? staged + col[j] : c.codes + t * H + col[j];
                ckpt_values8(*reinterpret_cast<const uint2 *>(p), byte, a.format, v);
            } else {
                const uint32_t code = c.codes[t * H + col[j]];
                v[0] = (a.format == MHC_CKPT_E4M3 ? ckpt_value<MHC_CKPT_E4M3>(code) : ckpt_value<MHC_CKPT_INT8>(code)) *
                       ckpt_unit(byte);
            }
        };
        auto load_y = [&](int j, float (&v)[VEC]) {
            if (!a.y) held(a.ck_y, st, now.by[j], j, v);
            else load_run<VEC>(MODE == ROWS_RING ? reinterpret_cast<const TY *>(st) + col[j]
                                                 : static_cast<const TY *>(a.y) + t * a.y_stride + col[j], v);
        };
        auto load_r = [&](int j, float (&v)[VEC]) {
            if (!a.residual) held(a.ck_r, st_r, now.br[j], j, v);
            else load_run<VEC>(MODE == ROWS_RING ? reinterpret_cast<const TR *>(st_r) + col[j]
                                                 : static_cast<const TR *>(a.residual) + t * a.r_stride + col[j], v);
        };
        auto load_z = [&](int j, float (&v)[VEC]) {
            const void *const row = MODE == ROWS_RING
                ? static_cast<const void *>(st_g) : static_cast<const uint8_t *>(f.gate) + t * f.gate_stride * ge;
            load_params<VEC>(row, f.gate_dtype, col[j], v);
        };

        float sum[3] = {0.f, 0.f, 0.f};
        float ev[RUNS][VEC];                        // d_ro + rstd_pre d_h w2
#pragma unroll
        for (int j = 0; j < RUNS; ++j) {
            if (!in[j]) continue;
            float y[VEC], r[VEC], v[VEC], w[VEC], ro[VEC];
            load_y(j, y);
            load_r(j, r);
            load_run<VEC>(gw + col[j], w);
            if (full_gate) {
                load_z(j, v);
                gate_values<VEC>(v, f.gate_act);
#pragma unroll
                for (int e = 0; e < VEC; ++e) w[e] *= v[e];
            }
            load_scale<VEC>(f, col[j], v);
            const float tr = token * rstd1;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                y[e] *= w[e];                       // g w1 y, without a token's gate
                ro[e] = fmaf(y[e], tr, v[e] * r[e]);
            }
            // d_h, then d_h w2
            load_run<VEC>(MODE == ROWS_RING ? reinterpret_cast<const TY *>(st_h) + col[j]
                                            : static_cast<const TY *>(a.d_h) + t * a.d_h_stride + col[j], r);
            load_weights<VEC>(f.w_pre, f.w_pre_dtype, f.weight_offset, col[j], w);
            if (a.d_ro)
                load_run<VEC>(MODE == ROWS_RING ? reinterpret_cast<const TR *>(st_f) + col[j]
                                                : static_cast<const TR *>(a.d_ro) + t * a.d_ro_stride + col[j], v);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                acc1[j][e] = fmaf(r[e] * rstd2, ro[e], acc1[j][e]);
                const float dv = r[e] * w[e];
                ev[j][e] = fmaf(rstd2, dv, a.d_ro ? v[e] : 0.f);
                sum[0] = fmaf(dv, ro[e], sum[0]);
                sum[1] = fmaf(y[e], ev[j][e], sum[1]);
                sum[2] = fmaf(y[e], ro[e], sum[2]);
            }
        }
        group_sum<3>(sum, red[grp & (kMaxGroups / 2 - 1)][which], 1 + (grp & 7), warp, warps);
        which ^= 1;
        if (MODE == ROWS_RING) {
            // every thread of the group is past the row before: its stage is free
            if (warps == 1) __syncwarp();
            const long long ahead_row = t + (ring.stages - 1) * row_step;
            if (tid == 0 && last >= 0 && ahead_row < f.T && ok) fetch(ahead_row, last);
            last = s;
            if (++s == ring.stages) {
                s = 0;
                phase ^= 1;
            }
        }
        const float q = rstd2 * (rstd2 * (rstd2 * (sum[0] * f.inv_h)));
        const float c1 = fmaf(-q, sum[2], sum[1]);
        const float p = f.post_norm ? rstd1 * (rstd1 * (rstd1 * (token * c1 * f.inv_h))) : 0.f;
#pragma unroll
        for (int j = 0; j < RUNS; ++j) {
            if (!in[j]) continue;
            float y[VEC], v[VEC], w[VEC], o[VEC];
            const float tr = token * rstd1;
            load_y(j, y);
            load_run<VEC>(gw + col[j], w);
            load_r(j, v);
            load_scale<VEC>(f, col[j], o);
            if (full_gate) {
                float z[VEC];
                load_z(j, z);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    float g, slope;
                    gate_both(z[e], f.gate_act, &g, &slope);
                    const float u = y[e] * rstd1;
                    const float D = fmaf(-q, fmaf(g * w[e], u, o[e] * v[e]), ev[j][e]);
                    acc0[j][e] = fmaf(g * D, u, acc0[j][e]);
                    z[e] = slope * (w[e] * u * D);                                      // d_gate
                    y[e] = fmaf(-p, y[e], rstd1 * (g * w[e] * D));                      // d_y
                    ev[j][e] = D;
                }
                if (a.d_gate) {
                    if (f.gate_dtype == MHC_F32) store_run<VEC>(static_cast<float *>(a.d_gate) + t * H + col[j], z);
                    else store_run<VEC>(static_cast<TY *>(a.d_gate) + t * H + col[j], z);
                }
            } else {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float D = fmaf(-q, fmaf(y[e] * w[e], tr, o[e] * v[e]), ev[j][e]);
                    acc0[j][e] = fmaf(D * y[e], tr, acc0[j][e]);
                    y[e] = fmaf(-p, y[e], tr * (w[e] * D));
                    ev[j][e] = D;
                }
            }
            store_run<VEC>(static_cast<TY *>(a.d_y) + t * H + col[j], y);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float d = v[e] * ev[j][e];
                if (f.scale_form == MHC_SCALE_CHANNEL) acc2[j][e] += d;
                else scale_sum += d;
                o[e] *= ev[j][e];
            }
            store_run<VEC>(static_cast<TR *>(a.d_r) + t * H + col[j], o);
        }
        if (token_gate && a.d_gate && tid == 0) static_cast<float *>(a.d_gate)[t] = token_slope * rstd1 * c1;
    }
    if (MODE == ROWS_RING && !ok && tid == 0) {
        // copies that may still be in flight, before the CTA's memory goes
        int gave_up = 0;
        for (int k = 0; k < ring.stages; ++k) {
            const uint32_t b = smem_addr(&bar[k]);
            mbar_wait(b, k < s ? phase ^ 1 : phase, &gave_up, ring.timeout_ns, ring.status, SITE_BWD_ROW);
        }
    }

    // the groups' sums, one group after the other (gw's place), then out
    __syncthreads();
    float *const out = a.sums + static_cast<long long>(blockIdx.x) * kBackSums * H;
    auto leave = [&](const float (&acc)[RUNS][VEC], int k) {
        if (ring.groups == 1) {
#pragma unroll
            for (int j = 0; j < RUNS; ++j)
                if (in[j])
#pragma unroll
                    for (int e = 0; e < VEC; ++e) out[static_cast<long long>(k) * H + col[j] + e] = acc[j][e];
            return;
        }
        for (int g = 0; g < ring.groups; ++g) {
            if (g == grp)
#pragma unroll
                for (int j = 0; j < RUNS; ++j)
                    if (in[j])
#pragma unroll
                        for (int e = 0; e < VEC; ++e)
                            gw[col[j] + e] = g == 0 ? acc[j][e] : gw[col[j] + e] + acc[j][e];
            __syncthreads();
        }
        for (int c = threadIdx.x; c < H; c += blockDim.x) out[static_cast<long long>(k) * H + c] = gw[c];
        __syncthreads();
    };
    leave(acc0, 0);
    leave(acc1, 1);
    if (f.scale_form == MHC_SCALE_CHANNEL) leave(acc2, 2);
    float total[1] = {scale_sum};
    block_sum<1>(total, scale_red);
    if (threadIdx.x == 0) a.scale_sums[blockIdx.x] = total[0];
}

template <class TY, class TR, int MODE>
cudaError_t bwd_rows(const BlockBwdArgs &a, const BwdRing &ring, unsigned grid, int threads, size_t smem, bool pdl,
                     cudaStream_t s) {
    static SmemGrant grant;
    if (cudaError_t e = grant_smem(block_bwd_kernel<TY, TR, MODE>, grant, smem, kSmemMost)) return e;
    return launch_block_kernel(block_bwd_kernel<TY, TR, MODE>, grid, threads * ring.groups, smem, pdl, s, a, ring);
}

template <class TY, class TR>
cudaError_t bwd(const BlockBwdArgs &a, int dtype, int r_dtype, int sms, bool pdl, int *parts, cudaStream_t s) {
    const BlockForm &f = a.f;
    const int H = f.H;
    if (H > kCols * kMaxThreads) return launch_block_bwd_loop(a, dtype, r_dtype, pdl, parts, s);
    const bool full = f.gate_form == MHC_GATE_FULL;
    auto codes_fit = [&](const Ckpt &c) { return (reinterpret_cast<uintptr_t>(c.codes) & 15u) == 0; };
    const bool vec = H % 8 == 0 && (a.y ? rows16(a.y, a.y_stride, H, sizeof(TY), f.T) : codes_fit(a.ck_y)) &&
                     (a.residual ? rows16(a.residual, a.r_stride, H, sizeof(TR), f.T) : codes_fit(a.ck_r)) &&
                     (!a.d_ro || rows16(a.d_ro, a.d_ro_stride, H, sizeof(TR), f.T)) &&
                     rows16(a.d_h, a.d_h_stride, H, sizeof(TY), f.T) && rows16(a.d_y, H, H, sizeof(TY), f.T) &&
                     rows16(a.d_r, H, H, sizeof(TR), f.T) && params16(f) &&
                     (!full || (rows16(f.gate, f.gate_stride, H, elem_bytes(f.gate_dtype), f.T) &&
                                (!a.d_gate || rows16(a.d_gate, H, H, elem_bytes(f.gate_dtype), f.T))));
    BwdRing ring = {};
    const int threads = row_threads(H, kCols);
    // as many groups as fit, but no more than give every SM a row
    long long groups = kMaxThreads / threads, rows = (f.T + sms - 1) / sms;
    if (groups > kMaxGroups) groups = kMaxGroups;
    ring.groups = static_cast<int>(rows < groups ? rows : groups);
    const long long ctas = (f.T + ring.groups - 1) / ring.groups;
    const unsigned grid = static_cast<unsigned>(ctas < sms ? ctas : sms);
    *parts = static_cast<int>(grid);
    size_t smem = (static_cast<size_t>(H) * 4 + 127) / 128 * 128;
    if (!vec) return bwd_rows<TY, TR, ROWS_ANY>(a, ring, grid, threads, smem, pdl, s);
    ring.bytes[0] = H * (a.y ? sizeof(TY) : 1);
    ring.bytes[1] = H * (a.residual ? sizeof(TR) : 1);
    ring.bytes[2] = a.d_ro ? H * sizeof(TR) : 0;
    ring.bytes[3] = H * sizeof(TY);
    ring.bytes[4] = full ? H * elem_bytes(f.gate_dtype) : 0;
    for (uint32_t b : ring.bytes) ring.stage_bytes += b;
    const size_t room = kSmemMost - smem;
    long long stages = static_cast<long long>(room / (static_cast<size_t>(ring.stage_bytes) * ring.groups));
    if (stages > kMaxStages) stages = kMaxStages;
    // codes' rows on 16-byte boundaries, more than a row a group, and two stages at least
    const bool ringed = ((a.y && a.residual) || H % 16 == 0) && ctas > sms && stages >= 2;
    if (!ringed) return bwd_rows<TY, TR, ROWS_VEC>(a, ring, grid, threads, smem, pdl, s);
    ring.stages = static_cast<int>(stages);
    smem += static_cast<size_t>(ring.stage_bytes) * ring.groups * ring.stages;
    int n = 0;
    if (require_device(&n, &ring.status)) return cudaErrorUnknown;
    ring.timeout_ns = wait_timeout_ns();
    return bwd_rows<TY, TR, ROWS_RING>(a, ring, grid, threads, smem, pdl, s);
}

// Sums over the row kernel's CTAs, in an order that their number fixes: 32 columns a block, a warp
// every 16th CTA, the warps' sums then in turn.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(32 * kSumWarps) block_sums_kernel(const BlockSumArgs a) {
    __shared__ float part[kSumWarps][32];
    griddep_wait();
    const BlockForm &f = a.f;
    const int H = f.H, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = blockIdx.y;
    const int c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < H) {
#pragma unroll 4
        for (int p = warp; p < a.parts; p += kSumWarps)
            v += a.sums[(static_cast<long long>(p) * kBackSums + k) * H + c];
    }
    part[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < H) {
        v = 0.f;
#pragma unroll
        for (int w = 0; w < kSumWarps; ++w) v += part[w][lane];
        if (k == 0) {
            float g = 1.f, slope = 1.f;
            if (f.gate_form == MHC_GATE_CHANNEL) gate_both(load_any(f.gate, f.gate_dtype, c), f.gate_act, &g, &slope);
            if (a.d_w_post) a.d_w_post[c] = g * v;
            if (a.d_gate) a.d_gate[c] = slope * weight_at(f.w_post, f.w_post_dtype, f.weight_offset, c) * v;
        } else if (k == 1) {
            if (a.d_w_pre) a.d_w_pre[c] = v;
        } else {
            a.d_res_scale[c] = v;
        }
    }
    if (k == 0 && blockIdx.x == 0 && a.d_res_scale && f.scale_form == MHC_SCALE_ONE && warp == 1) {
        v = 0.f;
        for (int p = lane; p < a.parts; p += 32) v += a.scale_sums[p];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) a.d_res_scale[0] = v;
    }
}

}  // namespace

cudaError_t launch_block_bwd(const BlockBwdArgs &a, int dtype, int r_dtype, int sms, bool pdl, int *parts,
                             cudaStream_t s) {
    if (dtype == MHC_F32) return bwd<float, float>(a, dtype, r_dtype, sms, pdl, parts, s);
    if (dtype == MHC_BF16)
        return r_dtype == MHC_F32 ? bwd<__nv_bfloat16, float>(a, dtype, r_dtype, sms, pdl, parts, s)
                                  : bwd<__nv_bfloat16, __nv_bfloat16>(a, dtype, r_dtype, sms, pdl, parts, s);
    return r_dtype == MHC_F32 ? bwd<__half, float>(a, dtype, r_dtype, sms, pdl, parts, s)
                              : bwd<__half, __half>(a, dtype, r_dtype, sms, pdl, parts, s);
}

cudaError_t launch_block_sums(const BlockSumArgs &a, bool pdl, cudaStream_t s) {
    const unsigned kinds = a.d_res_scale && a.f.scale_form == MHC_SCALE_CHANNEL ? 3 : 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.f.H + 31) / 32), kinds);
    cfg.blockDim = dim3(32 * kSumWarps);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, block_sums_kernel, a);
}

}  // namespace mhc
