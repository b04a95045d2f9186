// The product with its epilogue for up to 64 rows (the tokens of a decode step): bound by reading the
// weights once. The weights take the place of the tensor core's 128 rows and the tokens that of its
// columns, so a CTA streams 128 rows of weights (16 KB for 64 of k) beside a few KB of tokens through
// as many stages as shared memory holds. To have every SM read, the k of a tile is split over
// the CTAs of a cluster, whose sums meet in distributed shared memory, in the order of the CTAs: no
// second kernel, and the same result run to run. 1 x 7168 into 4096 bf16: 13.1 us among weights that L2 does not hold, 4.5 TB/s;
// 7168 into 7168 19, 5.4 TB/s; 64 tokens 16.6.
// Across the weights' rows (the gradient of the input, 4096 into 7168): 13.2 for a token, 14.2 for 16, 17.3 for 64.
#include <atomic>

#include "epilogue.cuh"
#include "mhc_internal.h"
#include "pair_mma.cuh"

namespace mhc {
namespace {

constexpr int kRows = 128;                          // of weights by a cluster
constexpr int kWeightBytes = 2 * kPairBoxBytes;
constexpr int kThreads = 192;                       // loads, products, four epilogue warps
constexpr int kMaxStages = 6;
constexpr int kStageBudget = 100 * 1024;             // two CTAs an SM: 1 x 7168 into 4096 15.6 -> 13.6 us, 1 x 2048 into 2048 10.0 -> 6.0
constexpr int kMaxSplit = 8;
// Steps of one sum in tensor memory, as in the other products. What an instruction cuts adds up where the products have one sign: 8 steps of
// an fp32 result lose 9e-7 of it (fp16 operands 2.8e-6, their products having more bits to be cut), 64 of a 16-bit one some 8 times that, a
// twentieth of fp16's half step. (Without a limit 65536 of k lose 4e-4, four fifths of it, and are no faster: 16 x 20000 into 20000
// 129.6 us, by 64 130.1.)
constexpr int kChainExact = 8, kChain = 64;

enum FewSite : int { SITE_F_EMPTY = 90, SITE_F_FULL, SITE_F_ACC, SITE_F_DRAIN, SITE_F_ACC_EMPTY };

struct FewArgs {
    int m, n, width;                // tokens, rows of weights, tokens rounded up to 16
    int steps, per, split, stages;  // steps of 64 of k, of a CTA, CTAs of a cluster
    int chain;                      // steps of one sum in tensor memory
    int tmem_cols, w_turned;
    uint32_t idesc;
    unsigned int *status;
    unsigned long long timeout_ns;
    EpilogueArgs e;
};

template <int KIND>
__global__ void __launch_bounds__(kThreads, 2)
few_tokens_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                  const __grid_constant__ FewArgs a) {
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    uint8_t *const basep = raw + (base - smem_addr(raw));
    const int stage_bytes = kWeightBytes + a.width * 128;
    const uint32_t bars = base + a.stages * stage_bytes;
    const uint32_t full = bars, empty = bars + 8 * kMaxStages, acc_full = bars + 16 * kMaxStages, acc_empty = acc_full + 16,
                   drain = acc_full + 32;
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(basep + a.stages * stage_bytes + 16 * kMaxStages + 40);
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    // the sums, [tokens][128], over the stages once nothing is on its way to them
    float *const sums = reinterpret_cast<float *>(basep);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int tile = blockIdx.x / a.split, rank = blockIdx.x - tile * a.split;
    // steps of 64 of k in turn: what a cluster reads at a time lies together
    const int mine = (a.steps - rank + a.split - 1) / a.split;

    if (threadIdx.x == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full + 8 * b, 1);
            mbar_init(acc_empty + 8 * b, 4);        // the epilogue warps
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&map_x);
        tma_prefetch_desc(&map_w);
    }
    if (warp == 2) {
        tmem_alloc(smem_addr(tmem_slot), a.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();

    if (warp == 0 && elect_one()) {
        const uint64_t policy = policy_evict_first();      // weights: past L2 before they come again
        int it = 0;
        bool ok = true;
        for (; it < mine; ++it) {
            const int s = it % a.stages, ph = (it / a.stages) & 1, k = (it * a.split + rank) * kPairStep;
            if (!mbar_wait(empty + 8 * s, ph ^ 1, abort_flag, a.timeout_ns, a.status, SITE_F_EMPTY)) {
                ok = false;
                break;
            }
            const uint32_t bar = full + 8 * s, dst = base + s * stage_bytes;
            mbar_arrive_expect_tx(bar, stage_bytes);
            if (a.w_turned) {
                tma_load_3d(dst, &map_w, tile * kRows, k, 0, bar, policy);
                tma_load_3d(dst + kPairBoxBytes, &map_w, tile * kRows + 64, k, 0, bar, policy);
            } else {
                tma_load_3d(dst, &map_w, k, tile * kRows, 0, bar, policy);
            }
            tma_load_3d(dst + kWeightBytes, &map_x, k, 0, 0, bar, policy);
        }
        // the last products' releases of their stages have arrived before this CTA may exit
        for (int k = it > a.stages ? it - a.stages : 0; k < it && ok; ++k)
            ok = mbar_wait(empty + 8 * (k % a.stages), (k / a.stages) & 1, abort_flag, a.timeout_ns, a.status, SITE_F_EMPTY);
        if (!ok) {
            // gave up: the copies still in flight land before this CTA exits
            int gave_up = 0;
            for (int k = it > a.stages ? it - a.stages : 0; k < it; ++k)
                mbar_wait(full + 8 * (k % a.stages), (k / a.stages) & 1, &gave_up, a.timeout_ns, a.status, SITE_F_DRAIN);
        }
    } else if (warp == 1 && elect_one()) {
        bool ok = true;
        int in_chain = 0, done = 0;
        for (int it = 0; it < mine && ok; ++it) {
            const int s = it % a.stages, buf = done & 1;
            if (in_chain == 0) ok = mbar_wait(acc_empty + 8 * buf, ((done >> 1) & 1) ^ 1, abort_flag, a.timeout_ns, a.status, SITE_F_ACC_EMPTY);
            if (ok) ok = mbar_wait(full + 8 * s, (it / a.stages) & 1, abort_flag, a.timeout_ns, a.status, SITE_F_FULL);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sw = base + s * stage_bytes, acc = tmem + buf * a.width;
            const uint64_t dw = a.w_turned ? desc_columns(sw) : desc_rows(sw), nw = a.w_turned ? 2048 >> 4 : 32 >> 4;
            const uint64_t dx = desc_rows(sw + kWeightBytes);
#pragma unroll
            for (int q = 0; q < kPairStep / 16; ++q)
                tc_mma_bf16(acc, dw + q * nw, dx + q * (32 >> 4), a.idesc, in_chain > 0 || q > 0);
            tc_commit(empty + 8 * s);
            if (++in_chain == a.chain || it + 1 == mine) {
                tc_commit(acc_full + 8 * buf);
                in_chain = 0;
                ++done;
            }
        }
        if (!ok) {
            // the products issued end before tensor memory is freed
            int gave_up = 0;
            tc_commit(drain);
            mbar_wait(drain, 0, &gave_up, a.timeout_ns, a.status, SITE_F_DRAIN);
        }
    } else if (warp >= 2) {
        const int quad = warp & 3, row = quad * 32 + lane;
        bool ok = true;
        const int live = (mine + a.chain - 1) / a.chain;
        float v[kFewTokens / 16][16] = {};
        for (int p = 0; p < live; ++p) {
            const int buf = p & 1;
            ok = mbar_wait(acc_full + 8 * buf, (p >> 1) & 1, abort_flag, a.timeout_ns, a.status, SITE_F_ACC);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int q = 0; q < kFewTokens / 16; ++q) {
                if (16 * q >= a.width) break;
                uint32_t w[16];
                tmem_ld16_now(tmem + buf * a.width + 16 * q + (static_cast<uint32_t>(quad * 32) << 16), w);
#pragma unroll
                for (int e = 0; e < 16; ++e) v[q][e] += __uint_as_float(w[e]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty + 8 * buf);
        }
        // the last sum is there: so are all, and nothing is on its way to the stages
#pragma unroll
        for (int q = 0; q < kFewTokens / 16; ++q) {
            if (16 * q >= a.width || !ok) break;
#pragma unroll
            for (int e = 0; e < 16; ++e) sums[(16 * q + e) * kRows + row] = v[q][e];
        }
        tc_fence_before();
    }
    __syncwarp();
    __syncthreads();
    __syncwarp();
    // The sums are in shared memory: no columns are held while this CTA waits for others of its cluster, which may themselves wait
    // for columns that other kernels' clusters hold.
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, a.tmem_cols);
    }
    __syncwarp();
    if (a.split > 1) cluster_sync();
    // each CTA the same rows of every token
    const int rows = kRows / a.split, r0 = rank * rows;
    if (!*abort_flag) {
        // four elements of a thread at a time, what they are combined with on its way beside the sums
        constexpr int kAtOnce = 4;
        const int shift = 31 - __clz(rows), count = a.m << shift;
        for (int q0 = threadIdx.x; q0 < count; q0 += kAtOnce * kThreads) {
            float x[kAtOnce], extra[kAtOnce], bias[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int q = q0 + u * kThreads, t = q >> shift, r = r0 + (q & (rows - 1)), j = tile * kRows + r;
                x[u] = extra[u] = bias[u] = 0.f;
                if (q >= count || j >= a.n) continue;
                if constexpr (KIND == EPI_LINEAR) {
                    if (a.e.bias) bias[u] = load_any(a.e.bias, a.e.bias_dtype, j);
                    if (a.e.residual) extra[u] = load_any(a.e.residual, a.e.residual_dtype, t * a.e.residual_stride + j);
                } else {
                    extra[u] = load_any(a.e.z, a.e.z_dtype, t * a.e.z_stride + j);
                }
                if (a.split == 1) {
                    x[u] = sums[t * kRows + r];
                } else {
                    float part[kMaxSplit];
                    const uint32_t at = smem_addr(sums + t * kRows + r);
#pragma unroll
                    for (int p = 0; p < kMaxSplit; ++p) part[p] = p < a.split ? load_at_rank(at, p) : 0.f;
#pragma unroll
                    for (int p = 0; p < kMaxSplit; ++p) x[u] += part[p];
                }
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int q = q0 + u * kThreads, t = q >> shift, j = tile * kRows + r0 + (q & (rows - 1));
                if (q >= count || j >= a.n) continue;
                const long long to = static_cast<long long>(t) * a.n + j;
                if constexpr (KIND == EPI_LINEAR) {
                    x[u] += bias[u];
                    if (a.e.z) store_any(a.e.z, a.e.z_dtype, to, x[u]);
                    with_act(a.e.act, [&](auto act) { x[u] = act_value<decltype(act)::value>(x[u]); });
                    x[u] += extra[u];
                } else {
                    with_act(a.e.act, [&](auto act) { x[u] *= act_slope<decltype(act)::value>(extra[u]); });
                }
                store_any(a.e.out, a.e.out_dtype, to, x[u]);
            }
        }
    }
    __syncwarp();
    if (a.split > 1) cluster_sync();        // no CTA's sums go while another reads them
}

std::atomic<int> g_smem[64];

}  // namespace

int launch_few_tokens(const Product &p, int sms, unsigned int *status, bool pdl, cudaStream_t s) {
    FewArgs a = {};
    a.m = static_cast<int>(p.m);
    a.n = p.n;
    a.width = (a.m + 15) / 16 * 16;
    a.steps = static_cast<int>((p.k + kPairStep - 1) / kPairStep);
    const int tiles = (p.n + kRows - 1) / kRows;
    a.split = 1;
    // also where there is nothing to split, so that more CTAs finish many tokens (512 elements of a CTA at least)
    while (a.split < kMaxSplit && 2 * a.split * tiles <= 2 * sms && (a.steps >= 2 * a.split || a.m * kRows / a.split >= 1024)) a.split *= 2;
    a.per = (a.steps + a.split - 1) / a.split;
    // Longer sums go in pieces through two places of tensor memory in turn. At
    // most 128 columns of it a CTA: two CTAs of different clusters lie on an SM, and one that waited for the other's
    // columns while its own cluster waits for it would wait for ever.
    const int most = p.exact ? kChainExact : kChain;
    a.chain = a.per > most ? most : a.per;
    a.tmem_cols = 32;
    while (a.tmem_cols < (a.per > a.chain ? 2 : 1) * a.width) a.tmem_cols *= 2;
    const int stage_bytes = kWeightBytes + a.width * 128;
    a.stages = kStageBudget / stage_bytes < kMaxStages ? kStageBudget / stage_bytes : kMaxStages;
    a.w_turned = p.b.turned;
    const uint32_t fmt = p.bf16 ? 1u : 0u;
    a.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((p.b.turned ? 1u : 0u) << 15) |
              (static_cast<uint32_t>(a.width >> 3) << 17) | (static_cast<uint32_t>(kRows >> 4) << 24);
    a.status = status;
    a.timeout_ns = wait_timeout_ns();
    a.e = p.epi;
    CUtensorMap mx, mw;
    if (!encode_matrices16(&mx, p.bf16, p.a.p, p.k, p.m, 1, p.a.pitch * 2, 0, a.width) ||
        !(p.b.turned ? encode_matrices16(&mw, p.bf16, p.b.p, p.n, p.k, 1, p.b.pitch * 2, 0, kPairStep)
                     : encode_matrices16(&mw, p.bf16, p.b.p, p.k, p.n, 1, p.b.pitch * 2, 0, kRows)))
        return MHC_ERR_CUDA;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MHC_ERR_CUDA;
    constexpr int smem_most = kStageBudget + 1024 + 16 * kMaxStages + 64;
    auto *const kern = p.kind == EPI_SLOPE ? few_tokens_kernel<EPI_SLOPE> : few_tokens_kernel<EPI_LINEAR>;
    if (!g_smem[dev & 63].load(std::memory_order_acquire)) {
        for (auto k : {few_tokens_kernel<EPI_SLOPE>, few_tokens_kernel<EPI_LINEAR>})
            if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_most) != cudaSuccess) return MHC_ERR_CUDA;
        g_smem[dev & 63].store(1, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles) * a.split);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(a.stages) * stage_bytes + 1024 + 16 * kMaxStages + 64;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(a.split);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return note_launch(cudaLaunchKernelEx(&cfg, kern, mx, mw, a));
}

}  // namespace mhc
