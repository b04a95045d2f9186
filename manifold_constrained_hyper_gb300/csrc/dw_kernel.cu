// Weight gradient of a projection from its checkpointed input,
// d_w[i][j] = sum_t d_out[t][i] * x[t][j], on the 5th-generation tensor cores.
//
// The checkpoint's values are exact in bf16, so a first kernel writes them
// out in 16 bits (3 bytes of traffic a value) and the product runs on plain
// 16-bit operands: unpacking them inside it would convert every value once
// per 256 rows of d_w, and pass it twice more through shared memory, which
// the operands' own traffic already fills. The same kernel copies a d_out whose
// rows TMA cannot read.
//
// Both operands lie with the long axis (tokens) outermost, so a box of 64
// columns x 64 tokens lands in shared memory as 64 rows of 128 bytes and the
// MMA reads both "transposed" (the M and N axes contiguous). A pair of CTAs
// (cta_group::2) forms a 256 x 256 tile of d_w: each holds 128 columns of
// d_out and 128 of x per step of 64 tokens (32 KB, six steps in flight), and
// its half of the sums in tensor memory, in two buffers, so that what one
// holds is read and stored under the products into the other. With an fp16
// d_out (both operands of a product have one type) x goes to fp16, whose range
// does not hold a checkpoint's: every 32 columns of every piece of the sums (below)
// give up the power of two of their largest scale, which their sums get back. Where there are
// too few tiles for the machine the tokens are split, and a second kernel
// adds the splits in their order.
//
// Measured: 8192 tokens, 7168 x 4096 bf16, with the unpacking: 268 us in a burst, 1796 TFLOP/s (0.94 of a
// library product's burst rate), 300 in a long run at the power cap, 1600 (0.93 of its sustained one); with an
// fp16 d_out and an fp32 d_w 310. 4096 tokens, 2048 x 2048 fp32: 35.4 us, with an fp16 d_out 36.9: preparing x
// takes 7.8 us where unpacking it to bf16 takes 5.0.
#include <atomic>

#include "mhc_internal.h"
#include "vec_io.cuh"

namespace mhc {
namespace {

constexpr int kTile = 256;                          // rows of d_w by a pair of CTAs, and columns at most
constexpr int kHalf = kTile / 2;                    // what one CTA loads of either operand at most
constexpr int kStep = 64;                           // tokens per pipeline stage
constexpr int kBoxBytes = kStep * 128;              // 64 columns x 64 tokens, 16 bits
constexpr int kStageBytes = 4 * kBoxBytes;          // two boxes of either operand
constexpr int kStages = 6;
constexpr int kSumWarps = 8;                        // epilogue: two to a quadrant of tensor-memory lanes
constexpr int kThreads = 64 + 32 * kSumWarps;       // loads, products, epilogue
// Steps of 64 tokens that tensor memory adds up by itself. The tensor cores cut
// what an addition shifts out, so a long chain of them drifts (4096 tokens in
// one: 4.2e-6 of the result, in pieces of 16 steps 9e-7, of 8 steps 4.2e-7); the epilogue
// adds the pieces in fp32 registers, rounded to nearest, while the next piece's
// products run into the other buffer. A d_w of 16 bits is rounded by up to 2^-9 or 2^-11
// of itself at the end, so longer pieces do there.
constexpr int kChain32 = 8, kChain16 = 64;
// With fp16 operands a piece is also what shares a power of two: shorter ones for a 16-bit d_w too,
// so that preparing x has work for every SM.
constexpr int kChainF16 = 16;
constexpr int kBars = 2 * kStages + 5;
constexpr int kTurnBytes = kSumWarps * 32 * 33 * 4;         // a 32 x 32 piece of the sums for each epilogue warp
constexpr int kSmem = kStages * kStageBytes + 1024 /* alignment */ + 256 /* barriers */ + kTurnBytes;
constexpr int kTmemCols = 512;
// Rows of tiles that are walked together (8192 tokens, 4096 x 7168: 296 us; one by one 309, 4 302, 16 298).
constexpr int kBand = 8;

enum DwSite : int { SITE_DW_EMPTY = 60, SITE_DW_FULL, SITE_DW_ACC_EMPTY, SITE_DW_ACC_FULL, SITE_DW_DRAIN };

struct GemmArgs {
    long long T;
    int n, k;
    int tiles_n, tiles_k, splits, steps_per_split, steps;
    int tile_k;                     // columns of a tile: 256, or 128 for few tiles
    int chain;                      // steps between two additions in registers
    void *out;                      // d_w, or the splits' fp32 sums [splits][n][k]
    int out_dtype, accumulate, wide;    // wide: rows of out lie on 32-byte boundaries
    unsigned int *status;
    unsigned long long timeout_ns;
};
// fp16: the largest scale byte of x's groups of columns in a piece.
struct TopArgs {
    const uint8_t *top;             // [splits * pieces][groups]
    int pieces, groups, shift;      // pieces of a split at most
};

__device__ __forceinline__ void dw_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t dw_cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t dw_map_to_rank(uint32_t addr, uint32_t rank) {
    uint32_t d;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(addr), "r"(rank));
    return d;
}
__device__ __forceinline__ void arrive_at_rank(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar) : "memory");
}
// A box into this CTA's shared memory, its bytes counted at a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap *m, int c0, int c1,
                                              uint32_t cluster_bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(cluster_bar) : "memory");
}
__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}"
        ::"r"(d_tmem), "l"(ad), "l"(bd), "r"(idesc), "r"(add) : "memory");
}
// Arrive at `bar` in both CTAs when every product issued so far is done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
        ::"r"(bar), "h"(static_cast<uint16_t>(3)) : "memory");
}
// Columns contiguous, 128-byte rows in the 128-byte swizzle: 8 tokens an
// atom of 1024 bytes, the next 64 columns a box further on.
__device__ __forceinline__ uint64_t desc_columns(uint32_t addr) {
    return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | (static_cast<uint64_t>(kBoxBytes >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}
// 32, or 16, columns of this warp's 32 lanes, there when it returns.
__device__ __forceinline__ void tmem_ld32_now(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint64_t *v) {
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        w[2 * e] = static_cast<uint32_t>(v[e]);
        w[2 * e + 1] = static_cast<uint32_t>(v[e] >> 32);
    }
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};"
        ::"r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "r"(w[8]), "r"(w[9]),
          "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15]), "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_ld16_now(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr) : "memory");
}

// 2^(top - 127 - shift), what sums of fp16 operands are multiplied by; top >= 1 and shift < 23, so
// that it is subnormal at the least.
__device__ __forceinline__ float top_unit(int top, int shift) {
    const int e = top - shift;
    return __uint_as_float(e > 0 ? static_cast<uint32_t>(e) << 23 : 1u << (22 + e));
}

// Columns [j, j + 32) of one row of out on a 32-byte boundary, `row` its first
// element. k is a multiple of 8 here: groups of 8 columns are in or out as a whole.
__device__ __forceinline__ void store_row(const GemmArgs &a, long long row, int j, const uint32_t (&v)[32]) {
#pragma unroll
    for (int c = 0; c < 32; c += 8) {
        if (j + c >= a.k) break;
        Run r;
#pragma unroll
        for (int i = 0; i < 4; ++i) r.p[i] = (static_cast<uint64_t>(v[c + 2 * i + 1]) << 32) | v[c + 2 * i];
        const long long at = row + j + c;
        auto put = [&](auto *p) {
            if (a.accumulate) {
                const Run old = load8(p);
#pragma unroll
                for (int i = 0; i < 4; ++i) r.p[i] = add2(old.p[i], r.p[i]);
            }
            store8(p, r);
        };
        if (a.out_dtype == MHC_F32) put(static_cast<float *>(a.out) + at);
        else if (a.out_dtype == MHC_BF16) put(static_cast<__nv_bfloat16 *>(a.out) + at);
        else put(static_cast<__half *>(a.out) + at);
    }
}

// Work item -> tile row, tile column, split. Tiles are walked in bands of
// kBand rows, so that the tiles in flight share columns of both operands in L2.
__device__ __forceinline__ void item_place(const GemmArgs &a, int item, int *ti, int *tj, int *split) {
    const int tiles = a.tiles_n * a.tiles_k;
    *split = item / tiles;
    const int r = item - *split * tiles;
    const int band = r / (kBand * a.tiles_k), first = band * kBand;
    const int rows = a.tiles_n - first < kBand ? a.tiles_n - first : kBand;
    const int q = r - band * kBand * a.tiles_k;
    *tj = q / rows;
    *ti = first + q - *tj * rows;
}

template <bool F16>
__global__ void __launch_bounds__(kThreads, 1)
dw_gemm_kernel(const __grid_constant__ CUtensorMap map_d, const __grid_constant__ CUtensorMap map_x,
               const GemmArgs a, const TopArgs b) {
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    uint8_t *const basep = raw + (base - smem_addr(raw));
    const uint32_t bars = base + kStages * kStageBytes;
    const uint32_t full = bars, empty = bars + 8 * kStages, acc_full = bars + 16 * kStages,
                   acc_empty = acc_full + 16, drain = acc_full + 32;
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(basep + kStages * kStageBytes + 8 * kBars);
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *const turn = reinterpret_cast<float *>(basep + kStages * kStageBytes + 256);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = dw_cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int items = a.tiles_n * a.tiles_k * a.splits;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + 8 * s, 1);             // the leader's: its own announcement of both CTAs' bytes
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full + 8 * b, 1);
            mbar_init(acc_empty + 8 * b, 2 * kSumWarps);    // the leader's: the epilogue warps of either CTA
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&map_d);
        tma_prefetch_desc(&map_x);
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(tmem_slot)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    dw_cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();

    if (warp == 0 && lane == 0) {
        // ------------------------------------------------ loads, either CTA its halves
        uint32_t it = 0;
        bool ok = true;
        for (int item = pair; item < items && ok; item += pairs) {
            int ti, tj, split;
            item_place(a, item, &ti, &tj, &split);
            const int s0 = split * a.steps_per_split;
            const int s1 = s0 + a.steps_per_split < a.steps ? s0 + a.steps_per_split : a.steps;
            const int ci = ti * kTile + static_cast<int>(rank) * kHalf, cj = tj * a.tile_k + static_cast<int>(rank) * (a.tile_k / 2);
            for (int st = s0; st < s1; ++st, ++it) {
                const uint32_t s = it % kStages, ph = (it / kStages) & 1;
                if (!mbar_wait(empty + 8 * s, ph ^ 1, abort_flag, a.timeout_ns, a.status, SITE_DW_EMPTY)) {
                    ok = false;
                    break;
                }
                if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, kBoxBytes * (a.tile_k == kTile ? 8 : 6));
                const uint32_t bar = dw_map_to_rank(full + 8 * s, 0), dst = base + s * kStageBytes;
                const int t = st * kStep;
                tma_load_pair(dst, &map_d, ci, t, bar);
                tma_load_pair(dst + kBoxBytes, &map_d, ci + 64, t, bar);
                tma_load_pair(dst + 2 * kBoxBytes, &map_x, cj, t, bar);
                if (a.tile_k == kTile) tma_load_pair(dst + 3 * kBoxBytes, &map_x, cj + 64, t, bar);
            }
        }
        // every stage's last release has arrived before this CTA may exit
        for (uint32_t k = it > kStages ? it - kStages : 0; k < it && ok; ++k)
            ok = mbar_wait(empty + 8 * (k % kStages), (k / kStages) & 1, abort_flag, a.timeout_ns, a.status,
                           SITE_DW_EMPTY);
        if (!ok && rank == 0) {
            // gave up: both CTAs' copies still in flight land before they exit
            int gave_up = 0;
            for (uint32_t k = it > kStages ? it - kStages : 0; k < it; ++k)
                mbar_wait(full + 8 * (k % kStages), (k / kStages) & 1, &gave_up, a.timeout_ns, a.status, SITE_DW_DRAIN);
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ------------------------------------------------ products, the leader for both
        const uint32_t fmt = F16 ? 0u : 1u;
        const uint32_t idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | (1u << 15) | (1u << 16) |
                               (static_cast<uint32_t>(a.tile_k >> 3) << 17) | (static_cast<uint32_t>(kTile >> 4) << 24);
        uint32_t it = 0, done = 0;
        bool ok = true;
        for (int item = pair; item < items && ok; item += pairs) {
            int ti, tj, split;
            item_place(a, item, &ti, &tj, &split);
            const int s0 = split * a.steps_per_split;
            const int s1 = s0 + a.steps_per_split < a.steps ? s0 + a.steps_per_split : a.steps;
            for (int c0 = s0; c0 < s1 && ok; c0 += a.chain, ++done) {
                const uint32_t buf = done & 1, acc = tmem + buf * kTile;
                if (!mbar_wait(acc_empty + 8 * buf, ((done >> 1) & 1) ^ 1, abort_flag, a.timeout_ns, a.status,
                               SITE_DW_ACC_EMPTY)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int c1 = c0 + a.chain < s1 ? c0 + a.chain : s1;
                for (int st = c0; st < c1; ++st, ++it) {
                    const uint32_t s = it % kStages;
                    if (!mbar_wait(full + 8 * s, (it / kStages) & 1, abort_flag, a.timeout_ns, a.status, SITE_DW_FULL)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = base + s * kStageBytes, sb = sa + 2 * kBoxBytes;
#pragma unroll
                    for (int q = 0; q < kStep / 16; ++q)
                        mma_pair(acc, desc_columns(sa + q * 2048), desc_columns(sb + q * 2048), idesc, st > c0 || q > 0);
                    commit_pair(empty + 8 * s);
                }
                if (ok) commit_pair(acc_full + 8 * buf);
            }
        }
        if (!ok) {
            // the products issued end before tensor memory is freed
            int gave_up = 0;
            commit_pair(drain);
            mbar_wait(drain, 0, &gave_up, a.timeout_ns, a.status, SITE_DW_DRAIN);
        }
    } else if (warp >= 2) {
        // ------------------------------------------------ epilogue, either CTA its 128 rows
        const int quad = warp & 3;                  // the tensor-memory lanes this warp may read
        const int width = a.tile_k / 2;             // the columns it sums: the tile's first or second half
        const int first = (warp - 2) / 4 * width;
        float *const piece = turn + (warp - 2) * 32 * 33;
        uint32_t done = 0;
        bool ok = true;
        for (int item = pair; item < items && ok; item += pairs) {
            int ti, tj, split;
            item_place(a, item, &ti, &tj, &split);
            const int s0 = split * a.steps_per_split;
            const int s1 = s0 + a.steps_per_split < a.steps ? s0 + a.steps_per_split : a.steps;
            uint64_t sum[4][16];
#pragma unroll
            for (int p = 0; p < 4; ++p)
#pragma unroll
                for (int e = 0; e < 16; ++e) sum[p][e] = 0ull;
            uint32_t part = 0;
            float unit[4] = {1.f, 1.f, 1.f, 1.f};      // fp16: the power of two that each 32 columns get back
            auto more = [](uint64_t sum, uint64_t v, float u) { return F16 ? fma2(v, splat2(u), sum) : add2(sum, v); };
            for (int c0 = s0; c0 < s1; c0 += a.chain, ++done) {
                const uint32_t buf = done & 1;
                const bool last = c0 + a.chain >= s1;
                if constexpr (F16) {
                    // on their way while the products go on
                    const uint8_t *const top = b.top + static_cast<long long>(split * b.pieces + (c0 - s0) / a.chain) * b.groups;
                    const int g = (tj * a.tile_k + first) / kCkptGroup;
#pragma unroll
                    for (int p = 0; p < 4; ++p)
                        if (32 * p < width && g + p < b.groups) unit[p] = top_unit(top[g + p], b.shift);
                }
                ok = mbar_wait(acc_full + 8 * buf, (done >> 1) & 1, abort_flag, a.timeout_ns, a.status, SITE_DW_ACC_FULL);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                part = tmem + buf * kTile + first + (static_cast<uint32_t>(quad * 32) << 16);
                if (c0 > s0 || !last) {
                    // one of several pieces; the last one's place takes the sum
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        if (32 * p >= width) break;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t v[16];
                            tmem_ld16_now(part + 32 * p + 16 * h, v);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                sum[p][8 * h + e] = more(sum[p][8 * h + e], (static_cast<uint64_t>(v[2 * e + 1]) << 32) | v[2 * e], unit[p]);
                            if (last) tmem_st16(part + 32 * p + 16 * h, &sum[p][8 * h]);
                        }
                    }
                    if (last) tmem_st_wait();
                    if constexpr (F16) {
                        // the pieces' powers of two are in the sum
#pragma unroll
                        for (int p = 0; p < 4; ++p) unit[p] = 1.f;
                    }
                }
                if (last) break;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_at_rank(dw_map_to_rank(acc_empty + 8 * buf, 0));
            }
            if (!ok) break;
            const int i = ti * kTile + static_cast<int>(rank) * kHalf + quad * 32 + lane;
            const long long row = (static_cast<long long>(split) * a.n + i) * a.k;
#pragma unroll 1
            for (int c = 0; c < width; c += 32) {
                const int j = tj * a.tile_k + first + c;
                if (j >= a.k) break;
                uint32_t v[32];
                tmem_ld32_now(part + c, v);
                if constexpr (F16) {
                    const float u = c == 0 ? unit[0] : c == 32 ? unit[1] : c == 64 ? unit[2] : unit[3];
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * u);
                }
                if (a.wide) {
                    if (i < a.n) store_row(a, row, j, v);
                    continue;
                }
                // rows on any boundary: the piece turned in shared memory, then a row a store
#pragma unroll
                for (int e = 0; e < 32; ++e) piece[lane * 33 + e] = __uint_as_float(v[e]);
                __syncwarp();
                const int i0 = i - lane, rows = a.n - i0 < 32 ? a.n - i0 : 32;
                if (j + lane < a.k) {
                    const long long at = row - static_cast<long long>(lane) * a.k + j + lane;
#pragma unroll 4
                    for (int r = 0; r < rows; ++r) {
                        float x = piece[r * 33 + lane];
                        const long long q = at + static_cast<long long>(r) * a.k;
                        if (a.accumulate) x += load_any(a.out, a.out_dtype, q);
                        store_any(a.out, a.out_dtype, q, x);
                    }
                }
                __syncwarp();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_at_rank(dw_map_to_rank(acc_empty + 8 * (done & 1), 0));
            ++done;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    dw_cluster_sync();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// d_w from the splits' sums, in their order (none: zeros). VEC elements a thread (4 where the
// splits' sums lie on 16-byte boundaries, else 1), the loads of eight splits in flight: few elements of
// many splits are bound by latency.
template <int VEC>
__global__ void __launch_bounds__(256) dw_join_kernel(const float *parts, int splits, long long count, void *d_w,
                                                      int dtype, int accumulate) {
    griddep_wait();
    const long long step = static_cast<long long>(gridDim.x) * 256 * VEC;
    for (long long i = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) * VEC; i < count; i += step) {
        float v[VEC] = {};
        for (int s0 = 0; s0 < splits; s0 += 8) {
            alignas(16) float w[8][VEC];
#pragma unroll
            for (int s = 0; s < 8; ++s) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) w[s][e] = 0.f;
                if (s0 + s >= splits) continue;
                const float *const p = parts + (s0 + s) * count + i;
                if constexpr (VEC == 4) *reinterpret_cast<float4 *>(w[s]) = *reinterpret_cast<const float4 *>(p);
                else w[s][0] = *p;
            }
#pragma unroll
            for (int s = 0; s < 8; ++s)
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[e] += w[s][e];
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            store_any(d_w, dtype, i + e, accumulate ? load_any(d_w, dtype, i + e) + v[e] : v[e]);
    }
}
cudaError_t launch_join(const float *parts, int splits, long long count, void *d_w, int dtype, int accumulate, int sms, bool pdl,
                        cudaStream_t s) {
    const int vec = splits && count % 4 == 0 ? 4 : 1;
    const long long need = (count + 256 * vec - 1) / (256 * vec), cap = static_cast<long long>(sms) * 16;
    return launch_block_kernel(vec == 4 ? dw_join_kernel<4> : dw_join_kernel<1>, static_cast<unsigned>(need < cap ? need : cap), 256,
                               0, pdl, s, parts, splits, count, d_w, dtype, accumulate);
}

// The operands as the products read them: the checkpoint's values in 16 bits,
// and, where its rows do not allow 16-byte loads, d_out; each in rows on 16-byte
// boundaries. Eight columns a lane, kRuns of them in flight; past a row's
// end stands 0 (the copies above cut rows at their length).
struct PrepareArgs {
    Ckpt x;
    long long T;
    int k, n;                       // n: columns of d_out to copy, 0 where none are
    uint16_t *x16, *d16;
    long long x_pitch, d_pitch;
    const uint16_t *d_out;
    long long d_stride;
};
constexpr int kRuns = 4;
template <class T, int FMT, class I>
__global__ void __launch_bounds__(256) dw_prepare_kernel(const PrepareArgs a) {
    griddep_wait();
    const I per_x = static_cast<I>((a.k + 7) / 8), per_d = static_cast<I>((a.n + 7) / 8);
    const I total_x = static_cast<I>(a.T) * per_x, total = total_x + static_cast<I>(a.T) * per_d;
    const int groups = (a.k + 31) / 32;
    for (I i0 = static_cast<I>(blockIdx.x) * (256 * kRuns) + threadIdx.x; i0 < total;
         i0 += static_cast<I>(gridDim.x) * (256 * kRuns)) {
        uint4 w[kRuns];
        uint32_t byte[kRuns];
#pragma unroll
        for (int r = 0; r < kRuns; ++r) {
            const I i = i0 + r * 256;
            w[r] = make_uint4(0u, 0u, 0u, 0u);
            byte[r] = 0;
            if (i < total_x) {
                const I t = i / per_x;
                const int c = static_cast<int>(i - t * per_x) * 8;
                byte[r] = a.x.scales[static_cast<long long>(t) * groups + c / 32];
                const uintptr_t row = reinterpret_cast<uintptr_t>(a.x.codes) + static_cast<uintptr_t>(t) * a.k;
                uint64_t v[1];
                load_words<1>(row + c, row + a.k, v);
                w[r].x = static_cast<uint32_t>(v[0]);
                w[r].y = static_cast<uint32_t>(v[0] >> 32);
            } else if (i < total) {
                const I t = (i - total_x) / per_d;
                const int c = static_cast<int>(i - total_x - t * per_d) * 8;
                const uintptr_t row = reinterpret_cast<uintptr_t>(a.d_out + static_cast<long long>(t) * a.d_stride);
                uint64_t v[2];
                load_words<2>(row + 2 * c, row + 2 * static_cast<uintptr_t>(a.n), v);
                w[r] = make_uint4(static_cast<uint32_t>(v[0]), static_cast<uint32_t>(v[0] >> 32), static_cast<uint32_t>(v[1]),
                                  static_cast<uint32_t>(v[1] >> 32));
            }
        }
#pragma unroll
        for (int r = 0; r < kRuns; ++r) {
            const I i = i0 + r * 256;
            if (i < total_x) {
                const I t = i / per_x;
                const int c = static_cast<int>(i - t * per_x) * 8;
                const Run v = ckpt_values8(make_uint2(w[r].x, w[r].y), byte[r], FMT);
                store8(reinterpret_cast<T *>(a.x16 + static_cast<long long>(t) * a.x_pitch + c), v);
            } else if (i < total) {
                const I t = (i - total_x) / per_d;
                const int c = static_cast<int>(i - total_x - t * per_d) * 8;
                *reinterpret_cast<uint4 *>(a.d16 + static_cast<long long>(t) * a.d_pitch + c) = w[r];
            }
        }
    }
}
template <class T, int FMT>
cudaError_t launch_prepare(const PrepareArgs &a, int sms, bool pdl, cudaStream_t s) {
    const long long total = a.T * ((a.k + 7) / 8 + (a.n + 7) / 8);
    const long long need = (total + 256 * kRuns - 1) / (256 * kRuns), cap = static_cast<long long>(sms) * 8;
    return launch_block_kernel(total < (1ll << 31) ? dw_prepare_kernel<T, FMT, unsigned>
                                                   : dw_prepare_kernel<T, FMT, unsigned long long>,
                               static_cast<unsigned>(need < cap ? need : cap), 256, 0, pdl, s, a);
}

// The same with fp16 operands. A CTA takes the columns of one or two groups through the tokens of
// one piece: the largest scale byte of either first (255, not a number, left out, 1 at least), while the
// first codes are on their way, then x * 2^-(its k) * 2^shift, where the largest code is below
// fp16's largest value: 448 * 2^7, 127 * 2^9. The CTAs past x's copy d_out.
struct PieceArgs {
    int steps, steps_per_split, chain, pieces;
    int columns, column_blocks;     // of a CTA: 32 or 64; CTAs a piece
    long long x_blocks;
    uint8_t *top;
    int shift, plain;               // plain: codes on boundaries of 8
};
constexpr int kPieceTokens = kStep * kChainF16;
template <int FMT>
__global__ void __launch_bounds__(256) dw_prepare_f16_kernel(const PrepareArgs a, const PieceArgs b) {
    __shared__ uint8_t bytes[2 * kPieceTokens];
    __shared__ uint32_t red[2][8];
    griddep_wait();
    if (blockIdx.x >= b.x_blocks) {
        const long long per_d = (a.n + 7) / 8, total = a.T * per_d;
        for (long long i = (blockIdx.x - b.x_blocks) * 256 + threadIdx.x; i < total; i += (gridDim.x - b.x_blocks) * 256) {
            const long long t = i / per_d;
            const int c = static_cast<int>(i - t * per_d) * 8;
            const uintptr_t row = reinterpret_cast<uintptr_t>(a.d_out + t * a.d_stride);
            uint64_t v[2];
            load_words<2>(row + 2 * c, row + 2 * static_cast<uintptr_t>(a.n), v);
            *reinterpret_cast<uint4 *>(a.d16 + t * a.d_pitch + c) =
                make_uint4(static_cast<uint32_t>(v[0]), static_cast<uint32_t>(v[0] >> 32), static_cast<uint32_t>(v[1]),
                           static_cast<uint32_t>(v[1] >> 32));
        }
        return;
    }
    const int piece = static_cast<int>(blockIdx.x / b.column_blocks), block = static_cast<int>(blockIdx.x - static_cast<long long>(piece) * b.column_blocks);
    const int split = piece / b.pieces, s0 = split * b.steps_per_split + (piece - split * b.pieces) * b.chain;
    const int s1 = min(min(s0 + b.chain, (split + 1) * b.steps_per_split), b.steps);
    if (s0 >= s1) return;
    const long long t0 = static_cast<long long>(s0) * kStep;
    const int tokens = static_cast<int>((static_cast<long long>(s1) * kStep < a.T ? static_cast<long long>(s1) * kStep : a.T) - t0);
    const int groups = (a.k + 31) / 32, g0 = block * (b.columns / 32), mine = min(b.columns / 32, groups - g0);
    // a thread 8 columns of a token, `lanes` of them a token
    const int lanes = b.columns / 8, rows = 256 / lanes, row0 = threadIdx.x / lanes, lane = threadIdx.x - row0 * lanes;
    const int c = g0 * 32 + lane * 8, g = lane / 4;
    auto load = [&](int first, uint2 (&w)[kRuns]) {
#pragma unroll
        for (int q = 0; q < kRuns; ++q) {
            const int r = first + q * rows;
            if (r >= tokens || c >= a.k) continue;
            const uintptr_t row = reinterpret_cast<uintptr_t>(a.x.codes) + static_cast<uintptr_t>(t0 + r) * a.k;
            if (b.plain) {
                w[q] = *reinterpret_cast<const uint2 *>(row + c);
            } else {
                uint64_t v[1];
                load_words<1>(row + c, row + a.k, v);
                w[q] = make_uint2(static_cast<uint32_t>(v[0]), static_cast<uint32_t>(v[0] >> 32));
            }
        }
    };
    uint2 w[kRuns], next[kRuns];
    load(row0, w);
    uint32_t most[2] = {1u, 1u};
    for (int i = threadIdx.x; i < tokens; i += 256) {
        const uint8_t *const scales = a.x.scales + (t0 + i) * groups + g0;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (e >= mine) break;
            const uint32_t byte = scales[e];
            bytes[2 * i + e] = static_cast<uint8_t>(byte);
            if (byte != 255u) most[e] = max(most[e], byte);
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        most[e] = __reduce_max_sync(0xffffffffu, most[e]);
        if ((threadIdx.x & 31) == 0) red[e][threadIdx.x >> 5] = most[e];
    }
    __syncthreads();
    uint32_t top = 1u;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, red[g][i]);
    if (row0 == 0 && lane % 4 == 0 && g < mine) b.top[static_cast<long long>(piece) * groups + g0 + g] = static_cast<uint8_t>(top);
    const int add = b.shift + 127 - static_cast<int>(top);
    for (int first = row0; first < tokens; first += kRuns * rows) {
        load(first + kRuns * rows, next);
#pragma unroll
        for (int q = 0; q < kRuns; ++q) {
            const int r = first + q * rows;
            if (r < tokens && c < a.k) {
                // the scale byte of 2^(k - top + shift): 0 stands for 0, below all that fp16 holds of a code
                uint32_t byte = bytes[2 * r + g];
                if (byte != 255u) byte = static_cast<uint32_t>(max(static_cast<int>(byte) + add, 0));
                store8(reinterpret_cast<__half *>(a.x16 + (t0 + r) * a.x_pitch + c), ckpt_values8(w[q], byte, FMT));
            }
            w[q] = next[q];
        }
    }
}

std::atomic<int> g_dw_smem[64];

long long pitch16(int w) { return (w + 7) / 8 * 8; }
size_t up256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }

// How a call runs: the splits of the tokens and the workspace's parts.
struct DwPlan {
    int tile_k, tiles_n, tiles_k, steps, splits, steps_per_split;
    size_t x_bytes, d_bytes, part_bytes, top_bytes;
};

// Tiles of 128 columns where those of 256 would leave half of the pairs of CTAs
// idle (333 tokens into 519 x 1096 9.6 us, with 256 11.1; 154 into 1568 x 592 7.3 and 8.6). Splits: with fewer tiles
// than pairs, as many as give every pair an item of at least 4 steps (256 tokens), from 12 steps on: below,
// the second kernel costs about what the steps save (520 tokens into 2048 x 512: 11.1 us in two splits,
// 10.4 in one; 700 into 512 x 512 9.8 and 10.6; 1230 into 587 x 216 10.8 in five, 12.5 in two).
DwPlan dw_plan(long long T, int n, int k, bool d_aligned) {
    DwPlan p;
    p.tiles_n = (n + kTile - 1) / kTile;
    p.tile_k = static_cast<long long>(p.tiles_n) * ((k + kTile - 1) / kTile) <= kGridCap / 4 ? kTile / 2 : kTile;
    p.tiles_k = (k + p.tile_k - 1) / p.tile_k;
    p.steps = static_cast<int>((T + kStep - 1) / kStep);
    const long long tiles = static_cast<long long>(p.tiles_n) * p.tiles_k;
    long long s = (kGridCap / 2) / tiles;
    if (s > p.steps / 4) s = p.steps / 4;
    if (p.steps < 12) s = 1;
    if (s < 1) s = 1;
    p.steps_per_split = p.steps ? static_cast<int>((p.steps + s - 1) / s) : 0;
    p.splits = p.steps ? (p.steps + p.steps_per_split - 1) / p.steps_per_split : 0;
    p.x_bytes = up256(static_cast<size_t>(T) * pitch16(k) * 2);
    p.d_bytes = d_aligned ? 0 : up256(static_cast<size_t>(T) * pitch16(n) * 2);
    p.part_bytes = p.splits > 1 ? static_cast<size_t>(p.splits) * n * k * 4 : 0;
    p.top_bytes = static_cast<size_t>(p.splits) * ((p.steps_per_split + kChain32 - 1) / kChain32) * ckpt_groups(k);
    return p;
}

}  // namespace

bool dw_rows_aligned(const void *d_out, long long stride, long long T, int n) {
    return (reinterpret_cast<uintptr_t>(d_out) & 15u) == 0 &&
           (T == 1 || (stride % 8 == 0 && stride >= n && stride < (1ll << 38)));
}

size_t dw_workspace(long long T, int n, int k, bool d_aligned) {
    if (T == 0) return 0;
    const DwPlan p = dw_plan(T, n, k, d_aligned);
    return p.x_bytes + p.d_bytes + p.part_bytes + p.top_bytes;
}

int launch_dw(const DwArgs &a, bool d_aligned, int sms, unsigned int *status, bool pdl, cudaStream_t s) {
    const DwPlan p = dw_plan(a.T, a.n, a.k, d_aligned);
    const long long count = static_cast<long long>(a.n) * a.k;
    if (p.steps == 0) return note_launch(launch_join(nullptr, 0, count, a.d_w, a.d_w_dtype, 0, sms, pdl, s));
    uint8_t *ws = static_cast<uint8_t *>(a.workspace);
    void *const x16 = ws;
    void *const d16 = ws + p.x_bytes;
    float *const parts = reinterpret_cast<float *>(ws + p.x_bytes + p.d_bytes);
    const long long xp = pitch16(a.k), dp = d_aligned ? (a.T == 1 ? pitch16(a.n) : a.d_out_stride) : pitch16(a.n);
    const PrepareArgs u = {a.x, a.T, a.k, d_aligned ? 0 : a.n, static_cast<uint16_t *>(x16), static_cast<uint16_t *>(d16), xp,
                           pitch16(a.n), static_cast<const uint16_t *>(a.d_out), a.d_out_stride};
    // a third faster where there is nothing but runs of 8 of the checkpoint
    const bool plain = d_aligned && a.k % 8 == 0 && (reinterpret_cast<uintptr_t>(a.x.codes) & 7u) == 0, e4m3 = a.format == MHC_CKPT_E4M3;
    const CkptArgs c = {nullptr, x16, xp, a.T, a.k, a.x};
    PieceArgs b = {};
    if (a.dtype == MHC_F16) {
        b.steps = p.steps;
        b.steps_per_split = p.steps_per_split;
        b.chain = a.d_w_dtype == MHC_F32 ? kChain32 : kChainF16;
        b.pieces = (p.steps_per_split + b.chain - 1) / b.chain;
        b.top = ws + p.x_bytes + p.d_bytes + p.part_bytes;
        b.shift = e4m3 ? 7 : 9;
        b.plain = a.k % 8 == 0 && (reinterpret_cast<uintptr_t>(a.x.codes) & 7u) == 0;
        // rows of 64 bytes where that leaves CTAs for every SM
        const long long pieces = static_cast<long long>(p.splits) * b.pieces;
        b.columns = pieces * ((a.k + 63) / 64) >= 2 * sms ? 64 : 32;
        b.column_blocks = (a.k + b.columns - 1) / b.columns;
        b.x_blocks = pieces * b.column_blocks;
        const long long need = (a.T * ((u.n + 7) / 8) + 255) / 256, cap = static_cast<long long>(sms) * 8;
        const unsigned grid = static_cast<unsigned>(b.x_blocks + (need < cap ? need : cap));
        if (int e = note_launch(launch_block_kernel(e4m3 ? dw_prepare_f16_kernel<MHC_CKPT_E4M3> : dw_prepare_f16_kernel<MHC_CKPT_INT8>,
                                                    grid, 256, 0, pdl, s, u, b)))
            return e;
    } else {
        auto prepare = e4m3 ? launch_prepare<__nv_bfloat16, MHC_CKPT_E4M3> : launch_prepare<__nv_bfloat16, MHC_CKPT_INT8>;
        if (int e = note_launch(plain ? launch_ckpt_unpack(c, a.dtype, a.format, sms, pdl, s) : prepare(u, sms, pdl, s)))
            return e;
    }
    CUtensorMap md, mx;
    if (!encode_rows16(&md, a.dtype == MHC_BF16, d_aligned ? a.d_out : d16, a.n, a.T, dp * 2, kStep) ||
        !encode_rows16(&mx, a.dtype == MHC_BF16, x16, a.k, a.T, xp * 2, kStep))
        return MHC_ERR_CUDA;
    GemmArgs g = {};
    g.T = a.T;
    g.n = a.n;
    g.k = a.k;
    g.tile_k = p.tile_k;
    g.tiles_n = p.tiles_n;
    g.tiles_k = p.tiles_k;
    g.splits = p.splits;
    g.steps_per_split = p.steps_per_split;
    g.steps = p.steps;
    g.out = p.splits > 1 ? static_cast<void *>(parts) : a.d_w;
    g.out_dtype = p.splits > 1 ? MHC_F32 : a.d_w_dtype;
    g.accumulate = p.splits > 1 ? 0 : a.accumulate;
    g.chain = a.d_w_dtype == MHC_F32 ? kChain32 : a.dtype == MHC_F16 ? kChainF16 : kChain16;
    const TopArgs top = {b.top, b.pieces, static_cast<int>(ckpt_groups(a.k)), b.shift};
    g.wide = a.k % 8 == 0 && (reinterpret_cast<uintptr_t>(g.out) & 31u) == 0;
    g.status = status;
    g.timeout_ns = wait_timeout_ns();
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MHC_ERR_CUDA;
    if (!g_dw_smem[dev & 63].load(std::memory_order_acquire)) {
        for (auto kern : {dw_gemm_kernel<false>, dw_gemm_kernel<true>})
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) return MHC_ERR_CUDA;
        g_dw_smem[dev & 63].store(1, std::memory_order_release);
    }
    const long long items = static_cast<long long>(p.tiles_n) * p.tiles_k * p.splits, pairs = sms / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * static_cast<unsigned>(items < pairs ? items : pairs));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    if (int e = note_launch(cudaLaunchKernelEx(&cfg, a.dtype == MHC_F16 ? dw_gemm_kernel<true> : dw_gemm_kernel<false>, md, mx, g, top))) return e;
    if (p.splits == 1) return MHC_OK;
    return note_launch(launch_join(parts, p.splits, count, a.d_w, a.d_w_dtype, a.accumulate, sms, pdl, s));
}

}  // namespace mhc
