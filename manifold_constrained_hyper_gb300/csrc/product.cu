// Products of 16-bit matrices with an epilogue, D[i][j] = sum_k A(i, k) B(j, k), on the 5th-generation
// tensor cores: the projection, its two gradients, and the products of the orthogonalised update.
//
// A pair of CTAs (cta_group::2) forms a 256 x 256 tile of D (256 x 128 where there are few tiles): each
// loads 128 rows of A and half of the tile's of B for every 64 elements of k (32 KB, six steps in
// flight), and holds its half of the sums in tensor memory, in two buffers, so that the epilogue of
// one tile runs under the products of the next. Either operand may lie with k contiguous or outermost:
// TMA brings both into the layout that the tensor core reads, so nothing is transposed beforehand. An
// operand in two fp16 parts (hi + lo, 22 bits) takes three products a step, hi hi, hi lo and lo hi, into
// the same sums.
#include <atomic>

#include "epilogue.cuh"
#include "mhc_internal.h"
#include "pair_mma.cuh"

namespace mhc {
namespace {

constexpr int kTile = 256;
constexpr int kHalf = kTile / 2;
constexpr int kStep = kPairStep;
constexpr int kBoxBytes = kPairBoxBytes;
constexpr int kStageBytes = 4 * kBoxBytes;
constexpr int kStages = 6;
constexpr int kSumWarps = 8;                        // epilogue: two to a quadrant of tensor-memory lanes
constexpr int kThreads = 64 + 32 * kSumWarps;       // loads, products, epilogue
// Steps that tensor memory adds up by itself: the tensor cores cut what an addition shifts out, and a
// chain of 64 steps drifts by 4e-6 of the result, one of 8 by 4e-7. The epilogue adds the pieces in fp32.
constexpr int kChainExact = 8, kChain = 64;
constexpr int kBars = 2 * kStages + 5;
constexpr int kTurnBytes = kSumWarps * 32 * 33 * 4;
constexpr int kSmem = kStages * kStageBytes + 1024 + 256 + kTurnBytes;
constexpr int kTmemCols = 512;
constexpr int kBand = 8;                            // rows of tiles that are walked together

enum ProductSite : int { SITE_P_EMPTY = 80, SITE_P_FULL, SITE_P_ACC_EMPTY, SITE_P_ACC_FULL, SITE_P_DRAIN };

struct Args {
    long long m;
    int n;
    int tiles_m, tiles_n, splits, steps_per_split, steps;
    int tile_n;                     // 256 or 128
    int chain;                      // steps between two additions in registers
    int passes;                     // products a step: 1, or 3 of operands in two parts
    int symmetric;                  // tiles left of the diagonal are mirrored, not formed
    int items;
    int a_turned, b_turned;
    uint32_t idesc;
    unsigned int *status;
    unsigned long long timeout_ns;
    EpilogueArgs e;
};
struct Maps {
    CUtensorMap a[2], b[2];         // hi, lo
};
struct Place {
    int batch, split, ti, tj;
};

// Work item -> its matrix, part of the summed axis and tile. Tiles are walked in bands of kBand rows, so
// that those in flight share columns of both operands in L2; symmetric ones row by row from the diagonal.
__device__ __forceinline__ Place place_of(const Args &a, int item) {
    Place p;
    if (a.symmetric) {
        const int ratio = kTile / a.tile_n;
        const int tiles = a.tiles_m * a.tiles_n - ratio * (a.tiles_m * (a.tiles_m - 1) / 2);
        p.batch = item / tiles;
        int r = item - p.batch * tiles;
        p.split = p.ti = 0;
        while (r >= a.tiles_n - ratio * p.ti) r -= a.tiles_n - ratio * p.ti++;
        p.tj = ratio * p.ti + r;
        return p;
    }
    const int tiles = a.tiles_m * a.tiles_n, which = item / tiles;
    p.batch = which / a.splits;
    p.split = which - p.batch * a.splits;
    const int r = item - which * tiles, band = r / (kBand * a.tiles_n), first = band * kBand;
    const int rows = a.tiles_m - first < kBand ? a.tiles_m - first : kBand;
    const int q = r - band * kBand * a.tiles_n;
    p.tj = q / rows;
    p.ti = first + q - p.tj * rows;
    return p;
}

__device__ __forceinline__ uint64_t pair_of(const uint32_t (&v)[32], int e) {
    return (static_cast<uint64_t>(v[e + 1]) << 32) | v[e];
}
// PAIR: columns [j, j + 32) of row i as hi + lo; mirror: at the transposed place too, a column a store
// of 32 rows. x: the row's 16 words of hi, then of lo, where there is an x.
__device__ __forceinline__ void load_pair(Raw &x, const Args &a, int batch, long long i, int j) {
    const EpilogueArgs &e = a.e;
    if (!e.x_hi || i >= a.m) return;
    const long long at = static_cast<long long>(batch) * e.batch_stride + i * e.pitch + j;
    const Piece p = {true, a.n - j};
    Raw lo = {};
    load_raw(x, p, e.x_hi, MHC_F16, at, 0);
    load_raw(lo, p, e.x_lo, MHC_F16, at, 0);
#pragma unroll
    for (int q = 0; q < 16; ++q) x.w[16 + q] = lo.w[q];
}
__device__ __forceinline__ void finish_pair(const Args &a, int batch, long long i, int j, bool mirror, const uint32_t (&v)[32], const Raw &x) {
    const EpilogueArgs &e = a.e;
    const long long base = static_cast<long long>(batch) * e.batch_stride;
    __half *const hi = static_cast<__half *>(e.hi) + base, *const lo = static_cast<__half *>(e.lo) + base;
    const uint64_t unit = splat2(e.unit);
    uint32_t hw[16], lw[16];
#pragma unroll
    for (int q = 0; q < 16; ++q) {
        uint64_t r = mul2(pair_of(v, 2 * q), unit);
        if (e.x_hi) {
            const __half *const tag = nullptr;
            r = fma2(add2(unpack2(x.w[q], tag), unpack2(x.w[16 + q], tag)), splat2(e.of_x), r);
            // the unit matrix
            r = add2(r, f2_pack(i == j + 2 * q ? e.of_unit : 0.f, i == j + 2 * q + 1 ? e.of_unit : 0.f));
        }
        hw[q] = pack2(r, static_cast<const __half *>(nullptr));
        lw[q] = pack2(fma2(unpack2(hw[q], static_cast<const __half *>(nullptr)), splat2(-1.f), r), static_cast<const __half *>(nullptr));
    }
    if (i >= a.m) return;
    const long long at = i * e.pitch + j;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (j + 8 * c >= a.n) break;
        *reinterpret_cast<uint4 *>(hi + at + 8 * c) = make_uint4(hw[4 * c], hw[4 * c + 1], hw[4 * c + 2], hw[4 * c + 3]);
        *reinterpret_cast<uint4 *>(lo + at + 8 * c) = make_uint4(lw[4 * c], lw[4 * c + 1], lw[4 * c + 2], lw[4 * c + 3]);
    }
    if (!mirror) return;
    uint16_t *h = reinterpret_cast<uint16_t *>(hi) + j * e.pitch + i, *l = reinterpret_cast<uint16_t *>(lo) + j * e.pitch + i;
    const long long step = here(e.pitch);
#pragma unroll
    for (int q = 0; q < 32; ++q, h += step, l += step) {
        if (j + q >= a.n) break;
        *h = static_cast<uint16_t>(hw[q >> 1] >> (q & 1) * 16);
        *l = static_cast<uint16_t>(lw[q >> 1] >> (q & 1) * 16);
    }
}

template <int KIND>
__global__ void __launch_bounds__(kThreads, 1)
product_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Args a) {
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    uint8_t *const basep = raw + (base - smem_addr(raw));
    const uint32_t bars = base + kStages * kStageBytes;
    const uint32_t full = bars, empty = bars + 8 * kStages, acc_full = bars + 16 * kStages,
                   acc_empty = acc_full + 16, drain = acc_full + 32;
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(basep + kStages * kStageBytes + 8 * kBars);
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *const turn = reinterpret_cast<float *>(basep + kStages * kStageBytes + 256);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

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
        tma_prefetch_desc(&maps.a[0]);
        tma_prefetch_desc(&maps.b[0]);
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_addr(tmem_slot)), "r"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();

    if (warp == 0 && elect_one()) {
        // ------------------------------------------------ loads, either CTA its halves
        uint32_t it = 0;
        bool ok = true;
        for (int item = pair; item < a.items && ok; item += pairs) {
            const Place p = place_of(a, item);
            const int s0 = p.split * a.steps_per_split;
            const int s1 = s0 + a.steps_per_split < a.steps ? s0 + a.steps_per_split : a.steps;
            const int half = a.tile_n / 2;
            const int ci = p.ti * kTile + static_cast<int>(rank) * kHalf, cj = p.tj * a.tile_n + static_cast<int>(rank) * half;
            for (int st = s0; st < s1; ++st, ++it) {
                const uint32_t s = it % kStages, ph = (it / kStages) & 1;
                if (!mbar_wait(empty + 8 * s, ph ^ 1, abort_flag, a.timeout_ns, a.status, SITE_P_EMPTY)) {
                    ok = false;
                    break;
                }
                if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, kBoxBytes * (a.tile_n == kTile ? 8 : 6));
                const uint32_t bar = map_to_rank(full + 8 * s, 0), dst = base + s * kStageBytes, db = dst + 2 * kBoxBytes;
                int k = st * kStep, part = 0;
                if (a.passes == 3) {
                    const int kb = st / 3;
                    k = kb * kStep;
                    part = st - 3 * kb;
                }
                const CUtensorMap *const ma = &maps.a[part == 2], *const mb = &maps.b[part == 1];
                if (a.a_turned) {
                    tma_load_pair_3d(dst, ma, ci, k, p.batch, bar);
                    tma_load_pair_3d(dst + kBoxBytes, ma, ci + 64, k, p.batch, bar);
                } else {
                    tma_load_pair_3d(dst, ma, k, ci, p.batch, bar);
                }
                if (a.b_turned) {
                    tma_load_pair_3d(db, mb, cj, k, p.batch, bar);
                    if (half == kHalf) tma_load_pair_3d(db + kBoxBytes, mb, cj + 64, k, p.batch, bar);
                } else {
                    tma_load_pair_3d(db, mb, k, cj, p.batch, bar);
                }
            }
        }
        // every stage's last release has arrived before this CTA may exit
        for (uint32_t k = it > kStages ? it - kStages : 0; k < it && ok; ++k)
            ok = mbar_wait(empty + 8 * (k % kStages), (k / kStages) & 1, abort_flag, a.timeout_ns, a.status, SITE_P_EMPTY);
        if (!ok && rank == 0) {
            // gave up: both CTAs' copies still in flight land before they exit
            int gave_up = 0;
            for (uint32_t k = it > kStages ? it - kStages : 0; k < it; ++k)
                mbar_wait(full + 8 * (k % kStages), (k / kStages) & 1, &gave_up, a.timeout_ns, a.status, SITE_P_DRAIN);
        }
    } else if (warp == 1 && rank == 0 && elect_one()) {
        // ------------------------------------------------ products, the leader for both
        uint32_t it = 0, done = 0;
        bool ok = true;
        for (int item = pair; item < a.items && ok; item += pairs) {
            const Place p = place_of(a, item);
            const int s0 = p.split * a.steps_per_split;
            const int s1 = s0 + a.steps_per_split < a.steps ? s0 + a.steps_per_split : a.steps;
            for (int c0 = s0; c0 < s1 && ok; c0 += a.chain, ++done) {
                const uint32_t buf = done & 1, acc = tmem + buf * kTile;
                if (!mbar_wait(acc_empty + 8 * buf, ((done >> 1) & 1) ^ 1, abort_flag, a.timeout_ns, a.status,
                               SITE_P_ACC_EMPTY)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int c1 = c0 + a.chain < s1 ? c0 + a.chain : s1;
                for (int st = c0; st < c1; ++st, ++it) {
                    const uint32_t s = it % kStages;
                    if (!mbar_wait(full + 8 * s, (it / kStages) & 1, abort_flag, a.timeout_ns, a.status, SITE_P_FULL)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = base + s * kStageBytes, sb = sa + 2 * kBoxBytes;
                    // the next 16 elements of k: 16 rows on, or 32 bytes within the rows
                    const uint64_t da = a.a_turned ? desc_columns(sa) : desc_rows(sa), na = a.a_turned ? 2048 >> 4 : 32 >> 4;
                    const uint64_t db = a.b_turned ? desc_columns(sb) : desc_rows(sb), nb = a.b_turned ? 2048 >> 4 : 32 >> 4;
#pragma unroll
                    for (int q = 0; q < kStep / 16; ++q)
                        mma_pair(acc, da + q * na, db + q * nb, a.idesc, st > c0 || q > 0);
                    commit_pair(empty + 8 * s);
                }
                if (ok) commit_pair(acc_full + 8 * buf);
            }
        }
        if (!ok) {
            // the products issued end before tensor memory is freed
            int gave_up = 0;
            commit_pair(drain);
            mbar_wait(drain, 0, &gave_up, a.timeout_ns, a.status, SITE_P_DRAIN);
        }
    } else if (warp >= 2) {
        // ------------------------------------------------ epilogue, either CTA its 128 rows
        const int quad = warp & 3;                  // the tensor-memory lanes this warp may read
        const int width = a.tile_n / 2;             // the columns it sums: the tile's first or second half
        const int first = (warp - 2) / 4 * width;
        float *const piece = turn + (warp - 2) * 32 * 33;
        uint32_t done = 0;
        bool ok = true;
        for (int item = pair; item < a.items && ok; item += pairs) {
            const Place p = place_of(a, item);
            const int s0 = p.split * a.steps_per_split;
            const int s1 = s0 + a.steps_per_split < a.steps ? s0 + a.steps_per_split : a.steps;
            const long long i = static_cast<long long>(p.ti) * kTile + static_cast<int>(rank) * kHalf + quad * 32 + lane;
            // the output's matrices follow one another, and so do the splits' sums
            const long long row = ((static_cast<long long>(p.batch) * a.splits + p.split) * a.m + i) * a.n;
            const int j0 = p.tj * a.tile_n + first;
            auto piece_at = [&](int j) {
                if (a.e.wide) return Piece{true, i < a.m ? a.n - j : 0};
                const long long rows = a.m - (i - lane);
                return Piece{false, j + lane >= a.n ? 0 : rows < 32 ? static_cast<int>(rows) : 32};
            };
            // what the piece from column j on is combined with
            auto ahead = [&](Raw &r, float &bias, int j) {
                if constexpr (KIND == EPI_PAIR) {
                    load_pair(r, a, p.batch, i, j);
                } else {
                    const bool wide = a.e.wide;
                    if (KIND == EPI_LINEAR && a.e.bias && j + lane < a.n) bias = load_any(a.e.bias, a.e.bias_dtype, j + lane);
                    load_extra<KIND>(r, piece_at(j), a.e, wide ? i : i - lane, wide ? j : j + lane,
                                     wide ? row + j : row - static_cast<long long>(lane) * a.n + j + lane, a.n);
                }
            };
            uint64_t sum[4][16];
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 16; ++e) sum[q][e] = 0ull;
            uint32_t part = 0;
            for (int c0 = s0; c0 < s1; c0 += a.chain, ++done) {
                const uint32_t buf = done & 1;
                const bool last = c0 + a.chain >= s1;
                ok = mbar_wait(acc_full + 8 * buf, (done >> 1) & 1, abort_flag, a.timeout_ns, a.status, SITE_P_ACC_FULL);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                part = tmem + buf * kTile + first + (static_cast<uint32_t>(quad * 32) << 16);
                if (c0 > s0 || !last) {
                    // one of several pieces; the last one's place takes the sum
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (32 * q >= width) break;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t v[16];
                            tmem_ld16_now(part + 32 * q + 16 * h, v);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                sum[q][8 * h + e] = add2(sum[q][8 * h + e], (static_cast<uint64_t>(v[2 * e + 1]) << 32) | v[2 * e]);
                            if (last) tmem_st16(part + 32 * q + 16 * h, &sum[q][8 * h]);
                        }
                    }
                    if (last) tmem_st_wait();
                }
                if (last) break;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_at_rank(map_to_rank(acc_empty + 8 * buf, 0));
            }
            if (!ok) break;
            // the sums' registers are free from here on: a piece's operands are on their way while the one
            // before is finished
            Raw extra = {};
            float bias = 0.f;
            if (j0 < a.n) ahead(extra, bias, j0);
            const bool mirror = a.symmetric && p.tj * a.tile_n >= (p.ti + 1) * kTile;
#pragma unroll 1
            for (int c = 0; c < width; c += 32) {
                const int j = j0 + c;
                if (j >= a.n) break;
                uint32_t v[32];
                tmem_ld32_now(part + c, v);
                Raw next = {};
                float next_bias = 0.f;
                if (c + 32 < width && j + 32 < a.n) ahead(next, next_bias, j + 32);
                if constexpr (KIND == EPI_PAIR) {
                    finish_pair(a, p.batch, i, j, mirror, v, extra);
                } else {
                    float f[32];
                    if (a.e.wide) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(v[e]);
                    } else {
                        // rows on any boundary: turned in shared memory, then a column a lane
#pragma unroll
                        for (int e = 0; e < 32; ++e) piece[lane * 33 + e] = __uint_as_float(v[e]);
                        __syncwarp();
#pragma unroll
                        for (int e = 0; e < 32; ++e) f[e] = piece[e * 33 + lane];
                        __syncwarp();
                    }
                    finish_piece<KIND>(piece_at(j), a.e, a.e.wide ? row + j : row - static_cast<long long>(lane) * a.n + j + lane, a.n, bias, f, extra);
                }
                extra = next;
                bias = next_bias;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_at_rank(map_to_rank(acc_empty + 8 * (done & 1), 0));
            ++done;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    cluster_sync();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
}

// The splits' sums in their order, then the epilogue. VEC elements of a row a thread (8 where every row
// lies on the boundaries of runs, else 1).
template <int KIND, int VEC>
__global__ void __launch_bounds__(256) product_join_kernel(const float *parts, int splits, long long m, int n, EpilogueArgs e) {
    griddep_wait();
    const long long count = m * n, step = static_cast<long long>(gridDim.x) * 256 * VEC;
    for (long long at = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) * VEC; at < count; at += step) {
        float v[VEC] = {};
        for (int s0 = 0; s0 < splits; s0 += 4) {
            alignas(16) float w[4][VEC];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (s0 + s >= splits) break;
                const float *const p = parts + (s0 + s) * count + at;
                if constexpr (VEC == 8) {
                    *reinterpret_cast<float4 *>(w[s]) = *reinterpret_cast<const float4 *>(p);
                    *reinterpret_cast<float4 *>(w[s] + 4) = *reinterpret_cast<const float4 *>(p + 4);
                } else {
                    w[s][0] = *p;
                }
            }
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (s0 + s >= splits) break;
#pragma unroll
                for (int q = 0; q < VEC; ++q) v[q] += w[s][q];
            }
        }
        const long long i = at / n;
        const int j = static_cast<int>(at - i * n);
        if constexpr (VEC == 1) {
            finish_element<KIND>(e, i, at, j, v[0]);
        } else {
            Run r = run_of(v);
            if constexpr (KIND == EPI_LINEAR) {
                const uint64_t unit = splat2(e.unit);
                const Run b = e.bias ? load_run(e.bias, e.bias_dtype, j) : run_splat(0.f);
#pragma unroll
                for (int q = 0; q < 4; ++q) r.p[q] = add2(mul2(r.p[q], unit), b.p[q]);
                if (e.z) store_run(e.z, e.z_dtype, at, r);
                with_act(e.act, [&](auto act) {
                    constexpr int ACT = decltype(act)::value;
#pragma unroll
                    for (int q = 0; q < 4; ++q) r.p[q] = f2_pack(act_value<ACT>(f2_lo(r.p[q])), act_value<ACT>(f2_hi(r.p[q])));
                });
                if (e.residual) {
                    const Run x = load_run(e.residual, e.residual_dtype, i * e.residual_stride + j);
#pragma unroll
                    for (int q = 0; q < 4; ++q) r.p[q] = add2(r.p[q], x.p[q]);
                }
            } else if constexpr (KIND == EPI_SLOPE) {
                const Run z = load_run(e.z, e.z_dtype, i * e.z_stride + j);
                with_act(e.act, [&](auto act) {
                    constexpr int ACT = decltype(act)::value;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        r.p[q] = mul2(r.p[q], f2_pack(act_slope<ACT>(f2_lo(z.p[q])), act_slope<ACT>(f2_hi(z.p[q]))));
                });
            } else if (e.accumulate) {
                const Run x = load_run(e.out, e.out_dtype, at);
#pragma unroll
                for (int q = 0; q < 4; ++q) r.p[q] = add2(x.p[q], r.p[q]);
            }
            store_run(e.out, e.out_dtype, at, r);
        }
    }
}

// Rows of either job in runs of 8, the second job's after the first's.
__global__ void __launch_bounds__(256) copy_rows16_kernel(const CopyJob a, const CopyJob b) {
    griddep_wait();
    const long long per_a = (a.n + 7) / 8, per_b = (b.n + 7) / 8, first = a.rows * per_a, total = first + b.rows * per_b;
    for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<long long>(gridDim.x) * 256) {
        const bool second = i >= first;
        const CopyJob &job = second ? b : a;
        const long long k = second ? i - first : i, per_row = second ? per_b : per_a;
        const long long t = total < (1ll << 31) ? static_cast<unsigned>(k) / static_cast<unsigned>(per_row) : k / per_row;
        const int c = static_cast<int>(k - t * per_row) * 8;
        const uintptr_t row = reinterpret_cast<uintptr_t>(static_cast<const uint16_t *>(job.src) + t * job.stride);
        uint64_t v[2];
        load_words<2>(row + 2 * c, row + 2 * static_cast<uintptr_t>(job.n), v);
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(job.dst) + t * job.pitch + c) =
            make_uint4(static_cast<uint32_t>(v[0]), static_cast<uint32_t>(v[0] >> 32), static_cast<uint32_t>(v[1]),
                       static_cast<uint32_t>(v[1] >> 32));
    }
}

// Sums over rows: a cluster of CTAs takes 64 columns (8 lanes of 8 each, 32 rows at a time), each a share of
// the rows; their sums meet in distributed shared memory, in the order of the shares.
constexpr int kSumColumns = 64, kSumSplit = 8;
template <class T>
__global__ void __launch_bounds__(256) column_sums_kernel(const T *x, long long stride, long long rows, int n, bool runs, float *out,
                                                          int accumulate) {
    __shared__ float red[32][kSumColumns + 1], mine[kSumColumns];
    griddep_wait();
    const int rank = blockIdx.x % kSumSplit, first = blockIdx.x / kSumSplit * kSumColumns;
    const int lane = threadIdx.x & 7, row0 = threadIdx.x >> 3, c = first + lane * 8;
    const long long share = (rows + kSumSplit - 1) / kSumSplit, r0 = share * rank, r1 = r0 + share < rows ? r0 + share : rows;
    Run s = run_splat(0.f);
    if (c < n) {
        if (runs) {
#pragma unroll 8
            for (long long r = r0 + row0; r < r1; r += 32) {
                const Run v = load8(x + r * stride + c);
#pragma unroll
                for (int q = 0; q < 4; ++q) s.p[q] = add2(s.p[q], v.p[q]);
            }
        } else {
#pragma unroll 4
            for (long long r = r0 + row0; r < r1; r += 32) {
                const Run v = load8_any(x + r * stride, c, n);
#pragma unroll
                for (int q = 0; q < 4; ++q) s.p[q] = add2(s.p[q], v.p[q]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) red[row0][lane * 8 + e] = run_at(s, e);
    __syncthreads();
    if (threadIdx.x < kSumColumns) {
        float v = 0.f;
#pragma unroll
        for (int r = 0; r < 32; ++r) v += red[r][threadIdx.x];
        mine[threadIdx.x] = v;
    }
    __syncthreads();
    cluster_sync();
    constexpr int kEach = kSumColumns / kSumSplit;
    if (threadIdx.x < kEach) {
        const int k = rank * kEach + threadIdx.x;
        float part[kSumSplit], v = 0.f;
#pragma unroll
        for (int p = 0; p < kSumSplit; ++p) part[p] = load_at_rank(smem_addr(mine + k), p);
#pragma unroll
        for (int p = 0; p < kSumSplit; ++p) v += part[p];
        if (first + k < n) out[first + k] = accumulate ? out[first + k] + v : v;
    }
    __syncwarp();
    cluster_sync();         // no CTA's sums go while another reads them
}

std::atomic<int> g_smem[64];

// How a product runs.
struct Plan {
    int tile_n, tiles_m, tiles_n, steps, splits, steps_per_split;
};
// Tiles of 128 columns where those of 256 would leave half of the pairs of CTAs idle; with fewer tiles
// than pairs the summed axis is split, as many times as give every pair an item of at least 4 steps.
Plan plan_of(long long m, int n, long long k, int batch, int passes, bool symmetric, bool may_split) {
    Plan p;
    p.tiles_m = static_cast<int>((m + kTile - 1) / kTile);
    auto tiles = [&](int tile_n) {
        const long long c = (n + tile_n - 1) / tile_n, all = static_cast<long long>(p.tiles_m) * c;
        return batch * (symmetric ? all - static_cast<long long>(kTile / tile_n) * p.tiles_m * (p.tiles_m - 1) / 2 : all);
    };
    p.tile_n = tiles(kTile) <= kGridCap / 4 ? kTile / 2 : kTile;
    p.tiles_n = (n + p.tile_n - 1) / p.tile_n;
    p.steps = static_cast<int>((k + kStep - 1) / kStep) * passes;
    long long s = may_split ? kGridCap / 2 / tiles(p.tile_n) : 1;
    if (s > p.steps / 4) s = p.steps / 4;
    if (p.steps < 12 || s < 1) s = 1;
    p.steps_per_split = static_cast<int>((p.steps + s - 1) / s);
    p.splits = (p.steps + p.steps_per_split - 1) / p.steps_per_split;
    return p;
}

bool encode_operand(CUtensorMap *m, const Product &p, const Operand &o, const void *ptr, long long rows, int box_rows) {
    return o.turned ? encode_matrices16(m, p.bf16, ptr, rows, p.k, p.batch, o.pitch * 2, o.batch_stride * 2, kStep)
                    : encode_matrices16(m, p.bf16, ptr, p.k, rows, p.batch, o.pitch * 2, o.batch_stride * 2, box_rows);
}

template <int KIND>
int launch_join(const float *parts, int splits, const Product &p, int sms, bool pdl, cudaStream_t s) {
    const int vec = p.epi.wide ? 8 : 1;
    const long long need = (p.m * p.n + 256 * vec - 1) / (256 * vec), cap = static_cast<long long>(sms) * 16;
    return note_launch(launch_block_kernel(vec == 8 ? product_join_kernel<KIND, 8> : product_join_kernel<KIND, 1>,
                                           static_cast<unsigned>(need < cap ? need : cap), 256, 0, pdl, s, parts, splits, p.m, p.n,
                                           p.epi));
}

}  // namespace

size_t product_parts_bytes(long long m, int n, long long k) {
    if (m <= 0) return 0;
    const Plan q = plan_of(m, n, k, 1, 1, false, true);
    return q.splits > 1 ? static_cast<size_t>(q.splits) * m * n * 4 : 0;
}

int launch_product(const Product &p, int sms, unsigned int *status, bool pdl, cudaStream_t s) {
    if (p.k == 0) return launch_join<EPI_SUMS>(nullptr, 0, p, sms, pdl, s);
    const int passes = p.a.lo ? 3 : 1;
    const Plan q = plan_of(p.m, p.n, p.k, p.batch, passes, p.symmetric, p.parts != nullptr);
    Maps maps;
    if (!encode_operand(&maps.a[0], p, p.a, p.a.hi, p.m, kHalf) || !encode_operand(&maps.b[0], p, p.b, p.b.hi, p.n, q.tile_n / 2) ||
        !encode_operand(&maps.a[1], p, p.a, p.a.lo ? p.a.lo : p.a.hi, p.m, kHalf) ||
        !encode_operand(&maps.b[1], p, p.b, p.b.lo ? p.b.lo : p.b.hi, p.n, q.tile_n / 2))
        return MHC_ERR_CUDA;
    Args a = {};
    a.m = p.m;
    a.n = p.n;
    a.tiles_m = q.tiles_m;
    a.tiles_n = q.tiles_n;
    a.splits = q.splits;
    a.steps_per_split = q.steps_per_split;
    a.steps = q.steps;
    a.tile_n = q.tile_n;
    a.chain = p.exact ? kChainExact : kChain;
    a.passes = passes;
    a.symmetric = p.symmetric;
    const long long all = static_cast<long long>(q.tiles_m) * q.tiles_n;
    const long long items = p.symmetric ? p.batch * (all - static_cast<long long>(kTile / q.tile_n) * q.tiles_m * (q.tiles_m - 1) / 2)
                                        : p.batch * all * q.splits;
    if (items > INT32_MAX - 1024) return MHC_ERR_UNSUPPORTED;
    a.items = static_cast<int>(items);
    a.a_turned = p.a.turned;
    a.b_turned = p.b.turned;
    const uint32_t fmt = p.bf16 ? 1u : 0u;
    a.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((p.a.turned ? 1u : 0u) << 15) | ((p.b.turned ? 1u : 0u) << 16) |
              (static_cast<uint32_t>(q.tile_n >> 3) << 17) | (static_cast<uint32_t>(kTile >> 4) << 24);
    a.status = status;
    a.timeout_ns = wait_timeout_ns();
    a.e = p.epi;
    Epilogue kind = p.kind;
    if (q.splits > 1) {
        kind = EPI_SUMS;
        a.e.out = p.parts;
        a.e.out_dtype = MHC_F32;
        a.e.accumulate = 0;
        a.e.wide = p.n % 8 == 0 && (reinterpret_cast<uintptr_t>(p.parts) & 31u) == 0;
    }
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MHC_ERR_CUDA;
    void (*const kernels[])(const Maps, const Args) = {product_kernel<EPI_SUMS>, product_kernel<EPI_LINEAR>,
                                                       product_kernel<EPI_SLOPE>, product_kernel<EPI_PAIR>};
    if (!g_smem[dev & 63].load(std::memory_order_acquire)) {
        for (auto kern : kernels)
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) return MHC_ERR_CUDA;
        g_smem[dev & 63].store(1, std::memory_order_release);
    }
    const long long pairs = sms / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * static_cast<unsigned>(a.items < pairs ? a.items : pairs));
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
    if (int e = note_launch(cudaLaunchKernelEx(&cfg, kernels[kind], maps, a))) return e;
    if (q.splits == 1) return MHC_OK;
    return p.kind == EPI_SUMS     ? launch_join<EPI_SUMS>(p.parts, q.splits, p, sms, pdl, s)
           : p.kind == EPI_LINEAR ? launch_join<EPI_LINEAR>(p.parts, q.splits, p, sms, pdl, s)
                                  : launch_join<EPI_SLOPE>(p.parts, q.splits, p, sms, pdl, s);
}

cudaError_t launch_copy_rows16(const CopyJob &a, const CopyJob &b, int sms, bool pdl, cudaStream_t s) {
    const long long need = (a.rows * ((a.n + 7) / 8) + b.rows * ((b.n + 7) / 8) + 255) / 256, cap = static_cast<long long>(sms) * 8;
    return launch_block_kernel(copy_rows16_kernel, static_cast<unsigned>(need < cap ? need : cap), 256, 0, pdl, s, a, b);
}

int launch_column_sums(const void *x, long long stride, int dtype, long long rows, int n, float *out, int accumulate, bool pdl,
                       cudaStream_t s) {
    const bool runs = n % 8 == 0 && stride % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15u) == 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((n + kSumColumns - 1) / kSumColumns * kSumSplit);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kSumSplit;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return note_launch(dtype == MHC_BF16 ? cudaLaunchKernelEx(&cfg, column_sums_kernel<__nv_bfloat16>, static_cast<const __nv_bfloat16 *>(x),
                                                              stride, rows, n, runs, out, accumulate)
                                         : cudaLaunchKernelEx(&cfg, column_sums_kernel<__half>, static_cast<const __half *>(x), stride,
                                                              rows, n, runs, out, accumulate));
}

}  // namespace mhc
