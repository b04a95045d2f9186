// Products of 16-bit matrices with an epilogue, D[i][j] = sum_k A(i, k) B(j, k), on the 5th-generation
// tensor cores: the projection and its two gradients.
//
// A pair of CTAs (cta_group::2) forms a 256 x 256 or 256 x 128 tile of D, or, where there are few tiles, one
// CTA a 128 x 128 or 128 x 64 one: each loads 128 rows of A and its part of the tile's of B for every 64
// elements of k (32 KB at most, six steps in flight), and holds its sums in tensor memory, in two buffers,
// so that the epilogue of one tile runs under the products of the next. Either operand may lie with k
// contiguous or outermost: TMA brings both into the layout that the tensor core reads, so nothing is
// transposed beforehand. The products are issued by an elected thread: by one that a comparison of lane
// numbers picks, each takes 80 ns, of which 256 x 256 sums hide all and 256 x 128 half (8192 x 4096 x 7168: 300 us
// against 278).
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
// Epilogue: two to a quadrant of tensor-memory lanes. With four, 96 registers a thread and five stages are left (8192 x 4096 x 7168
// 283 -> 307 us, 4195 x 254 x 1216 with gelu 28 -> 34).
constexpr int kSumWarps = 8;
constexpr int kThreads = 64 + 32 * kSumWarps;       // loads, products, epilogue
// Steps that tensor memory adds up by itself: the tensor cores cut what an addition shifts out, and a
// chain of 64 steps drifts by 4e-6 of the result, one of 8 by 4e-7 (fp16 operands, whose products have more bits to be cut, by 1e-5 and
// 1.2e-6). The epilogue adds the pieces in fp32.
constexpr int kChainExact = 8, kChain = 64;
constexpr int kBars = 2 * kStages + 5;
constexpr int kTurnBytes = kSumWarps * 32 * 32 * 4;     // a piece each, to turn it or to store it by rows
constexpr int kSmem = kStages * kStageBytes + 1024 + 256 + kTurnBytes;
constexpr int kTmemCols = 512;                      // all of it: shared memory has no room for another kernel's CTA that takes some
constexpr int kBand = 8;                            // rows of tiles that are walked together

enum ProductSite : int { SITE_P_EMPTY = 80, SITE_P_FULL, SITE_P_ACC_EMPTY, SITE_P_ACC_FULL, SITE_P_DRAIN };

struct Args {
    long long m;
    int n;
    int tiles_m, tiles_n, splits, steps_per_split, steps;
    int tile_n;                     // 256 or 128 of a pair of CTAs, 128 or 64 of one
    int chain;                      // steps between two additions in registers
    int items;
    int a_turned, b_turned;
    uint32_t idesc;
    unsigned int *status;
    unsigned long long timeout_ns;
    EpilogueArgs e;
    const void *rows;               // where the sums over k of A's rows are wanted: A [k][m], turned
    long long row_pitch, k;
    float *row_sums;
    int bf16, add_row_sums;
};
struct Place {
    int split, ti, tj;
};

// Work item -> its part of the summed axis and tile. Tiles are walked in bands of kBand rows, so that those
// in flight share columns of both operands in L2.
__device__ __forceinline__ Place place_of(const Args &a, int item) {
    const int tiles = a.tiles_m * a.tiles_n;
    Place p;
    p.split = item / tiles;
    const int r = item - p.split * tiles, band = r / (kBand * a.tiles_n), first = band * kBand;
    const int rows = a.tiles_m - first < kBand ? a.tiles_m - first : kBand;
    const int q = r - band * kBand * a.tiles_n;
    p.tj = q / rows;
    p.ti = first + q - p.tj * rows;
    return p;
}

// Sums over k of A's rows (a bias's gradient), by the epilogue's warps while the first tile's products are on: a CTA takes
// 32 of the rows, four lanes of 8, 64 of k at a time. `red`: 2 x 8 x 32 floats, the first warp's own once this returns.
template <class T>
__device__ __forceinline__ void sum_rows(const Args &a, float *red, int w, int lane) {
    const T *const x = static_cast<const T *>(a.rows);
    constexpr int kRowsAtOnce = 8 * kSumWarps;
    const int m = static_cast<int>(a.m);
    int turn = 0;
    for (int first = 32 * blockIdx.x; first < m; first += 32 * gridDim.x, turn ^= 1) {
        const int c = first + (lane & 3) * 8;
        Run s = run_splat(0.f);
        const T *from = x + (8 * w + (lane >> 2)) * a.row_pitch + c;
        long long left = a.k - 8 * w - (lane >> 2);
        // eight loads of a thread on their way at once; a run past the last column lies in its row's pitch, or past the last row in the
        // 16 bytes that hold its end, and its columns are not written
        for (; c < m && left > 0; left -= 8 * kRowsAtOnce, from += 8 * kRowsAtOnce * a.row_pitch) {
            uint4 v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                v[u] = make_uint4(0u, 0u, 0u, 0u);
                if (left > u * kRowsAtOnce) v[u] = *reinterpret_cast<const uint4 *>(from + u * kRowsAtOnce * a.row_pitch);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const Run t = unpack8(v[u], x);
#pragma unroll
                for (int q = 0; q < 4; ++q) s.p[q] = add2(s.p[q], t.p[q]);
            }
        }
        float *const here = red + turn * kSumWarps * 32;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float v = run_at(s, e);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane < 4) here[w * 32 + lane * 8 + e] = v;
        }
        named_barrier_sync(1, kSumWarps * 32);
        if (w == 0 && first + lane < m) {
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < kSumWarps; ++k) v += here[k * 32 + lane];
            float *const to = a.row_sums + first + lane;
            *to = a.add_row_sums ? *to + v : v;
        }
    }
    __syncwarp();
}

template <int KIND, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const __grid_constant__ Args a) {
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    uint8_t *const basep = raw + (base - smem_addr(raw));
    const uint32_t bars = base + kStages * kStageBytes + kTurnBytes;
    const uint32_t full = bars, empty = bars + 8 * kStages, acc_full = bars + 16 * kStages,
                   acc_empty = acc_full + 16, drain = acc_full + 32;
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(basep + (bars - base) + 8 * kBars);
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    float *const turn = reinterpret_cast<float *>(basep + kStages * kStageBytes);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    constexpr int kCtas = PAIR ? 2 : 1, kRows = kCtas * kHalf;      // of a tile
    const uint32_t rank = PAIR ? cluster_rank() : 0;
    const int pair = blockIdx.x / kCtas, pairs = gridDim.x / kCtas;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + 8 * s, 1);             // the leader's: its own announcement of both CTAs' bytes
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full + 8 * b, 1);
            mbar_init(acc_empty + 8 * b, kCtas * kSumWarps);    // the leader's: the epilogue warps of either CTA
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&map_a);
        tma_prefetch_desc(&map_b);
    }
    if (warp == 2) {
        unit_tmem_alloc<PAIR>(smem_addr(tmem_slot), kTmemCols);
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (PAIR) cluster_sync();
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
            const int half = a.tile_n / kCtas;
            const int ci = p.ti * kRows + static_cast<int>(rank) * kHalf, cj = p.tj * a.tile_n + static_cast<int>(rank) * half;
            for (int st = s0; st < s1; ++st, ++it) {
                const uint32_t s = it % kStages, ph = (it / kStages) & 1;
                if (!mbar_wait(empty + 8 * s, ph ^ 1, abort_flag, a.timeout_ns, a.status, SITE_P_EMPTY)) {
                    ok = false;
                    break;
                }
                if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, kCtas * (2 * kBoxBytes + half * 128));
                const uint32_t bar = PAIR ? map_to_rank(full + 8 * s, 0) : full + 8 * s, dst = base + s * kStageBytes, db = dst + 2 * kBoxBytes;
                const int k = st * kStep;
                if (a.a_turned) {
                    unit_load<PAIR>(dst, &map_a, ci, k, bar);
                    unit_load<PAIR>(dst + kBoxBytes, &map_a, ci + 64, k, bar);
                } else {
                    unit_load<PAIR>(dst, &map_a, k, ci, bar);
                }
                if (a.b_turned) {
                    unit_load<PAIR>(db, &map_b, cj, k, bar);
                    if (half == kHalf) unit_load<PAIR>(db + kBoxBytes, &map_b, cj + 64, k, bar);
                } else {
                    unit_load<PAIR>(db, &map_b, k, cj, bar);
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
                        unit_multiply<PAIR>(acc, da + q * na, db + q * nb, a.idesc, st > c0 || q > 0);
                    unit_commit<PAIR>(empty + 8 * s);
                }
                if (ok) unit_commit<PAIR>(acc_full + 8 * buf);
            }
        }
        if (!ok) {
            // the products issued end before tensor memory is freed
            int gave_up = 0;
            unit_commit<PAIR>(drain);
            mbar_wait(drain, 0, &gave_up, a.timeout_ns, a.status, SITE_P_DRAIN);
        }
    } else if (warp >= 2) {
        // ------------------------------------------------ epilogue, either CTA its 128 rows
        const int quad = warp & 3;                  // the tensor-memory lanes this warp may read
        const int width = a.tile_n / 2;             // the columns it sums: the tile's first or second half
        const int first = (warp - 2) / 4 * width;
        float *const piece = turn + (warp - 2) * 32 * 32;
        if constexpr (KIND == EPI_SUMS) {
            if (a.row_sums) {
                if (a.bf16) sum_rows<__nv_bfloat16>(a, turn, warp - 2, lane);
                else sum_rows<__half>(a, turn, warp - 2, lane);
            }
        }
        uint32_t done = 0;
        bool ok = true;
        for (int item = pair; item < a.items && ok; item += pairs) {
            const Place p = place_of(a, item);
            const int s0 = p.split * a.steps_per_split;
            const int s1 = s0 + a.steps_per_split < a.steps ? s0 + a.steps_per_split : a.steps;
            const long long i0 = static_cast<long long>(p.ti) * kRows + static_cast<int>(rank) * kHalf + quad * 32;
            const long long row = (p.split * a.m + i0) * a.n;    // the splits' sums follow one another
            const int j0 = p.tj * a.tile_n + first, rows = a.m - i0 >= 32 ? 32 : a.m > i0 ? static_cast<int>(a.m - i0) : 0;
            const bool wide = a.e.wide;
            const uint32_t buf = smem_addr(piece);
            auto piece_at = [&](int j) {
                if (wide) return Piece{true, rows, a.n - j};
                return Piece{false, j + lane >= a.n ? 0 : rows, 1};
            };
            // what the piece from column j on is combined with
            auto ahead = [&](Raw &r, float &bias, int j) {
                if (KIND == EPI_LINEAR && a.e.bias && j + lane < a.n) bias = load_any(a.e.bias, a.e.bias_dtype, j + lane);
                load_extra<KIND>(r, piece_at(j), a.e, i0, wide ? j : j + lane, row + (wide ? j : j + lane), a.n);
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
                if (lane == 0) unit_arrive<PAIR>(acc_empty + 8 * buf);
            }
            if (!ok) break;
// the sums' registers are free from here on: a piece's operands are on their way while the one before is finished
            Raw extra = {};
            float bias = 0.f;
            if (j0 < a.n) ahead(extra, bias, j0);
#pragma unroll 1
            for (int c = 0; c < width; c += 32) {
                const int j = j0 + c;
                if (j >= a.n) break;
                Raw next = {};
                float next_bias = 0.f;
                if (c + 32 < width && j + 32 < a.n) ahead(next, next_bias, j + 32);
                if constexpr (KIND == EPI_SUMS) {
                    if (wide) {
                        finish_sums(piece_at(j), a.e, row + j, a.n, part + c, extra, buf, [](uint32_t at, uint32_t (&u)[16]) { tmem_ld16_now(at, u); });
                        extra = next;
                        continue;
                    }
                }
                uint32_t v[32];
                tmem_ld32_now(part + c, v);
                float f[32];
                if (KIND != EPI_SUMS && wide) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(v[e]);
                } else {
                    // rows on any boundary: turned in shared memory, then a column a lane
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 32; ++e) piece[lane * 32 + (e ^ lane)] = __uint_as_float(v[e]);
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 32; ++e) f[e] = piece[e * 32 + (lane ^ e)];
                }
                finish_piece<KIND>(piece_at(j), a.e, row + (wide ? j : j + lane), a.n, bias, f, extra, buf);
                extra = next;
                bias = next_bias;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) unit_arrive<PAIR>(acc_empty + 8 * (done & 1));
            ++done;
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    if constexpr (PAIR) cluster_sync();
    if (warp == 2) unit_tmem_free<PAIR>(tmem, kTmemCols);
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
                if (e.bias) {
                    const Run b = load_run(e.bias, e.bias_dtype, j);
#pragma unroll
                    for (int q = 0; q < 4; ++q) r.p[q] = add2(r.p[q], b.p[q]);
                }
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

// Rows of either job in runs of 8, the second job's after the first's, by `blocks` CTAs of 256 threads.
__device__ __forceinline__ void copy_rows(const CopyJob &a, const CopyJob &b, int block, int blocks) {
    const long long per_a = (a.n + 7) / 8, per_b = (b.n + 7) / 8, first = a.rows * per_a, total = first + b.rows * per_b;
    for (long long i = static_cast<long long>(block) * 256 + threadIdx.x; i < total; i += static_cast<long long>(blocks) * 256) {
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
__global__ void __launch_bounds__(256) copy_rows16_kernel(const CopyJob a, const CopyJob b) {
    griddep_wait();
    copy_rows(a, b, blockIdx.x, gridDim.x);
}

// Sums over rows: a cluster of CTAs takes 64 columns (8 lanes of 8 each, 32 rows at a time), each a share of
// the rows; their sums meet in distributed shared memory, in the order of the shares. The clusters past
// the columns copy rows.
constexpr int kSumColumns = 64, kSumSplit = 8;
template <class T>
__global__ void __launch_bounds__(256) column_sums_kernel(const T *x, long long stride, long long rows, int n, bool runs, float *out,
                                                          int accumulate, const CopyJob a, const CopyJob b) {
    __shared__ float red[32][kSumColumns + 1], mine[kSumColumns];
    griddep_wait();
    const int summing = (n + kSumColumns - 1) / kSumColumns * kSumSplit;
    if (blockIdx.x >= summing) return copy_rows(a, b, blockIdx.x - summing, gridDim.x - summing);
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
    bool pair;
    int tile_n, tiles_m, tiles_n, steps, splits, steps_per_split;
};
// The cheapest form, by what was measured on one GB300: a step of 64 takes 0.33 us where a pair's 256 x 256
// products keep the tensor cores busy, else what it takes to issue and to load; a tile's epilogue runs
// under the next tile's products, the last one's alone; splitting the summed axis costs writing and reading
// the parts in fp32 and a launch. k > 0.
Plan plan_of(long long m, int n, long long k, bool may_split) {
    struct Form {
        bool pair;
        int tile_n;
        double step, epilogue;
    };
    constexpr Form forms[] = {{true, 256, 0.33, 5.2}, {true, 128, 0.22, 2.6}, {false, 128, 0.20, 2.6}, {false, 64, 0.17, 1.3}};
    Plan best = {};
    double least = 1e300;
    for (const Form &f : forms) {
        Plan p = {f.pair, f.tile_n, 0, 0, 0, 0, 0};
        const int rows = f.pair ? kTile : kHalf, places = f.pair ? kGridCap / 2 : kGridCap;
        p.tiles_m = static_cast<int>((m + rows - 1) / rows);
        p.tiles_n = (n + f.tile_n - 1) / f.tile_n;
        p.steps = static_cast<int>((k + kStep - 1) / kStep);
        const long long tiles = static_cast<long long>(p.tiles_m) * p.tiles_n;
        long long most = may_split ? places / tiles : 1;
        if (most > p.steps / 4) most = p.steps / 4;
        for (long long s : {1LL, most}) {
            if (s < 1) continue;
            p.steps_per_split = static_cast<int>((p.steps + s - 1) / s);
            p.splits = (p.steps + p.steps_per_split - 1) / p.steps_per_split;
            const double rounds = static_cast<double>((tiles * p.splits + places - 1) / places), products = p.steps_per_split * f.step;
            const double parts = p.splits > 1 ? 4. + static_cast<double>(m) * n * 4 * (p.splits + 1) / 6e6 : 0.;
            const double cost = (rounds - 1) * (products > f.epilogue ? products : f.epilogue) + products + f.epilogue + parts;
            if (cost < least) {
                least = cost;
                best = p;
            }
        }
    }
    return best;
}

bool encode_operand(CUtensorMap *m, const Product &p, const Operand &o, long long rows, int box_rows) {
    return o.turned ? encode_rows16(m, p.bf16, o.p, rows, p.k, o.pitch * 2, kStep) : encode_rows16(m, p.bf16, o.p, p.k, rows, o.pitch * 2, box_rows);
}

template <int KIND>
int launch_join(const float *parts, int splits, const Product &p, int sms, bool pdl, cudaStream_t s) {
    const int vec = p.epi.wide && p.epi.extra_runs && p.epi.bias_runs ? 8 : 1;
    const long long need = (p.m * p.n + 256 * vec - 1) / (256 * vec), cap = static_cast<long long>(sms) * 16;
    return note_launch(launch_block_kernel(vec == 8 ? product_join_kernel<KIND, 8> : product_join_kernel<KIND, 1>,
                                           static_cast<unsigned>(need < cap ? need : cap), 256, 0, pdl, s, parts, splits, p.m, p.n,
                                           p.epi));
}

}  // namespace

size_t product_parts_bytes(long long m, int n, long long k) {
    if (m <= 0 || k <= 0) return 0;     // a sum over nothing is written by the joining kernel alone
    const Plan q = plan_of(m, n, k, true);
    return q.splits > 1 ? static_cast<size_t>(q.splits) * m * n * 4 : 0;
}

// Up to 96 rounds of 64 of k a CTA, which the first tile's products hide, or which take less than a launch (777 x 1000 x 2048 8.9 us
// against 11.8 by a kernel of their own, 6000 x 1000 x 1000 38.4 against 42.7, 1024 x 16384 x 128 12.3 against 24.0;
// 4096 x 64 x 64 10.4 against 9.7). Longer ones wait behind the products' loads: 8192 x 2048 x 2048 60.9 against 54.8.
bool product_sums_rows(long long m, int n, long long k) {
    const Plan q = plan_of(m, n, k, true);
    const long long items = static_cast<long long>(q.tiles_m) * q.tiles_n * q.splits, ctas = q.pair ? 2 : 1;
    const long long grid = items * ctas < kGridCap ? items * ctas : kGridCap, groups = (m + 31) / 32;
    return (groups + grid - 1) / grid * ((k + 63) / 64) <= 96;
}

int launch_product(const Product &p, int sms, unsigned int *status, bool pdl, cudaStream_t s) {
    if (p.k == 0) return launch_join<EPI_SUMS>(nullptr, 0, p, sms, pdl, s);
    const Plan q = plan_of(p.m, p.n, p.k, p.parts != nullptr);
    const int ctas = q.pair ? 2 : 1;
    CUtensorMap ma, mb;
    if (!encode_operand(&ma, p, p.a, p.m, kHalf) || !encode_operand(&mb, p, p.b, p.n, q.tile_n / ctas)) return MHC_ERR_CUDA;
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
    const long long items = static_cast<long long>(q.tiles_m) * q.tiles_n * q.splits;
    if (items > INT32_MAX - 1024) return MHC_ERR_UNSUPPORTED;
    a.items = static_cast<int>(items);
    a.a_turned = p.a.turned;
    a.b_turned = p.b.turned;
    const uint32_t fmt = p.bf16 ? 1u : 0u;
    a.idesc = (1u << 4) | (fmt << 7) | (fmt << 10) | ((p.a.turned ? 1u : 0u) << 15) | ((p.b.turned ? 1u : 0u) << 16) |
              (static_cast<uint32_t>(q.tile_n >> 3) << 17) | (static_cast<uint32_t>(ctas * kHalf >> 4) << 24);
    a.status = status;
    a.timeout_ns = wait_timeout_ns();
    a.e = p.epi;
    if (p.row_sums) {
        a.rows = p.a.p;
        a.row_pitch = p.a.pitch;
        a.k = p.k;
        a.row_sums = p.row_sums;
        a.bf16 = p.bf16;
        a.add_row_sums = p.add_row_sums;
    }
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
    void (*const kernels[2][3])(const CUtensorMap, const CUtensorMap, const Args) = {
        {product_kernel<EPI_SUMS, false>, product_kernel<EPI_LINEAR, false>, product_kernel<EPI_SLOPE, false>},
        {product_kernel<EPI_SUMS, true>, product_kernel<EPI_LINEAR, true>, product_kernel<EPI_SLOPE, true>}};
    if (!g_smem[dev & 63].load(std::memory_order_acquire)) {
        for (auto &row : kernels)
            for (auto kern : row)
                if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) return MHC_ERR_CUDA;
        g_smem[dev & 63].store(1, std::memory_order_release);
    }
    const long long places = sms / ctas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas * static_cast<unsigned>(a.items < places ? a.items : places));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    if (int e = note_launch(cudaLaunchKernelEx(&cfg, kernels[q.pair][kind], ma, mb, a))) return e;
    if (q.splits == 1) return MHC_OK;
    return p.kind == EPI_SUMS     ? launch_join<EPI_SUMS>(p.parts, q.splits, p, sms, pdl, s)
           : p.kind == EPI_LINEAR ? launch_join<EPI_LINEAR>(p.parts, q.splits, p, sms, pdl, s)
                                  : launch_join<EPI_SLOPE>(p.parts, q.splits, p, sms, pdl, s);
}

namespace {
unsigned copy_blocks(const CopyJob &a, const CopyJob &b, int sms) {
    const long long need = (a.rows * ((a.n + 7) / 8) + b.rows * ((b.n + 7) / 8) + 255) / 256, cap = static_cast<long long>(sms) * 8;
    return static_cast<unsigned>(need < cap ? need : cap);
}
}  // namespace

cudaError_t launch_copy_rows16(const CopyJob &a, const CopyJob &b, int sms, bool pdl, cudaStream_t s) {
    return launch_block_kernel(copy_rows16_kernel, copy_blocks(a, b, sms), 256, 0, pdl, s, a, b);
}

int launch_column_sums(const void *x, long long stride, int dtype, long long rows, int n, float *out, int accumulate, const CopyJob &a,
                       const CopyJob &b, int sms, bool pdl, cudaStream_t s) {
    const bool runs = n % 8 == 0 && stride % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15u) == 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((n + kSumColumns - 1) / kSumColumns * kSumSplit + (copy_blocks(a, b, sms) + kSumSplit - 1) / kSumSplit * kSumSplit);
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
                                                              stride, rows, n, runs, out, accumulate, a, b)
                                         : cudaLaunchKernelEx(&cfg, column_sums_kernel<__half>, static_cast<const __half *>(x), stride,
                                                              rows, n, runs, out, accumulate, a, b));
}

}  // namespace mhc
