// All the products of an orthogonalised update in one cooperative launch: CTAs, or pairs of them, stay on their
// SMs and walk the products one after another, a barrier of the grid between two. Products with few
// tiles split the summed axis over the CTAs; those of a tile wait for one another's parts, and each
// then adds them, in their order, for some of the tile's columns. Every wait has a limit.
//
// A pair forms a 256 x 256 or 256 x 128 tile, a CTA 128 rows of 128, 64 or 32 columns, as the products with an epilogue do (64 of k
// a stage, five stages, two buffers of sums in tensor memory). Every operand is two fp16 parts: a step of 64 is one stage of both
// operands' hi and one of their lo, and three products (with a stage for each product hi came twice: 2048 x 1024 took 9 % longer,
// 2944 x 1760 23 %).
//
// 4096 x 7168 3.28 ms in a burst, 3.55 with the tensor cores at the power cap; 2048 x 1024 201 us (15 launches 450), where a
// product takes some 5.5 us beside its own steps: 0.6 until the first stage is there, 1 to 3 the epilogue, 0.4 until the
// CTA's warps have met, 1.5 to 2.3 the barrier; split, 3 more for the parts.
// A symmetric result's tiles left of the diagonal are not formed: those right of it are stored twice,
// the second time a column a store, which is contiguous across a warp's lanes.
#include <atomic>
#include <cmath>

#include "epilogue.cuh"
#include "mhc_internal.h"
#include "orthogonal.h"
#include "pair_mma.cuh"

namespace mhc {
namespace {

constexpr int kHalf = 128;                          // rows of a tile by a CTA
constexpr int kStageBytes = 4 * kPairBoxBytes;
constexpr int kStages = 5;
constexpr int kSumWarps = 8;
constexpr int kThreads = 64 + 32 * kSumWarps;
constexpr int kBars = 2 * kStages + 7;
constexpr int kOutBytes = 32 * 128;                 // 32 rows of 64 columns of 16 bits, of hi or of lo
constexpr int kSmem = kStages * kStageBytes + 1024 + 2 * kSumWarps * kOutBytes + 256;
constexpr int kTmemCols = 512;                      // all of it: shared memory has no room for another kernel's CTA that takes some
constexpr int kBand = 8;

enum NsSite : int { SITE_N_EMPTY = 100, SITE_N_FULL, SITE_N_ACC_EMPTY, SITE_N_ACC_FULL, SITE_N_DRAIN, SITE_N_GRID, SITE_N_GO, SITE_N_MEET, SITE_N_PARTS };

// The matrices [p][p] of a step: A and P, and where two steps are one, P A (then the two P's product) and the
// second P.
enum NsMatrix : int { M_A, M_P, M_T, M_R, M_COUNT };
enum NsRole : int { R_GRAM, R_SQUARE, R_APPLY };
// One product.
struct Phase {
    int role;                       // GRAM: of X with itself; SQUARE: of two matrices; APPLY: of one with X
    int a, b, out, add;             // matrices; add: what is added times of_add (-1: nothing)
    int m, n, tiles_m, tiles_n, tile_n, steps, splits, per, items;
    int symmetric, ratio, a_turned, b_turned;       // ratio: of a tile's rows to its columns
    uint32_t idesc;
    float of_sum, of_add, of_unit;  // of_unit: on the diagonal
};
constexpr int kPairPhases = 7, kStepPhases = 3, kPhases = kPairPhases + kStepPhases;
static_assert(kNsCounters == 32 + kPhases * kNsMostCtas, "a counter for each tile of each phase");
struct NsArgs {
    // two steps as one (`pairs` times), then a step (`singles` times, once at least)
    Phase phase[kPhases];
    int pairs, singles;
    int wide;                       // X is the second operand where it is applied to, else the first
    __half *x[2][2], *mat[M_COUNT][2];      // [turn][hi, lo]
    long long x_pitch, x_size, p_pitch, p_size;
    float of_out;
    void *out;
    int out_dtype, out_wide;
    float *parts;
    unsigned int *counters;         // [0]: the grid's barrier; from 32 on, parts of a tile that are there
    unsigned int *status;
    unsigned long long timeout_ns;
};
struct NsMaps {
    CUtensorMap gram_a[2][2], gram_b[2][2], apply_x[2][2];      // [turn][hi, lo]
    CUtensorMap mat_a[M_COUNT][2], mat_b[M_COUNT][2];
};
// Which of the phases the ph-th product is, how many like it came before, and X's turn.
struct Step {
    int phase, round, x;
};
__device__ __forceinline__ Step step_of(const NsArgs &a, int ph) {
    const int in_pairs = kPairPhases * a.pairs;
    Step s;
    if (ph < in_pairs) {
        s.round = ph / kPairPhases;
        s.phase = ph - s.round * kPairPhases;
        s.x = s.round & 1;
        return s;
    }
    ph -= in_pairs;
    s.round = ph / kStepPhases;
    s.phase = kPairPhases + ph - s.round * kStepPhases;
    s.x = (a.pairs + s.round) & 1;
    return s;
}

struct Place {
    int batch, split, ti, tj, tile;
};
__device__ __forceinline__ Place place_of(const Phase &f, int item) {
    Place p;
    const int ratio = f.ratio;
    const int tiles = f.tiles_m * f.tiles_n - (f.symmetric ? ratio * (f.tiles_m * (f.tiles_m - 1) / 2) : 0);
    p.tile = item / f.splits;
    p.split = item - p.tile * f.splits;
    p.batch = p.tile / tiles;
    int r = p.tile - p.batch * tiles;
    if (f.symmetric) {
        p.ti = 0;
        while (r >= f.tiles_n - ratio * p.ti) r -= f.tiles_n - ratio * p.ti++;
        p.tj = ratio * p.ti + r;
        return p;
    }
    const int band = r / (kBand * f.tiles_n), first = band * kBand;
    const int rows = f.tiles_m - first < kBand ? f.tiles_m - first : kBand;
    const int q = r - band * kBand * f.tiles_n;
    p.tj = q / rows;
    p.ti = first + q - p.tj * rows;
    return p;
}

// Whether the count has come to `target`, within the limit.
__device__ __forceinline__ bool count_wait(const unsigned int *count, unsigned int target, const NsArgs &a, volatile int *abort_flag, int site) {
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        unsigned int v;
        asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
        if (v >= target) return true;
        if (*abort_flag) return false;
        if (globaltimer_ns() - t0 > a.timeout_ns) {
            record_failure(a.status, 7, site);
            *abort_flag = 1;
            return false;
        }
    }
}

// Where a product's sums go: as hi + lo (and the mirrored place), or to the output.
struct Target {
    __half *hi, *lo;
    long long pitch;
    float unit;
    const __half *x_hi, *x_lo;      // what is added, times of_x, and of_unit on the diagonal; or NULL
    float of_x, of_unit;            // of_unit: where there is no x too
    bool mirror, final;
    int m, n;
};
// 8 columns of a row of x.
__device__ __forceinline__ void load_x8(uint4 &h, uint4 &l, const Target &t, int i, int j) {
    h = l = make_uint4(0u, 0u, 0u, 0u);
    if (!t.x_hi || i >= t.m || j >= t.n) return;
    const long long at = static_cast<long long>(i) * t.pitch + j;
    h = __ldcg(reinterpret_cast<const uint4 *>(t.x_hi + at));
    l = __ldcg(reinterpret_cast<const uint4 *>(t.x_lo + at));
}
// Eight sums of row i from column j on in two parts.
__device__ __forceinline__ void pair8(const Target &t, int i, int j, const float *v, const uint4 &xh, const uint4 &xl, uint4 *hi, uint4 *lo) {
    const __half *const tag = nullptr;
    const uint32_t h4[4] = {xh.x, xh.y, xh.z, xh.w}, l4[4] = {xl.x, xl.y, xl.z, xl.w};
    uint32_t hw[4], lw[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        uint64_t r = mul2(f2_pack(v[2 * q], v[2 * q + 1]), splat2(t.unit));
        if (t.x_hi) r = fma2(add2(unpack2(h4[q], tag), unpack2(l4[q], tag)), splat2(t.of_x), r);
        if (t.of_unit != 0.f) r = add2(r, f2_pack(i == j + 2 * q ? t.of_unit : 0.f, i == j + 2 * q + 1 ? t.of_unit : 0.f));
        // hi: the leading 11 bits, cut, not rounded (two masks where a conversion back would take four
        // times as long); lo, up to 2^-10 of it, holds 11 more
        const uint64_t h = r & 0xFFFFE000FFFFE000ull;
        hw[q] = pack2(h, tag);
        lw[q] = pack2(fma2(h, splat2(-1.f), r), tag);
    }
    *hi = make_uint4(hw[0], hw[1], hw[2], hw[3]);
    *lo = make_uint4(lw[0], lw[1], lw[2], lw[3]);
}
// The same eight at the mirrored place: a column of the warp's 32 rows a store.
__device__ __forceinline__ void mirror8(const Target &t, int i, int j, const uint4 &hi, const uint4 &lo) {
    const uint32_t hw[4] = {hi.x, hi.y, hi.z, hi.w}, lw[4] = {lo.x, lo.y, lo.z, lo.w};
    const long long step = here(t.pitch);
    uint16_t *h = reinterpret_cast<uint16_t *>(t.hi) + j * step + i, *l = reinterpret_cast<uint16_t *>(t.lo) + j * step + i;
#pragma unroll
    for (int q = 0; q < 8; ++q, h += step, l += step) {
        if (j + q >= t.n) break;
        *h = static_cast<uint16_t>(hw[q >> 1] >> (q & 1) * 16);
        *l = static_cast<uint16_t>(lw[q >> 1] >> (q & 1) * 16);
    }
}
// The warp's 32 x 64 elements of 16 bits at `held` (a row a 128-byte line, its 16 bytes c at c ^ (row & 7)) to whole lines.
__device__ __forceinline__ void put_lines(uint8_t *to, long long pitch_bytes, int rows, int columns, uint32_t held) {
    const int lane = threadIdx.x & 31, c = lane & 7;
    const long long step = here(4 * pitch_bytes);
    uint8_t *q = to + (lane >> 3) * pitch_bytes + 16 * c;
#pragma unroll
    for (int k = 0; k < 8; ++k, q += step) {
        const int row = 4 * k + (lane >> 3);
        const uint4 v = ld_shared_v4(held + row * 128 + ((c ^ (row & 7)) << 4));
        if (row < rows && 8 * c < columns) *reinterpret_cast<uint4 *>(q) = v;
    }
}
// 64 columns (width: or 32) of the warp's 32 rows, through shared memory: a row a lane to global memory would be 32 lines
// a store (by TMA from there: 1 us more until the stores are complete). `sums`: in tensor memory.
__device__ __forceinline__ void put_piece(const NsArgs &a, const Target &t, int batch, int i0, int j, int width, uint32_t sums, uint32_t held) {
    const int lane = threadIdx.x & 31, i = i0 + lane;
    __syncwarp();       // the piece before has been read
    // sixteen columns at a time: a short loop, whose instructions are fetched once
#pragma unroll 1
    for (int c0 = 0; c0 < width; c0 += 16) {
        uint4 xh[2], xl[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) load_x8(xh[k], xl[k], t, i, j + c0 + 8 * k);
        uint32_t u[16];
        tmem_ld16_now(sums + c0, u);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int c = c0 + 8 * k;
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(u[8 * k + e]);
            const uint32_t at = held + lane * 128 + (((c >> 3) ^ (lane & 7)) << 4);
            if (t.final) {
                uint32_t o[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint64_t r = f2_pack(v[2 * q] * a.of_out, v[2 * q + 1] * a.of_out);
                    o[q] = a.out_dtype == MHC_BF16 ? bf2_pack_rn(r) : pack2(r, static_cast<const __half *>(nullptr));
                }
                st_shared_v4(at, make_uint4(o[0], o[1], o[2], o[3]));
            } else {
                uint4 hw, lw;
                pair8(t, i, j + c, v, xh[k], xl[k], &hw, &lw);
                st_shared_v4(at, hw);
                st_shared_v4(at + kOutBytes, lw);
                if (t.mirror && i < t.m && j + c < t.n) mirror8(t, i, j + c, hw, lw);
            }
        }
    }
    __syncwarp();
    const int rows = t.m - i0, columns = t.n - j < width ? t.n - j : width;
    if (t.final) {
        put_lines(static_cast<uint8_t *>(a.out) + ((static_cast<long long>(batch) * t.m + i0) * t.n + j) * 2, static_cast<long long>(t.n) * 2, rows,
                  columns, held);
        return;
    }
    const long long at = static_cast<long long>(i0) * t.pitch + j;
    put_lines(reinterpret_cast<uint8_t *>(t.hi + at), t.pitch * 2, rows, columns, held);
    put_lines(reinterpret_cast<uint8_t *>(t.lo + at), t.pitch * 2, rows, columns, held + kOutBytes);
}
// Columns [j, j + 8) of the warp's 32 rows from i0 on, a row a lane; `piece`: 32 x 9 floats of the warp.
__device__ __forceinline__ void put8(const NsArgs &a, const Target &t, int batch, int i0, int j, float (&v)[8], float *piece) {
    const int lane = threadIdx.x & 31, i = i0 + lane;
    if (!t.final) {
        if (i >= t.m || j >= t.n) return;
        uint4 xh, xl, hw, lw;
        load_x8(xh, xl, t, i, j);
        pair8(t, i, j, v, xh, xl, &hw, &lw);
        const long long at = static_cast<long long>(i) * t.pitch + j;
        *reinterpret_cast<uint4 *>(t.hi + at) = hw;
        *reinterpret_cast<uint4 *>(t.lo + at) = lw;
        if (t.mirror) mirror8(t, i, j, hw, lw);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= a.of_out;
    const long long row0 = static_cast<long long>(batch) * t.m + i0;
    if (a.out_wide) {
        if (i >= t.m || j >= t.n) return;
        with_type(a.out_dtype, [&](auto tag) {
            using T = std::remove_const_t<std::remove_pointer_t<decltype(tag)>>;
            store8(static_cast<T *>(a.out) + (row0 + lane) * t.n + j, run_of(v));
        });
        return;
    }
    // rows on any boundary: turned in shared memory, 8 columns of four rows a store
#pragma unroll
    for (int e = 0; e < 8; ++e) piece[lane * 9 + e] = v[e];
    __syncwarp();
    const int rows = t.m - i0 < 32 ? t.m - i0 : 32, col = lane & 7;
    if (j + col < t.n)
#pragma unroll
        for (int r = 0; r < 32; r += 4)
            if (r + (lane >> 3) < rows)
                store_any(a.out, a.out_dtype, (row0 + r + (lane >> 3)) * t.n + j + col, piece[(r + (lane >> 3)) * 9 + col]);
    __syncwarp();
}

template <bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
ns_kernel(const __grid_constant__ NsMaps maps, const __grid_constant__ NsArgs a) {
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    uint8_t *const basep = raw + (base - smem_addr(raw));
    const uint32_t bars = base + kStages * kStageBytes + 2 * kSumWarps * kOutBytes;
    const uint32_t full = bars, empty = bars + 8 * kStages, acc_full = bars + 16 * kStages,
                   acc_empty = acc_full + 16, drain = acc_full + 32,
                   go = acc_full + 40 /* the grid's barrier is passed */, together = acc_full + 48 /* the epilogue's warps */;
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(basep + (bars - base) + 8 * kBars);
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    constexpr int kCtas = PAIR ? 2 : 1, kTile = kCtas * kHalf;
    const uint32_t rank = PAIR ? cluster_rank() : 0;
    const int unit = blockIdx.x / kCtas, units = gridDim.x / kCtas;
    const int phases = kPairPhases * a.pairs + kStepPhases * a.singles;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(acc_full + 8 * b, 1);
            mbar_init(acc_empty + 8 * b, kCtas * kSumWarps);
        }
        mbar_init(drain, 1);
        mbar_init(go, 1);
        mbar_init(together, kSumWarps);
        *abort_flag = 0;
        fence_mbar_init();
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
        for (int ph = 0; ph < phases && ok; ++ph) {
            const Step at = step_of(a, ph);
            const Phase &f = a.phase[at.phase];
            if (ph) {
                // one thread a CTA asks, for the epilogue too
                ok = count_wait(a.counters, ph * gridDim.x, a, abort_flag, SITE_N_GRID);
                if (!ok) break;
                fence_proxy_async_global();
                mbar_arrive(go);
            }
            const CUtensorMap *const ma = f.role == R_GRAM                ? maps.gram_a[at.x]
                                          : f.role == R_APPLY && !a.wide ? maps.apply_x[at.x]
                                                                         : maps.mat_a[f.a];
            const CUtensorMap *const mb = f.role == R_GRAM               ? maps.gram_b[at.x]
                                          : f.role == R_APPLY && a.wide ? maps.apply_x[at.x]
                                                                        : maps.mat_b[f.b];
            const int half = f.tile_n / kCtas;
            for (int item = unit; item < f.items && ok; item += units) {
                const Place p = place_of(f, item);
                const int s0 = p.split * f.per, s1 = s0 + f.per < f.steps ? s0 + f.per : f.steps;
                const int ci = p.ti * kTile + static_cast<int>(rank) * kHalf, cj = p.tj * f.tile_n + static_cast<int>(rank) * half;
                for (int st = 2 * s0; st < 2 * s1; ++st, ++it) {
                    const uint32_t s = it % kStages, turn_of = (it / kStages) & 1;
                    if (!mbar_wait(empty + 8 * s, turn_of ^ 1, abort_flag, a.timeout_ns, a.status, SITE_N_EMPTY)) {
                        ok = false;
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, kCtas * (2 * kPairBoxBytes + half * 128));
                    const uint32_t bar = PAIR ? map_to_rank(full + 8 * s, 0) : full + 8 * s, da = base + s * kStageBytes, db = da + 2 * kPairBoxBytes;
                    const int part = st & 1, k = (st >> 1) * kPairStep;
                    const CUtensorMap *const am = ma + part, *const bm = mb + part;
                    if (f.a_turned) {
                        unit_load<PAIR>(da, am, ci, k, p.batch, bar);
                        unit_load<PAIR>(da + kPairBoxBytes, am, ci + 64, k, p.batch, bar);
                    } else {
                        unit_load<PAIR>(da, am, k, ci, p.batch, bar);
                    }
                    if (f.b_turned) {
                        unit_load<PAIR>(db, bm, cj, k, p.batch, bar);
                        if (half == kHalf) unit_load<PAIR>(db + kPairBoxBytes, bm, cj + 64, k, p.batch, bar);
                    } else {
                        unit_load<PAIR>(db, bm, k, cj, p.batch, bar);
                    }
                }
            }
        }
        // every stage's last release has arrived before this CTA may exit
        for (uint32_t k = it > kStages ? it - kStages : 0; k < it && ok; ++k)
            ok = mbar_wait(empty + 8 * (k % kStages), (k / kStages) & 1, abort_flag, a.timeout_ns, a.status, SITE_N_EMPTY);
        if (!ok && rank == 0) {
            // gave up: both CTAs' copies still in flight land before they exit
            int gave_up = 0;
            for (uint32_t k = it > kStages ? it - kStages : 0; k < it; ++k)
                mbar_wait(full + 8 * (k % kStages), (k / kStages) & 1, &gave_up, a.timeout_ns, a.status, SITE_N_DRAIN);
        }
    } else if (warp == 1 && rank == 0 && elect_one()) {
        // ------------------------------------------------ products, the leader for both
        uint32_t it = 0, done = 0;
        bool ok = true;
        for (int ph = 0; ph < phases && ok; ++ph) {
            const Phase &f = a.phase[step_of(a, ph).phase];
            const uint64_t na = f.a_turned ? 2048 >> 4 : 32 >> 4, nb = f.b_turned ? 2048 >> 4 : 32 >> 4;
            for (int item = unit; item < f.items && ok; item += units, ++done) {
                const int split = item % f.splits, s0 = split * f.per, s1 = s0 + f.per < f.steps ? s0 + f.per : f.steps;
                const uint32_t buf = done & 1, acc = tmem + buf * 256;
                // a barrier of the grid may lie between: as long as it may take
                if (!mbar_wait(acc_empty + 8 * buf, ((done >> 1) & 1) ^ 1, abort_flag, a.timeout_ns, a.status, SITE_N_ACC_EMPTY)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                for (int st = s0; st < s1; ++st) {
                    // hi of both; then lo, and the products of hi with it
                    uint32_t held[2], a_at[2], b_at[2];
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        const uint32_t s = it % kStages;
                        ok = mbar_wait(full + 8 * s, (it / kStages) & 1, abort_flag, 2 * a.timeout_ns, a.status, SITE_N_FULL);
                        if (!ok) break;
                        ++it;
                        tc_fence_after();
                        held[part] = s;
                        a_at[part] = base + s * kStageBytes;
                        b_at[part] = a_at[part] + 2 * kPairBoxBytes;
                        auto multiply = [&](uint32_t left, uint32_t right, bool add) {
                            const uint64_t da = f.a_turned ? desc_columns(left) : desc_rows(left), db = f.b_turned ? desc_columns(right) : desc_rows(right);
#pragma unroll
                            for (int q = 0; q < kPairStep / 16; ++q) unit_multiply<PAIR>(acc, da + q * na, db + q * nb, f.idesc, add || q > 0);
                        };
                        if (part == 0) {
                            multiply(a_at[0], b_at[0], st > s0);
                        } else {
                            multiply(a_at[0], b_at[1], true);
                            multiply(a_at[1], b_at[0], true);
                        }
                    }
                    if (!ok) break;
#pragma unroll
                    for (int part = 0; part < 2; ++part) unit_commit<PAIR>(empty + 8 * held[part]);
                }
                if (ok) unit_commit<PAIR>(acc_full + 8 * buf);
            }
        }
        if (!ok) {
            // the products issued end before tensor memory is freed
            int gave_up = 0;
            unit_commit<PAIR>(drain);
            mbar_wait(drain, 0, &gave_up, a.timeout_ns, a.status, SITE_N_DRAIN);
        }
    } else if (warp >= 2) {
        // ------------------------------------------------ epilogue, either CTA its 128 rows
        const int quad = warp & 3, w = warp - 2;
        const uint32_t held = base + kStages * kStageBytes + 2 * w * kOutBytes;     // this warp's hi, then lo
        float *const piece = reinterpret_cast<float *>(basep + (held - base));
        uint32_t done = 0, met = 0;
        bool ok = true;
        // the epilogue's warps wait for one another, within the limit
        auto meet = [&] {
            __syncwarp();
            if (lane == 0) mbar_arrive(together);
            const bool all = mbar_wait(together, met++ & 1, abort_flag, 2 * a.timeout_ns, a.status, SITE_N_MEET);
            return __all_sync(0xffffffffu, all) != 0;
        };
        for (int ph = 0; ph < phases && ok; ++ph) {
            const Step st = step_of(a, ph);
            const bool final = ph + 1 == phases;
            const Phase &f = a.phase[st.phase];
            const int width = f.tile_n / 2, first = w / 4 * width;
            if (ph) {
                ok = mbar_wait(go, (ph - 1) & 1, abort_flag, 2 * a.timeout_ns, a.status, SITE_N_GO);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
            }
            for (int item = unit; item < f.items && ok; item += units, ++done) {
                const Place p = place_of(f, item);
                const uint32_t buf = done & 1;
                const int i0 = p.ti * kTile + static_cast<int>(rank) * kHalf + quad * 32, j0 = p.tj * f.tile_n;
                Target t;
                const bool to_x = f.role == R_APPLY;
                const long long at = p.batch * (to_x ? a.x_size : a.p_size);
                __half *const *const to_pair = to_x ? a.x[st.x ^ 1] : a.mat[f.out];
                t.hi = to_pair[0] + at;
                t.lo = to_pair[1] + at;
                t.pitch = to_x ? a.x_pitch : a.p_pitch;
                t.unit = f.of_sum;
                t.x_hi = f.add < 0 ? nullptr : a.mat[f.add][0] + at;
                t.x_lo = f.add < 0 ? nullptr : a.mat[f.add][1] + at;
                t.of_x = f.of_add;
                t.of_unit = f.of_unit;
                t.mirror = f.symmetric && j0 >= (p.ti + 1) * kTile;
                t.final = final;
                t.m = f.m;
                t.n = f.n;
                ok = mbar_wait(acc_full + 8 * buf, (done >> 1) & 1, abort_flag, 2 * a.timeout_ns, a.status, SITE_N_ACC_FULL);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint32_t sums = tmem + buf * 256 + first + (static_cast<uint32_t>(quad * 32) << 16);
                if (f.splits == 1) {
#pragma unroll 1
                    for (int c = 0; c < width && i0 < f.m && j0 + first + c < f.n; c += 64) {
                        if (!final || a.out_wide) {
                            put_piece(a, t, p.batch, i0, j0 + first + c, width < 64 ? width : 64, sums + c, held);
                            continue;
                        }
#pragma unroll 1
                        for (int k = c; k < c + 64 && k < width && j0 + first + k < f.n; k += 8) {
                            uint32_t u[8];
                            tmem_ld8_now(sums + k, u);
                            float v[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(u[e]);
                            put8(a, t, p.batch, i0, j0 + first + k, v, piece);
                        }
                    }
                } else {
                    // the tile's parts, [split][column][128 rows], a column of 32 rows a store
                    const long long part_size = static_cast<long long>(f.tile_n) * kHalf;
                    float *const parts = a.parts + (static_cast<long long>(p.tile) * kCtas + rank) * f.splits * part_size + quad * 32 + lane;
                    float *const to = parts + p.split * part_size + first * kHalf;
#pragma unroll 1
                    for (int c = 0; c < width; c += 32) {
                        uint32_t u[32];
                        tmem_ld32_now(sums + c, u);
#pragma unroll
                        for (int e = 0; e < 32; ++e) __stcg(to + (c + e) * kHalf, __uint_as_float(u[e]));
                    }
                    // every part of the tile is there (its CTAs are all resident); each finishes some columns. The release of the
                    // thread that the warps met with carries what they all wrote; a fence of each beside it is 0.7 us more.
                    ok = meet();
                    if (!ok) break;
                    if (threadIdx.x == 64) {
                        unsigned int *const count = a.counters + 32 + st.phase * kNsMostCtas + p.tile * kCtas + rank;
                        asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(count) : "memory");
                        count_wait(count, f.splits * (st.round + 1), a, abort_flag, SITE_N_PARTS);
                    }
                    ok = meet() && !*abort_flag;
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    for (int g = p.split + f.splits * (w / 4); g < f.tile_n / 8; g += 2 * f.splits) {
                        const int j = p.tj * f.tile_n + 8 * g;
                        if (j >= f.n) break;
                        float v[8] = {};
                        for (int s0 = 0; s0 < f.splits; s0 += 4) {
                            float u[4][8];
#pragma unroll
                            for (int q = 0; q < 4; ++q)
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    u[q][e] = s0 + q < f.splits ? __ldcg(parts + (s0 + q) * part_size + (8 * g + e) * kHalf) : 0.f;
#pragma unroll
                            for (int q = 0; q < 4; ++q)
#pragma unroll
                                for (int e = 0; e < 8; ++e) v[e] += u[q][e];
                        }
                        put8(a, t, p.batch, i0, j, v, piece);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) unit_arrive<PAIR>(acc_empty + 8 * buf);
            }
            if (!ok || final) break;
            // what this CTA wrote, before it arrives: seen by other CTAs' loads of either kind
            fence_proxy_async_global();
            ok = meet();
            if (ok && threadIdx.x == 64) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(a.counters) : "memory");
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    if constexpr (PAIR) cluster_sync();
    if (warp == 2) unit_tmem_free<PAIR>(tmem, kTmemCols);
}

// Pairs of CTAs, and CTAs, that the device holds at once: 0 before it was asked.
std::atomic<int> g_units[2][64];

template <bool PAIR>
int resident_units(int *units) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return MHC_ERR_CUDA;
    constexpr int kCtas = PAIR ? 2 : 1;
    int n = g_units[PAIR][dev & 63].load(std::memory_order_acquire);
    if (!n) {
        if (cudaFuncSetAttribute(ns_kernel<PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess) return MHC_ERR_CUDA;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kCtas);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = kCtas;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, ns_kernel<PAIR>, &cfg) != cudaSuccess || n < 1) return MHC_ERR_CUDA;
        if (n > kNsMostCtas / kCtas) n = kNsMostCtas / kCtas;
        g_units[PAIR][dev & 63].store(n, std::memory_order_release);
    }
    *units = n;
    return MHC_OK;
}

// A product by `units` pairs of CTAs, or CTAs. The cheapest of both tiles' widths and of splitting or not, by what was
// measured on one GB300: three products of 64 take 0.95 us with a pair's 256 columns, where the tensor cores are busy, else
// what it takes to load them, more where every SM loads for several tiles in turn (3 x 1408 x 6436 by CTAs' tiles takes 14 % longer than by pairs');
// finishing 64 columns of a tile by a warp 3 us; writing parts and waiting for the others'
// 3.1 (256 columns 5.3), and finishing 8 columns of s parts 0.4 + 0.1 s. (By 16 columns, with half as many parts: 5331 x 149 took 15 %
// longer, 628 x 392 11 %.)
Phase phase_of(int role, int m, int n, int k, int batch, bool a_turned, bool b_turned, bool pair, int units, double *cost) {
    Phase f = {};
    const bool symmetric = role != R_APPLY;
    const int rows = pair ? 2 * kHalf : kHalf;
    f.role = role;
    f.add = -1;
    f.of_sum = 1.f / kNsScale;
    f.m = m;
    f.n = n;
    f.symmetric = symmetric;
    f.a_turned = a_turned;
    f.b_turned = b_turned;
    f.tiles_m = (m + rows - 1) / rows;
    f.steps = (k + kPairStep - 1) / kPairStep;
    auto tiles = [&](int tile_n) {
        const long long c = (n + tile_n - 1) / tile_n, all = f.tiles_m * c;
        return batch * (symmetric ? all - rows / tile_n * (static_cast<long long>(f.tiles_m) * (f.tiles_m - 1) / 2) : all);
    };
    double best = 1e300;
    long long count = 0;
    for (int tile_n : {rows, rows / 2, 32}) {
        // 32 columns where there are few tiles, with half the epilogue of 64 (256 x 256 takes 9 % less, 400 x 416 10 %).
        // (Read across k a tile's columns come by 64.)
        if (tile_n == 32 && (pair || b_turned)) continue;
        const long long c = tiles(tile_n);
        const int form = tile_n == 256 ? 0 : pair ? 1 : tile_n == 128 ? 2 : tile_n == 64 ? 3 : 4;
        constexpr double kThree[] = {0.95, 0.52, 0.55, 0.42, 0.38}, kBusy[] = {0.95, 0.62, 0.68, 0.55, 0.50};
        int most = static_cast<int>(c <= units ? units / c : 1);
        if (most > f.steps / 2) most = f.steps / 2;
        if (most > tile_n / 8) most = tile_n / 8;       // each of them finishes 8 columns at least
        if (tile_n == 32) most = 1;
        for (int s : {1, most}) {
            if (s < 1) continue;
            const int per = (f.steps + s - 1) / s;
            const double rounds = static_cast<double>((c * s + units - 1) / units), finish = 3. * tile_n / 128;
            const double work = per * (rounds > 1. ? kBusy[form] : kThree[form]);
            const double all = s > 1 ? work + (tile_n == 256 ? 5.3 : 3.1) + (0.4 + 0.1 * s) * ((tile_n / 8 + 2 * s - 1) / (2 * s))
                                     : (rounds - 1) * (work > finish ? work : finish) + work + finish;
            if (all >= best) continue;
            best = all;
            count = c;
            f.tile_n = tile_n;
            f.per = per;
            f.splits = (f.steps + per - 1) / per;
        }
    }
    f.ratio = rows / f.tile_n;
    f.tiles_n = (n + f.tile_n - 1) / f.tile_n;
    f.items = static_cast<int>(count * f.splits);
    f.idesc = (1u << 4) | ((a_turned ? 1u : 0u) << 15) | ((b_turned ? 1u : 0u) << 16) | (static_cast<uint32_t>(f.tile_n >> 3) << 17) |
              (static_cast<uint32_t>(rows >> 4) << 24);
    *cost = best;
    return f;
}

}  // namespace

int launch_ns(const NsCall &c, unsigned int *status, cudaStream_t s) {
    const int p = c.m < c.n ? c.m : c.n, q = c.m < c.n ? c.n : c.m;
    const bool wide = c.m <= c.n;
    NsArgs a = {};
    // Two steps as one, X <- (P1 P0) X with A1 = P0 P0 A: two products of X less, three of matrices [p][p] more. The product
    // of two P has to stay below 16. (Where squared singular values pass 2 and it does not, the A after it is above 16 too, in either form.) 4096 x 7168: 15 % fewer operations; small matrices are bound by the number of products.
    double largest = 0.;
    for (int i = 0; i <= 64; ++i) {
        const double l = i / 32., v = std::fabs(c.a + l * (c.b + l * c.c));
        if (v > largest) largest = v;
    }
    a.wide = wide;
    // by pairs of CTAs or by CTAs, whichever makes a step the cheaper
    int units[2] = {};
    if (int e = resident_units<false>(&units[0])) return e;
    if (int e = resident_units<true>(&units[1])) return e;
    double cost[2][3];
    Phase forms[2][3];
    for (int k = 0; k < 2; ++k) {
        forms[k][0] = phase_of(R_GRAM, p, p, q, c.batch, !wide, !wide, k, units[k], &cost[k][0]);
        forms[k][1] = phase_of(R_SQUARE, p, p, p, c.batch, false, false, k, units[k], &cost[k][1]);
        forms[k][2] = phase_of(R_APPLY, c.m, c.n, p, c.batch, false, wide, k, units[k], &cost[k][2]);
    }
    const bool pair = cost[1][0] + cost[1][1] + cost[1][2] <= cost[0][0] + cost[0][1] + cost[0][2];
    const int ctas = pair ? 2 : 1, places = units[pair];
    const Phase gram = forms[pair][0], square = forms[pair][1], apply = forms[pair][2];
    const bool two = p >= 2048 && q >= p + p / 4 && largest <= 3.8 && square.tile_n == apply.tile_n;
    a.pairs = two ? (c.steps - 1) / 2 : 0;
    a.singles = c.steps - 2 * a.pairs;
    auto poly = [&](Phase f, int out, const NsPolynomial &n) {
        f.a = f.b = M_A;
        f.out = out;
        f.of_sum = n.of_square / kNsScale;
        f.add = n.of_a != 0.f ? M_A : -1;
        f.of_add = n.of_a;
        f.of_unit = n.of_unit * kNsScale;
        return f;
    };
    const NsPolynomial plain = ns_polynomial(c.a, c.b, c.c, false), complete = ns_polynomial(c.a, c.b, c.c, true);
    auto times = [&](Phase f, int x, int y, int out) {
        f.a = x;
        f.b = y;
        f.out = out;
        return f;
    };
    Phase *f = a.phase;
    *f++ = times(gram, 0, 0, M_A);
    *f++ = poly(square, M_P, plain);
    *f++ = times(square, M_P, M_A, M_T);
    *f++ = times(square, M_P, M_T, M_A);
    *f++ = poly(square, M_R, plain);
    *f++ = times(square, M_R, M_P, M_T);
    *f++ = times(apply, M_T, M_T, 0);
    Phase shifted = times(gram, 0, 0, M_A);
    shifted.of_unit = complete.shift * kNsScale;
    *f++ = shifted;
    *f++ = poly(square, M_P, complete);
    *f++ = times(apply, M_P, M_P, 0);
    for (int k = 0; k < 2; ++k) {
        a.x[0][k] = c.x[0][k];
        a.x[1][k] = c.x[1][k];
        for (int t = 0; t < M_COUNT; ++t) a.mat[t][k] = c.mat[t][k];
    }
    a.x_pitch = c.x_pitch;
    a.x_size = c.x_size;
    a.p_pitch = c.p_pitch;
    a.p_size = c.p_size;
    a.of_out = 1.f / (kNsScale * kNsScale);
    a.out = c.out;
    a.out_dtype = c.out_dtype;
    a.out_wide = c.n % 8 == 0 && (reinterpret_cast<uintptr_t>(c.out) & 15u) == 0;
    a.parts = c.parts;
    a.counters = c.counters;
    a.status = status;
    a.timeout_ns = wait_timeout_ns();
    NsMaps maps = {};
    auto rows = [&](CUtensorMap *m, const __half *x, int inner, int count, long long pitch, long long size, int box) {
        return encode_matrices16(m, false, x, inner, count, c.batch, pitch * 2, size * 2, box);
    };
    bool ok = true;
    for (int k = 0; k < 2; ++k) {
        for (int t = 0; t < 2; ++t) {
            const __half *const x = c.x[t][k];
            ok = ok && rows(&maps.gram_a[t][k], x, c.n, c.m, c.x_pitch, c.x_size, wide ? kHalf : kPairStep);
            ok = ok && rows(&maps.gram_b[t][k], x, c.n, c.m, c.x_pitch, c.x_size, wide ? gram.tile_n / ctas : kPairStep);
            ok = ok && rows(&maps.apply_x[t][k], x, c.n, c.m, c.x_pitch, c.x_size, wide ? kPairStep : kHalf);
        }
        // without pairs A is squared and P applied, no more
        for (int t = 0; t < (a.pairs ? M_COUNT : M_T); ++t) {
            const __half *const x = c.mat[t][k];
            // where it is the second operand it has the rows of the tile's columns: of a square, or applied to a tall X
            const bool applied = a.pairs ? false : t == M_P;
            ok = ok && rows(&maps.mat_a[t][k], x, p, p, c.p_pitch, c.p_size, kHalf);
            ok = ok && rows(&maps.mat_b[t][k], x, p, p, c.p_pitch, c.p_size, (applied ? apply.tile_n : square.tile_n) / ctas);
        }
    }
    if (!ok) return MHC_ERR_CUDA;
    int most = 0;
    for (const Phase &f : a.phase) most = most > f.items ? most : f.items;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas * static_cast<unsigned>(most < places ? most : places));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeCooperative;
    attr[1].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return note_launch(cudaLaunchKernelEx(&cfg, pair ? ns_kernel<true> : ns_kernel<false>, maps, a));
}

}  // namespace mhc
