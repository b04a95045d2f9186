// The whole orthogonalised update of matrices with a side of at most 128, a cluster of CTAs a matrix and
// one launch: no product leaves the SMs. X lies with its short side as rows (128 of them, zeros past the
// end), 64 or 128 of its columns in each CTA's shared memory, in two fp16 parts and in the layout that the
// tensor core reads, both along k (for A = X X^T) and across it (for P X). A side of at most 64, or 32, leaves room for
// two, or four, stretches of the columns, one below the other: A is the sum of what comes out on the diagonal, and stands there
// as often (1024 x 64 60 -> 44 us, a batch of 46 237 -> 101, 32 x 8192 147 -> 53). Per step:
//   each CTA's part of A over its columns, in fp32, to its shared memory;
//   each CTA adds some rows of A over the CTAs, in their order, and writes them to all of them
//     (distributed shared memory, a row a warp: whole lines; 16 bytes here and there took eight times as long);
//   each CTA forms P, the same everywhere, and its columns of P X, which take X's place.
// Two barriers of the cluster a step, some 8 us in all (6 x 128 x 500: 49 us), where a barrier of the grid and a trip
// through L2 after each of the three products come to 28 (143).
#include <atomic>

#include "epilogue.cuh"
#include "mhc_internal.h"
#include "orthogonal.h"
#include "pair_mma.cuh"

namespace mhc {
namespace {

constexpr int kP = 128;                             // rows of X, sides of A and P
constexpr int kThreads = 256;
constexpr int kBox = kP * 128;                      // 128 rows of 64 columns of 16 bits
constexpr int kPitch = kP + 4;                      // floats of a row of the sums
constexpr int kMost = 16;                           // CTAs of a cluster
constexpr int kTmemCols = 2 * kP;
// X hi, lo (two boxes each), A and then P hi, lo, sums
constexpr int kXAt = 0, kMAt = 4 * kBox, kSumsAt = 8 * kBox, kSmallBars = kSumsAt + kP * kPitch * 4;
constexpr int kSmem = kSmallBars + 256 + 1024;

enum SmallSite : int { SITE_S_MMA = 130 };

struct SmallArgs {
    const void *g;
    int dtype, tall;
    long long row_stride, batch_stride;
    int p, q, width, ctas, steps;
    int stretch;                    // columns of a stretch
    float eps, of_sum, of_square, of_a, shift, of_unit;     // of_a: what is added of A; shift: what A has on its diagonal
    void *out;
    int out_dtype;
    unsigned int *status;
    unsigned long long timeout_ns;
};

__device__ __forceinline__ uint4 load16_at_rank(uint32_t addr, uint32_t rank) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(map_to_rank(addr, rank)) : "memory");
    return v;
}
__device__ __forceinline__ void store8_at_rank(uint32_t addr, uint32_t rank, uint32_t x, uint32_t y) {
    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(map_to_rank(addr, rank)), "r"(x), "r"(y) : "memory");
}
// Where run c (8 columns) of a row lies in a matrix of boxes of 64 columns in the 128-byte swizzle.
__device__ __forceinline__ uint32_t run_at_box(int row, int c) {
    return (c >> 3) * kBox + row * 128 + (((c & 7) ^ (row & 7)) << 4);
}
// Two values as hi (cut) and lo.
__device__ __forceinline__ void two_parts(float v0, float v1, uint32_t *hi, uint32_t *lo) {
    const __half *const tag = nullptr;
    const uint64_t r = f2_pack(v0, v1), h = r & 0xFFFFE000FFFFE000ull;
    *hi = pack2(h, tag);
    *lo = pack2(fma2(h, splat2(-1.f), r), tag);
}
__device__ __forceinline__ void two_parts(const float (&v)[8], uint4 *hi, uint4 *lo) {
    two_parts(v[0], v[1], &hi->x, &lo->x);
    two_parts(v[2], v[3], &hi->y, &lo->y);
    two_parts(v[4], v[5], &hi->z, &lo->z);
    two_parts(v[6], v[7], &hi->w, &lo->w);
}
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }
// The columns' descriptor, the next 64 columns a box of 128 rows further on.
__device__ __forceinline__ uint64_t desc_across(uint32_t addr) {
    return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | (static_cast<uint64_t>(kBox >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

// SHIFT: log2 of the rows of a stretch, 5 to 7.
template <int SHIFT>
__global__ void __launch_bounds__(kThreads, 1) ns_small_kernel(const __grid_constant__ SmallArgs a) {
    extern __shared__ uint8_t raw[];
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    uint8_t *const basep = raw + (base - smem_addr(raw));
    float *const sums = reinterpret_cast<float *>(basep + kSumsAt);
    const uint32_t bar = base + kSmallBars;
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(basep + kSmallBars + 16);
    volatile int *const abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    double *const squares = reinterpret_cast<double *>(basep + kSmallBars + 32);      // [0]: of the CTA; then of the warps
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = blockIdx.x % a.ctas, batch = blockIdx.x / a.ctas, j0 = rank * a.width;
    const int live = min(a.width, a.stretch - j0);  // of the CTA's columns of every stretch
    constexpr int rows_p = 1 << SHIFT;
    // element (r, j) of the CTA's X: row r & (rows_p - 1) of the matrix, and this column of it, or -1
    auto column_of = [&](int r, int j) {
        const int c = (rows_p == kP ? 0 : (r >> SHIFT) * a.stretch) + j0 + j;
        return (r & (rows_p - 1)) < a.p && j < live && (rows_p == kP || c < a.q) ? c : -1;
    };

    if (threadIdx.x == 0) {
        mbar_init(bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    // After the kernel before, and half of the columns: a CTA of another kernel's cluster with little shared memory may lie on the
    // SM, and neither may wait for the other's columns while the rest of its cluster waits for it.
    griddep_wait();
    if (warp == 0) {
        tmem_alloc(smem_addr(tmem_slot), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;       // A, and in its place P X; P

    // ------------------------------------------------ X's columns, in fp32 to the sums' place, and their squares
    {
        const long long at = batch * a.batch_stride;
        float f = 0.f;
        // the axis that is contiguous in memory across the lanes, 16 loads of each on their way at once
        const int shift = a.tall || a.width == kP ? 7 : 6, mask = (1 << shift) - 1, count = kP * a.width;
        with_type(a.dtype, [&](auto tag) {
            const auto *const g = static_cast<decltype(tag)>(a.g) + at;
#pragma unroll 1
            for (int e0 = threadIdx.x; e0 < count; e0 += 16 * kThreads) {
                float v[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const int e = e0 + k * kThreads, o = e >> shift, c = e & mask, r = a.tall ? c : o, j = column_of(r, a.tall ? o : c), i = r & (rows_p - 1);
                    v[k] = 0.f;
                    if (j >= 0) v[k] = to_f32(g[a.tall ? j * a.row_stride + i : i * a.row_stride + j]);
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const int e = e0 + k * kThreads, o = e >> shift, c = e & mask;
                    sums[(a.tall ? c : o) * kPitch + (a.tall ? o : c)] = v[k];
                    f = fmaf(v[k], v[k], f);
                }
            }
        });
        // the warp's in fp32, unless that leaves its range, or its accurate part: then all again in double
        float all = f;
#pragma unroll
        for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        double s = all;
        if (!(all < 1e30f && all > 1e-30f)) {
            s = 0.;
            for (int e = threadIdx.x; e < count; e += kThreads) {
                const int o = e >> shift, c = e & mask;
                const double v = sums[(a.tall ? c : o) * kPitch + (a.tall ? o : c)];
                s += v * v;
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        }
        if (lane == 0) squares[1 + warp] = s;
        __syncthreads();
        if (threadIdx.x == 0) {
            s = 0.;
            for (int w = 0; w < kThreads / 32; ++w) s += squares[1 + w];
            squares[0] = s;
        }
        __syncthreads();
        cluster_sync();
        // one thread finds the factor: double precision is slow here
        float *const factor = reinterpret_cast<float *>(squares + 10);
        if (warp == 0) {
            s = 0.;
            if (lane < a.ctas)
                asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(s) : "r"(map_to_rank(smem_addr(squares), lane)) : "memory");
#pragma unroll
            for (int o = 8; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0) {
                const double norm = sqrt(s) + static_cast<double>(a.eps);
                // by a power of two first where fp32 does not hold the factor; a matrix of zeros, with no eps, stays one
                factor[0] = norm > 0x1p100 ? 0x1p-100f : norm < 0x1p-100 ? 0x1p100f : 1.f;
                factor[1] = norm == 0. ? 0.f : static_cast<float>(kNsScale / (norm * factor[0]));
            }
        }
        __syncthreads();
        const float first = factor[0], second = factor[1];
        for (int u = threadIdx.x; u < kP * (a.width / 8); u += kThreads) {
            const int i = u & (kP - 1), c = u / kP;
            const float4 lo4 = *reinterpret_cast<const float4 *>(sums + i * kPitch + 8 * c), hi4 = *reinterpret_cast<const float4 *>(sums + i * kPitch + 8 * c + 4);
            float v[8] = {lo4.x, lo4.y, lo4.z, lo4.w, hi4.x, hi4.y, hi4.z, hi4.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = v[e] * first * second;
            uint4 h, l;
            two_parts(v, &h, &l);
            st_shared_v4(base + kXAt + run_at_box(i, c), h);
            st_shared_v4(base + kXAt + 2 * kBox + run_at_box(i, c), l);
        }
    }
    // beside the diagonal A is zero, and what follows from it too
    if (rows_p < kP)
        for (int u = threadIdx.x; u < 4 * kBox / 16; u += kThreads) st_shared_v4(base + kMAt + 16 * u, make_uint4(0u, 0u, 0u, 0u));
    fence_proxy_async_smem();
    __syncthreads();

    const uint32_t x = base + kXAt, m = base + kMAt;
    const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(kP >> 4) << 24);
    const uint32_t square = idesc | (static_cast<uint32_t>(kP >> 3) << 17), across = idesc | (1u << 16) | (static_cast<uint32_t>(a.width >> 3) << 17);
    uint32_t turns = 0;
    // hi hi, hi lo and lo hi, one after another into the same sums; B along k, or across it
    auto multiply = [&](uint32_t acc, uint32_t left, uint32_t right, int k, bool along) {
        if (warp == 0 && elect_one()) {
            tc_fence_after();
            for (int part = 0; part < 3; ++part) {
                const uint32_t l = left + (part == 2 ? 2 * kBox : 0), r = right + (part == 1 ? 2 * kBox : 0);
                for (int q = 0; q < k; q += 16) {
                    const uint32_t inside = (q >> 6) * kBox + (q & 63) * 2;
                    tc_mma_bf16(acc, desc_rows(l + inside), along ? desc_rows(r + inside) : desc_across(r + q * 128), along ? square : across,
                                part > 0 || q > 0);
                }
            }
            tc_commit(bar);
        }
        __syncwarp();
        // on a wait that ran out the rest goes on without its values, so that every barrier is met
        mbar_wait(bar, turns++ & 1, abort_flag, a.timeout_ns, a.status, SITE_S_MMA);
        __syncwarp();
        tc_fence_after();
    };
    const int quad = warp & 3, half = warp >> 2, row = quad * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    // the warp's half of the columns of sums, eight at a time
    auto each8 = [&](uint32_t acc, int width, auto &&f) {
#pragma unroll 1
        for (int c = half * (width / 2); c < (half + 1) * (width / 2); c += 8) {
            uint32_t u[8];
            tmem_ld8_now(acc + c + lanes, u);
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(u[e]);
            f(c, v);
        }
        tc_fence_before();
    };

    for (int step = 0; step < a.steps; ++step) {
        // A, over this CTA's columns
        multiply(tmem, x, x, a.width, true);
        each8(tmem, kP, [&](int c, float (&v)[8]) {
            float *const to = sums + row * kPitch + c;
            *reinterpret_cast<float4 *>(to) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4 *>(to + 4) = make_float4(v[4], v[5], v[6], v[7]);
        });
        __syncthreads();
        cluster_sync();
        // over all columns: every ctas-th row from this CTA's on, a warp a row (of every stretch), four columns a lane, to every CTA
        // (two rows of a warp at a time)
        const int next_row = a.ctas * (kThreads / 32), below = 4 * lane >> SHIFT << SHIFT;      // the lane's stretch
        for (int i0 = rank + a.ctas * warp; i0 < rows_p; i0 += 2 * next_row) {
            float v[2][4] = {};
            for (int r0 = 0; r0 < a.ctas; r0 += 8) {
                uint4 w[2][8];
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int r = 0; r < 8; ++r)
                        w[k][r] = r0 + r < a.ctas && i0 + k * next_row < rows_p
                                      ? load16_at_rank(base + kSumsAt + ((below + i0 + k * next_row) * kPitch + 4 * lane) * 4, r0 + r)
                                      : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        v[k][0] += __uint_as_float(w[k][r].x);
                        v[k][1] += __uint_as_float(w[k][r].y);
                        v[k][2] += __uint_as_float(w[k][r].z);
                        v[k][3] += __uint_as_float(w[k][r].w);
                    }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int i = below + i0 + k * next_row;
                if (i0 + k * next_row >= rows_p) break;
                // the stretches', the same in every lane that holds them
#pragma unroll
                for (int o = rows_p / 4; o < 32; o <<= 1)
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[k][e] += __shfl_xor_sync(0xffffffffu, v[k][e], o);
#pragma unroll
                for (int e = 0; e < 4; ++e) v[k][e] = v[k][e] * a.of_sum + (i == 4 * lane + e ? a.shift : 0.f);
                uint32_t h[2], l[2];
                two_parts(v[k][0], v[k][1], &h[0], &l[0]);
                two_parts(v[k][2], v[k][3], &h[1], &l[1]);
                const uint32_t to = m + run_at_box(i, lane >> 1) + (lane & 1) * 8;
                for (int r = 0; r < a.ctas; ++r) {
                    store8_at_rank(to, r, h[0], h[1]);
                    store8_at_rank(to + 2 * kBox, r, l[0], l[1]);
                }
            }
        }
        fence_proxy_async_all();        // the tensor cores of other CTAs read what this one wrote
        __syncthreads();
        cluster_sync();
        fence_proxy_async_all();
        __syncthreads();
        // P, in A's place
        multiply(tmem + kP, m, m, kP, true);
        each8(tmem + kP, kP, [&](int c, float (&v)[8]) {
            const uint32_t to = m + run_at_box(row, c >> 3);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = v[e] * a.of_square + (row == c + e ? a.of_unit : 0.f);
            if (a.of_a != 0.f) {
                const __half *const tag = nullptr;
                const uint4 h = ld_shared_v4(to), l = ld_shared_v4(to + 2 * kBox);
                const uint32_t hw[4] = {h.x, h.y, h.z, h.w}, lw[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint64_t s = add2(unpack2(hw[q], tag), unpack2(lw[q], tag));
                    v[2 * q] = fmaf(a.of_a, f2_lo(s), v[2 * q]);
                    v[2 * q + 1] = fmaf(a.of_a, f2_hi(s), v[2 * q + 1]);
                }
            }
            uint4 h, l;
            two_parts(v, &h, &l);
            st_shared_v4(to, h);
            st_shared_v4(to + 2 * kBox, l);
        });
        fence_proxy_async_smem();
        __syncthreads();
        // P X, in X's place
        multiply(tmem, m, x, kP, false);
        if (step + 1 == a.steps) break;
        each8(tmem, a.width, [&](int c, float (&v)[8]) {
            const uint32_t to = x + run_at_box(row, c >> 3);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] *= a.of_sum;
            uint4 h, l;
            two_parts(v, &h, &l);
            st_shared_v4(to, h);
            st_shared_v4(to + 2 * kBox, l);
        });
        fence_proxy_async_smem();
        __syncthreads();
    }
    // ------------------------------------------------ the output, through the sums' place
    const float of_out = a.of_sum * a.of_sum;
    each8(tmem, a.width, [&](int c, float (&v)[8]) {
        float *const to = sums + row * kPitch + c;
        *reinterpret_cast<float4 *>(to) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4 *>(to + 4) = make_float4(v[4], v[5], v[6], v[7]);
    });
    __syncthreads();
    const long long out_at = static_cast<long long>(batch) * a.p * a.q;
    const int shift = a.tall || a.width == kP ? 7 : 6, mask = (1 << shift) - 1;
    with_type(a.out_dtype, [&](auto tag) {
        using T = std::remove_const_t<std::remove_pointer_t<decltype(tag)>>;
        T *const out = static_cast<T *>(a.out) + out_at;
#pragma unroll 8
        for (int e = threadIdx.x; e < kP * a.width; e += kThreads) {
            const int o = e >> shift, c = e & mask, r = a.tall ? c : o, at = a.tall ? o : c, j = column_of(r, at), i = r & (rows_p - 1);
            if (j >= 0)
                out[a.tall ? static_cast<long long>(j) * a.p + i : static_cast<long long>(i) * a.q + j] =
                    from_f32<T>(sums[r * kPitch + at] * of_out);
        }
    });
    tc_fence_before();
    __syncthreads();
    cluster_sync();         // nothing of this CTA is read or written any more
    if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

using SmallKernel = void (*)(const SmallArgs);
const SmallKernel kKernels[] = {ns_small_kernel<5>, ns_small_kernel<6>, ns_small_kernel<7>};
// The largest cluster of at most kMost CTAs that the device holds, asked once a device: 0 before, and where it cannot be launched at all -1.
std::atomic<int> g_most[64];
int most_ctas() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return kMost;       // without a device: sizes for the one that the library is for
    }
    int most = g_most[dev & 63].load(std::memory_order_acquire);
    if (most) return most;
    most = -1;
    bool ready = true;
    for (auto kern : kKernels)
        ready = ready && cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) == cudaSuccess &&
                cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
    for (int ctas = kMost; ready && ctas && most < 0; ctas /= 2) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(ctas));
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = kSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kKernels[0], &cfg) == cudaSuccess && n > 0) most = ctas;
    }
    cudaGetLastError();
    g_most[dev & 63].store(most, std::memory_order_release);
    return most;
}

}  // namespace

namespace {
int shift_of(int p) { return p <= 32 ? 5 : p <= 64 ? 6 : 7; }
int stretch_of(int p, int q) { return (q + (kP >> shift_of(p)) - 1) / (kP >> shift_of(p)); }
}  // namespace

bool ns_small_fits_in(int m, int n, int ctas) {
    const int p = m < n ? m : n, q = m < n ? n : m;
    return p <= kP && stretch_of(p, q) <= kP * ctas;
}
bool ns_small_fits(int m, int n) { return ns_small_fits_in(m, n, kMost) && ns_small_fits_in(m, n, most_ctas()); }

int launch_ns_small(const OrthogonalArgs &o, const NsPolynomial &f, unsigned int *status, bool pdl, cudaStream_t s) {
    SmallArgs a = {};
    a.g = o.g;
    a.dtype = o.dtype;
    a.tall = o.m > o.n;
    a.row_stride = o.row_stride;
    a.batch_stride = o.batch_stride;
    a.p = a.tall ? o.n : o.m;
    a.q = a.tall ? o.m : o.n;
    const int most = most_ctas();
    a.stretch = stretch_of(a.p, a.q);
    // the width by how many clusters the GPU holds at once, and by a matrix's time: 128 columns a CTA take a seventh longer than
    // 64 in a cluster of at most 8, and less than 64 in a larger one (128 x 1024 8 % less; 64 x 128 x 512, 115 us, less than half)
    double least = 1e300;
    for (int width : {64, 128}) {
        const int ctas = (a.stretch + width - 1) / width, at_once = kGridCap / ctas;
        const double cost = (width == 128 ? 1.15 : ctas <= 8 ? 1. : 1.25) * ((o.batch + at_once - 1) / at_once);
        if (ctas > most || cost >= least) continue;
        least = cost;
        a.width = width;
        a.ctas = ctas;
    }
    a.steps = o.steps;
    a.eps = o.eps;
    a.of_sum = 1.f / kNsScale;
    a.of_square = f.of_square / kNsScale;
    a.of_a = f.of_a;
    a.shift = f.shift * kNsScale;
    a.of_unit = f.of_unit * kNsScale;
    a.out = o.out;
    a.out_dtype = o.out_dtype;
    a.status = status;
    a.timeout_ns = wait_timeout_ns();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(o.batch) * a.ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(a.ctas);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return note_launch(cudaLaunchKernelEx(&cfg, kKernels[shift_of(a.p) - 5], a));
}

}  // namespace mhc
