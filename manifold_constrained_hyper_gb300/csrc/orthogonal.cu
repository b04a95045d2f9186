// The orthogonalised update: X = G / (|G| + eps), then `steps` times
//   A = X X^T,   P = a I + b A + c A A,   X <- P X          (rows and columns exchanged where G is tall),
// an odd polynomial of G's singular values that drives them towards 1. Bound by its products: with p the
// shorter side and q the longer, 2 p^2 q + 2 p^3 + 2 p^2 q operations a step, of which the two symmetric
// products form half.
//
// What is lost in a weak direction at the first step is amplified with it, by a^steps (480 for five
// steps of 3.4445) against the strong ones, so 11 or 8 bits of X do not give 16-bit results. Every
// matrix is held in two fp16 parts, hi + lo, 22 bits, and every product takes three on the tensor
// cores; sums are fp32. That holds for the last step of a bf16 result too. (By the leading parts alone it took 3 to 15 % less, 4096 x
// 7168 3.0 ms against 3.5, but lost up to 1.7e-3 of the result with the usual coefficients, as much as its rounding, and 3e-2 with (3, -30, 2),
// where b / 2c on A's diagonal all but cancels.) Elements are at most 1 (X), about 1.5 (A) or a (P): a factor of 2^12 in all of them
// keeps what matters of lo above fp16's smallest values, and leaves room for 16 times 1.
//
// By size: orthogonal_small.cu where a side is at most 128 and the other not too long, else this file's two kernels (the norm; X in two parts) and
// orthogonal_kernel.cu's one. 4096 x 7168 3.28 ms in a burst, 2048 x 1024 201 us, 256 x 256 99, 6 x 128 x 500 49.
//
// G may lie in strided rows. A tall G is not turned: its Gram matrix is X^T X, the product reading both
// operands with the summed axis outermost.
#include "orthogonal.h"
#include "vec_io.cuh"

namespace mhc {
namespace {

constexpr float kScale = kNsScale;
constexpr int kNormParts = 64;                      // shares of a matrix's squares
constexpr int kRuns = 4;

struct Shape {
    int p, q;                       // the shorter and the longer side
    long long x_pitch, p_pitch;     // elements of a row of X, of A and P
    long long x_size, p_size;       // elements of one matrix
    size_t parts_at, x_at, a_at, sums_at, counters_at, total;
};
long long pitch8(long long w) { return (w + 7) / 8 * 8; }
size_t up256(size_t b) { return (b + 255) & ~static_cast<size_t>(255); }
Shape shape_of(int batch, int m, int n) {
    Shape s;
    s.p = m < n ? m : n;
    s.q = m < n ? n : m;
    s.x_pitch = pitch8(n);
    s.p_pitch = pitch8(s.p);
    s.x_size = up256(static_cast<size_t>(m) * s.x_pitch * 2) / 2;
    s.p_size = up256(static_cast<size_t>(s.p) * s.p_pitch * 2) / 2;
    s.parts_at = 0;
    s.x_at = up256(static_cast<size_t>(batch) * kNormParts * 8);
    s.a_at = s.x_at + 4 * static_cast<size_t>(batch) * s.x_size * 2;
    s.sums_at = s.a_at + 8 * static_cast<size_t>(batch) * s.p_size * 2;
    s.counters_at = s.sums_at + kNsPartsBytes;
    s.total = s.counters_at + up256(kNsCounters * 4);
    return s;
}

// A share of the sum of one matrix's squares, in double between threads. A share that
// leaves fp32's range, or its accurate part, is formed again in double throughout.
template <class T>
__global__ void __launch_bounds__(256) ns_norm_kernel(const T *g, long long row_stride, long long batch_stride, int m, int n, bool runs,
                                                      double *parts, unsigned int *counters) {
    __shared__ double red[8];
    griddep_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int i = threadIdx.x; i < kNsCounters; i += 256) counters[i] = 0;
    const long long per_row = (n + 7) / 8, total = per_row * m;
    const T *const x = g + blockIdx.y * batch_stride;
    const long long step = static_cast<long long>(gridDim.x) * 256;
    auto load = [&](long long i) {
        const long long t = i / per_row;
        const int c = static_cast<int>(i - t * per_row) * 8;
        return runs ? load8(x + t * row_stride + c) : load8_any(x + t * row_stride, c, n);
    };
    double s = 0.;
    for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < total; i += step * kRuns) {
        Run v[kRuns];
#pragma unroll
        for (int r = 0; r < kRuns; ++r) {
            v[r] = run_splat(0.f);
            if (i + r * step < total) v[r] = load(i + r * step);
        }
        uint64_t q2 = 0ull;
#pragma unroll
        for (int r = 0; r < kRuns; ++r)
#pragma unroll
            for (int q = 0; q < 4; ++q) q2 = fma2(v[r].p[q], v[r].p[q], q2);
        const float f = f2_lo(q2) + f2_hi(q2);
        if (f < 1e30f && f > 1e-30f) {
            s += f;
        } else {
#pragma unroll
            for (int r = 0; r < kRuns; ++r)
#pragma unroll
                for (int e = 0; e < 8; ++e) s += static_cast<double>(run_at(v[r], e)) * run_at(v[r], e);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x) return;
    s = 0.;
    for (int w = 0; w < 8; ++w) s += red[w];
    parts[blockIdx.y * kNormParts + blockIdx.x] = s;
}

// X in two fp16 parts, times 2^12.
template <class T>
__global__ void __launch_bounds__(256) ns_split_kernel(const T *g, long long row_stride, long long batch_stride, int m, int n, bool runs,
                                                       float eps, const double *parts, int count, __half *hi, __half *lo, long long pitch,
                                                       long long size) {
    __shared__ float factor[2];
    griddep_wait();
    if (threadIdx.x < 32) {
        double s = 0.;
        for (int p = threadIdx.x; p < count; p += 32) s += parts[blockIdx.y * kNormParts + p];
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (threadIdx.x == 0) {
            // by a power of two first where fp32 does not hold the factor
            const double norm = sqrt(s) + static_cast<double>(eps);
            const float first = norm > 0x1p100 ? 0x1p-100f : norm < 0x1p-100 ? 0x1p100f : 1.f;
            factor[0] = first;
            // a matrix of zeros, with no eps, stays one
            factor[1] = norm == 0. ? 0.f : static_cast<float>(kScale / (norm * first));
        }
    }
    __syncthreads();
    const float f0 = factor[0], f1 = factor[1];
    const long long per_row = (n + 7) / 8, total = per_row * m;
    const T *const x = g + blockIdx.y * batch_stride;
    hi += blockIdx.y * size;
    lo += blockIdx.y * size;
    for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < total; i += static_cast<long long>(gridDim.x) * 256) {
        const long long t = i / per_row;
        const int c = static_cast<int>(i - t * per_row) * 8;
        const Run v = runs ? load8(x + t * row_stride + c) : load8_any(x + t * row_stride, c, n);
        uint4 hw, lw;
        uint32_t *const hp = &hw.x, *const lp = &lw.x;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint64_t y = mul2(mul2(v.p[q], splat2(f0)), splat2(f1));
            hp[q] = pack2(y, static_cast<const __half *>(nullptr));
            lp[q] = pack2(fma2(unpack2(hp[q], static_cast<const __half *>(nullptr)), splat2(-1.f), y), static_cast<const __half *>(nullptr));
        }
        *reinterpret_cast<uint4 *>(hi + t * pitch + c) = hw;
        *reinterpret_cast<uint4 *>(lo + t * pitch + c) = lw;
    }
}

template <class T>
int launch_start(const OrthogonalArgs &a, const Shape &sh, const NsCall &c, int sms, bool pdl, cudaStream_t s) {
    const T *const g = static_cast<const T *>(a.g);
    const bool runs = a.n % 8 == 0 && a.row_stride % 8 == 0 && a.batch_stride % 8 == 0 &&
                      (reinterpret_cast<uintptr_t>(g) & (sizeof(T) == 4 ? 31u : 15u)) == 0;
    double *const parts = reinterpret_cast<double *>(static_cast<uint8_t *>(a.workspace) + sh.parts_at);
    const long long all = static_cast<long long>(a.m) * ((a.n + 7) / 8);
    // shares of 1024 runs at least, and not more of them than fill the machine four times
    long long count = (all + 1023) / 1024, most = (4LL * sms + a.batch - 1) / a.batch;
    if (most > kNormParts) most = kNormParts;
    if (count > most) count = most;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(count), a.batch);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    if (int e = note_launch(cudaLaunchKernelEx(&cfg, ns_norm_kernel<T>, g, a.row_stride, a.batch_stride, a.m, a.n, runs, parts, c.counters))) return e;
    long long blocks = (all + 255) / 256, cap = (8LL * sms + a.batch - 1) / a.batch;
    if (blocks > cap) blocks = cap;
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), a.batch);
    return note_launch(cudaLaunchKernelEx(&cfg, ns_split_kernel<T>, g, a.row_stride, a.batch_stride, a.m, a.n, runs, a.eps,
                                          static_cast<const double *>(parts), static_cast<int>(count), c.x[0][0], c.x[0][1], sh.x_pitch, sh.x_size));
}

}  // namespace

size_t orthogonal_workspace(int batch, int m, int n) { return ns_small_fits(m, n) ? 0 : shape_of(batch, m, n).total; }

int launch_orthogonal(const OrthogonalArgs &a, int sms, unsigned int *status, bool pdl, cudaStream_t s) {
    if (ns_small_fits(a.m, a.n)) return launch_ns_small(a, ns_polynomial(a.a, a.b, a.c, true), status, pdl, s);
    const Shape sh = shape_of(a.batch, a.m, a.n);
    uint8_t *const ws = static_cast<uint8_t *>(a.workspace);
    __half *const x = reinterpret_cast<__half *>(ws + sh.x_at), *const p = reinterpret_cast<__half *>(ws + sh.a_at);
    const long long xs = sh.x_size * a.batch, ps = sh.p_size * a.batch;
    NsCall c = {a.batch, a.m, a.n, a.steps, a.a, a.b, a.c, {{x, x + xs}, {x + 2 * xs, x + 3 * xs}}, {{p, p + ps}, {p + 2 * ps, p + 3 * ps}, {p + 4 * ps, p + 5 * ps}, {p + 6 * ps, p + 7 * ps}},
                sh.x_pitch, sh.x_size, sh.p_pitch, sh.p_size, a.out, a.out_dtype, reinterpret_cast<float *>(ws + sh.sums_at),
                reinterpret_cast<unsigned int *>(ws + sh.counters_at)};
    const int e = a.dtype == MHC_F32    ? launch_start<float>(a, sh, c, sms, pdl, s)
                  : a.dtype == MHC_BF16 ? launch_start<__nv_bfloat16>(a, sh, c, sms, pdl, s)
                                        : launch_start<__half>(a, sh, c, sms, pdl, s);
    return e ? e : launch_ns(c, status, s);
}

}  // namespace mhc
