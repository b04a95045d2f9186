// 8-bit activation checkpoints: packing and reading back. Both are bound by
// memory: 2 bytes in and 1 + 1/32 out for a 16-bit value, and the reverse.
#include "vec_io.cuh"

namespace mhc {
namespace {

constexpr int kThreads = 256;

// A warp per group of 32 values: any width, stride and alignment.
template <class T>
__global__ void ckpt_pack_kernel(const CkptArgs a, int format) {
    griddep_wait();
    const int groups = (a.H + 31) / 32, lane = threadIdx.x & 31;
    const long long total = a.T * groups, step = static_cast<long long>(gridDim.x) * (kThreads / 32);
    for (long long i = static_cast<long long>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; i < total;
         i += step) {
        const long long t = i / groups;
        const int g = static_cast<int>(i - t * groups), c = g * 32 + lane;
        const float x = c < a.H ? to_f32(static_cast<const T *>(a.x)[t * a.stride + c]) : 0.f;
        ckpt_store_lane(a.c, format, t, a.H, groups, g, lane, x);
    }
}

template <class T>
__global__ void ckpt_unpack_kernel(const CkptArgs a, int format) {
    griddep_wait();
    const int groups = (a.H + 31) / 32, lane = threadIdx.x & 31;
    const long long total = a.T * groups, step = static_cast<long long>(gridDim.x) * (kThreads / 32);
    for (long long i = static_cast<long long>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; i < total;
         i += step) {
        const long long t = i / groups;
        const int g = static_cast<int>(i - t * groups), c = g * 32 + lane;
        if (c < a.H)
            static_cast<T *>(a.out)[t * a.stride + c] = from_f32<T>(ckpt_load(a.c, format, t, a.H, groups, c));
    }
}

// Eight values a lane, four lanes a group, for rows on boundaries of 8 elements
// with H a multiple of 8. A lane has kRuns runs in flight, each a block's width
// from the next; the lanes past a row's end (where H is no multiple of 32)
// hold zeros, so that every lane takes part in its group's maximum.
constexpr int kRuns = 4;

// Run i of the call -> its row and column; false past the end or the row's end.
template <class I>
__device__ __forceinline__ bool run_place(I i, I total, I per_row, int H, long long *t, int *c) {
    const I row = i / per_row;
    *t = static_cast<long long>(row);
    *c = static_cast<int>(i - row * per_row) * 8;
    return i < total && *c < H;
}

template <class T, int FMT, class I>
__global__ void __launch_bounds__(kThreads) ckpt_pack_vec_kernel(const CkptArgs a) {
    griddep_wait();
    const I per_row = static_cast<I>((a.H + 31) / 32) * 4, total = static_cast<I>(a.T) * per_row;
    const I step = static_cast<I>(gridDim.x) * (kThreads * kRuns);
    const int groups = (a.H + 31) / 32;
    // whole warps enter: a warp's runs start at a multiple of 32, and total is one of 4
    for (I i0 = static_cast<I>(blockIdx.x) * (kThreads * kRuns) + (threadIdx.x & ~31u); i0 < total; i0 += step) {
        Run v[kRuns];
        long long t[kRuns];
        int c[kRuns];
        bool in[kRuns];
#pragma unroll
        for (int r = 0; r < kRuns; ++r) {
            in[r] = run_place<I>(i0 + r * kThreads + (threadIdx.x & 31), total, per_row, a.H, &t[r], &c[r]);
            v[r] = run_splat(0.f);
            if (in[r]) v[r] = load8(static_cast<const T *>(a.x) + t[r] * a.stride + c[r]);
        }
#pragma unroll
        for (int r = 0; r < kRuns; ++r) {
            const uint32_t byte = ckpt_byte_quad<FMT>(v[r]);
            if (!in[r]) continue;
            *reinterpret_cast<uint2 *>(a.c.codes + t[r] * a.H + c[r]) = ckpt_codes8<FMT>(v[r], byte);
            if ((threadIdx.x & 3) == 0) a.c.scales[t[r] * groups + c[r] / 32] = static_cast<uint8_t>(byte);
        }
    }
}

template <class T, int FMT, class I>
__global__ void __launch_bounds__(kThreads) ckpt_unpack_vec_kernel(const CkptArgs a) {
    griddep_wait();
    const I per_row = static_cast<I>(a.H / 8), total = static_cast<I>(a.T) * per_row;
    const I step = static_cast<I>(gridDim.x) * (kThreads * kRuns);
    const int groups = (a.H + 31) / 32;
    for (I i0 = static_cast<I>(blockIdx.x) * (kThreads * kRuns) + threadIdx.x; i0 < total; i0 += step) {
        uint2 w[kRuns];
        uint32_t byte[kRuns];
        long long t[kRuns];
        int c[kRuns];
        bool in[kRuns];
#pragma unroll
        for (int r = 0; r < kRuns; ++r) {
            in[r] = run_place<I>(i0 + r * kThreads, total, per_row, a.H, &t[r], &c[r]);
            if (!in[r]) continue;
            w[r] = *reinterpret_cast<const uint2 *>(a.c.codes + t[r] * a.H + c[r]);
            byte[r] = a.c.scales[t[r] * groups + c[r] / 32];
        }
#pragma unroll
        for (int r = 0; r < kRuns; ++r) {
            if (!in[r]) continue;
            store8(static_cast<T *>(a.out) + t[r] * a.stride + c[r], ckpt_values8(w[r], byte[r], FMT));
        }
    }
}

// Whether the runs of 8 are there: rows of x on boundaries of 8 elements, of codes on 8-byte ones.
bool runs_fit(const CkptArgs &a, const void *x, int elem) {
    return a.H % 8 == 0 && reinterpret_cast<uintptr_t>(x) % (8 * elem) == 0 &&
           (reinterpret_cast<uintptr_t>(a.c.codes) & 7u) == 0 && (a.T == 1 || a.stride % 8 == 0);
}
// The index type: 32 bits where the runs and a grid's step past them fit.
bool small_index(const CkptArgs &a) { return a.T * ckpt_groups(a.H) * 4 < (1ll << 31); }
unsigned runs_grid(const CkptArgs &a, int sms) {
    const long long runs = a.T * ckpt_groups(a.H) * 4;
    const long long need = (runs + kThreads * kRuns - 1) / (kThreads * kRuns), cap = static_cast<long long>(sms) * 8;
    return static_cast<unsigned>(need < cap ? need : cap);
}
template <class T, int FMT>
cudaError_t pack_vec(const CkptArgs &a, int sms, bool pdl, cudaStream_t s) {
    return launch_block_kernel(small_index(a) ? ckpt_pack_vec_kernel<T, FMT, unsigned>
                                              : ckpt_pack_vec_kernel<T, FMT, unsigned long long>,
                               runs_grid(a, sms), kThreads, 0, pdl, s, a);
}
template <class T, int FMT>
cudaError_t unpack_vec(const CkptArgs &a, int sms, bool pdl, cudaStream_t s) {
    return launch_block_kernel(small_index(a) ? ckpt_unpack_vec_kernel<T, FMT, unsigned>
                                              : ckpt_unpack_vec_kernel<T, FMT, unsigned long long>,
                               runs_grid(a, sms), kThreads, 0, pdl, s, a);
}
template <class T>
cudaError_t pack_any(const CkptArgs &a, int format, int sms, bool pdl, cudaStream_t s) {
    return format == MHC_CKPT_E4M3 ? pack_vec<T, MHC_CKPT_E4M3>(a, sms, pdl, s) : pack_vec<T, MHC_CKPT_INT8>(a, sms, pdl, s);
}
template <class T>
cudaError_t unpack_any(const CkptArgs &a, int format, int sms, bool pdl, cudaStream_t s) {
    return format == MHC_CKPT_E4M3 ? unpack_vec<T, MHC_CKPT_E4M3>(a, sms, pdl, s)
                                   : unpack_vec<T, MHC_CKPT_INT8>(a, sms, pdl, s);
}

unsigned grid_for(long long groups, int sms) {
    const long long need = (groups + kThreads / 32 - 1) / (kThreads / 32), cap = static_cast<long long>(sms) * 8;
    return static_cast<unsigned>(need < cap ? need : cap);
}

}  // namespace

cudaError_t launch_ckpt_pack(const CkptArgs &a, int dtype, int format, int sms, bool pdl, cudaStream_t s) {
    if (runs_fit(a, a.x, dtype == MHC_F32 ? 4 : 2))
        return dtype == MHC_F32 ? pack_any<float>(a, format, sms, pdl, s)
               : dtype == MHC_BF16 ? pack_any<__nv_bfloat16>(a, format, sms, pdl, s)
                                   : pack_any<__half>(a, format, sms, pdl, s);
    const unsigned grid = grid_for(a.T * ckpt_groups(a.H), sms);
    auto kern = dtype == MHC_F32 ? ckpt_pack_kernel<float>
                : dtype == MHC_BF16 ? ckpt_pack_kernel<__nv_bfloat16> : ckpt_pack_kernel<__half>;
    return launch_block_kernel(kern, grid, kThreads, 0, pdl, s, a, format);
}

cudaError_t launch_ckpt_unpack(const CkptArgs &a, int dtype, int format, int sms, bool pdl, cudaStream_t s) {
    if (runs_fit(a, a.out, dtype == MHC_F32 ? 4 : 2))
        return dtype == MHC_F32 ? unpack_any<float>(a, format, sms, pdl, s)
               : dtype == MHC_BF16 ? unpack_any<__nv_bfloat16>(a, format, sms, pdl, s)
                                   : unpack_any<__half>(a, format, sms, pdl, s);
    const unsigned grid = grid_for(a.T * ckpt_groups(a.H), sms);
    auto kern = dtype == MHC_F32 ? ckpt_unpack_kernel<float>
                : dtype == MHC_BF16 ? ckpt_unpack_kernel<__nv_bfloat16> : ckpt_unpack_kernel<__half>;
    return launch_block_kernel(kern, grid, kThreads, 0, pdl, s, a, format);
}

}  // namespace mhc
