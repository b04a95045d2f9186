// 8-bit activation checkpoints: packing and reading back. Both are bound by
// memory: 2 bytes in and 1 + 1/32 out for a 16-bit value, and the reverse.
#include "vec_io.cuh"

namespace mhc {
namespace {

constexpr int kThreads = 256;

// Eight values a lane, four lanes a group. A lane has kRuns runs in flight, each a block's width
// from the next; the lanes past a row's end (where H is no multiple of 32)
// hold zeros, so that every lane takes part in its group's maximum. Rows and codes on
// boundaries of 8 elements (EVEN) by one access; else loads of the words that hold a run and, where
// what is written lies elsewhere, stores of two elements or one (packing and reading back 8192 x 7168
// bf16: 57.6 us, 0.92 of a copy's rate; strided by 7171 81 us, a warp a group 222; 7170 wide 100, 7169 243).
constexpr int kRuns = 4;

// Run i of the call -> its row and column; false past the end or the row's end.
template <class I>
__device__ __forceinline__ bool run_place(I i, I total, I per_row, int H, long long *t, int *c) {
    const I row = i / per_row;
    *t = static_cast<long long>(row);
    *c = static_cast<int>(i - row * per_row) * 8;
    return i < total && *c < H;
}

template <class T, int FMT, class I, bool EVEN>
__global__ void __launch_bounds__(kThreads) ckpt_pack_kernel(const CkptArgs a, int unit) {
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
            if (!in[r]) continue;
            const T *const row = static_cast<const T *>(a.x) + t[r] * a.stride;
            if constexpr (EVEN) v[r] = load8(row + c[r]);
            else v[r] = load8_any(row, c[r], a.H);
        }
#pragma unroll
        for (int r = 0; r < kRuns; ++r) {
            const uint32_t byte = ckpt_byte_quad<FMT>(v[r]);
            if (!in[r]) continue;
            uint8_t *const codes = a.c.codes + t[r] * a.H + c[r];
            const uint2 w = ckpt_codes8<FMT>(v[r], byte);
            if (EVEN || unit == 8) {
                *reinterpret_cast<uint2 *>(codes) = w;
            } else {
                const uint64_t word[1] = {static_cast<uint64_t>(w.y) << 32 | w.x};
                store_words<1>(codes, word, unit == 2, a.H - c[r] < 8 ? a.H - c[r] : 8);
            }
            if ((threadIdx.x & 3) == 0) a.c.scales[t[r] * groups + c[r] / 32] = static_cast<uint8_t>(byte);
        }
    }
}

template <class T, int FMT, class I, bool EVEN>
__global__ void __launch_bounds__(kThreads) ckpt_unpack_kernel(const CkptArgs a, int unit) {
    griddep_wait();
    const I per_row = static_cast<I>((a.H + 7) / 8), total = static_cast<I>(a.T) * per_row;
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
            const uint8_t *const codes = a.c.codes + t[r] * a.H;
            if constexpr (EVEN) {
                w[r] = *reinterpret_cast<const uint2 *>(codes + c[r]);
            } else {
                uint64_t word[1];
                load_words<1>(reinterpret_cast<uintptr_t>(codes + c[r]), reinterpret_cast<uintptr_t>(codes + a.H), word);
                w[r] = make_uint2(static_cast<uint32_t>(word[0]), static_cast<uint32_t>(word[0] >> 32));
            }
            byte[r] = a.c.scales[t[r] * groups + c[r] / 32];
        }
#pragma unroll
        for (int r = 0; r < kRuns; ++r) {
            if (!in[r]) continue;
            T *const out = static_cast<T *>(a.out) + t[r] * a.stride + c[r];
            const Run v = ckpt_values8(w[r], byte[r], FMT);
            if (EVEN || unit == 8) store8(out, v);
            else store8_any(out, v, unit == 2, a.H - c[r] < 8 ? a.H - c[r] : 8);
        }
    }
}

// Elements that the address of every run of 8 is a multiple of: 8, 2 or 1.
int unit_of(const void *p, int elem, long long stride, int H, long long T) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if (H % 8 == 0 && at % (8 * elem) == 0 && (T == 1 || stride % 8 == 0)) return 8;
    return at % (2 * elem) == 0 && (T == 1 || stride % 2 == 0) ? 2 : 1;
}
// The index type: 32 bits where the runs and a grid's step past them fit.
bool small_index(const CkptArgs &a) { return a.T * ckpt_groups(a.H) * 4 < (1ll << 31); }
unsigned runs_grid(const CkptArgs &a, int sms) {
    const long long runs = a.T * ckpt_groups(a.H) * 4;
    const long long need = (runs + kThreads * kRuns - 1) / (kThreads * kRuns), cap = static_cast<long long>(sms) * 8;
    return static_cast<unsigned>(need < cap ? need : cap);
}
template <class T, int FMT>
cudaError_t pack(const CkptArgs &a, int sms, bool pdl, cudaStream_t s) {
    const int unit = unit_of(a.c.codes, 1, a.H, a.H, a.T);
    auto kern = unit == 8 && unit_of(a.x, sizeof(T), a.stride, a.H, a.T) == 8
                    ? (small_index(a) ? ckpt_pack_kernel<T, FMT, unsigned, true> : ckpt_pack_kernel<T, FMT, unsigned long long, true>)
                    : (small_index(a) ? ckpt_pack_kernel<T, FMT, unsigned, false> : ckpt_pack_kernel<T, FMT, unsigned long long, false>);
    return launch_block_kernel(kern, runs_grid(a, sms), kThreads, 0, pdl, s, a, unit);
}
template <class T, int FMT>
cudaError_t unpack(const CkptArgs &a, int sms, bool pdl, cudaStream_t s) {
    const int unit = unit_of(a.out, sizeof(T), a.stride, a.H, a.T);
    auto kern = unit == 8 && unit_of(a.c.codes, 1, a.H, a.H, a.T) == 8
                    ? (small_index(a) ? ckpt_unpack_kernel<T, FMT, unsigned, true> : ckpt_unpack_kernel<T, FMT, unsigned long long, true>)
                    : (small_index(a) ? ckpt_unpack_kernel<T, FMT, unsigned, false> : ckpt_unpack_kernel<T, FMT, unsigned long long, false>);
    return launch_block_kernel(kern, runs_grid(a, sms), kThreads, 0, pdl, s, a, unit);
}
template <class T>
cudaError_t pack(const CkptArgs &a, int format, int sms, bool pdl, cudaStream_t s) {
    return format == MHC_CKPT_E4M3 ? pack<T, MHC_CKPT_E4M3>(a, sms, pdl, s) : pack<T, MHC_CKPT_INT8>(a, sms, pdl, s);
}
template <class T>
cudaError_t unpack(const CkptArgs &a, int format, int sms, bool pdl, cudaStream_t s) {
    return format == MHC_CKPT_E4M3 ? unpack<T, MHC_CKPT_E4M3>(a, sms, pdl, s) : unpack<T, MHC_CKPT_INT8>(a, sms, pdl, s);
}

}  // namespace

cudaError_t launch_ckpt_pack(const CkptArgs &a, int dtype, int format, int sms, bool pdl, cudaStream_t s) {
    auto run = dtype == MHC_F32 ? pack<float> : dtype == MHC_BF16 ? pack<__nv_bfloat16> : pack<__half>;
    return run(a, format, sms, pdl, s);
}

cudaError_t launch_ckpt_unpack(const CkptArgs &a, int dtype, int format, int sms, bool pdl, cudaStream_t s) {
    // what a finite value's checkpoint stands for may lie past fp16's largest (65504: 65536), and stays finite
    auto run = dtype == MHC_F32 ? unpack<float> : dtype == MHC_BF16 ? unpack<__nv_bfloat16> : unpack<FiniteHalf>;
    return run(a, format, sms, pdl, s);
}

}  // namespace mhc
