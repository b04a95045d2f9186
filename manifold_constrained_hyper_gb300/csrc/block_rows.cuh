// What the row kernels of the gated residual block share: which columns a
// thread holds, group-wide sums, rows staged in shared memory by bulk copies.
#pragma once
#include <atomic>

#include "mhc_internal.h"
#include "vec_io.cuh"

namespace mhc {

// How a row kernel gets its rows.
enum RowMode : int {
    ROWS_RING = 0,      // staged ahead of use by bulk copies (rows on 16-byte boundaries)
    ROWS_VEC = 1,       // 16-byte loads (the same, or a few rows only)
    ROWS_ANY = 2        // single elements, any boundary
};
// A thread's COLS columns: run j covers VEC of them from (j * threads + thread) * VEC.
template <int MODE, int COLS>
struct Runs {
    static constexpr int kVec = MODE == ROWS_ANY ? 1 : 8;
    static constexpr int kRuns = COLS / kVec;
};
inline int row_threads(int H, int cols) { return ((H + cols - 1) / cols + 31) / 32 * 32; }

// Sums of N values over a group of `warps` whole warps that share the named
// barrier `bar`, in one fixed order, for every thread of it. `red`: 32 N floats of the
// group's own; the caller alternates between two, so that a value is read by
// all before it is written again.
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float *red, int bar, int warp, int warps) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (warps == 1) return;
    if (lane == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) red[k * 32 + warp] = v[k];
    }
    named_barrier_sync(bar, warps * 32);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        v[k] = lane < warps ? red[k * 32 + lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
}

// VEC parameters (weights, scales) of a run; past the row's end `fill`.
template <int VEC>
__device__ __forceinline__ void load_params(const void *p, int dtype, int c, float (&v)[VEC]) {
    if (dtype == MHC_F32) load_run<VEC>(static_cast<const float *>(p) + c, v);
    else if (dtype == MHC_BF16) load_run<VEC>(static_cast<const __nv_bfloat16 *>(p) + c, v);
    else load_run<VEC>(static_cast<const __half *>(p) + c, v);
}
template <int VEC>
__device__ __forceinline__ void load_weights(const void *w, int dtype, float offset, int c, float (&v)[VEC]) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = 1.f;
        return;
    }
    load_params<VEC>(w, dtype, c, v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] += offset;
}
template <int VEC>
__device__ __forceinline__ void load_scale(const BlockForm &f, int c, float (&v)[VEC]) {
    if (f.scale_form == MHC_SCALE_CHANNEL) {
        load_run<VEC>(f.res_scale + c, v);
        return;
    }
    const float a = f.scale_form == MHC_SCALE_ONE ? *f.res_scale : 1.f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = a;
}
template <int VEC>
__device__ __forceinline__ void gate_values(float (&v)[VEC], int act) {
    if (act == MHC_ACT_NONE) return;
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = gate_value(v[e], act);
}

// A row's bytes are a multiple of 16 and so are its address and stride.
inline bool rows16(const void *p, long long stride, int H, int elem, long long T) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && static_cast<long long>(H) * elem % 16 == 0 &&
           (T == 1 || stride * elem % 16 == 0);
}
inline int elem_bytes(int dtype) { return dtype == MHC_F32 ? 4 : 2; }
// Weights and scales can be read 8 at a time.
inline bool params16(const BlockForm &f) {
    const void *const p[] = {f.w_post, f.w_pre, f.scale_form == MHC_SCALE_CHANNEL ? f.res_scale : nullptr,
                             f.gate_form == MHC_GATE_CHANNEL ? f.gate : nullptr};
    for (const void *q : p)
        if (reinterpret_cast<uintptr_t>(q) & 15u) return false;
    return true;
}

// Opts a kernel in to `smem` bytes of dynamic shared memory (all of its calls: at most `most`), once per device.
struct SmemGrant {
    std::atomic<int> bytes[64];
};
template <class K>
inline cudaError_t grant_smem(K kern, SmemGrant &g, size_t smem, size_t most) {
    if (smem <= 48 * 1024) return cudaSuccess;
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    std::atomic<int> &cur = g.bytes[dev & 63];
    if (cur.load(std::memory_order_acquire)) return cudaSuccess;
    if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most)))
        return e;
    cur.store(1, std::memory_order_release);
    return cudaSuccess;
}

}  // namespace mhc
