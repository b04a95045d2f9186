// Layer norm's row kernels share: a group of warps holds a row, eight consecutive columns a run.
#pragma once
#include <atomic>

#include "linear_internal.h"
#include "vec_io.cuh"

namespace mhc {

constexpr int kLnThreads = 512;                     // of a CTA: as many groups as fit
constexpr int kLnMaxHeld = 8192;                    // columns that a group holds in registers

// Sums over a group of `warps` warps (whole ones), the same in every thread. red: [2][16][N] floats of the
// group; `turn` alternates between calls, so that one barrier a call is enough.
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], int warps, int warp, int lane, int barrier, float *red, int *turn) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] += __shfl_xor_sync(0xffffffffu, v[e], o);
    if (warps == 1) return;
    float *const here = red + *turn * 16 * N;
    *turn ^= 1;
    if (lane == 0)
#pragma unroll
        for (int e = 0; e < N; ++e) here[warp * N + e] = v[e];
    named_barrier_sync(barrier, warps * 32);
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = lane < warps ? here[lane * N + e] : 0.f;
#pragma unroll
    for (int o = 8; o; o >>= 1)
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] += __shfl_xor_sync(0xffffffffu, v[e], o);
    // lanes 16 and up hold the sum of nothing
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = __shfl_sync(0xffffffffu, v[e], 0);
}
template <bool RUNS, class T>
__device__ __forceinline__ Run ln_load(const T *row, int c, int H) {
    if constexpr (RUNS) return load8(row + c);
    else return load8_any(row, c, H);
}
template <bool RUNS, class T>
__device__ __forceinline__ void ln_store(T *row, int c, int H, const Run &r) {
    if constexpr (RUNS) store8(row + c, r);
    else store8_any(row + c, r, (reinterpret_cast<uintptr_t>(row + c) & (2 * sizeof(T) - 1)) == 0, H - c < 8 ? H - c : 8);
}
// 8 parameters from column c on; `otherwise` where there are none.
template <bool RUNS>
__device__ __forceinline__ Run ln_param(const void *p, int dtype, int c, int H, float otherwise) {
    if (!p) return run_splat(otherwise);
    if (dtype == MHC_F32) return ln_load<RUNS>(static_cast<const float *>(p), c, H);
    if (dtype == MHC_BF16) return ln_load<RUNS>(static_cast<const __nv_bfloat16 *>(p), c, H);
    return ln_load<RUNS>(static_cast<const __half *>(p), c, H);
}
// Lanes past the row's end hold 0 of v.
__device__ __forceinline__ Run ln_masked(Run v, int c, int H) {
    if (c + 8 <= H) return v;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = c + e < H ? run_at(v, e) : 0.f;
    return run_of(f);
}
__device__ __forceinline__ float run_sum(const Run &r) {
    const uint64_t s = add2(add2(r.p[0], r.p[1]), add2(r.p[2], r.p[3]));
    return f2_lo(s) + f2_hi(s);
}

// ---------------------------------------------------------------- staged rows
// Rows on the way to shared memory by bulk copies while others are worked on: each group of warps has
// `stages` places of its own, filled in turn; row k of the group is the k/stages-th filling of place
// k % stages, and thread 0 of the group orders the next one when the group has the row in registers. A wait
// that runs out raises the flag, after which none waits: the CTA then goes through its rows without
// their values, so that no thread misses a barrier, and the status says so.
constexpr int kLnArrays = 3;
struct LnRing {
    int stages, row_bytes[kLnArrays], stage_bytes;      // of each array (a multiple of 16), 0 where there is none
    unsigned int *status;
    unsigned long long timeout_ns;
};
// The kernels' limit of shared memory, set once a device and kernel (each has its own `done`).
inline cudaError_t ln_allow_smem(const void *kern, int bytes, std::atomic<uint64_t> *done) {
    int dev = 0;
    if (cudaError_t e = cudaGetDevice(&dev)) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
    if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) return e;
    done->fetch_or(bit, std::memory_order_release);
    return cudaSuccess;
}
enum LnSite : int { SITE_LN_ROW = 120, SITE_LN_DRAIN };

struct LnStages {
    const LnRing &ring;
    uint32_t bars, base;                            // of the group
    uint8_t *basep;
    volatile int *abort_flag;

    __device__ __forceinline__ void order(int k, const void *const (&src)[kLnArrays]) const {
        const int s = k % ring.stages;
        uint32_t total = 0, dst = base + s * ring.stage_bytes;
#pragma unroll
        for (int i = 0; i < kLnArrays; ++i) total += ring.row_bytes[i];
        mbar_arrive_expect_tx(bars + 8 * s, total);
        const uint64_t policy = policy_evict_first();
#pragma unroll
        for (int i = 0; i < kLnArrays; ++i) {
            if (!ring.row_bytes[i]) continue;
            bulk_load(dst, src[i], ring.row_bytes[i], bars + 8 * s, policy);
            dst += ring.row_bytes[i];
        }
    }
    __device__ __forceinline__ void wait(int k) const {
        mbar_wait(bars + 8 * (k % ring.stages), (k / ring.stages) & 1, abort_flag, ring.timeout_ns, ring.status, SITE_LN_ROW);
    }
    // Gave up: the copies still on their way land before the CTA exits. `ordered`: how many rows were.
    __device__ __forceinline__ void drain(int ordered) const {
        int gave_up = 0;
        for (int k = ordered > ring.stages ? ordered - ring.stages : 0; k < ordered; ++k)
            mbar_wait(bars + 8 * (k % ring.stages), (k / ring.stages) & 1, &gave_up, ring.timeout_ns, ring.status, SITE_LN_DRAIN);
    }
    __device__ __forceinline__ const uint8_t *row(int k, int array) const {
        int at = k % ring.stages * ring.stage_bytes;
        for (int i = 0; i < array; ++i) at += ring.row_bytes[i];
        return basep + at;
    }
};

}  // namespace mhc
