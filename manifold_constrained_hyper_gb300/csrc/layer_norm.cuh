// Layer norm's row kernels share: a group of warps holds a row, eight consecutive columns a run.
#pragma once
#include <atomic>

#include "layer_norm_shape.h"
#include "linear_internal.h"
#include "vec_io.cuh"

namespace mhc {

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
// runs: the row that is written lies on them even where those that are read do not.
template <bool RUNS, class T>
__device__ __forceinline__ void ln_store(T *row, int c, int H, const Run &r, bool runs) {
    if (RUNS || runs) store8(row + c, r);
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
// `stages` places of its own, filled in turn by a lane of the CTA's last warp, which does nothing else
// (ordering a row takes some 600 cycles, too long for a thread that others wait for). A place is free again when
// each warp of the group has said so. A wait that runs out raises the flag, after which none waits:
// the CTA then goes through its rows without their values, so that no thread misses a barrier, and the
// status says so. A row on no boundary of 16 bytes comes with the 16-byte words that hold its ends.
struct LnRing {
    int stages, row_bytes[kLnArrays], place[kLnArrays + 1];     // bytes of a row of each array (0: none), where they lie in a stage; its size
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
enum LnSite : int { SITE_LN_ROW = 120, SITE_LN_FREE, SITE_LN_DRAIN };

// The next filling of a group's places: 16 bytes of barriers each (filled, free), then the rows.
struct LnPlace {
    uint32_t bars, base;
    int at, turn;
    __device__ __forceinline__ uint32_t full() const { return bars + 16 * at; }
    __device__ __forceinline__ uint32_t empty() const { return bars + 16 * at + 8; }
    __device__ __forceinline__ void next(const LnRing &ring) {
        if (++at == ring.stages) {
            at = 0;
            turn ^= 1;
        }
    }
};
__device__ __forceinline__ void ln_bars_init(uint32_t bars, int places, int warps) {
    for (int s = 0; s < places; ++s) {
        mbar_init(bars + 16 * s, 1);
        mbar_init(bars + 16 * s + 8, warps);
    }
    fence_mbar_init();
}
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// One row on its way to a place.
__device__ __forceinline__ void ln_order(const LnRing &ring, const LnPlace &p, const void *const (&src)[kLnArrays], uint64_t policy) {
    uint32_t bytes[kLnArrays], total = 0;
    uintptr_t from[kLnArrays];
#pragma unroll
    for (int i = 0; i < kLnArrays; ++i) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(src[i]), low = static_cast<uintptr_t>(15);
        from[i] = at & ~low;
        bytes[i] = ring.row_bytes[i] ? static_cast<uint32_t>(((at + ring.row_bytes[i] + 15) & ~low) - from[i]) : 0;
        total += bytes[i];
    }
    mbar_arrive_expect_tx(p.full(), total);
#pragma unroll
    for (int i = 0; i < kLnArrays; ++i)
        if (bytes[i])
            bulk_load(p.base + p.at * ring.place[kLnArrays] + ring.place[i], reinterpret_cast<const void *>(from[i]), bytes[i], p.full(), policy);
}
// Gave up: the copies still on their way land before the CTA exits. p: the next place to be filled, after k rows.
__device__ __forceinline__ void ln_drain(const LnRing &ring, const LnPlace &p, int k) {
    int gave_up = 0;
    LnPlace q = p;
    for (int back = k < ring.stages ? k : ring.stages; back > 0; --back) {
        q.at = p.at - back;
        q.turn = p.turn;
        if (q.at < 0) {
            q.at += ring.stages;
            q.turn ^= 1;
        }
        mbar_wait(q.full(), q.turn, &gave_up, ring.timeout_ns, ring.status, SITE_LN_DRAIN);
    }
}
// The last warp: lane g fills group g's places with `rows` rows, sources(k, src) naming the k-th's arrays.
template <class F>
__device__ __forceinline__ void ln_fill(const LnRing &ring, LnPlace p, bool mine, int rows, int *abort_flag, F &&sources) {
    const uint64_t policy = policy_evict_first();
    uint64_t t0 = globaltimer_ns();
    int k = 0;
    while (true) {
        const bool todo = mine && k < rows && !*reinterpret_cast<volatile int *>(abort_flag);
        if (!__any_sync(0xffffffffu, todo)) break;
        if (todo && mbar_test(p.empty(), p.turn ^ 1)) {
            const void *src[kLnArrays];
            sources(k, src);
            ln_order(ring, p, src, policy);
            p.next(ring);
            ++k;
            t0 = globaltimer_ns();
        } else if (todo && globaltimer_ns() - t0 > ring.timeout_ns) {
            record_failure(ring.status, 7, SITE_LN_FREE);
            *reinterpret_cast<volatile int *>(abort_flag) = 1;
        }
    }
    if (mine && *reinterpret_cast<volatile int *>(abort_flag)) ln_drain(ring, p, k);
}
// Columns [c, c + 8) of a staged row, `skew` bytes into its first word; RUNS: none. Past the row's end 0.
template <bool RUNS, class T>
__device__ __forceinline__ Run ln_staged(const uint8_t *row, uint32_t skew, int c, int H, const T *tag) {
    if constexpr (RUNS) return load8_shared(reinterpret_cast<const T *>(row) + c);
    else return ln_masked(load8_skewed(reinterpret_cast<const uint4 *>(row + c * sizeof(T)), skew, tag), c, H);
}
template <class T>
__device__ __forceinline__ uint32_t ln_skew(const T *p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u;
}
// A parameter's H values, zeros up to Hp, to shared memory by the CTA's first `threads` threads, eight loads of each on their way at once.
__device__ __forceinline__ void ln_stage_param(float *to, const void *p, int dtype, int H, int Hp, float otherwise, int threads) {
    for (int c0 = threadIdx.x; c0 < Hp; c0 += 8 * threads) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = c0 + e * threads;
            v[e] = c >= H ? 0.f : p ? load_any(p, dtype, c) : otherwise;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c0 + e * threads < Hp) to[c0 + e * threads] = v[e];
    }
}

}  // namespace mhc
