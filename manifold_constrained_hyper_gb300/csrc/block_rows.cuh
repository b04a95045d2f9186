// What the row kernels of the gated residual block share: which columns a
// thread holds, group-wide sums, rows staged in shared memory by bulk copies.
#pragma once
#include <atomic>

#include "vec_io.cuh"

namespace mhc {

// How a row kernel gets its rows.
enum RowMode : int {
    ROWS_RING = 0,      // staged ahead of use by bulk copies, runs of 8 (rows on boundaries of 8 elements)
    ROWS_VEC = 1,       // runs of 8 from global memory: a few rows only, or rows too wide for two stages
    ROWS_ANY = 2,       // staged, single elements: any boundary
    ROWS_SKEW = 3       // staged, runs of 8 of inputs on any boundary; what is written is on boundaries of 8 elements
};
// A thread holds RUNS runs of 8 columns of its group's row: with vector loads
// run j is the columns from (j * threads + thread) * 8, with single ones the
// columns (8 j + e) * threads + thread.
inline int row_threads(int H, int runs) { return ((H + 8 * runs - 1) / (8 * runs) + 31) / 32 * 32; }

struct Place {
    int thread, threads, H;                         // of the group
};
template <int MODE>
__device__ __forceinline__ int run_col(const Place &p, int j) {
    return MODE == ROWS_ANY ? j * 8 * p.threads + p.thread : (j * p.threads + p.thread) * 8;
}
// Past a row's end a staged thread reads zeros that lie behind it: no load needs a guard, and the row's
// sums and a checkpoint's group that the end cuts are what they are without them. (The row's last run again,
// times a weight of 0, would be NaN of an infinity there, and through the sums the whole row.) From global
// memory it reads the last run again, which run_in leaves out of the sums and run_within of parameters. A
// group that the end cuts is the last run's own, whose maximum that leaves as it is.
__device__ __forceinline__ int run_read_col(const Place &p, int j) {
    const int c = run_col<ROWS_VEC>(p, j);
    return c < p.H ? c : p.H - 8;
}
template <int MODE>
__device__ __forceinline__ bool run_in(const Place &p, int j) { return run_col<MODE>(p, j) < p.H; }
// Run j of a row in global memory, and of a type known at run time.
template <class T>
__device__ __forceinline__ Run load_run(const T *row, const Place &p, int j) {
    return load8(row + run_read_col(p, j));
}
__device__ __forceinline__ Run load_run_any(const void *row, int dtype, const Place &p, int j) {
    if (dtype == MHC_F32) return load_run(static_cast<const float *>(row), p, j);
    if (dtype == MHC_BF16) return load_run(static_cast<const __nv_bfloat16 *>(row), p, j);
    return load_run(static_cast<const __half *>(row), p, j);
}
template <int MODE, class T>
__device__ __forceinline__ void store_run(T *row, const Place &p, int j, const Run &r) {
    const int c = run_col<MODE>(p, j);
    if constexpr (MODE != ROWS_ANY) {
        if (c < p.H) store8(row + c, r);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e * p.threads < p.H) row[c + e * p.threads] = from_f32<T>(run_at(r, e));
    }
}
// Zeros at the end of a row's place in a stage (zero_place_end), which no copy reaches: behind a row that
// begins where its place does, those of one run; on any boundary kPlaceEnd bytes.
constexpr int kRunEnd = 32, kPlaceEnd = 64;
// Run j of a row staged in shared memory; AGAIN: past the row's end its last run.
template <bool AGAIN = false, class T>
__device__ __forceinline__ Run staged_run(const T *row, const Place &p, int j) {
    return load8_shared(row + (AGAIN ? run_read_col(p, j) : min(run_col<ROWS_RING>(p, j), p.H)));
}
// The same `skew` bytes into its place; what it reads past the row's end begins 16 bytes (32 of fp32) on.
template <class T>
__device__ __forceinline__ Run staged_skewed(const uint8_t *place, uint32_t skew, const Place &p, int j) {
    const int c = run_col<ROWS_SKEW>(p, j);
    return load8_skewed(reinterpret_cast<const uint4 *>(place + (c < p.H ? c : p.H + 8) * sizeof(T)), skew, static_cast<const T *>(nullptr));
}
// The same on any boundary, single elements: one element of the zeros for every row, however skewed, and
// every type, so that one index serves all of a row's tensors.
template <class T>
__device__ __forceinline__ Run staged_single(const T *row, const Place &p, int j) {
    const int c = run_col<ROWS_ANY>(p, j), zero = (2 * p.H + 30) / 16 * 8;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = to_f32(row[c + e * p.threads < p.H ? c + e * p.threads : zero]);
    return run_of(v);
}
__device__ __forceinline__ void zero_place_end(uint8_t *place, uint32_t bytes, bool any) {
    if (!bytes) return;
#pragma unroll
    for (int i = 16; i <= kPlaceEnd; i += 16)
        if (any || i <= kRunEnd) *reinterpret_cast<uint4 *>(place + bytes - i) = make_uint4(0u, 0u, 0u, 0u);
}
// A run with what lies past the row's end set to 0.
template <int MODE>
__device__ __forceinline__ Run run_within(const Run &r, const Place &p, int j) {
    const int c = run_col<MODE>(p, j);
    if constexpr (MODE != ROWS_ANY) {
        return c < p.H ? r : run_splat(0.f);
    } else {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c + e * p.threads < p.H ? run_at(r, e) : 0.f;
        return run_of(v);
    }
}
// Bulk copies start and end on 16-byte boundaries: a row that does not is
// copied with what shares its first and last 16 bytes (within the allocation,
// which begins and ends on such a boundary), and begins `skew` bytes into its place.
__device__ __forceinline__ uint32_t skew16(const void *p) { return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & 15u; }
__device__ __forceinline__ uint32_t skewed_bytes(const void *p, uint32_t bytes) { return (skew16(p) + bytes + 15u) & ~15u; }
__device__ __forceinline__ void bulk_load_row(uint32_t dst, const void *p, uint32_t bytes, uint32_t bar, uint64_t policy) {
    bulk_load(dst, static_cast<const uint8_t *>(p) - skew16(p), skewed_bytes(p, bytes), bar, policy);
}
// A row's place in a stage. On any boundary copies write (bytes + 30) / 16 * 16 at most, and the zeros
// follow. Single elements: element (2 H + 30) / 16 * 8 of a row up to 14 (or 12) bytes into its place lies
// in them whole: of 2 bytes it begins where they do or up to 14 bytes on, of 4 between 4 H + 30 and 4 H + 72,
// and they reach from 4 H + 30 at most to 4 H + 79 at least. Runs of 8 (H a multiple of 8): those from
// element H + 8 on, 32 bytes or 48, begin there or 16 bytes on.
inline uint32_t row_place(int H, int elem, bool any) {
    const uint32_t bytes = static_cast<uint32_t>(H) * elem;
    return any ? (bytes + 15 + 15) / 16 * 16 + kPlaceEnd : bytes + kRunEnd;
}
__device__ __forceinline__ Run staged_run_any(const void *row, int dtype, const Place &p, int j) {
    if (dtype == MHC_F32) return staged_run(static_cast<const float *>(row), p, j);
    if (dtype == MHC_BF16) return staged_run(static_cast<const __nv_bfloat16 *>(row), p, j);
    return staged_run(static_cast<const __half *>(row), p, j);
}
// What a thread keeps in shared memory of its own columns for every row: run j
// in two halves of 16 bytes, each half of all threads together (no two of a
// warp's eight on the same banks). RUNS * 8 * threads floats an array.
__device__ __forceinline__ Run kept_run(const float *kept, const Place &p, int j) {
    const ulonglong2 *const q = reinterpret_cast<const ulonglong2 *>(kept) + 2 * j * p.threads + p.thread;
    const ulonglong2 a = q[0], b = q[p.threads];
    Run r;
    r.p[0] = a.x;
    r.p[1] = a.y;
    r.p[2] = b.x;
    r.p[3] = b.y;
    return r;
}
__device__ __forceinline__ void keep_run(float *kept, const Place &p, int j, const Run &r) {
    ulonglong2 *const q = reinterpret_cast<ulonglong2 *>(kept) + 2 * j * p.threads + p.thread;
    q[0] = make_ulonglong2(r.p[0], r.p[1]);
    q[p.threads] = make_ulonglong2(r.p[2], r.p[3]);
}
// A run in tensor memory: 8 columns of the warp's 32 lanes. Whole warps. The load leaves its
// registers undefined until the wait, so they stand as they are in between: only the wait, which
// takes them, gives a run.
struct LoadingRun {
    uint32_t v[8];
};
__device__ __forceinline__ void tmem_run_load(uint32_t taddr, LoadingRun &r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r.v[0]), "=r"(r.v[1]), "=r"(r.v[2]), "=r"(r.v[3]), "=r"(r.v[4]), "=r"(r.v[5]), "=r"(r.v[6]), "=r"(r.v[7])
                 : "r"(taddr) : "memory");
}
__device__ __forceinline__ Run tmem_run_wait(LoadingRun &l) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(l.v[0]), "+r"(l.v[1]), "+r"(l.v[2]), "+r"(l.v[3]), "+r"(l.v[4]), "+r"(l.v[5]), "+r"(l.v[6]), "+r"(l.v[7])
                 :: "memory");
    Run r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = (static_cast<uint64_t>(l.v[2 * i + 1]) << 32) | l.v[2 * i];
    return r;
}
__device__ __forceinline__ void tmem_run_store(uint32_t taddr, const Run &r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"r"(taddr), "r"(static_cast<uint32_t>(r.p[0])), "r"(static_cast<uint32_t>(r.p[0] >> 32)),
                   "r"(static_cast<uint32_t>(r.p[1])), "r"(static_cast<uint32_t>(r.p[1] >> 32)),
                   "r"(static_cast<uint32_t>(r.p[2])), "r"(static_cast<uint32_t>(r.p[2] >> 32)),
                   "r"(static_cast<uint32_t>(r.p[3])), "r"(static_cast<uint32_t>(r.p[3] >> 32)) : "memory");
}
__device__ __forceinline__ void run_gate(Run &r, int act) {
    if (act == MHC_ACT_NONE) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = f2_pack(gate_value(f2_lo(r.p[i]), act), gate_value(f2_hi(r.p[i]), act));
}
// Run j of a vector parameter as it lies in memory, of a type known at run time.
// Predicated loads, no branches: those of all parameters are in flight together,
// and a kernel's start goes by one latency instead of one for each of them.
struct RawParam {
    uint32_t w[8];
};
template <int MODE>
__device__ __forceinline__ RawParam raw_param(const void *p, int dtype, const Place &at, int j) {
    RawParam r = {};
    const int wide = p && dtype == MHC_F32, narrow = p && dtype != MHC_F32;
    if constexpr (MODE != ROWS_ANY) {
        const uint64_t a = reinterpret_cast<uint64_t>(p) + static_cast<uint64_t>(run_read_col(at, j)) * (wide ? 4 : 2);
        asm volatile(
            "{\n.reg .pred p, q;\nsetp.ne.b32 p, %9, 0;\nsetp.ne.b32 q, %10, 0;\n"
            "@p ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
            "@q ld.global.v4.b32 {%0, %1, %2, %3}, [%8];\n}"
            : "+r"(r.w[0]), "+r"(r.w[1]), "+r"(r.w[2]), "+r"(r.w[3]), "+r"(r.w[4]), "+r"(r.w[5]), "+r"(r.w[6]), "+r"(r.w[7])
            : "l"(a), "r"(wide), "r"(narrow) : "memory");
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint64_t c = static_cast<uint64_t>(min(run_col<ROWS_ANY>(at, j) + e * at.threads, at.H - 1));
            asm volatile(
                "{\n.reg .pred p, q;\nsetp.ne.b32 p, %2, 0;\nsetp.ne.b32 q, %3, 0;\n"
                "@p ld.global.b32 %0, [%1];\n@q ld.global.u16 %0, [%1];\n}"
                : "+r"(r.w[e]) : "l"(reinterpret_cast<uint64_t>(p) + c * (wide ? 4 : 2)), "r"(wide), "r"(narrow) : "memory");
        }
    }
    return r;
}
template <int MODE>
__device__ __forceinline__ Run param_run(const RawParam &r, int dtype) {
    float v[8];
    if (dtype == MHC_F32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(r.w[e]);
        return run_of(v);
    }
    if constexpr (MODE != ROWS_ANY) {
        const uint4 w = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
        return dtype == MHC_BF16 ? unpack8(w, static_cast<const __nv_bfloat16 *>(nullptr))
                                 : unpack8(w, static_cast<const __half *>(nullptr));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            v[e] = dtype == MHC_BF16 ? __uint_as_float(r.w[e] << 16)
                                     : __half2float(__ushort_as_half(static_cast<unsigned short>(r.w[e])));
        return run_of(v);
    }
}
// What every row of a block needs of run j: w1 = (w_post + offset) * act of a
// channel gate, w2 = w_pre + offset, the residual's scale (1 where there is
// none); past the row's end 0, so that what they multiply leaves the row's sums alone.
struct RowParams {
    Run w1, w2, sc;
};
template <int MODE>
__device__ __forceinline__ RowParams load_row_params(const BlockForm &f, const Place &at, int j) {
    const bool gated = f.gate_form == MHC_GATE_CHANNEL, scaled = f.scale_form == MHC_SCALE_CHANNEL;
    const RawParam r1 = raw_param<MODE>(f.w_post, f.w_post_dtype, at, j), r2 = raw_param<MODE>(f.w_pre, f.w_pre_dtype, at, j),
                   rg = raw_param<MODE>(gated ? f.gate : nullptr, f.gate_dtype, at, j),
                   rs = raw_param<MODE>(scaled ? f.res_scale : nullptr, MHC_F32, at, j);
    const float one = f.scale_form == MHC_SCALE_ONE ? *f.res_scale : 1.f;
    RowParams p;
    const uint64_t offset = splat2(f.weight_offset);
    p.w1 = run_splat(1.f);
    if (f.w_post) {
        p.w1 = param_run<MODE>(r1, f.w_post_dtype);
#pragma unroll
        for (int i = 0; i < 4; ++i) p.w1.p[i] = add2(p.w1.p[i], offset);
    }
    if (gated) {
        Run g = param_run<MODE>(rg, f.gate_dtype);
        run_gate(g, f.gate_act);
#pragma unroll
        for (int i = 0; i < 4; ++i) p.w1.p[i] = mul2(p.w1.p[i], g.p[i]);
    }
    p.w2 = run_splat(1.f);
    if (f.w_pre) {
        p.w2 = param_run<MODE>(r2, f.w_pre_dtype);
#pragma unroll
        for (int i = 0; i < 4; ++i) p.w2.p[i] = add2(p.w2.p[i], offset);
    }
    p.sc = scaled ? param_run<MODE>(rs, MHC_F32) : run_splat(one);
    p.w1 = run_within<MODE>(p.w1, at, j);
    p.w2 = run_within<MODE>(p.w2, at, j);
    p.sc = run_within<MODE>(p.sc, at, j);
    return p;
}
// Run j of a row's checkpoint. Whole warps call it.
template <int FMT, int MODE>
__device__ __forceinline__ void store_ckpt(const Ckpt &c, long long t, const Place &p, int j, const Run &r) {
    const int groups = (p.H + 31) / 32, col = run_col<MODE>(p, j);
    uint8_t *const codes = c.codes + t * p.H, *const scales = c.scales + t * groups;
    if constexpr (MODE != ROWS_ANY) {
        const uint32_t byte = ckpt_byte_quad<FMT>(r);
        if (col >= p.H) return;
        *reinterpret_cast<uint2 *>(codes + col) = ckpt_codes8<FMT>(r, byte);
        if ((threadIdx.x & 3) == 0) scales[col / 32] = static_cast<uint8_t>(byte);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int i = col + e * p.threads;
            uint32_t byte;
            const uint32_t code = ckpt_encode_lane<FMT>(run_at(r, e), &byte);
            if (i < p.H) codes[i] = static_cast<uint8_t>(code);
            if (i < p.H && (threadIdx.x & 31) == 0) scales[i / 32] = static_cast<uint8_t>(byte);
        }
    }
}
template <int MODE>
__device__ __forceinline__ void store_ckpt(const Ckpt &c, int format, long long t, const Place &p, int j, const Run &r) {
    if (format == MHC_CKPT_E4M3) store_ckpt<MHC_CKPT_E4M3, MODE>(c, t, p, j, r);
    else store_ckpt<MHC_CKPT_INT8, MODE>(c, t, p, j, r);
}

// Wait for a stage's row. The groups of a CTA share its stages and run at their
// own pace: one may come to a stage whose row before last has not yet landed, where the parity of
// its own phase would read as passed. `armed` says which filling the stage is in; a filling
// begins only when the one before has been read. Bounded, like mbar_wait.
__device__ __forceinline__ bool stage_wait(volatile int *armed, int filling, uint32_t bar, volatile int *abort_flag,
                                           uint64_t timeout_ns, unsigned int *status, int site) {
    if (*armed != filling) {
        const uint64_t t0 = globaltimer_ns();
        while (*armed != filling) {
            if (*abort_flag) return false;
            if (globaltimer_ns() - t0 > timeout_ns) {
                record_failure(status, 7, site);
                *abort_flag = 1;
                return false;
            }
        }
    }
    return mbar_wait(bar, filling & 1, abort_flag, timeout_ns, status, site);
}
// Begin a filling: its bytes announced to the barrier, then the stage marked.
__device__ __forceinline__ void stage_arm(volatile int *armed, int filling, uint32_t bar, uint32_t bytes) {
    mbar_arrive_expect_tx(bar, bytes);
    __threadfence_block();
    *armed = filling;
}

// Sums of N values (1 or 3) over a group of up to MAXW whole warps that share
// the named barrier `bar`, in one fixed order, for every thread of it. Within a
// warp by shuffles (of three sums two at a time: after the first two steps a
// lane carries one of them); across warps every thread adds all of them itself
// (16-byte broadcasts: half the latency of a second round of shuffles). `red`:
// N MAXW floats of the group's own on a 16-byte boundary, zero beyond its
// warps; the caller alternates between two, so that a value is read by all
// before it is written again.
template <int N, int MAXW>
__device__ __forceinline__ void group_sum(float (&v)[N], float *red, int bar, int warp, int warps) {
    const int lane = threadIdx.x & 31;
    float x = v[0];
    if constexpr (N == 3) {
        // lane bit 4 picks v0 or v1 (with v2 beside v0), bit 3 then v0 or v2
        const bool up = lane & 16, mid = lane & 8;
        const float give = up ? v[0] : v[1], keep = up ? v[1] : v[0];
        const float a = keep + __shfl_xor_sync(0xffffffffu, give, 16);
        const float b = v[2] + __shfl_xor_sync(0xffffffffu, v[2], 16);
        const float give2 = mid ? a : b, keep2 = mid ? b : a;
        // lanes 0-7: v0, 8-15: v2, 16-23: v1, 24-31: v2 once more
        x = keep2 + __shfl_xor_sync(0xffffffffu, give2, 8);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (warps == 1) {
            v[0] = __shfl_sync(0xffffffffu, x, 0);
            v[1] = __shfl_sync(0xffffffffu, x, 16);
            v[2] = __shfl_sync(0xffffffffu, x, 8);
            return;
        }
        if ((lane & 7) == 0 && lane < 24) red[(lane == 0 ? 0 : lane == 16 ? 1 : 2) * MAXW + warp] = x;
    } else {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        v[0] = x;
        if (warps == 1) return;
        if (lane == 0) red[warp] = x;
    }
    named_barrier_sync(bar, warps * 32);
#pragma unroll
    for (int k = 0; k < N; ++k) {
        uint64_t s[MAXW / 4];
#pragma unroll
        for (int i = 0; i < MAXW / 4; ++i) {
            const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(red + k * MAXW + 4 * i);
            s[i] = add2(w.x, w.y);
        }
#pragma unroll
        for (int n = MAXW / 8; n > 0; n >>= 1)
#pragma unroll
            for (int i = 0; i < n; ++i) s[i] = add2(s[i], s[i + n]);
        v[k] = f2_lo(s[0]) + f2_hi(s[0]);
    }
}

// Rows of runs: 8 elements a multiple of what a row's address and stride are
// multiples of (16 bytes; 32 for fp32).
inline bool rows_of_runs(const void *p, long long stride, int elem, long long T) {
    return reinterpret_cast<uintptr_t>(p) % (8 * elem) == 0 && (T == 1 || stride % 8 == 0);
}
inline int elem_bytes(int dtype) { return dtype == MHC_F32 ? 4 : 2; }
// Weights and scales can be read 8 at a time.
inline bool params_of_runs(const BlockForm &f) {
    const void *const p[] = {f.w_post, f.w_pre, f.scale_form == MHC_SCALE_CHANNEL ? f.res_scale : nullptr,
                             f.gate_form == MHC_GATE_CHANNEL ? f.gate : nullptr};
    for (const void *q : p)
        if (reinterpret_cast<uintptr_t>(q) & 31u) return false;
    return true;
}

// Opts a kernel in to `smem` bytes of dynamic shared memory (all of its calls: at most `most`), once per device.
struct SmemGrant {
    std::atomic<int> bytes[64];
};
template <class K>
inline cudaError_t grant_smem(K kern, SmemGrant &g, size_t smem, size_t most) {
    if (smem <= 32 * 1024) return cudaSuccess;      // with the kernels' static arrays, below 48 KB
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
