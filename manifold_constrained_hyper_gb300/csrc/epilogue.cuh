// What the products' kernels do to one element, or to runs of 8, of the sums.
#pragma once
#include "act.cuh"
#include "linear_internal.h"
#include "vec_io.cuh"

namespace mhc {

__device__ __forceinline__ Run load_run(const void *p, int dtype, long long i) {
    if (dtype == MHC_F32) return load8(static_cast<const float *>(p) + i);
    if (dtype == MHC_BF16) return load8(static_cast<const __nv_bfloat16 *>(p) + i);
    return load8(static_cast<const __half *>(p) + i);
}
__device__ __forceinline__ void store_run(void *p, int dtype, long long i, const Run &r) {
    if (dtype == MHC_F32) store8(static_cast<float *>(p) + i, r);
    else if (dtype == MHC_BF16) store8(static_cast<__nv_bfloat16 *>(p) + i, r);
    else store8(static_cast<__half *>(p) + i, r);
}
// f(a null pointer of the type)
template <class F>
__device__ __forceinline__ void with_type(int dtype, F &&f) {
    if (dtype == MHC_F32) f(static_cast<const float *>(nullptr));
    else if (dtype == MHC_BF16) f(static_cast<const __nv_bfloat16 *>(nullptr));
    else f(static_cast<const __half *>(nullptr));
}

// A piece of 32 x 32 sums, as the 32 lanes of a warp hold it: `wide`, a row a lane, 32 columns, of which
// `n` (a multiple of 8) are in the matrix; else turned, a column a lane, 32 rows, of which `n` are in
// it (none of a lane past the last column). at: the first element's index, of a matrix whose rows are
// `pitch` apart.
struct Piece {
    bool wide;
    int n;
};
// The compiler would keep the 32 rows' distances in registers from the kernel's start on.
__device__ __forceinline__ long long here(long long pitch) {
    asm volatile("" : "+l"(pitch));
    return pitch;
}
// What it is combined with, as it lies in memory: on its way while the products go on, or while the
// piece before is stored.
struct Raw {
    uint32_t w[32];
};
__device__ __forceinline__ void load_raw(Raw &r, const Piece &p, const void *from, int dtype, long long at, long long pitch) {
    if (p.wide) {
        if (dtype == MHC_F32) {
            const uint4 *const q = reinterpret_cast<const uint4 *>(static_cast<const float *>(from) + at);
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (4 * c < p.n) {
                    const uint4 t = q[c];
                    r.w[4 * c] = t.x, r.w[4 * c + 1] = t.y, r.w[4 * c + 2] = t.z, r.w[4 * c + 3] = t.w;
                }
        } else {
            const uint4 *const q = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(from) + at);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (8 * c < p.n) {
                    const uint4 t = q[c];
                    r.w[4 * c] = t.x, r.w[4 * c + 1] = t.y, r.w[4 * c + 2] = t.z, r.w[4 * c + 3] = t.w;
                }
        }
        return;
    }
    pitch = here(pitch);
    if (dtype == MHC_F32) {
        const uint32_t *q = static_cast<const uint32_t *>(from) + at;
#pragma unroll
        for (int c = 0; c < 32; ++c, q += pitch)
            if (c < p.n) r.w[c] = *q;
    } else {
        const uint16_t *q = static_cast<const uint16_t *>(from) + at;
#pragma unroll
        for (int c = 0; c < 32; ++c, q += pitch)
            if (c < p.n) r.w[c] = *q;
    }
}
// Value e of it.
__device__ __forceinline__ float raw_at(const Raw &r, bool, int e, const float *) { return __uint_as_float(r.w[e]); }
__device__ __forceinline__ float raw_at(const Raw &r, bool wide, int e, const __nv_bfloat16 *) {
    return __uint_as_float(!wide ? r.w[e] << 16 : e & 1 ? r.w[e >> 1] & 0xFFFF0000u : r.w[e >> 1] << 16);
}
__device__ __forceinline__ float raw_at(const Raw &r, bool wide, int e, const __half *) {
    const uint32_t w = !wide ? r.w[e] : e & 1 ? r.w[e >> 1] >> 16 : r.w[e >> 1];
    return __half2float(__ushort_as_half(static_cast<unsigned short>(w)));
}
// f(e, the value) for each of the 32.
template <class F>
__device__ __forceinline__ void each_raw(const Raw &r, bool wide, int dtype, F &&f) {
    with_type(dtype, [&](auto tag) {
        if (wide) {
#pragma unroll
            for (int e = 0; e < 32; ++e) f(e, raw_at(r, true, e, tag));
        } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) f(e, raw_at(r, false, e, tag));
        }
    });
}
__device__ __forceinline__ void store_piece(const Piece &p, void *to, int dtype, long long at, long long pitch, const float (&v)[32]) {
    with_type(dtype, [&](auto tag) {
        using T = std::remove_const_t<std::remove_pointer_t<decltype(tag)>>;
        T *q = static_cast<T *>(to) + at;
        if (p.wide) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (8 * c >= p.n) break;
                Run r;
#pragma unroll
                for (int k = 0; k < 4; ++k) r.p[k] = f2_pack(v[8 * c + 2 * k], v[8 * c + 2 * k + 1]);
                store8(q + 8 * c, r);
            }
        } else {
            const long long step = here(pitch);
#pragma unroll
            for (int c = 0; c < 32; ++c, q += step)
                if (c < p.n) *q = from_f32<T>(v[c]);
        }
    });
}
// What finish_piece combines a piece with: loaded ahead of it.
template <int KIND>
__device__ __forceinline__ void load_extra(Raw &r, const Piece &p, const EpilogueArgs &e, long long i, int j, long long at, int n) {
    if constexpr (KIND == EPI_LINEAR) {
        if (e.residual) load_raw(r, p, e.residual, e.residual_dtype, i * e.residual_stride + j, e.residual_stride);
    } else if constexpr (KIND == EPI_SLOPE) {
        load_raw(r, p, e.z, e.z_dtype, i * e.z_stride + j, e.z_stride);
    } else if constexpr (KIND == EPI_SUMS) {
        if (e.accumulate) load_raw(r, p, e.out, e.out_dtype, at, n);
    }
}
// The epilogue of a piece whose first element is (i, j), `at` its index in a contiguous output of n
// columns; bias: of column j + lane.
template <int KIND>
__device__ __forceinline__ void finish_piece(const Piece &p, const EpilogueArgs &e, long long at, int n, float bias, float (&v)[32],
                                             const Raw &r) {
    if constexpr (KIND == EPI_LINEAR) {
        if (e.bias) {
            if (p.wide) {
#pragma unroll
                for (int q = 0; q < 32; ++q) v[q] += __shfl_sync(0xffffffffu, bias, q);
            } else {
#pragma unroll
                for (int q = 0; q < 32; ++q) v[q] += bias;
            }
        }
        if (e.z) store_piece(p, e.z, e.z_dtype, at, n, v);
        if (e.act != MHC_LINEAR_NONE)
            with_act(e.act, [&](auto act) {
#pragma unroll
                for (int q = 0; q < 32; ++q) v[q] = act_value<decltype(act)::value>(v[q]);
            });
        if (e.residual) each_raw(r, p.wide, e.residual_dtype, [&](int q, float x) { v[q] += x; });
    } else if constexpr (KIND == EPI_SLOPE) {
        float z[32];
        each_raw(r, p.wide, e.z_dtype, [&](int q, float x) { z[q] = x; });
        with_act(e.act, [&](auto act) {
#pragma unroll
            for (int q = 0; q < 32; ++q) v[q] *= act_slope<decltype(act)::value>(z[q]);
        });
    } else {
        if (e.accumulate) each_raw(r, p.wide, e.out_dtype, [&](int q, float x) { v[q] += x; });
    }
    store_piece(p, e.out, e.out_dtype, at, n, v);
}
// One element on any boundary.
template <int KIND>
__device__ __forceinline__ void finish_element(const EpilogueArgs &e, long long i, long long at, int j, float x) {
    if constexpr (KIND == EPI_LINEAR) {
        if (e.bias) x += load_any(e.bias, e.bias_dtype, j);
        if (e.z) store_any(e.z, e.z_dtype, at, x);
        with_act(e.act, [&](auto act) { x = act_value<decltype(act)::value>(x); });
        if (e.residual) x += load_any(e.residual, e.residual_dtype, i * e.residual_stride + j);
    } else if constexpr (KIND == EPI_SLOPE) {
        const float z = load_any(e.z, e.z_dtype, i * e.z_stride + j);
        with_act(e.act, [&](auto act) { x *= act_slope<decltype(act)::value>(z); });
    } else if (e.accumulate) {
        x += load_any(e.out, e.out_dtype, at);
    }
    store_any(e.out, e.out_dtype, at, x);
}

}  // namespace mhc
