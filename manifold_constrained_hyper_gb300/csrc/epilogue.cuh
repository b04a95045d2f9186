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

// A piece of 32 x 32 sums, as the 32 lanes of a warp hold it: `wide`, a row a lane, 32 columns, where `rows` and `columns` (a
// multiple of 8) of it are in the matrix; else turned, a column a lane, 32 rows, of which the lane's column has `rows` in the
// matrix (none past the last column). `row0`: the index of the piece's first element, or, turned, of the lane's first,
// in a matrix whose rows are `pitch` apart. Between memory and a row a lane, wide pieces go through the warp's 4 KB
// of shared memory, `buf`, so that an access of the warp touches whole rows and not 32 lines.
struct Piece {
    bool wide;
    int rows, columns;
};
// The compiler would keep the 32 rows' distances in registers from the kernel's start on.
__device__ __forceinline__ long long here(long long pitch) {
    asm volatile("" : "+l"(pitch));
    return pitch;
}
// Where the 16 bytes `c` of a row lie in buf: 8 of them a row (fp32), or 4, so that neither lanes with a row each nor lanes
// along rows meet on a bank.
template <int PER_ROW>
__device__ __forceinline__ uint32_t buf_at(int row, int c) {
    return PER_ROW == 8 ? row * 128 + ((c ^ (row & 7)) << 4) : row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
}
// What a piece is combined with, as it lies in memory: on its way while the products go on.
struct Raw {
    uint32_t w[32];
};
template <int PER_ROW>
__device__ __forceinline__ void load_rows(Raw &r, const Piece &p, const uint8_t *from, long long pitch_bytes) {
    const int lane = threadIdx.x & 31, c = lane % PER_ROW;
    constexpr int kRowsAtOnce = 32 / PER_ROW, kSize = PER_ROW == 8 ? 4 : 2;
    const long long step = here(pitch_bytes * kRowsAtOnce);
    const uint8_t *q = from + lane / PER_ROW * pitch_bytes + 16 * c;
#pragma unroll
    for (int k = 0; k < PER_ROW; ++k, q += step)
        if (lane / PER_ROW + k * kRowsAtOnce < p.rows && c * 16 < p.columns * kSize) {
            const uint4 t = *reinterpret_cast<const uint4 *>(q);
            r.w[4 * k] = t.x, r.w[4 * k + 1] = t.y, r.w[4 * k + 2] = t.z, r.w[4 * k + 3] = t.w;
        }
}
// runs: the source's rows lie on the boundaries of runs of 8; others are read a column a lane, turned or not.
__device__ __forceinline__ void load_raw(Raw &r, const Piece &p, const void *from, int dtype, long long row0, long long pitch, bool runs) {
    const int size = dtype == MHC_F32 ? 4 : 2, lane = threadIdx.x & 31;
    if (p.wide) {
        const uint8_t *const first = static_cast<const uint8_t *>(from) + row0 * size;
        if (runs) {
            if (size == 4) load_rows<8>(r, p, first, pitch * 4);
            else load_rows<4>(r, p, first, pitch * 2);
            return;
        }
        if (lane >= p.columns) return;
        row0 += lane;
    }
    const long long step = here(pitch);
    if (size == 4) {
        const uint32_t *q = static_cast<const uint32_t *>(from) + row0;
#pragma unroll
        for (int c = 0; c < 32; ++c, q += step)
            if (c < p.rows) r.w[c] = *q;
    } else {
        const uint16_t *q = static_cast<const uint16_t *>(from) + row0;
#pragma unroll
        for (int c = 0; c < 32; ++c, q += step)
            if (c < p.rows) r.w[c] = *q;
    }
}
// From whole rows to a row a lane.
template <int PER_ROW>
__device__ __forceinline__ void spread_rows(Raw &r, uint32_t buf) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < PER_ROW; ++k)
        st_shared_v4(buf + buf_at<PER_ROW>(lane / PER_ROW + k * (32 / PER_ROW), lane % PER_ROW),
                     make_uint4(r.w[4 * k], r.w[4 * k + 1], r.w[4 * k + 2], r.w[4 * k + 3]));
    __syncwarp();
#pragma unroll
    for (int k = 0; k < PER_ROW; ++k) {
        const uint4 t = ld_shared_v4(buf + buf_at<PER_ROW>(lane, k));
        r.w[4 * k] = t.x, r.w[4 * k + 1] = t.y, r.w[4 * k + 2] = t.z, r.w[4 * k + 3] = t.w;
    }
}
__device__ __forceinline__ void st_shared_u32(uint32_t a, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
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
__device__ __forceinline__ void each_raw(Raw &r, bool wide, int dtype, bool runs, uint32_t buf, F &&f) {
    const int lane = threadIdx.x & 31;
    if (wide && runs) {
        if (dtype == MHC_F32) spread_rows<8>(r, buf);
        else spread_rows<4>(r, buf);
    }
    with_type(dtype, [&](auto tag) {
        if (wide && runs) {
#pragma unroll
            for (int e = 0; e < 32; ++e) f(e, raw_at(r, true, e, tag));
            return;
        }
        if (wide) {
            // from a column a lane to a row a lane
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 32; ++e) st_shared_u32(buf + (e * 32 + (lane ^ e)) * 4, __float_as_uint(raw_at(r, false, e, tag)));
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 32; ++e) f(e, __uint_as_float(ld_shared_u32(buf + (lane * 32 + (e ^ lane)) * 4)));
            return;
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) f(e, raw_at(r, false, e, tag));
    });
}
// A row a lane, in words, to whole rows.
template <int PER_ROW>
__device__ __forceinline__ void store_rows(const Piece &p, uint8_t *to, long long pitch_bytes, const uint4 (&v)[PER_ROW], uint32_t buf) {
    const int lane = threadIdx.x & 31, c = lane % PER_ROW;
    constexpr int kRowsAtOnce = 32 / PER_ROW, kSize = PER_ROW == 8 ? 4 : 2;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < PER_ROW; ++k) st_shared_v4(buf + buf_at<PER_ROW>(lane, k), v[k]);
    __syncwarp();
    const long long step = here(pitch_bytes * kRowsAtOnce);
    uint8_t *q = to + lane / PER_ROW * pitch_bytes + 16 * c;
#pragma unroll
    for (int k = 0; k < PER_ROW; ++k, q += step) {
        const int row = lane / PER_ROW + k * kRowsAtOnce;
        const uint4 t = ld_shared_v4(buf + buf_at<PER_ROW>(row, c));
        if (row < p.rows && c * 16 < p.columns * kSize) *reinterpret_cast<uint4 *>(q) = t;
    }
}
__device__ __forceinline__ void store_piece(const Piece &p, void *to, int dtype, long long row0, long long pitch, const float (&v)[32], uint32_t buf) {
    with_type(dtype, [&](auto tag) {
        using T = std::remove_const_t<std::remove_pointer_t<decltype(tag)>>;
        T *q = static_cast<T *>(to) + row0;
        if (p.wide) {
            constexpr int kPerRow = sizeof(T) == 4 ? 8 : 4;
            uint4 w[kPerRow];
#pragma unroll
            for (int c = 0; c < kPerRow; ++c) {
                if constexpr (sizeof(T) == 4)
                    w[c] = make_uint4(__float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]), __float_as_uint(v[4 * c + 2]), __float_as_uint(v[4 * c + 3]));
                else
                    w[c] = make_uint4(pack2(f2_pack(v[8 * c], v[8 * c + 1]), q), pack2(f2_pack(v[8 * c + 2], v[8 * c + 3]), q),
                                      pack2(f2_pack(v[8 * c + 4], v[8 * c + 5]), q), pack2(f2_pack(v[8 * c + 6], v[8 * c + 7]), q));
            }
            store_rows<kPerRow>(p, reinterpret_cast<uint8_t *>(q), pitch * static_cast<long long>(sizeof(T)), w, buf);
        } else {
            const long long step = here(pitch);
#pragma unroll
            for (int c = 0; c < 32; ++c, q += step)
                if (c < p.rows) *q = from_f32<T>(v[c]);
        }
    });
}
// What finish_piece combines a piece with: loaded ahead of it. (i, j): the piece's first element, or the lane's.
template <int KIND>
__device__ __forceinline__ void load_extra(Raw &r, const Piece &p, const EpilogueArgs &e, long long i, int j, long long row0, int n) {
    if constexpr (KIND == EPI_LINEAR) {
        if (e.residual) load_raw(r, p, e.residual, e.residual_dtype, i * e.residual_stride + j, e.residual_stride, e.extra_runs);
    } else if constexpr (KIND == EPI_SLOPE) {
        load_raw(r, p, e.z, e.z_dtype, i * e.z_stride + j, e.z_stride, e.extra_runs);
    } else if constexpr (KIND == EPI_SUMS) {
        if (e.accumulate) load_raw(r, p, e.out, e.out_dtype, row0, n, true);
    }
}
// The epilogue of a piece, `row0` as above in a contiguous output of n columns; bias: of column j + lane.
template <int KIND>
__device__ __forceinline__ void finish_piece(const Piece &p, const EpilogueArgs &e, long long row0, int n, float bias, float (&v)[32], Raw &r,
                                             uint32_t buf) {
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
        if (e.z) store_piece(p, e.z, e.z_dtype, row0, n, v, buf);
        if (e.act != MHC_LINEAR_NONE)
            with_act(e.act, [&](auto act) {
#pragma unroll
                for (int q = 0; q < 32; ++q) v[q] = act_value<decltype(act)::value>(v[q]);
            });
        if (e.residual) each_raw(r, p.wide, e.residual_dtype, e.extra_runs, buf, [&](int q, float x) { v[q] += x; });
    } else if constexpr (KIND == EPI_SLOPE) {
        float z[32];
        each_raw(r, p.wide, e.z_dtype, e.extra_runs, buf, [&](int q, float x) { z[q] = x; });
        with_act(e.act, [&](auto act) {
#pragma unroll
            for (int q = 0; q < 32; ++q) v[q] *= act_slope<decltype(act)::value>(z[q]);
        });
    } else {
        if (e.accumulate) each_raw(r, p.wide, e.out_dtype, true, buf, [&](int q, float x) { v[q] += x; });
    }
    store_piece(p, e.out, e.out_dtype, row0, n, v, buf);
}
// A wide piece of plain sums, sixteen columns at a time (weight gradients: 128 tokens, 4096 x 7168 38.9 -> 34.1 us, 1024, 4096 x 4096 38.2 -> 36.5;
// the projections' epilogue by 32 columns unrolled is 1 to 2 % faster). Between the loop and memory lie whole rows in buf; what
// the sums are added to lies there where the result goes.
template <int PER_ROW>
__device__ __forceinline__ void rows_to_buf(const Raw &r, uint32_t buf) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < PER_ROW; ++k)
        st_shared_v4(buf + buf_at<PER_ROW>(lane / PER_ROW + k * (32 / PER_ROW), lane % PER_ROW),
                     make_uint4(r.w[4 * k], r.w[4 * k + 1], r.w[4 * k + 2], r.w[4 * k + 3]));
}
template <int PER_ROW>
__device__ __forceinline__ void buf_to_rows(const Piece &p, uint8_t *to, long long pitch_bytes, uint32_t buf) {
    const int lane = threadIdx.x & 31, c = lane % PER_ROW;
    constexpr int kRowsAtOnce = 32 / PER_ROW, kSize = PER_ROW == 8 ? 4 : 2;
    __syncwarp();
    const long long step = here(pitch_bytes * kRowsAtOnce);
    uint8_t *q = to + lane / PER_ROW * pitch_bytes + 16 * c;
#pragma unroll
    for (int k = 0; k < PER_ROW; ++k, q += step) {
        const int row = lane / PER_ROW + k * kRowsAtOnce;
        const uint4 t = ld_shared_v4(buf + buf_at<PER_ROW>(row, c));
        if (row < p.rows && c * 16 < p.columns * kSize) *reinterpret_cast<uint4 *>(q) = t;
    }
    __syncwarp();
}
// Eight columns of the lane's row in buf, as type T.
template <class T>
__device__ __forceinline__ Run buf_load(uint32_t buf, int c, const T *tag) {
    const int lane = threadIdx.x & 31;
    if constexpr (sizeof(T) == 4) {
        const uint4 a = ld_shared_v4(buf + buf_at<8>(lane, c >> 2)), b = ld_shared_v4(buf + buf_at<8>(lane, (c >> 2) + 1));
        const float f[8] = {__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w),
                            __uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w)};
        return run_of(f);
    } else {
        return unpack8(ld_shared_v4(buf + buf_at<4>(lane, c >> 3)), tag);
    }
}
template <class T>
__device__ __forceinline__ void buf_store(uint32_t buf, int c, const float *v, T *tag) {
    const int lane = threadIdx.x & 31;
    if constexpr (sizeof(T) == 4) {
        st_shared_v4(buf + buf_at<8>(lane, c >> 2), make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])));
        st_shared_v4(buf + buf_at<8>(lane, (c >> 2) + 1), make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])));
    } else {
        st_shared_v4(buf + buf_at<4>(lane, c >> 3), make_uint4(pack2(f2_pack(v[0], v[1]), tag), pack2(f2_pack(v[2], v[3]), tag),
                                                              pack2(f2_pack(v[4], v[5]), tag), pack2(f2_pack(v[6], v[7]), tag)));
    }
}
// sums: the piece's in tensor memory; load16(address, values)
template <class Load>
__device__ __forceinline__ void finish_sums(const Piece &p, const EpilogueArgs &e, long long row0, int n, uint32_t sums, const Raw &r, uint32_t buf,
                                            Load &&load16) {
    with_type(e.out_dtype, [&](auto tag) {
        using T = std::remove_const_t<std::remove_pointer_t<decltype(tag)>>;
        constexpr int kPerRow = sizeof(T) == 4 ? 8 : 4;
        __syncwarp();
        if (e.accumulate) {
            rows_to_buf<kPerRow>(r, buf);
            __syncwarp();
        }
#pragma unroll 1
        for (int c0 = 0; c0 < 32; c0 += 16) {
            uint32_t u[16];
            load16(sums + c0, u);
            float v[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) v[q] = __uint_as_float(u[q]);
#pragma unroll
            for (int h = 0; h < 16; h += 8) {
                if (e.accumulate) {
                    const Run x = buf_load(buf, c0 + h, tag);
#pragma unroll
                    for (int q = 0; q < 8; ++q) v[h + q] += run_at(x, q);
                }
                buf_store(buf, c0 + h, v + h, static_cast<T *>(nullptr));
            }
        }
        buf_to_rows<kPerRow>(p, static_cast<uint8_t *>(e.out) + row0 * static_cast<long long>(sizeof(T)), n * static_cast<long long>(sizeof(T)), buf);
    });
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
