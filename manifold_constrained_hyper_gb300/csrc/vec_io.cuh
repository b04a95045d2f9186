// Runs of VEC consecutive elements of a row as fp32 values: VEC 8 by 16-byte
// loads and stores (which need the row on a 16-byte boundary), VEC 1 by
// single elements, for rows on any boundary.
#pragma once
#include "block_common.cuh"

namespace mhc {

template <int VEC>
__device__ __forceinline__ void load_run(const float *p, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = p[e];
    }
}
__device__ __forceinline__ float2 unpack2(uint32_t w, const __nv_bfloat16 *) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, const __half *) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
__device__ __forceinline__ uint32_t pack2(float a, float b, const __nv_bfloat16 *) {
    return bf2_pack_rn(f2_pack(a, b));
}
__device__ __forceinline__ uint32_t pack2(float a, float b, const __half *) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
template <int VEC, class T>
__device__ __forceinline__ void unpack_run(const uint4 &w, float (&v)[VEC], const T *tag) {
    static_assert(VEC == 8, "eight 16-bit values a vector");
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = unpack2(u[e], tag);
        v[2 * e] = f.x;
        v[2 * e + 1] = f.y;
    }
}
template <int VEC, class T>
__device__ __forceinline__ void load_run(const T *p, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        unpack_run<VEC>(*reinterpret_cast<const uint4 *>(p), v, p);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = to_f32(p[e]);
    }
}
template <int VEC>
__device__ __forceinline__ void store_run(float *p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) p[e] = v[e];
    }
}
template <int VEC, class T>
__device__ __forceinline__ void store_run(T *p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(pack2(v[0], v[1], p), pack2(v[2], v[3], p),
                                                   pack2(v[4], v[5], p), pack2(v[6], v[7], p));
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) p[e] = from_f32<T>(v[e]);
    }
}

// ---------------------------------------------------------------- checkpoints
// Four codes in a word, from four scaled values.
template <int FMT>
__device__ __forceinline__ uint32_t ckpt_code4(float a, float b, float c, float d) {
    if (FMT == MHC_CKPT_E4M3) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
        return lo | (hi << 16);
    }
    // x + 1.5 * 2^23 rounds x to a whole number, ties to even, in its lowest byte
    const uint32_t w0 = __float_as_uint(a + 12582912.f), w1 = __float_as_uint(b + 12582912.f);
    const uint32_t w2 = __float_as_uint(c + 12582912.f), w3 = __float_as_uint(d + 12582912.f);
    return __byte_perm(__byte_perm(w0, w1, 0x0040), __byte_perm(w2, w3, 0x0040), 0x5410);
}
// Four codes' values, unscaled.
template <int FMT>
__device__ __forceinline__ void ckpt_value4(uint32_t w, float (&v)[4]) {
    if (FMT == MHC_CKPT_E4M3) {
        const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xFFFFu), __NV_E4M3);
        const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3);
        const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
        v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    } else {
        // code + 128 in the low byte of 2^23: minus 2^23 + 128 is the code
        const uint32_t u = w ^ 0x80808080u;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440u | e)) - 8388736.f;
    }
}
// Scale byte of the group of which this lane holds 8 values and its 3
// neighbours (lanes 4 i .. 4 i + 3) the rest; `m` the largest magnitude of the
// lane's own, as bits.
template <int FMT>
__device__ __forceinline__ uint32_t ckpt_byte_quad(const float (&v)[8], unsigned mask) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t b = __float_as_uint(v[e]) & 0x7FFFFFFFu;
        m = m > b ? m : b;
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        const uint32_t n = __shfl_xor_sync(mask, m, o);
        m = m > n ? m : n;
    }
    return ckpt_scale_byte<FMT>(m);
}
template <int FMT>
__device__ __forceinline__ uint2 ckpt_codes8(const float (&v)[8], uint32_t byte) {
    if (byte == 255u) return make_uint2(0u, 0u);
    const float s = ckpt_inverse(byte);
    return make_uint2(ckpt_code4<FMT>(v[0] * s, v[1] * s, v[2] * s, v[3] * s),
                      ckpt_code4<FMT>(v[4] * s, v[5] * s, v[6] * s, v[7] * s));
}
__device__ __forceinline__ void ckpt_values8(uint2 w, uint32_t byte, int format, float (&v)[8]) {
    float a[4], b[4];
    if (format == MHC_CKPT_E4M3) {
        ckpt_value4<MHC_CKPT_E4M3>(w.x, a);
        ckpt_value4<MHC_CKPT_E4M3>(w.y, b);
    } else {
        ckpt_value4<MHC_CKPT_INT8>(w.x, a);
        ckpt_value4<MHC_CKPT_INT8>(w.y, b);
    }
    const float s = ckpt_unit(byte);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        v[e] = a[e] * s;
        v[4 + e] = b[e] * s;
    }
}

}  // namespace mhc
