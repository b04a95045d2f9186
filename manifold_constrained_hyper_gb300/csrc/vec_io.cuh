// Runs of 8 values of a row as 4 packed pairs of fp32 (f32x2 arithmetic), and
// their 8-bit checkpoints.
#pragma once
#include "block_common.cuh"

namespace mhc {

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

struct Run {
    uint64_t p[4];
};
__device__ __forceinline__ uint64_t splat2(float v) { return f2_pack(v, v); }
__device__ __forceinline__ float run_at(const Run &r, int e) { return e & 1 ? f2_hi(r.p[e >> 1]) : f2_lo(r.p[e >> 1]); }
__device__ __forceinline__ Run run_of(const float (&v)[8]) {
    Run r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = f2_pack(v[2 * i], v[2 * i + 1]);
    return r;
}
__device__ __forceinline__ Run run_splat(float v) {
    Run r;
    r.p[0] = r.p[1] = r.p[2] = r.p[3] = splat2(v);
    return r;
}

__device__ __forceinline__ uint64_t unpack2(uint32_t w, const __nv_bfloat16 *) { return bf2_unpack(w); }
__device__ __forceinline__ uint64_t unpack2(uint32_t w, const __half *) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return f2_pack(f.x, f.y);
}
__device__ __forceinline__ uint32_t pack2(uint64_t v, const __nv_bfloat16 *) { return bf2_pack_rn(v); }
__device__ __forceinline__ uint32_t pack2(uint64_t v, const __half *) {
    const __half2 h = __floats2half2_rn(f2_lo(v), f2_hi(v));
    return *reinterpret_cast<const uint32_t *>(&h);
}
// An fp16 element that is written as the largest finite one where the value lies past it; NaN stays.
struct FiniteHalf {
    uint16_t bits;
};
__device__ __forceinline__ uint32_t pack2(uint64_t v, const FiniteHalf *) {
    uint32_t w;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(f2_hi(v)), "f"(f2_lo(v)));
    return w;
}
// 8 consecutive values of a row in global memory: 16-bit ones from a 16-byte
// boundary, fp32 from a 32-byte one.
__device__ __forceinline__ Run load8(const float *p) {
    Run r;
    asm volatile("ld.global.v4.b64 {%0, %1, %2, %3}, [%4];"
                 : "=l"(r.p[0]), "=l"(r.p[1]), "=l"(r.p[2]), "=l"(r.p[3])
                 : "l"(reinterpret_cast<uint64_t>(p)) : "memory");
    return r;
}
template <class T>
__device__ __forceinline__ Run unpack8(const uint4 &w, const T *tag) {
    Run r;
    r.p[0] = unpack2(w.x, tag);
    r.p[1] = unpack2(w.y, tag);
    r.p[2] = unpack2(w.z, tag);
    r.p[3] = unpack2(w.w, tag);
    return r;
}
template <class T>
__device__ __forceinline__ Run load8(const T *p) {
    return unpack8(*reinterpret_cast<const uint4 *>(p), p);
}
// The same from shared memory. fp32: neighbouring threads' 32 bytes would put
// two of every eight on the same banks; every other four threads read their
// second half first.
__device__ __forceinline__ Run load8_shared(const float *p) {
    const ulonglong2 *const q = reinterpret_cast<const ulonglong2 *>(p);
    const int swap = (threadIdx.x >> 2) & 1;
    const ulonglong2 a = q[swap], b = q[swap ^ 1];
    Run r;
    r.p[0] = swap ? b.x : a.x;
    r.p[1] = swap ? b.y : a.y;
    r.p[2] = swap ? a.x : b.x;
    r.p[3] = swap ? a.y : b.y;
    return r;
}
template <class T>
__device__ __forceinline__ Run load8_shared(const T *p) {
    return unpack8(*reinterpret_cast<const uint4 *>(p), p);
}
// 8 values that begin `skew` bytes past a 16-byte boundary `p`: the aligned words
// around them, picked by the bits of skew (the same for a whole row).
template <class T>
__device__ __forceinline__ Run load8_skewed(const uint4 *p, uint32_t skew, const T *tag) {
    const uint4 a = p[0], b = p[1];
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t t[6], u[5];
#pragma unroll
    for (int j = 0; j < 6; ++j) t[j] = skew & 8 ? w[j + 2] : w[j];
#pragma unroll
    for (int j = 0; j < 5; ++j) u[j] = skew & 4 ? t[j + 1] : t[j];
    const uint32_t bits = (skew & 2) * 8;
    return unpack8(make_uint4(__funnelshift_r(u[0], u[1], bits), __funnelshift_r(u[1], u[2], bits),
                              __funnelshift_r(u[2], u[3], bits), __funnelshift_r(u[3], u[4], bits)), tag);
}
__device__ __forceinline__ Run load8_skewed(const uint4 *p, uint32_t skew, const float *) {
    const uint4 a = p[0], b = p[1], c = p[2];
    const uint32_t w[12] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
    uint32_t t[9];
#pragma unroll
    for (int j = 0; j < 9; ++j) t[j] = skew & 8 ? w[j + 2] : w[j];
    Run r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t lo = skew & 4 ? t[2 * i + 1] : t[2 * i], hi = skew & 4 ? t[2 * i + 2] : t[2 * i + 1];
        r.p[i] = (static_cast<uint64_t>(hi) << 32) | lo;
    }
    return r;
}
// Bytes [addr, addr + 8 N) of a row that ends at `end`, from the aligned 8-byte words
// that hold them (a word that holds none of the row is not read).
template <int N>
__device__ __forceinline__ void load_words(uintptr_t addr, uintptr_t end, uint64_t (&out)[N]) {
    const uintptr_t first = addr & ~static_cast<uintptr_t>(7);
    const uint32_t bits = static_cast<uint32_t>(addr - first) * 8;
    uint64_t w[N + 1];
#pragma unroll
    for (int i = 0; i <= N; ++i)
        w[i] = first + 8 * i < end ? *reinterpret_cast<const uint64_t *>(first + 8 * i) : 0ull;
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = bits ? (w[i] >> bits) | (w[i + 1] << (64 - bits)) : w[i];
}
// Values [c, c + 8) of a row of H on any boundary; past its end 0.
template <class T>
__device__ __forceinline__ Run load8_any(const T *row, int c, int H) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row);
    Run r;
    if constexpr (sizeof(T) == 4) {
        load_words<4>(at + 4 * static_cast<uintptr_t>(c), at + 4 * static_cast<uintptr_t>(H), r.p);
    } else {
        uint64_t w[2];
        load_words<2>(at + 2 * static_cast<uintptr_t>(c), at + 2 * static_cast<uintptr_t>(H), w);
        r = unpack8(make_uint4(static_cast<uint32_t>(w[0]), static_cast<uint32_t>(w[0] >> 32), static_cast<uint32_t>(w[1]),
                               static_cast<uint32_t>(w[1] >> 32)), row);
    }
    if (c + 8 > H) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c + e < H ? run_at(r, e) : 0.f;
        r = run_of(v);
    }
    return r;
}
// The first `n` of 8 elements of ELEM bytes each, held in w, to any boundary; two at a time
// where `pairs` (the address is a multiple of two elements).
template <int ELEM>
__device__ __forceinline__ void store_words(uint8_t *p, const uint64_t (&w)[ELEM], bool pairs, int n) {
    if (pairs && n == 8) {
#pragma unroll
        for (int b = 0; b < 8 * ELEM; b += 2 * ELEM) {
            const uint64_t two = w[b / 8] >> (b % 8 * 8);
            if constexpr (ELEM == 4) *reinterpret_cast<uint64_t *>(p + b) = two;
            else if constexpr (ELEM == 2) *reinterpret_cast<uint32_t *>(p + b) = static_cast<uint32_t>(two);
            else *reinterpret_cast<uint16_t *>(p + b) = static_cast<uint16_t>(two);
        }
        return;
    }
#pragma unroll
    for (int b = 0; b < 8 * ELEM; b += ELEM) {
        if (b >= n * ELEM) break;
        const uint64_t one = w[b / 8] >> (b % 8 * 8);
        if constexpr (ELEM == 4) *reinterpret_cast<uint32_t *>(p + b) = static_cast<uint32_t>(one);
        else if constexpr (ELEM == 2) *reinterpret_cast<uint16_t *>(p + b) = static_cast<uint16_t>(one);
        else p[b] = static_cast<uint8_t>(one);
    }
}
template <class T>
__device__ __forceinline__ void store8_any(T *p, const Run &r, bool pairs, int n) {
    if constexpr (sizeof(T) == 4) {
        store_words<4>(reinterpret_cast<uint8_t *>(p), r.p, pairs, n);
    } else {
        const uint64_t w[2] = {static_cast<uint64_t>(pack2(r.p[1], p)) << 32 | pack2(r.p[0], p),
                               static_cast<uint64_t>(pack2(r.p[3], p)) << 32 | pack2(r.p[2], p)};
        store_words<2>(reinterpret_cast<uint8_t *>(p), w, pairs, n);
    }
}
__device__ __forceinline__ void store8(float *p, const Run &r) {
    asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};"
                 ::"l"(reinterpret_cast<uint64_t>(p)), "l"(r.p[0]), "l"(r.p[1]), "l"(r.p[2]), "l"(r.p[3]) : "memory");
}
template <class T>
__device__ __forceinline__ void store8(T *p, const Run &r) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack2(r.p[0], p), pack2(r.p[1], p), pack2(r.p[2], p), pack2(r.p[3], p));
}

// ---------------------------------------------------------------- checkpoints
// Four codes in a word, from four scaled values.
template <int FMT>
__device__ __forceinline__ uint32_t ckpt_code4(uint64_t a, uint64_t b) {
    if (FMT == MHC_CKPT_E4M3) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f2_lo(a), f2_hi(a)), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f2_lo(b), f2_hi(b)), __NV_SATFINITE, __NV_E4M3);
        return lo | (hi << 16);
    }
    // x + 1.5 * 2^23 rounds x to a whole number, ties to even, in its lowest byte
    const uint64_t one = splat2(12582912.f);
    const uint64_t u = add2(a, one), v = add2(b, one);
    return __byte_perm(__byte_perm(static_cast<uint32_t>(u), static_cast<uint32_t>(u >> 32), 0x0040),
                       __byte_perm(static_cast<uint32_t>(v), static_cast<uint32_t>(v >> 32), 0x0040), 0x5410);
}
// Four codes' values, unscaled.
template <int FMT>
__device__ __forceinline__ void ckpt_value4(uint32_t w, uint64_t *a, uint64_t *b) {
    if (FMT == MHC_CKPT_E4M3) {
        const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w & 0xFFFFu), __NV_E4M3);
        const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> 16), __NV_E4M3);
        const float2 f = __half22float2(__half2(lo)), g = __half22float2(__half2(hi));
        *a = f2_pack(f.x, f.y);
        *b = f2_pack(g.x, g.y);
    } else {
        // code + 128 in the low byte of 2^23: minus 2^23 + 128 is the code
        const uint32_t u = w ^ 0x80808080u;
        const uint64_t off = splat2(-8388736.f);
        *a = add2((static_cast<uint64_t>(__byte_perm(u, 0x4B000000u, 0x7441)) << 32) | __byte_perm(u, 0x4B000000u, 0x7440), off);
        *b = add2((static_cast<uint64_t>(__byte_perm(u, 0x4B000000u, 0x7443)) << 32) | __byte_perm(u, 0x4B000000u, 0x7442), off);
    }
}
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// Scale byte of the group of which this lane holds 8 values and its 3
// neighbours (lanes 4 i .. 4 i + 3) the rest. Whole warps call it.
template <int FMT>
__device__ __forceinline__ uint32_t ckpt_byte_quad(const Run &r) {
    // three at a time, a NaN winning (its bits are above infinity's)
    float x = max3_abs(run_at(r, 0), run_at(r, 1), run_at(r, 2));
    x = max3_abs(x, run_at(r, 3), run_at(r, 4));
    x = max3_abs(x, run_at(r, 5), run_at(r, 6));
    uint32_t m = __float_as_uint(max3_abs(x, x, run_at(r, 7)));
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        const uint32_t n = __shfl_xor_sync(0xffffffffu, m, o);
        m = m > n ? m : n;
    }
    return ckpt_scale_byte<FMT>(m);
}
template <int FMT>
__device__ __forceinline__ uint2 ckpt_codes8(const Run &r, uint32_t byte) {
    if (byte == 255u) return make_uint2(0u, 0u);
    const uint64_t s = splat2(ckpt_inverse(byte));
    return make_uint2(ckpt_code4<FMT>(mul2(r.p[0], s), mul2(r.p[1], s)),
                      ckpt_code4<FMT>(mul2(r.p[2], s), mul2(r.p[3], s)));
}
__device__ __forceinline__ Run ckpt_values8(uint2 w, uint32_t byte, int format) {
    Run r;
    if (format == MHC_CKPT_E4M3) {
        ckpt_value4<MHC_CKPT_E4M3>(w.x, &r.p[0], &r.p[1]);
        ckpt_value4<MHC_CKPT_E4M3>(w.y, &r.p[2], &r.p[3]);
    } else {
        ckpt_value4<MHC_CKPT_INT8>(w.x, &r.p[0], &r.p[1]);
        ckpt_value4<MHC_CKPT_INT8>(w.y, &r.p[2], &r.p[3]);
    }
    const uint64_t s = splat2(ckpt_unit(byte));
#pragma unroll
    for (int i = 0; i < 4; ++i) r.p[i] = mul2(r.p[i], s);
    return r;
}

}  // namespace mhc
