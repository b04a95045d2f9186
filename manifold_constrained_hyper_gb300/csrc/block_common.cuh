// Element types, the gate, block-wide sums and the 8-bit checkpoint format,
// shared by the gated residual block's kernels.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cfloat>

#include "block_internal.h"
#include "ptx.cuh"

namespace mhc {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// An element of a tensor whose type is known at run time only.
__device__ __forceinline__ float load_any(const void *p, int dtype, long long i) {
    if (dtype == MHC_F32) return static_cast<const float *>(p)[i];
    if (dtype == MHC_BF16) return to_f32(static_cast<const __nv_bfloat16 *>(p)[i]);
    return to_f32(static_cast<const __half *>(p)[i]);
}
__device__ __forceinline__ void store_any(void *p, int dtype, long long i, float v) {
    if (dtype == MHC_F32) static_cast<float *>(p)[i] = v;
    else if (dtype == MHC_BF16) static_cast<__nv_bfloat16 *>(p)[i] = from_f32<__nv_bfloat16>(v);
    else static_cast<__half *>(p)[i] = from_f32<__half>(v);
}
__device__ __forceinline__ float weight_at(const void *w, int dtype, float offset, int i) {
    return w ? load_any(w, dtype, i) + offset : 1.f;
}

// act(z). The sigmoid from e = exp(-|z|) <= 1, as 1 / (1 + e) or e / (1 + e):
// no overflow, and the divisor stays in [1, 2], where the approximate division
// is off by 2 ulp. exp and tanh are CUDA's own, a few ulp, far below a
// 16-bit output's rounding and of the size of an fp32 one's.
__device__ __forceinline__ float gate_value(float z, int act) {
    if (act == MHC_ACT_SIGMOID) {
        const float e = expf(-fabsf(z));
        return __fdividef(z < 0.f ? e : 1.f, 1.f + e);
    }
    if (act == MHC_ACT_TANH) return tanhf(z);
    return z;
}
// act(z) and act'(z) together. The sigmoid's slope is e / (1 + e)^2, that of
// tanh four times the sigmoid's at 2 z: in these forms neither vanishes where
// the value has rounded to 1.
__device__ __forceinline__ void gate_both(float z, int act, float *g, float *slope) {
    *g = z;
    *slope = 1.f;
    if (act == MHC_ACT_SIGMOID) {
        const float e = expf(-fabsf(z)), s = __fdividef(1.f, 1.f + e);
        *g = z < 0.f ? e * s : s;
        *slope = e * s * s;
    } else if (act == MHC_ACT_TANH) {
        *g = tanhf(z);
        const float e = expf(-2.f * fabsf(z)), s = __fdividef(1.f, 1.f + e);
        *slope = 4.f * e * s * s;
    }
}

// ---------------------------------------------------------------- checkpoints
// Scale byte of a group whose largest magnitude has the bit pattern m: k + 127
// for the least k >= -126 with m <= Q 2^k. Q is 1.75 * 2^8 (E4M3) or
// 1.984375 * 2^6 (INT8): adding the distance of Q's mantissa from all ones
// carries into the exponent exactly when m's mantissa is above Q's. Subnormal
// m lie below Q 2^-126 and get the least k. 255 for infinity and NaN.
template <int FMT>
__device__ __forceinline__ uint32_t ckpt_scale_byte(uint32_t m) {
    if (m >= 0x7F800000u) return 255u;
    constexpr uint32_t up = FMT == MHC_CKPT_E4M3 ? 0x7FFFFFu - 0x600000u : 0x7FFFFFu - 0x7E0000u;
    constexpr int e = FMT == MHC_CKPT_E4M3 ? 8 : 6;
    const int k = static_cast<int>((m + up) >> 23) - e;
    return static_cast<uint32_t>(k < 1 ? 1 : k);
}
// 2^-k of a scale byte (a power of two, so that products with it are exact);
// NaN's byte gives 0: its codes are 0 once the caller has masked the values.
__device__ __forceinline__ float ckpt_inverse(uint32_t byte) {
    return byte == 255u ? 0.f : __uint_as_float((254u - byte) << 23);
}
__device__ __forceinline__ float ckpt_unit(uint32_t byte) {
    return byte == 255u ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(byte << 23);
}
// Code of v = x 2^-k, |v| <= Q.
template <int FMT>
__device__ __forceinline__ uint32_t ckpt_code(float v) {
    if (FMT == MHC_CKPT_E4M3) return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
    return static_cast<uint32_t>(__float2int_rn(v)) & 0xFFu;
}
template <int FMT>
__device__ __forceinline__ float ckpt_value(uint32_t code) {
    if (FMT == MHC_CKPT_E4M3) return __half2float(__half(__nv_cvt_fp8_to_halfraw(
                                   static_cast<__nv_fp8_storage_t>(code), __NV_E4M3)));
    return static_cast<float>(static_cast<signed char>(code));
}
__device__ __forceinline__ float ckpt_load(const Ckpt &c, int format, long long row, int H,
                                           int groups, int i) {
    const uint32_t code = c.codes[row * H + i], byte = c.scales[row * groups + i / kCkptGroup];
    const float v = format == MHC_CKPT_E4M3 ? ckpt_value<MHC_CKPT_E4M3>(code)
                                            : ckpt_value<MHC_CKPT_INT8>(code);
    return v * ckpt_unit(byte);
}
// One group by one warp: lane i holds the group's value i (0 past its end).
template <int FMT>
__device__ __forceinline__ uint32_t ckpt_encode_lane(float x, uint32_t *byte) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(x) & 0x7FFFFFFFu);
    *byte = ckpt_scale_byte<FMT>(m);
    return *byte == 255u ? 0u : ckpt_code<FMT>(x * ckpt_inverse(*byte));
}
__device__ __forceinline__ void ckpt_store_lane(const Ckpt &c, int format, long long row, int H,
                                                int groups, int g, int lane, float x) {
    const int i = g * kCkptGroup + lane;
    uint32_t byte, code;
    if (format == MHC_CKPT_E4M3) code = ckpt_encode_lane<MHC_CKPT_E4M3>(i < H ? x : 0.f, &byte);
    else code = ckpt_encode_lane<MHC_CKPT_INT8>(i < H ? x : 0.f, &byte);
    if (i < H) c.codes[row * H + i] = static_cast<uint8_t>(code);
    if (lane == 0) c.scales[row * groups + g] = static_cast<uint8_t>(byte);
}

// ---------------------------------------------------------------- sums
// The sums of N values over the block, in an order that its size fixes, for
// every thread. `red`: N * 32 floats of shared memory, free again at the
// caller's next call only if `red` alternates between two areas.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float *red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int warps = (blockDim.x + 31) >> 5;
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (warps == 1) return;
    if (lane == 0) {
#pragma unroll
        for (int k = 0; k < N; ++k) red[k * 32 + warp] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        v[k] = lane < warps ? red[k * 32 + lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
}

// A sum held as hi + lo, where lo gathers what each addition to hi rounded off (the error of an
// addition of two floats is a float, formed here by Knuth's two-sum): 48 bits. For the gradient of
// a single scale, a sum over all tokens and columns whose terms may all but cancel (2047 x 1102:
// 2.3 million terms). No infinity or NaN is lost: it stays in hi.
struct LongSum {
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float x) {
        const float t = __fadd_rn(hi, x), b = __fsub_rn(t, hi);
        lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(x, b));
        hi = t;
    }
    __device__ __forceinline__ void add(const LongSum &o) {
        add(o.hi);
        lo += o.lo;
    }
    __device__ __forceinline__ void add_warp() {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            LongSum other;
            other.hi = __shfl_xor_sync(0xffffffffu, hi, o);
            other.lo = __shfl_xor_sync(0xffffffffu, lo, o);
            add(other);
        }
    }
    __device__ __forceinline__ float value() const { return fabsf(hi) <= FLT_MAX ? hi + lo : hi; }
};
// Over the block, for its first warp. `red`: 64 floats of shared memory.
__device__ __forceinline__ void block_long_sum(LongSum &s, float *red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (blockDim.x + 31) >> 5;
    s.add_warp();
    if (lane == 0) {
        red[warp] = s.hi;
        red[32 + warp] = s.lo;
    }
    __syncthreads();
    if (warp) return;
    s.hi = lane < warps ? red[lane] : 0.f;
    s.lo = lane < warps ? red[32 + lane] : 0.f;
    s.add_warp();
}

// Launch of a kernel on `s`, as a programmatic dependent of the one before it
// when `pdl` (every kernel here waits for it before its first access).
template <class... P, class... A>
inline cudaError_t launch_block_kernel(void (*kern)(P...), unsigned grid, unsigned block, size_t smem,
                                       bool pdl, cudaStream_t s, A &&...a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, a...);
}

}  // namespace mhc
