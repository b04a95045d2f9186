// Dispatch of the gated residual block's row kernels by type, and the kernel that
// ends the backward pass: sums over tokens from the row kernel's CTAs.
#include "block_common.cuh"

namespace mhc {

#define MHC_ROWS(T)                                                                                              \
    cudaError_t block_fwd_##T(const BlockFwdArgs &, int, int, int, bool, cudaStream_t);                          \
    cudaError_t block_bwd_##T(const BlockBwdArgs &, int, int, int, bool, int *, cudaStream_t)
MHC_ROWS(bf16);
MHC_ROWS(bf16_f32);
MHC_ROWS(f16);
MHC_ROWS(f16_f32);
MHC_ROWS(f32);
#undef MHC_ROWS

namespace {

// Sums over the row kernel's CTAs, in an order that their number fixes: a warp
// every 16th CTA, the warps' sums then in turn. VEC columns a lane: 4 where H is
// a multiple of 4 (16-byte loads), else 1. Bound by L2: 152 CTAs leave 13 MB at H 7168.
constexpr int kSumWarps = 16;
template <int VEC>
__global__ void __launch_bounds__(32 * kSumWarps) block_sums_kernel(const BlockSumArgs a) {
    __shared__ float part[kSumWarps][32 * VEC];
    griddep_wait();
    const BlockForm &f = a.f;
    const int H = f.H, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = blockIdx.y;
    const int c0 = (blockIdx.x * 32 + lane) * VEC;
    float v[VEC] = {};
    if (c0 < H) {
#pragma unroll 5
        for (int p = warp; p < a.parts; p += kSumWarps) {
            const float *const src = a.sums + (static_cast<long long>(p) * kBackSums + k) * H + c0;
            if constexpr (VEC == 4) {
                const float4 w = *reinterpret_cast<const float4 *>(src);
                v[0] += w.x;
                v[1] += w.y;
                v[2] += w.z;
                v[3] += w.w;
            } else {
                v[0] += *src;
            }
        }
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) part[warp][e * 32 + lane] = v[e];
    __syncthreads();
    // a thread a column from here
    const int e = threadIdx.x / 32, c = (blockIdx.x * 32 + lane) * VEC + e;
    if (e < VEC && c < H) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kSumWarps; ++w) s += part[w][e * 32 + lane];
        if (k == 0) {
            float g = 1.f, slope = 1.f;
            if (f.gate_form == MHC_GATE_CHANNEL) gate_both(load_any(f.gate, f.gate_dtype, c), f.gate_act, &g, &slope);
            if (a.d_w_post) a.d_w_post[c] = g * s;
            if (a.d_gate) a.d_gate[c] = slope * weight_at(f.w_post, f.w_post_dtype, f.weight_offset, c) * s;
        } else if (k == 1) {
            if (a.d_w_pre) a.d_w_pre[c] = s;
        } else {
            a.d_res_scale[c] = s;
        }
    }
    if (k == 0 && blockIdx.x == 0 && a.d_res_scale && f.scale_form == MHC_SCALE_ONE && warp == kSumWarps - 1) {
        LongSum s;
        for (int p = lane; p < a.parts; p += 32) {
            LongSum part;
            part.hi = a.scale_sums[2 * p];
            part.lo = a.scale_sums[2 * p + 1];
            s.add(part);
        }
        s.add_warp();
        if (lane == 0) a.d_res_scale[0] = s.value();
    }
}

}  // namespace

cudaError_t launch_block_fwd(const BlockFwdArgs &a, int dtype, int r_dtype, int sms, bool pdl, cudaStream_t s) {
    const bool wide = r_dtype == MHC_F32;
    auto rows = dtype == MHC_F32 ? block_fwd_f32
                : dtype == MHC_BF16 ? (wide ? block_fwd_bf16_f32 : block_fwd_bf16)
                                    : (wide ? block_fwd_f16_f32 : block_fwd_f16);
    return rows(a, dtype, r_dtype, sms, pdl, s);
}

cudaError_t launch_block_bwd(const BlockBwdArgs &a, int dtype, int r_dtype, int sms, bool pdl, int *parts,
                             cudaStream_t s) {
    const bool wide = r_dtype == MHC_F32;
    auto rows = dtype == MHC_F32 ? block_bwd_f32
                : dtype == MHC_BF16 ? (wide ? block_bwd_bf16_f32 : block_bwd_bf16)
                                    : (wide ? block_bwd_f16_f32 : block_bwd_f16);
    return rows(a, dtype, r_dtype, sms, pdl, parts, s);
}

cudaError_t launch_block_sums(const BlockSumArgs &a, bool pdl, cudaStream_t s) {
    const int vec = a.f.H % 4 == 0 ? 4 : 1;         // the workspace is on 16 bytes
    const unsigned kinds = a.d_res_scale && a.f.scale_form == MHC_SCALE_CHANNEL ? 3 : 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((a.f.H + 32 * vec - 1) / (32 * vec)), kinds);
    cfg.blockDim = dim3(32 * kSumWarps);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, vec == 4 ? block_sums_kernel<4> : block_sums_kernel<1>, a);
}

}  // namespace mhc
