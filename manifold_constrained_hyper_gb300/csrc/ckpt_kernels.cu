// 8-bit activation checkpoints: packing and reading back.
#include "block_common.cuh"

namespace mhc {
namespace {

constexpr int kThreads = 256;

// A warp per group of 32 values: any width, stride and alignment.
template <class T>
__global__ void ckpt_pack_kernel(const CkptArgs a, int format) {
    griddep_wait();
    const int groups = (a.H + 31) / 32, lane = threadIdx.x & 31;
    const long long total = a.T * groups, step = static_cast<long long>(gridDim.x) * (kThreads / 32);
    for (long long i = static_cast<long long>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; i < total;
         i += step) {
        const long long t = i / groups;
        const int g = static_cast<int>(i - t * groups), c = g * 32 + lane;
        const float x = c < a.H ? to_f32(static_cast<const T *>(a.x)[t * a.stride + c]) : 0.f;
        ckpt_store_lane(a.c, format, t, a.H, groups, g, lane, x);
    }
}

template <class T>
__global__ void ckpt_unpack_kernel(const CkptArgs a, int format) {
    griddep_wait();
    const int groups = (a.H + 31) / 32, lane = threadIdx.x & 31;
    const long long total = a.T * groups, step = static_cast<long long>(gridDim.x) * (kThreads / 32);
    for (long long i = static_cast<long long>(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; i < total;
         i += step) {
        const long long t = i / groups;
        const int g = static_cast<int>(i - t * groups), c = g * 32 + lane;
        if (c < a.H)
            static_cast<T *>(a.out)[t * a.stride + c] = from_f32<T>(ckpt_load(a.c, format, t, a.H, groups, c));
    }
}

unsigned grid_for(long long groups, int sms) {
    const long long need = (groups + kThreads / 32 - 1) / (kThreads / 32), cap = static_cast<long long>(sms) * 8;
    return static_cast<unsigned>(need < cap ? need : cap);
}

}  // namespace

cudaError_t launch_ckpt_pack(const CkptArgs &a, int dtype, int format, int sms, bool pdl, cudaStream_t s) {
    const unsigned grid = grid_for(a.T * ckpt_groups(a.H), sms);
    auto kern = dtype == MHC_F32 ? ckpt_pack_kernel<float>
                : dtype == MHC_BF16 ? ckpt_pack_kernel<__nv_bfloat16> : ckpt_pack_kernel<__half>;
    return launch_block_kernel(kern, grid, kThreads, 0, pdl, s, a, format);
}

cudaError_t launch_ckpt_unpack(const CkptArgs &a, int dtype, int format, int sms, bool pdl, cudaStream_t s) {
    const unsigned grid = grid_for(a.T * ckpt_groups(a.H), sms);
    auto kern = dtype == MHC_F32 ? ckpt_unpack_kernel<float>
                : dtype == MHC_BF16 ? ckpt_unpack_kernel<__nv_bfloat16> : ckpt_unpack_kernel<__half>;
    return launch_block_kernel(kern, grid, kThreads, 0, pdl, s, a, format);
}

}  // namespace mhc
