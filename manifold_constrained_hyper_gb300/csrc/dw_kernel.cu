// Weight gradient of a projection from its checkpointed input:
// d_w[i][j] = sum_t d_out[t][i] * x[t][j].
#include "block_common.cuh"

namespace mhc {
namespace {

constexpr int kTile = 64, kStep = 16;

// 64 x 64 outputs a CTA, 4 x 4 a thread, 16 tokens a step.
__global__ void __launch_bounds__(256) dw_tile_kernel(const DwArgs a) {
    __shared__ float sd[kStep][kTile], sx[kStep][kTile];
    griddep_wait();
    const int tiles_k = (a.k + kTile - 1) / kTile, groups = (a.k + 31) / 32;
    const int i0 = static_cast<int>(blockIdx.x / tiles_k) * kTile, j0 = static_cast<int>(blockIdx.x % tiles_k) * kTile;
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (long long t0 = 0; t0 < a.T; t0 += kStep) {
        for (int e = threadIdx.x; e < kStep * kTile; e += 256) {
            const long long t = t0 + e / kTile;
            const int i = i0 + e % kTile, j = j0 + e % kTile;
            sd[e / kTile][e % kTile] = t < a.T && i < a.n ? load_any(a.d_out, a.dtype, t * a.d_out_stride + i) : 0.f;
            float x = t < a.T && j < a.k ? ckpt_load(a.x, a.format, t, a.k, groups, j) : 0.f;
            if (a.dtype == MHC_F16) x = to_f32(from_f32<__half>(x));
            sx[e / kTile][e % kTile] = x;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kStep; ++k)
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    acc[r][c] = fmaf(sd[k][ty * 4 + r], sx[k][tx + 16 * c], acc[r][c]);
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int i = i0 + ty * 4 + r, j = j0 + tx + 16 * c;
            if (i >= a.n || j >= a.k) continue;
            const long long at = static_cast<long long>(i) * a.k + j;
            const float v = a.accumulate ? load_any(a.d_w, a.d_w_dtype, at) + acc[r][c] : acc[r][c];
            store_any(a.d_w, a.d_w_dtype, at, v);
        }
}

}  // namespace

cudaError_t launch_dw(const DwArgs &a, bool pdl, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>((a.n + kTile - 1) / kTile) * static_cast<unsigned>((a.k + kTile - 1) / kTile);
    return launch_block_kernel(dw_tile_kernel, grid, 256, 0, pdl, s, a);
}

}  // namespace mhc
