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
// One element on any boundary.
template <int KIND>
__device__ __forceinline__ void finish_element(const EpilogueArgs &e, long long i, long long at, int j, float x) {
    if constexpr (KIND == EPI_LINEAR) {
        x *= e.unit;
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
