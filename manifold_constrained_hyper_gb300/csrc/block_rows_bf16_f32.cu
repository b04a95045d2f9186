// The gated residual block's row kernels: y of __nv_bfloat16, residual of float.
#include "block_backward.cuh"
#include "block_forward.cuh"

namespace mhc {

cudaError_t block_fwd_bf16_f32(const BlockFwdArgs &a, int dtype, int r_dtype, int sms, bool pdl, cudaStream_t s) {
    return block_fwd<__nv_bfloat16, float>(a, dtype, r_dtype, sms, pdl, s);
}
cudaError_t block_bwd_bf16_f32(const BlockBwdArgs &a, int dtype, int r_dtype, int sms, bool pdl, int *parts, cudaStream_t s) {
    return block_bwd<__nv_bfloat16, float>(a, dtype, r_dtype, sms, pdl, parts, s);
}

}  // namespace mhc
