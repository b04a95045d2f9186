// The gated residual block's row kernels: y of __half, residual of float.
#include "block_backward.cuh"
#include "block_forward.cuh"

namespace mhc {

cudaError_t block_fwd_f16_f32(const BlockFwdArgs &a, int dtype, int r_dtype, int sms, bool pdl, cudaStream_t s) {
    return block_fwd<__half, float>(a, dtype, r_dtype, sms, pdl, s);
}
cudaError_t block_bwd_f16_f32(const BlockBwdArgs &a, int dtype, int r_dtype, int sms, bool pdl, int *parts, cudaStream_t s) {
    return block_bwd<__half, float>(a, dtype, r_dtype, sms, pdl, parts, s);
}

}  // namespace mhc
