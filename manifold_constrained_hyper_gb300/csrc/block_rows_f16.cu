// The gated residual block's row kernels: y of __half, residual of __half.
#include "block_backward.cuh"
#include "block_forward.cuh"

namespace mhc {

cudaError_t block_fwd_f16(const BlockFwdArgs &a, int dtype, int r_dtype, int sms, bool pdl, cudaStream_t s) {
    return block_fwd<__half, __half>(a, dtype, r_dtype, sms, pdl, s);
}
cudaError_t block_bwd_f16(const BlockBwdArgs &a, int dtype, int r_dtype, int sms, bool pdl, int *parts, cudaStream_t s) {
    return block_bwd<__half, __half>(a, dtype, r_dtype, sms, pdl, parts, s);
}

}  // namespace mhc
