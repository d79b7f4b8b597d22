// The backward of the residual norm with a 16-bit residual stream.
#include "residual_norm_bwd.cuh"

namespace gbssim {

cudaError_t residual_norm_bwd_16_status(unsigned *flags, bool clear)
{
    return exchange_status(flags, clear);
}

cudaError_t residual_norm_bwd_16_launch(const ResidualNormArgs &a, int blk, cudaStream_t s)
{
    return blk == GBSSIM_BF16 ? launch<bf16, bf16>(a, s) : launch<f16, f16>(a, s);
}

}  // namespace gbssim
