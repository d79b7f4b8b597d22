// The backward of the residual norm with a float32 residual stream.
#include "residual_norm_bwd.cuh"

namespace gbssim {

cudaError_t residual_norm_bwd_f32_status(unsigned *flags, bool clear)
{
    return exchange_status(flags, clear);
}

cudaError_t residual_norm_bwd_f32_launch(const ResidualNormArgs &a, int blk, cudaStream_t s)
{
    return blk == GBSSIM_F32    ? launch<float, float>(a, s)
           : blk == GBSSIM_BF16 ? launch<float, bf16>(a, s)
                                : launch<float, f16>(a, s);
}

}  // namespace gbssim
