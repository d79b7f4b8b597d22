// Host side: tensor maps of the tensor-copy unit.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <mutex>

namespace gbssim {

inline PFN_cuTensorMapEncodeTiled_v12000 heads_map_encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    });
    return encode;
}

// [batch][token][head][dim] of a 16-bit type, strides in elements; boxes of 64 columns
// x `box_heads` x `box_tokens` of one sample, with the 128-byte swizzle.  What lies
// outside the tensor reads as zeros.
inline bool encode_heads_map(CUtensorMap &m, const void *data, bool bf, int dim, int heads, int tokens,
                             int batch, long long head_stride, long long token_stride,
                             long long batch_stride, int box_heads, int box_tokens)
{
    const auto encode = heads_map_encoder();
    if (!encode) return false;
    const cuuint64_t dims[4] = {cuuint64_t(dim), cuuint64_t(heads), cuuint64_t(tokens), cuuint64_t(batch)};
    const cuuint64_t strides[3] = {cuuint64_t(head_stride) * 2, cuuint64_t(token_stride) * 2,
                                   cuuint64_t(batch_stride) * 2};
    const cuuint32_t box[4] = {64, cuuint32_t(box_heads), cuuint32_t(box_tokens), 1};
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    const auto once = [&] {
        return encode(&m, bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                      const_cast<void *>(data), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    if (once()) return true;
    // a host thread that has not used the device yet (autograd's, before its first
    // launch) has no current context, which this driver call does not make by itself
    int device = 0;
    return cudaGetDevice(&device) == cudaSuccess && cudaSetDevice(device) == cudaSuccess && once();
}

}  // namespace gbssim
