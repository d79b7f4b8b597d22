// The second kernel of the residual norm's backward: the parameters' gradients from
// the blocks' column sums.  Its reads are the partials, some megabytes at most;
// what it costs is the time of a few dependent loads, so a column's partials go
// to 64 threads.
#include <climits>

#include "residual_norm.cuh"

namespace gbssim {
namespace {

constexpr int kFinishCols = 8, kFinishLanes = 64;

__device__ __forceinline__ void store_param(const ParamGrad &g, int group, int dim, int col, float v)
{
    if (!g.p) return;
    const long long i = (g.per_sample ? (long long)group * dim : 0) + col;
    if (g.type == GBSSIM_F32) static_cast<float *>(g.p)[i] = v;
    else if (g.type == GBSSIM_BF16) static_cast<bf16 *>(g.p)[i] = from_f32<bf16>(v);
    else static_cast<f16 *>(g.p)[i] = from_f32<f16>(v);
}

// Adds the blocks' partials.  A block takes 8 columns (one sector of each
// partial), 64 threads of a column every 64th partial each, then their sums in a
// fixed order.  Part y < groups of the grid makes the gradients that each group has of its
// own, the last those shared by all.
__global__ void __launch_bounds__(kFinishCols * kFinishLanes)
    residual_norm_finish_kernel(const __grid_constant__ ResidualNormArgs a,
                                const __grid_constant__ ParamGrads g, int shared_part)
{
    constexpr int kWarps = kFinishCols * kFinishLanes / 32;
    __shared__ float part[5][kWarps][kFinishCols];
    const int cx = threadIdx.x % kFinishCols, lane = threadIdx.x / kFinishCols;
    const int across = (a.dim + kFinishCols - 1) / kFinishCols;  // blocks of a part
    const int y = int(blockIdx.x) / across, first = (int(blockIdx.x) - y * across) * kFinishCols;
    const int col = first + cx;
    const bool shared = y == shared_part;
    const int each = a.plan.classes * a.plan.splits;  // partials of a group
    const int p0 = shared ? 0 : y * each;
    const int p1 = shared ? a.plan.groups * each : p0 + each;
    const bool full = a.gate_rows.p != nullptr;
    // what turns A and F into the gradients
    const auto factors = [&](int group, float &gate, float &w, float &b) {
        gate = a.gate.p && !full ? param_at(a.gate, group, col) : 1.0f;
        w = a.w1.p ? param_at(a.w1, group, col) + a.offset : 1.0f;
        b = a.b1.p ? param_at(a.b1, group, col) : 0.0f;
    };
    // dg, dw1, db1, dw2, db2
    float v[5] = {};
    pdl_wait();
    if (col < a.dim && p0 < p1) {
        const bool vary = shared && (a.gate.stride || a.w1.stride || a.b1.stride);
        float gate, w, b;
        if (!vary) factors(p0 / each, gate, w, b);
        const long long pitch = (long long)a.sums * a.dim;
        const float *src = a.partials + (p0 + lane) * pitch + col;
#pragma unroll 4
        for (int p = p0 + lane; p < p1; p += kFinishLanes, src += kFinishLanes * pitch) {
            const float A = a.sum_a >= 0 ? __ldcg(src + (long long)a.sum_a * a.dim) : 0.0f;
            const float F = a.sum_f >= 0 ? __ldcg(src + (long long)a.sum_f * a.dim) : 0.0f;
            const float C = a.sum_c >= 0 ? __ldcg(src + (long long)a.sum_c * a.dim) : 0.0f;
            const float E = a.sum_e >= 0 ? __ldcg(src + (long long)a.sum_e * a.dim) : 0.0f;
            if (vary) factors(p / each, gate, w, b);
            v[0] += fmaf(w, A, b * F);
            v[1] = fmaf(gate, A, v[1]);
            v[2] = fmaf(gate, F, v[2]);
            v[3] += C;
            v[4] += E;
        }
    }
    // a warp holds four threads of each column
#pragma unroll
    for (int k = 0; k < 5; ++k) {
        v[k] += __shfl_xor_sync(0xffffffffu, v[k], 8);
        v[k] += __shfl_xor_sync(0xffffffffu, v[k], 16);
        if ((threadIdx.x & 31) < kFinishCols) part[k][threadIdx.x / 32][cx] = v[k];
    }
    __syncthreads();
    if (threadIdx.x < 5 * kFinishCols) {
        const int k = threadIdx.x / kFinishCols, x = threadIdx.x % kFinishCols;
        const int to = first + x;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += part[k][w][x];
        const ParamGrad &out = k == 0 ? g.gate : k == 1 ? g.w1 : k == 2 ? g.b1 : k == 3 ? g.w2 : g.b2;
        if (to < a.dim && bool(out.per_sample) != shared) store_param(out, y, a.dim, to, s);
    }
}

}  // namespace

cudaError_t residual_norm_bwd_launch(const ResidualNormArgs &a, int res, int blk,
                                     const ParamGrads &g, cudaStream_t s)
{
    cudaError_t e = cudaSuccess;
    if (a.plan.grid > 0) {
        e = res == GBSSIM_F32 ? residual_norm_bwd_f32_launch(a, blk, s)
                              : residual_norm_bwd_16_launch(a, blk, s);
    }
    if (e != cudaSuccess || a.sums == 0) return e;
    bool own = false, shared = false;
    for (const ParamGrad *p : {&g.gate, &g.w1, &g.b1, &g.w2, &g.b2})
        if (p->p) (p->per_sample ? own : shared) = true;
    const int shared_part = own ? a.plan.groups : 0;
    const long long blocks =
        (long long)((a.dim + kFinishCols - 1) / kFinishCols) * (shared_part + (shared ? 1 : 0));
    if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(kFinishCols * kFinishLanes);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, residual_norm_finish_kernel, a, g, shared_part);
}

}  // namespace gbssim
