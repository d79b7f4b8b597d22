// Forward of the residual norm: x' = s x + g post(y), u = pre(x').
//
// Bound by memory: x and y are read once, x' and u written once, and both
// norms' statistics are taken from the row held in registers, in float32.  u
// comes from x' before its rounding.
#include "residual_norm.cuh"

namespace gbssim {
namespace {

// Mean and 1 / deviation of the team's row; columns outside it must not count.
template <bool ALIGNED>
__device__ __forceinline__ float2 row_stats(const float (&v)[8], const Cols<ALIGNED> &c, int kind,
                                            const ResidualNormArgs &a, TeamSum &sum)
{
    if (kind == GBSSIM_ROW_NONE) return make_float2(0.0f, 1.0f);
    float mean = 0.0f;
    if (kind == GBSSIM_ROW_LAYER) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s += c.has(e) ? v[e] : 0.0f;
        mean = sum(make_float2(s, 0.0f)).x * a.inv_dim;
    }
    float q = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float d = c.has(e) ? v[e] - mean : 0.0f;
        q = fmaf(d, d, q);
    }
    const float var = sum(make_float2(q, 0.0f)).x * a.inv_dim;
    return make_float2(mean, 1.0f / sqrtf(var + a.eps));
}

template <typename R, typename Y, bool ALIGNED>
__global__ void __launch_bounds__(kMaxTeamThreads, 2)
    residual_norm_fwd_kernel(const __grid_constant__ ResidualNormArgs a)
{
    __shared__ float2 slots[2][16];
    __shared__ float2 cluster_slots[2][4];
    const Cols<ALIGNED> c(a);
    const BlockRows rows(a.plan);
    TeamSum sum{slots, cluster_slots, 0, a.plan.tpr, a.plan.teams > 1 ? 1 : a.plan.threads / 32,
                a.plan.cluster};
    const int team = a.plan.teams > 1 ? int(threadIdx.x) / a.plan.tpr : 0;
    // no block writes into another's shared memory before that block runs
    if (a.plan.cluster > 1) cooperative_groups::this_cluster().sync();

    // post and gate of a column in one factor and one summand, except that a
    // gate of its own per row stays apart
    float w1[8], b1[8], w2[8], b2[8];
    load_param(a.w1, rows.group, c, a.offset, 1.0f, w1);
    load_param(a.b1, rows.group, c, 0.0f, 0.0f, b1);
    load_param(a.w2, rows.group, c, a.offset, 1.0f, w2);
    load_param(a.b2, rows.group, c, 0.0f, 0.0f, b2);
    if (a.gate.p) {
        float g[8];
        load_param(a.gate, rows.group, c, 0.0f, 1.0f, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w1[e] *= g[e];
            b1[e] *= g[e];
        }
    }
    // every team of the block takes part in every sum, with a row or without
    for (int r0 = rows.r0; r0 < rows.r1; r0 += a.plan.teams) {
        const int r = r0 + team;
        const bool active = r < rows.r1;
        const int b = r / a.tokens, t = r - b * a.tokens;
        float x[8], y[8];
        load_row(static_cast<const R *>(a.x.p) + row_offset(a.x, b, t), c, active, x);
        float2 s1 = make_float2(0.0f, 1.0f);
        if (a.y.p) {
            load_row(static_cast<const Y *>(a.y.p) + row_offset(a.y, b, t), c, active, y);
            s1 = row_stats(y, c, a.post, a, sum);
            float g[8];
            if (a.gate_rows.p)
                load_row(static_cast<const Y *>(a.gate_rows.p) + row_offset(a.gate_rows, b, t), c,
                         active, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float z = fmaf((y[e] - s1.x) * s1.y, w1[e], b1[e]);
                if (a.gate_rows.p) z *= g[e];
                x[e] = fmaf(a.scale, x[e], z);
            }
            store_row(static_cast<R *>(a.x_out) + (long long)r * a.dim, c, active, x);
        }
        float2 s2 = make_float2(0.0f, 1.0f);
        if (a.u) {
            s2 = row_stats(x, c, a.pre, a, sum);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = fmaf((x[e] - s2.x) * s2.y, w2[e], b2[e]);
            store_row(static_cast<Y *>(a.u) + (long long)r * a.dim, c, active, x);
        }
        if (a.stats && active && c.t == 0 && c.first == 0)
            a.stats[r] = make_float4(s1.x, s1.y, s2.x, s2.y);
    }
}

template <typename R, typename Y, bool ALIGNED>
cudaError_t launch(const ResidualNormArgs &a, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.plan.grid);
    cfg.blockDim = dim3(unsigned(a.plan.threads));
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(a.plan.cluster);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.plan.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, residual_norm_fwd_kernel<R, Y, ALIGNED>, a);
}

template <typename R, typename Y>
cudaError_t launch(const ResidualNormArgs &a, cudaStream_t s)
{
    return a.plan.aligned ? launch<R, Y, true>(a, s) : launch<R, Y, false>(a, s);
}

}  // namespace

cudaError_t residual_norm_fwd_launch(const ResidualNormArgs &a, int res, int blk, cudaStream_t s)
{
    if (res == GBSSIM_F32) {
        if (blk == GBSSIM_F32) return launch<float, float>(a, s);
        if (blk == GBSSIM_BF16) return launch<float, bf16>(a, s);
        return launch<float, f16>(a, s);
    }
    return res == GBSSIM_BF16 ? launch<bf16, bf16>(a, s) : launch<f16, f16>(a, s);
}

}  // namespace gbssim
