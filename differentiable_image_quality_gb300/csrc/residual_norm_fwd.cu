// Forward of the residual norm: x' = s x + g post(y), u = pre(x').
//
// Bound by memory: x and y are read once, x' and u written once, and both
// norms' statistics are taken from the row held in registers, in float32.  u
// comes from x' before its rounding.
#include "residual_norm.cuh"

namespace gbssim {
namespace {

// (mean / deviation, 1 / deviation, mean) of the team's row, so that a normalised
// value is one fused multiply-add: v * y - x.
struct RowStats {
    float scaled_mean, rstd, mean;
};

// Columns that the row does not have hold zero: they add nothing to a sum of
// squares, but must not count about a mean.
template <bool ALIGNED>
__device__ __forceinline__ RowStats row_stats(const float (&v)[8], const Cols<ALIGNED> &c, int kind,
                                              const ResidualNormArgs &a, TeamSum &sum)
{
    if (kind == GBSSIM_ROW_NONE) return {0.0f, 1.0f, 0.0f};
    float q[1] = {0.0f}, mean = 0.0f;
    if (kind == GBSSIM_ROW_LAYER) {
        float s[1] = {0.0f};
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] += v[e];
        sum(s);
        mean = s[0] * a.inv_dim;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float d = c.has(e) ? v[e] - mean : 0.0f;
            q[0] = fmaf(d, d, q[0]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) q[0] = fmaf(v[e], v[e], q[0]);
    }
    sum(q);
    const float rstd = rsqrtf(fmaf(q[0], a.inv_dim, a.eps));
    return {mean * rstd, rstd, mean};
}

// BIAS: either norm has a bias.
template <typename R, typename Y, bool ALIGNED, bool BIAS>
__global__ void __launch_bounds__(kMaxTeamThreads, 2)
    residual_norm_fwd_kernel(const __grid_constant__ ResidualNormArgs a)
{
    using SR = Staged<R, ALIGNED>;
    using SY = Staged<Y, ALIGNED>;
    extern __shared__ uint4 ring[];
    __shared__ float slots[2][2][16];
    __shared__ float cluster_slots[2][2][4];
    const BlockRows rows(a);
    const Cols<ALIGNED> c(a, rows.shift);
    TeamSum sum{slots, cluster_slots, 0, a.plan.tpr, a.plan.teams > 1 ? 1 : a.plan.threads / 32,
                a.plan.cluster};
    const int team = a.plan.teams > 1 ? int(threadIdx.x) / a.plan.tpr : 0;
    const int threads = a.plan.threads, stages = a.plan.stages;
    const int stage_words = (SR::kUnits + SY::kUnits * (a.gate_rows.p ? 2 : 1)) * threads;
    uint4 *const mine = ring + threadIdx.x;
    // no block writes into another's shared memory before that block runs
    if (a.plan.cluster > 1) cooperative_groups::this_cluster().sync();

    const auto fetch = [&](int i, uint4 *slot) {
        if (i < rows.count && c.any()) {
            const int r = rows.first + i * rows.step;
            SR::fetch(a.x, row_of<R>(a.x, a.tokens, r), c, slot, threads);
            slot += SR::kUnits * threads;
            if (a.y.p) SY::fetch(a.y, row_of<Y>(a.y, a.tokens, r), c, slot, threads);
            slot += SY::kUnits * threads;
            if (a.gate_rows.p)
                SY::fetch(a.gate_rows, row_of<Y>(a.gate_rows, a.tokens, r), c, slot, threads);
        }
        staged_commit();
    };
    for (int i = 0; i < stages - 1; ++i) fetch(i * a.plan.teams + team, mine + i * stage_words);

    // post and gate of a column in one factor and one summand; a gate of its
    // own per row stays apart
    float w1[8], b1[8], w2[8], b2[8];
    load_param(a.w1, rows.group, c, a.offset, 1.0f, w1);
    load_param(a.w2, rows.group, c, a.offset, 1.0f, w2);
    if (BIAS) {
        load_param(a.b1, rows.group, c, 0.0f, 0.0f, b1);
        load_param(a.b2, rows.group, c, 0.0f, 0.0f, b2);
    }
    if (a.gate.p) {
        float g[8];
        load_param(a.gate, rows.group, c, 0.0f, 1.0f, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w1[e] *= g[e];
            if (BIAS) b1[e] *= g[e];
        }
    }
    int now = 0;
    // every team of the block takes part in every sum, with a row or without
    for (int i0 = 0; i0 < rows.count; i0 += a.plan.teams) {
        const int i = i0 + team, r = rows.first + i * rows.step;
        const bool active = i < rows.count;
        {
            const int ahead = now == 0 ? stages - 1 : now - 1;
            fetch(i + (stages - 1) * a.plan.teams, mine + ahead * stage_words);
        }
        staged_wait(stages);
        const uint4 *slot = mine + now * stage_words;
        now = now + 1 == stages ? 0 : now + 1;
        float x[8];
        SR::read(row_of<R>(a.x, a.tokens, r), c, active, slot, threads, x);
        slot += SR::kUnits * threads;
        RowStats s1 = {0.0f, 1.0f, 0.0f}, s2 = {0.0f, 1.0f, 0.0f};
        if (a.y.p) {
            float y[8];
            SY::read(row_of<Y>(a.y, a.tokens, r), c, active, slot, threads, y);
            s1 = row_stats(y, c, a.post, a, sum);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float h = fmaf(y[e], s1.rstd, -s1.scaled_mean);
                y[e] = BIAS ? fmaf(h, w1[e], b1[e]) : h * w1[e];
            }
            if (a.gate_rows.p) {
                float g[8];
                SY::read(row_of<Y>(a.gate_rows, a.tokens, r), c, active, slot + SY::kUnits * threads,
                         threads, g);
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] *= g[e];
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = fmaf(a.scale, x[e], y[e]);
            store_row(static_cast<R *>(a.x_out) + (long long)r * a.dim, c, active, x);
        }
        if (a.u) {
            s2 = row_stats(x, c, a.pre, a, sum);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float h = fmaf(x[e], s2.rstd, -s2.scaled_mean);
                x[e] = BIAS ? fmaf(h, w2[e], b2[e]) : h * w2[e];
            }
            store_row(static_cast<Y *>(a.u) + (long long)r * a.dim, c, active, x);
        }
        if (a.stats && active && c.first <= 0 && c.any())
            a.stats[r] = make_float4(s1.mean, s1.rstd, s2.mean, s2.rstd);
    }
}

template <typename R, typename Y, bool ALIGNED, bool BIAS>
cudaError_t launch(ResidualNormArgs a, cudaStream_t s)
{
    const int units = Staged<R, ALIGNED>::kUnits +
                      Staged<Y, ALIGNED>::kUnits * (a.gate_rows.p ? 2 : 1);
    return launch_staged(residual_norm_fwd_kernel<R, Y, ALIGNED, BIAS>, a, units, 2, s);
}

template <typename R, typename Y>
cudaError_t launch(const ResidualNormArgs &a, cudaStream_t s)
{
    const bool bias = a.b1.p || a.b2.p;
    if (a.plan.aligned) return bias ? launch<R, Y, true, true>(a, s) : launch<R, Y, true, false>(a, s);
    return bias ? launch<R, Y, false, true>(a, s) : launch<R, Y, false, false>(a, s);
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
