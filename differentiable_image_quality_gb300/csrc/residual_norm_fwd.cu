// Forward of the residual norm: x' = s x + g post(y), u = pre(x').
//
// Bound by memory: x and y are read once, x' and u written once, and both
// norms' statistics are taken from the row held in registers, in float32.  u
// comes from x' before its rounding.
#include "common.cuh"
#include "residual_norm.cuh"

namespace gbssim {
namespace {

struct RowStats {
    float mean, rstd;
};

// Mean and 1 / deviation of the team's row.  Columns that the row does not have
// hold zero: they add nothing to a sum of squares, but must not count about a mean.
template <bool ALIGNED>
__device__ __forceinline__ RowStats row_stats(const f32x2 (&v)[4], const Cols<ALIGNED> &c, int kind,
                                              const ResidualNormArgs &a, TeamSum &sum)
{
    if (kind == GBSSIM_ROW_NONE) return {0.0f, 1.0f};
    f32x2 q = 0;
    float mean = 0.0f;
    if (kind == GBSSIM_ROW_LAYER) {
        mean = sum.one(sum2(add2(add2(v[0], v[1]), add2(v[2], v[3])))) * a.inv_dim;
        const f32x2 m = both(-mean);
        if (c.all()) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f32x2 d = add2(v[e], m);
                q = fma2(d, d, q);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 h = halves(add2(v[e / 2], m));
                const float d = c.has(e) ? (e & 1 ? h.y : h.x) : 0.0f;
                q = fma2(pair(d, 0.0f), pair(d, 0.0f), q);
            }
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) q = fma2(v[e], v[e], q);
    }
    return {mean, rsqrtf(fmaf(sum.one(sum2(q)), a.inv_dim, a.eps))};
}

// BIAS: either norm has a bias.
template <typename R, typename Y, bool ALIGNED, bool BIAS>
__global__ void __launch_bounds__(kMaxTeamThreads, 2)
    residual_norm_fwd_kernel(const __grid_constant__ ResidualNormArgs a)
{
    using SR = Staged<R, ALIGNED>;
    using SY = Staged<Y, ALIGNED>;
    extern __shared__ uint4 ring[];
    __shared__ float2 slots[2][16];
    __shared__ float2 cluster_slots[2][4];
    const BlockRows rows(a);
    const Cols<ALIGNED> c(a, rows.shift);
    TeamSum sum{slots, cluster_slots, 0, a.plan.tpr, a.plan.teams > 1 ? 1 : a.plan.threads / 32,
                a.plan.cluster};
    const int team = a.plan.teams > 1 ? int(threadIdx.x) / a.plan.tpr : 0;
    const int step = rows.step * a.plan.teams;  // rows from one of the team's to its next
    const int pitch = a.plan.threads * 16, stages = a.plan.stages;
    const bool has_y = a.y.p, has_gates = a.gate_rows.p;
    const int stage_bytes = (SR::kUnits + SY::kUnits * (has_gates ? 2 : 1)) * pitch;
    const unsigned mine = smem_u32(ring) + threadIdx.x * 16, over = mine + stages * stage_bytes;
    // no block writes into another's shared memory before that block runs
    if (a.plan.cluster > 1) cooperative_groups::this_cluster().sync();

    int r = rows.first + team * rows.step, left = rows.count - team;  // the team's row; none if <= 0
    int ahead = r, ahead_left = left;
    unsigned to = mine;
    const auto fetch = [&] {
        if (ahead_left > 0 && c.any()) {
            SR::fetch(a.x, row_at<R>(a.x, a.tokens, ahead, c.first), c, to, pitch);
            if (has_y)
                SY::fetch(a.y, row_at<Y>(a.y, a.tokens, ahead, c.first), c, to + SR::kUnits * pitch,
                          pitch);
            if (has_gates)
                SY::fetch(a.gate_rows, row_at<Y>(a.gate_rows, a.tokens, ahead, c.first), c,
                          to + (SR::kUnits + SY::kUnits) * pitch, pitch);
        }
        staged_commit();
        ahead += step;
        ahead_left -= a.plan.teams;
        to += stage_bytes;
        if (to == over) to = mine;
    };
    for (int i = 0; i < stages - 1; ++i) fetch();

    // post and gate of a column in one factor and one summand; a gate of its
    // own per row stays apart
    f32x2 w1[4], b1[4], w2[4], b2[4];
    load_param(a.w1, rows.group, c, a.offset, 1.0f, w1);
    load_param(a.w2, rows.group, c, a.offset, 1.0f, w2);
    if (BIAS) {
        load_param(a.b1, rows.group, c, 0.0f, 0.0f, b1);
        load_param(a.b2, rows.group, c, 0.0f, 0.0f, b2);
    }
    if (a.gate.p) {
        f32x2 g[4];
        load_param(a.gate, rows.group, c, 0.0f, 1.0f, g);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w1[e] = mul2(w1[e], g[e]);
            if (BIAS) b1[e] = mul2(b1[e], g[e]);
        }
    }
    const f32x2 scale = both(a.scale);
    unsigned at = mine;
    // every team of the block takes part in every sum, with a row or without
    for (int i = 0; i < rows.count; i += a.plan.teams) {
        const bool active = left > 0;
        fetch();
        staged_wait(stages);
        f32x2 x[4];
        SR::read(a.x, a.tokens, r, c, active, at, pitch, x);
        RowStats s1 = {0.0f, 1.0f}, s2 = {0.0f, 1.0f};
        if (has_y) {
            f32x2 y[4];
            SY::read(a.y, a.tokens, r, c, active, at + SR::kUnits * pitch, pitch, y);
            s1 = row_stats(y, c, a.post, a, sum);
            const f32x2 v = both(s1.rstd), m = both(-s1.mean * s1.rstd);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[e] = fma2(y[e], v, m);
                y[e] = BIAS ? fma2(y[e], w1[e], b1[e]) : mul2(y[e], w1[e]);
            }
            if (has_gates) {
                f32x2 g[4];
                SY::read(a.gate_rows, a.tokens, r, c, active, at + (SR::kUnits + SY::kUnits) * pitch,
                         pitch, g);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = mul2(y[e], g[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = fma2(scale, x[e], y[e]);
            store_cols(static_cast<R *>(a.x_out) + ((long long)r * a.dim + c.first), c, active, x);
        }
        if (a.u) {
            s2 = row_stats(x, c, a.pre, a, sum);
            const f32x2 v = both(s2.rstd), m = both(-s2.mean * s2.rstd);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[e] = fma2(x[e], v, m);
                x[e] = BIAS ? fma2(x[e], w2[e], b2[e]) : mul2(x[e], w2[e]);
            }
            store_cols(static_cast<Y *>(a.u) + ((long long)r * a.dim + c.first), c, active, x);
        }
        if (a.stats && active && c.first <= 0 && c.any())
            a.stats[r] = make_float4(s1.mean, s1.rstd, s2.mean, s2.rstd);
        r += step;
        left -= a.plan.teams;
        at += stage_bytes;
        if (at == over) at = mine;
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
