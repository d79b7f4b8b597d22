// Forward of the residual norm: x' = s x + g post(y), u = pre(x').
//
// Bound by memory: x and y are read once, x' and u written once, and both
// norms' statistics are taken from the row held in registers, in float32.  u
// comes from x' before its rounding.  What has to be hidden is the chain of two
// sums over the row: by the rows of other blocks, and by copying the next row
// meanwhile.  65536 x 4096 bfloat16, root-mean-square norms: 332 to 359 us for
// 2.15 GB (88 to 95 % of the copy rate); 8192 x 1152 conditioned, float32
// stream: 29 us (57 %, instruction issue).
#include "residual_norm.cuh"

namespace gbssim {
namespace {

// 16-byte words a thread stages of a row: x, y and a gate per row.
template <typename R, typename Y, bool ALIGNED, bool ANY>
constexpr int fwd_units()
{
    return Staged<R, ALIGNED, ANY>::kUnits + Staged<Y, ALIGNED, ANY>::kUnits * (ANY ? 2 : 1);
}

template <typename R, typename Y, bool ALIGNED, bool ANY>
constexpr int fwd_stages()
{
    return stages_of(fwd_units<R, Y, ALIGNED, ANY>(), 2);
}

struct RowStats {
    float mean, rstd;
};

// Mean and 1 / deviation of the team's row.  Columns that the row does not have
// hold zero: they add nothing to a sum of squares, but must not count about a mean.
template <bool LAYER, bool ALIGNED, bool CLUSTER>
__device__ __forceinline__ RowStats row_stats(const f32x2 (&v)[4], const Cols<ALIGNED> &c, int kind,
                                              const ResidualNormArgs &a, TeamSum<CLUSTER> &sum)
{
    if (kind == GBSSIM_ROW_NONE) return {0.0f, 1.0f};
    if (!LAYER || kind == GBSSIM_ROW_RMS) {
        f32x2 q = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) q = fma2(v[e], v[e], q);
        return {0.0f, rsqrtf(fmaf(sum.one(sum2(q)), a.inv_dim, a.eps))};
    }
    // the squares about the mean of the lanes' own columns, in registers; the
    // lanes' means about the row's when the warps are joined
    float lanes = sum2(add2(add2(v[0], v[1]), add2(v[2], v[3])));
    lanes = sum.lanes(lanes);
    const f32x2 m = both(-lanes * sum.inv_columns);
    f32x2 q = 0;
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
    const float2 both_sums = sum.join_squares(lanes, sum.lanes(sum2(q)), a.inv_dim);
    return {both_sums.x * a.inv_dim, rsqrtf(fmaf(both_sums.y, a.inv_dim, a.eps))};
}

// NORMS: 0 neither subtracts a mean nor has a bias, 1 they may but for a bias of
// the post norm, 2 they may.  ANY: whatever a call may ask for; without it y and u
// are there, gates are columns', and one stride reaches every row.  CLUSTER: blocks
// may share rows.
template <typename R, typename Y, bool ALIGNED, int NORMS, bool ANY, bool CLUSTER>
__global__ void __launch_bounds__(kFwdThreads, 1)
    residual_norm_fwd_kernel(const __grid_constant__ ResidualNormArgs a)
{
    using SR = Staged<R, ALIGNED, ANY>;
    using SY = Staged<Y, ALIGNED, ANY>;
    constexpr int kStages = fwd_stages<R, Y, ALIGNED, ANY>();
    constexpr bool LAYER = NORMS > 0, BIAS1 = NORMS == 2;
    extern __shared__ uint4 ring[];
    __shared__ TeamSlots slots;
    const int cluster = CLUSTER ? a.plan.cluster : 1;
    const BlockRows rows(a, cluster);
    const Cols<ALIGNED> c(a, cluster, rows.shift);
    TeamSum<CLUSTER> sum(slots, a);
    if (LAYER) sum.count_columns(c.upto - c.from);
    const int team = a.plan.teams > 1 ? int(threadIdx.x) / a.plan.tpr : 0;
    const int step = rows.step * a.plan.teams;  // rows from one of the team's to its next
    const int pitch = a.plan.threads * 16;
    const bool has_y = !ANY || a.y.p, has_gates = ANY && a.gate_rows.p, has_u = !ANY || a.u;
    const int stage_bytes = fwd_units<R, Y, ALIGNED, ANY>() * pitch;
    const unsigned mine = smem_u32(ring) + threadIdx.x * 16, over = mine + kStages * stage_bytes;

    int r = rows.first + team * rows.step, left = rows.count - team;  // the team's row; none if <= 0
    const int shift_x = SR::shift_of(a.x, a.tokens, rows.first, -rows.shift),
              shift_y = SY::shift_of(a.y, a.tokens, rows.first, -rows.shift),
              shift_g = SY::shift_of(a.gate_rows, a.tokens, rows.first, -rows.shift);
    int ahead = r, ahead_left = left;
    unsigned to = mine;
    constexpr bool kShared = sizeof(R) == 4 || sizeof(Y) == 4;  // lanes copy for one another
    const auto fetch = [&] {
        if (kShared) __syncwarp();  // the stage has been read by all lanes
        if (ahead_left > 0) {
            SR::fetch(a.x, row_at<R, ANY>(a.x, a.tokens, ahead, c.first), c, to, pitch);
            if (has_y)
                SY::fetch(a.y, row_at<Y, ANY>(a.y, a.tokens, ahead, c.first), c,
                          to + SR::kUnits * pitch, pitch);
            if (has_gates)
                SY::fetch(a.gate_rows, row_at<Y, ANY>(a.gate_rows, a.tokens, ahead, c.first), c,
                          to + (SR::kUnits + SY::kUnits) * pitch, pitch);
        }
        staged_commit();
        ahead += step;
        ahead_left -= a.plan.teams;
        to += stage_bytes;
        if (to == over) to = mine;
    };
    for (int i = 0; i < kStages - 1; ++i) fetch();

    // post and gate of a column in one factor and one summand; a gate of its
    // own per row stays apart
    f32x2 w1[4], b1[4], w2[4], b2[4];
    {
        const RawParam rg = fetch_param(a.gate, rows.group, c), r1 = fetch_param(a.w1, rows.group, c),
                       r2 = fetch_param(a.w2, rows.group, c);
        RawParam rb1, rb2;
        if (BIAS1) rb1 = fetch_param(a.b1, rows.group, c);
        if (LAYER) rb2 = fetch_param(a.b2, rows.group, c);
        f32x2 g[4];
        param_values(a.gate, rg, c, 0.0f, 1.0f, g);
        param_values(a.w1, r1, c, a.offset, 1.0f, w1);
        param_values(a.w2, r2, c, a.offset, 1.0f, w2);
        if (BIAS1) param_values(a.b1, rb1, c, 0.0f, 0.0f, b1);
        if (LAYER) param_values(a.b2, rb2, c, 0.0f, 0.0f, b2);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w1[e] = mul2(w1[e], g[e]);
            if (BIAS1) b1[e] = mul2(b1[e], g[e]);
        }
    }
    const f32x2 scale = both(a.scale);
    unsigned at = mine;
    // every team of the block takes part in every sum, with a row or without
    for (int i = 0; i < rows.count; i += a.plan.teams) {
        const bool active = left > 0;
        fetch();
        staged_wait<kStages - 1>();
        if (kShared) __syncwarp();
        f32x2 x[4];
        SR::read(a.x, a.tokens, r, shift_x, c, active, at, pitch, x);
        RowStats s1 = {0.0f, 1.0f}, s2 = {0.0f, 1.0f};
        if (has_y) {
            f32x2 y[4];
            SY::read(a.y, a.tokens, r, shift_y, c, active, at + SR::kUnits * pitch, pitch, y);
            s1 = row_stats<LAYER>(y, c, a.post, a, sum);
            const f32x2 v = both(s1.rstd), m = both(-s1.mean * s1.rstd);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                y[e] = LAYER ? fma2(y[e], v, m) : mul2(y[e], v);
                y[e] = BIAS1 ? fma2(y[e], w1[e], b1[e]) : mul2(y[e], w1[e]);
            }
            if (has_gates) {
                f32x2 g[4];
                SY::read(a.gate_rows, a.tokens, r, shift_g, c, active, at + (SR::kUnits + SY::kUnits) * pitch,
                         pitch, g);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = mul2(y[e], g[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = fma2(scale, x[e], y[e]);
            store_cols(static_cast<R *>(a.x_out) + ((long long)r * a.dim + c.first), c, active, x);
        }
        if (has_u) {
            s2 = row_stats<LAYER>(x, c, a.pre, a, sum);
            const f32x2 v = both(s2.rstd), m = both(-s2.mean * s2.rstd);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[e] = LAYER ? fma2(fma2(x[e], v, m), w2[e], b2[e]) : mul2(mul2(x[e], v), w2[e]);
            store_cols(static_cast<Y *>(a.u) + ((long long)r * a.dim + c.first), c, active, x);
        }
        if (a.stats && active && c.first <= 0 && c.any())
            a.stats[r] = make_float4(s1.mean, s1.rstd, s2.mean, s2.rstd);
        r += step;
        left -= a.plan.teams;
        at += stage_bytes;
        if (at == over) at = mine;
    }
    sum.finish();
}

template <typename R, typename Y, bool ALIGNED, int NORMS, bool ANY, bool CLUSTER>
cudaError_t launch(const ResidualNormArgs &a, cudaStream_t s)
{
    static std::atomic<unsigned long long> asked{0};
    return launch_staged(residual_norm_fwd_kernel<R, Y, ALIGNED, NORMS, ANY, CLUSTER>, asked, a,
                         fwd_units<R, Y, ALIGNED, ANY>(), fwd_stages<R, Y, ALIGNED, ANY>(), s);
}

// A kernel that can do everything has to ask, row for row, what it is to do: the
// usual calls have kernels of their own.
template <typename R, typename Y, bool ALIGNED>
cudaError_t launch(const ResidualNormArgs &a, cudaStream_t s)
{
    const int norms = a.b1.p                                                                 ? 2
                      : a.post == GBSSIM_ROW_LAYER || a.pre == GBSSIM_ROW_LAYER || a.b2.p ? 1
                                                                                            : 0;
    if (!a.y.p || !a.u || a.gate_rows.p || a.tokens != 0 || a.plan.uneven)
        return launch<R, Y, ALIGNED, 2, true, true>(a, s);
    if (a.plan.cluster > 1)
        return norms > 0 ? launch<R, Y, ALIGNED, 2, false, true>(a, s)
                         : launch<R, Y, ALIGNED, 0, false, true>(a, s);
    return norms == 2   ? launch<R, Y, ALIGNED, 2, false, false>(a, s)
           : norms == 1 ? launch<R, Y, ALIGNED, 1, false, false>(a, s)
                        : launch<R, Y, ALIGNED, 0, false, false>(a, s);
}

template <typename R, typename Y>
cudaError_t launch(const ResidualNormArgs &a, cudaStream_t s)
{
    return a.plan.aligned ? launch<R, Y, true>(a, s) : launch<R, Y, false>(a, s);
}

}  // namespace

cudaError_t residual_norm_cluster_room(ClusterRoom *room)
{
    const auto kernel = residual_norm_fwd_kernel<float, float, true, 2, true, true>;
    constexpr int kAlone = 120 * 1024;  // shared memory that leaves an SM room for one block
    cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kStagedBlock);
    for (int size = 2; size <= 4 && e == cudaSuccess; size *= 2) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(unsigned(size));
        cfg.blockDim = dim3(512);
        cfg.dynamicSmemBytes = kAlone;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = unsigned(size);
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(size == 2 ? &room->of2 : &room->of4, kernel, &cfg);
    }
    return e;
}

cudaError_t residual_norm_fwd_status(unsigned *flags, bool clear) { return exchange_status(flags, clear); }

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
