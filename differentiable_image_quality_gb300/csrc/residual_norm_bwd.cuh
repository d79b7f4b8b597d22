// Backward of the residual norm.  With G = dL/dx', V = dL/du:
//   dx^ = V (w2 + o),  T = G + r2 (dx^ - mean(dx^) - x^ mean(dx^ x^)),   dx = s T,
//   q = T g,  dy^ = q (w1 + o),  dy = r1 (dy^ - mean(dy^) - y^ mean(dy^ y^)),
// (no mean(.) terms for the root-mean-square norm, dy = q without a post norm),
// and over the rows that share a parameter
//   dw2 = sum V x^,  db2 = sum V,  dw1 = sum q y^,  db1 = sum q,
//   dg = sum T (y^ (w1 + o) + b1).
// A gate that is shared by rows factors out of the sums: with A = sum T y^ and
// F = sum T, dg = (w1 + o) A + b1 F, dw1 = g A, db1 = g F -- two column sums
// serve three gradients.  A gate of its own per row has its gradient written
// row by row, and A = sum q y^, F = sum q.
//
// Bound by memory where rows are wide: x, y, G and V are read once, dx and dy
// written once.  x^ and y^ are formed again from x, y and the saved statistics,
// not stored.  Column sums stay in registers over a block's rows (float32), go
// to a partial per block, and a second kernel adds the partials in a fixed
// order.  32400 x 4096 bfloat16 with a gate per row: 385 us for 2.1 GB (81 % of
// the copy rate); 71050 x 964 bfloat16 199 us (61 %), 32400 x 1001 float16 133 us
// (42 %): instruction issue, and with 96 to 128 registers a thread only 16 to 20
// warps to cover a row's two sums.
#pragma once

#include "residual_norm.cuh"

namespace gbssim {
namespace {

// 16-byte words a thread stages of a row: x, G, y, V and a gate per row.
template <typename R, typename Y, bool ALIGNED, bool FULL>
constexpr int bwd_units()
{
    return 2 * Staged<R, ALIGNED, true>::kUnits + (FULL ? 3 : 2) * Staged<Y, ALIGNED, true>::kUnits;
}

template <typename R, typename Y, bool ALIGNED, bool FULL>
constexpr int bwd_stages()
{
    return stages_of(bwd_units<R, Y, ALIGNED, FULL>(), 1);
}

// One column sum of the block to its partial: over the block's teams first.
template <bool ALIGNED>
__device__ __forceinline__ void write_sum(const ResidualNormArgs &a, const Cols<ALIGNED> &c,
                                          int place, const f32x2 (&sums)[4], float *scratch)
{
    if (place < 0) return;
    float v[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 h = halves(sums[e]);
        v[2 * e] = h.x;
        v[2 * e + 1] = h.y;
    }
    const int item = int(blockIdx.x) / a.plan.cluster;
    float *dst = a.partials + ((long long)item * a.sums + place) * a.dim;
    if (a.plan.teams > 1) {
        // teams of a warp by shuffles, then the warps through shared memory
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tpr = a.plan.tpr;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            for (int o = tpr; o < 32; o <<= 1) v[e] += __shfl_xor_sync(0xffffffffu, v[e], o);
            if (lane < tpr) scratch[(warp * 32 + lane) * 8 + e] = v[e];
        }
        __syncthreads();
        if (int(threadIdx.x) < tpr) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float s = 0.0f;
                for (int w = 0; w < kSmallBlock / 32; ++w) s += scratch[(w * 32 + lane) * 8 + e];
                if (c.has(e)) dst[c.first + e] = s;
            }
        }
        __syncthreads();
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (c.has(e)) dst[c.first + e] = v[e];
}

// FULL: a gate of its own per row.  NORMS: 0 neither subtracts a mean nor has a
// bias, 1 they may but for a bias of the post norm, 2 they may.  ANY: whatever a call
// may ask for; without it all four inputs and both outputs are there and one stride
// reaches every row.  CLUSTER: blocks may share rows.
template <typename R, typename Y, bool ALIGNED, bool FULL, int NORMS, bool ANY, bool CLUSTER>
__global__ void __launch_bounds__(NORMS == 0 && !FULL && !CLUSTER ? kBwdResidentPlain : kBwdThreads, 1)
    residual_norm_bwd_kernel(const __grid_constant__ ResidualNormArgs a)
{
    using SR = Staged<R, ALIGNED, ANY>;
    using SY = Staged<Y, ALIGNED, ANY>;
    constexpr int kStages = bwd_stages<R, Y, ALIGNED, FULL>();
    constexpr bool LAYER = NORMS > 0, BIAS1 = NORMS == 2;
    extern __shared__ uint4 ring[];
    __shared__ TeamSlots slots;
    __shared__ float scratch[kSmallBlock * 8];
    if (a.sums) pdl_trigger();  // the kernel that adds the partials waits for all of this one
    const int cluster = CLUSTER ? a.plan.cluster : 1;
    const BlockRows rows(a, cluster);
    const Cols<ALIGNED> c(a, cluster, rows.shift);
    TeamSum<CLUSTER> sum(slots, a);
    const int team = a.plan.teams > 1 ? int(threadIdx.x) / a.plan.tpr : 0;
    const int step = rows.step * a.plan.teams;  // rows from one of the team's to its next
    const int pitch = a.plan.threads * 16;
    const bool has_y = !ANY || a.y.p, has_gx = !ANY || a.gx.p, has_gu = !ANY || a.gu.p;
    const bool wants_x = !ANY || a.dx, wants_y = !ANY || a.dy, wants_g = FULL && a.dgate_rows;
    // the words of a stage: x, G, y, V, gate
    const int at_gx = SR::kUnits * pitch, at_y = 2 * at_gx, at_gu = at_y + SY::kUnits * pitch,
              at_gate = at_gu + SY::kUnits * pitch;
    const int stage_bytes = bwd_units<R, Y, ALIGNED, FULL>() * pitch;
    const unsigned mine = smem_u32(ring) + threadIdx.x * 16, over = mine + kStages * stage_bytes;

    int r = rows.first + team * rows.step, left = rows.count - team;  // the team's row; none if <= 0
    const int shift_x = SR::shift_of(a.x, a.tokens, rows.first, -rows.shift),
              shift_y = SY::shift_of(a.y, a.tokens, rows.first, -rows.shift),
              shift_gx = SR::shift_of(a.gx, a.tokens, rows.first, -rows.shift),
              shift_gu = SY::shift_of(a.gu, a.tokens, rows.first, -rows.shift),
              shift_g = SY::shift_of(a.gate_rows, a.tokens, rows.first, -rows.shift);
    int ahead = r, ahead_left = left;
    unsigned to = mine;
    constexpr bool kShared = sizeof(R) == 4 || sizeof(Y) == 4;  // lanes copy for one another
    const auto fetch = [&] {
        if (kShared) __syncwarp();  // the stage has been read by all lanes
        if (ahead_left > 0) {
            SR::fetch(a.x, row_at<R, ANY>(a.x, a.tokens, ahead, c.first), c, to, pitch);
            if (has_gx)
                SR::fetch(a.gx, row_at<R, ANY>(a.gx, a.tokens, ahead, c.first), c, to + at_gx, pitch);
            if (has_y)
                SY::fetch(a.y, row_at<Y, ANY>(a.y, a.tokens, ahead, c.first), c, to + at_y, pitch);
            if (has_gu)
                SY::fetch(a.gu, row_at<Y, ANY>(a.gu, a.tokens, ahead, c.first), c, to + at_gu, pitch);
            if (FULL)
                SY::fetch(a.gate_rows, row_at<Y, ANY>(a.gate_rows, a.tokens, ahead, c.first), c,
                          to + at_gate, pitch);
        }
        staged_commit();
        ahead += step;
        ahead_left -= a.plan.teams;
        to += stage_bytes;
        if (to == over) to = mine;
    };
    for (int i = 0; i < kStages - 1; ++i) fetch();

    f32x2 w1[4], b1[4], w2[4];  // with the gate of the column in w1 and b1, unless FULL
    {
        const RawParam r1 = fetch_param(a.w1, rows.group, c), r2 = fetch_param(a.w2, rows.group, c);
        RawParam rg, rb1;
        if (!FULL) rg = fetch_param(a.gate, rows.group, c);
        if (BIAS1) rb1 = fetch_param(a.b1, rows.group, c);
        param_values(a.w1, r1, c, a.offset, 1.0f, w1);
        param_values(a.w2, r2, c, a.offset, 1.0f, w2);
        if (BIAS1) param_values(a.b1, rb1, c, 0.0f, 0.0f, b1);
        if (!FULL) {
            f32x2 g[4];
            param_values(a.gate, rg, c, 0.0f, 1.0f, g);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w1[e] = mul2(w1[e], g[e]);
                if (BIAS1) b1[e] = mul2(b1[e], g[e]);
            }
        }
    }
    const f32x2 scale = both(a.scale);
    unsigned at = mine;
    // Columns that a row does not have hold zeros of x, y, G, V and of w1 and b1:
    // whatever a mean makes of y^, x^ and T there meets a zero factor before it
    // enters a sum over the row, and their own sums are not stored.
    f32x2 sa[4] = {}, sf[4] = {}, sc[4] = {}, se[4] = {};
    // the statistics of the row after this one (neutral ones where there is none)
    float4 st_next = left > 0 ? a.stats[r] : make_float4(0.0f, 1.0f, 0.0f, 1.0f);
    for (int i = 0; i < rows.count; i += a.plan.teams) {
        const bool active = left > 0;
        const float4 st = st_next;
        st_next = left > a.plan.teams ? a.stats[r + step] : make_float4(0.0f, 1.0f, 0.0f, 1.0f);
        fetch();
        staged_wait<kStages - 1>();
        if (kShared) __syncwarp();

        f32x2 yh[4], xh[4], T[4], g[4];
        SR::read(a.x, a.tokens, r, shift_x, c, active, at, pitch, xh);
        if (has_y) {
            SY::read(a.y, a.tokens, r, shift_y, c, active, at + at_y, pitch, yh);
            if (FULL) SY::read(a.gate_rows, a.tokens, r, shift_g, c, active, at + at_gate, pitch, g);
            const f32x2 v = both(st.y), m = both(-st.x * st.y);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                yh[e] = LAYER ? fma2(yh[e], v, m) : mul2(yh[e], v);
                f32x2 z = BIAS1 ? fma2(yh[e], w1[e], b1[e]) : mul2(yh[e], w1[e]);
                if (FULL) z = mul2(z, g[e]);
                xh[e] = fma2(scale, xh[e], z);
            }
        }
        if (has_gx) {
            SR::read(a.gx, a.tokens, r, shift_gx, c, active, at + at_gx, pitch, T);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) T[e] = 0;
        }
        if (has_gu) {
            f32x2 V[4], q = 0;
            SY::read(a.gu, a.tokens, r, shift_gu, c, active, at + at_gu, pitch, V);
            const f32x2 v = both(st.w), m = both(-st.z * st.w);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                xh[e] = LAYER ? fma2(xh[e], v, m) : mul2(xh[e], v);
                sc[e] = fma2(V[e], xh[e], sc[e]);
                if (LAYER) se[e] = add2(se[e], V[e]);
                V[e] = mul2(V[e], w2[e]);
                q = fma2(V[e], xh[e], q);
            }
            float d[2] = {sum2(q), 0.0f};
            if (LAYER && a.pre == GBSSIM_ROW_LAYER) {
                d[1] = sum2(add2(add2(V[0], V[1]), add2(V[2], V[3])));
                sum(d);
            } else {
                d[0] = a.pre == GBSSIM_ROW_RMS ? sum.one(d[0]) : 0.0f;
            }
            // T += r2 (dx^ - mean(dx^) - x^ mean(dx^ x^))
            const f32x2 d0 = both(-d[0] * a.inv_dim), d1 = both(-d[1] * a.inv_dim);
#pragma unroll
            for (int e = 0; e < 4; ++e) T[e] = fma2(v, fma2(xh[e], d0, LAYER ? add2(V[e], d1) : V[e]), T[e]);
        }
        if (wants_x) {
            f32x2 dx[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) dx[e] = has_y ? mul2(scale, T[e]) : T[e];
            store_cols(static_cast<R *>(a.dx) + ((long long)r * a.dim + c.first), c, active, dx);
        }
        if (has_y) {
            if (wants_g) {
                f32x2 dg[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    dg[e] = mul2(T[e], BIAS1 ? fma2(yh[e], w1[e], b1[e]) : mul2(yh[e], w1[e]));
                store_cols(static_cast<Y *>(a.dgate_rows) + ((long long)r * a.dim + c.first), c, active, dg);
            }
            f32x2 q = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (FULL) T[e] = mul2(T[e], g[e]);
                sa[e] = fma2(T[e], yh[e], sa[e]);
                if (BIAS1) sf[e] = add2(sf[e], T[e]);
                T[e] = mul2(T[e], w1[e]);
                q = fma2(T[e], yh[e], q);
            }
            if (wants_y) {
                float d[2] = {sum2(q), 0.0f};
                if (LAYER && a.post == GBSSIM_ROW_LAYER) {
                    d[1] = sum2(add2(add2(T[0], T[1]), add2(T[2], T[3])));
                    sum(d);
                } else {
                    d[0] = a.post == GBSSIM_ROW_RMS ? sum.one(d[0]) : 0.0f;
                }
                const f32x2 v = both(st.y), d0 = both(-d[0] * a.inv_dim), d1 = both(-d[1] * a.inv_dim);
#pragma unroll
                for (int e = 0; e < 4; ++e) T[e] = mul2(v, fma2(yh[e], d0, LAYER ? add2(T[e], d1) : T[e]));
                store_cols(static_cast<Y *>(a.dy) + ((long long)r * a.dim + c.first), c, active, T);
            }
        }
        r += step;
        left -= a.plan.teams;
        at += stage_bytes;
        if (at == over) at = mine;
    }
    sum.finish();
    write_sum(a, c, a.sum_a, sa, scratch);
    write_sum(a, c, a.sum_c, sc, scratch);
    if (BIAS1) write_sum(a, c, a.sum_f, sf, scratch);
    if (LAYER) write_sum(a, c, a.sum_e, se, scratch);
}

template <typename R, typename Y, bool ALIGNED, bool FULL, int NORMS, bool ANY, bool CLUSTER>
cudaError_t launch(const ResidualNormArgs &a, cudaStream_t s)
{
    static std::atomic<unsigned long long> asked{0};
    return launch_staged(residual_norm_bwd_kernel<R, Y, ALIGNED, FULL, NORMS, ANY, CLUSTER>, asked, a,
                         bwd_units<R, Y, ALIGNED, FULL>(), bwd_stages<R, Y, ALIGNED, FULL>(), s);
}

// A kernel that can do everything has to ask, row for row, what it is to do: the
// usual calls have kernels of their own.
template <typename R, typename Y, bool ALIGNED>
cudaError_t launch(const ResidualNormArgs &a, cudaStream_t s)
{
    const bool any = residual_norm_bwd_any(a), cluster = a.plan.cluster > 1;
    const int norms = residual_norm_bwd_norms(a);
    if (a.gate_rows.p)
        return any || cluster ? launch<R, Y, ALIGNED, true, 2, true, true>(a, s)
               : norms > 0    ? launch<R, Y, ALIGNED, true, 2, false, false>(a, s)
                              : launch<R, Y, ALIGNED, true, 0, false, false>(a, s);
    if (any) return launch<R, Y, ALIGNED, false, 2, true, true>(a, s);
    if (cluster)
        return norms > 0 ? launch<R, Y, ALIGNED, false, 2, false, true>(a, s)
                         : launch<R, Y, ALIGNED, false, 0, false, true>(a, s);
    return norms == 2   ? launch<R, Y, ALIGNED, false, 2, false, false>(a, s)
           : norms == 1 ? launch<R, Y, ALIGNED, false, 1, false, false>(a, s)
                        : launch<R, Y, ALIGNED, false, 0, false, false>(a, s);
}

template <typename R, typename Y>
cudaError_t launch(const ResidualNormArgs &a, cudaStream_t s)
{
    return a.plan.aligned ? launch<R, Y, true>(a, s) : launch<R, Y, false>(a, s);
}

}  // namespace
}  // namespace gbssim
