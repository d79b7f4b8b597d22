// Shared parts of the residual-norm kernels: the norms before and after a
// residual block with its gate and residual scale, forward and backward.
//
//   y^ = (y - m1) r1,  z = y^ (w1 + o) + b1,  x' = s x + g z,
//   x^ = (x' - m2) r2, u = x^ (w2 + o) + b2,
// per row of D columns; m, r the row's mean (zero for the root-mean-square
// norm) and 1 / sqrt(mean((. - m)^2) + eps).
#pragma once

#include <cooperative_groups.h>

#include "gbssim.h"
#include "dtypes.cuh"

namespace gbssim {

// Every thread owns eight columns of a row for the whole kernel, so that the
// parameters of its columns and their gradients' sums stay in registers.  A row
// belongs to a team: `tpr` lanes of a warp (a power of two) for rows of up to
// 256 columns, a block of up to 512 threads for up to 4096, a cluster of two or
// four such blocks above.
constexpr int kColsPerThread = 8;
constexpr int kMaxTeamThreads = 512;
constexpr int kSmallBlock = 128;  // threads of a block that holds several teams
constexpr int kMaxDim = 4 * kMaxTeamThreads * kColsPerThread;

struct RowPtr {
    const void *p;
    long long sb, st;  // elements between batches and between tokens
};

struct ParamPtr {
    const void *p;
    int type, per_sample;
    long long stride;  // elements between samples; 0: one for all
};

// How rows and columns fall onto blocks.  Blocks (or clusters) take groups one
// after another, `splits` of them to a group of group_rows consecutive rows: a
// group is the rows that share the per-sample parameters, or all rows.
struct RowPlan {
    int aligned;       // 16-byte accesses everywhere
    int cluster;       // blocks of a cluster (1, 2, 4)
    int block_cols;    // columns of a block: a multiple of 8
    int tpr;           // threads of a team in a block
    int teams;         // teams of a block
    int groups, group_rows, splits;
    int threads;
    unsigned grid;     // groups * splits * cluster
};

struct ResidualNormArgs {
    RowPtr x, y, gate_rows;
    ParamPtr gate, w1, b1, w2, b2;
    int tokens, dim;
    int post, pre;     // gbssim_row_norm
    float scale, offset, eps, inv_dim;
    RowPlan plan;
    // forward
    void *x_out, *u;
    float4 *stats;     // (m1, r1, m2, r2) of each row
    // backward
    RowPtr gx, gu;
    void *dx, *dy, *dgate_rows;
    float *partials;   // [groups * splits][sums][dim]
    int sum_a, sum_f, sum_c, sum_e, sums;  // places of the column sums, -1: not wanted
};

// Outputs of the parameters' gradients.
struct ParamGrad {
    void *p;
    int type, per_sample;
};
struct ParamGrads {
    ParamGrad gate, w1, b1, w2, b2;
};

cudaError_t residual_norm_fwd_launch(const ResidualNormArgs &a, int res, int blk, cudaStream_t s);
cudaError_t residual_norm_bwd_launch(const ResidualNormArgs &a, int res, int blk,
                                     const ParamGrads &g, cudaStream_t s);

#ifdef __CUDACC__

// The columns of this thread: eight neighbours where rows are aligned, eight
// that lie a team's width apart otherwise (neighbouring lanes then still read
// neighbouring elements).
template <bool ALIGNED>
struct Cols {
    int first, n;  // the block's columns
    int t, tpr;
    __device__ __forceinline__ Cols(const ResidualNormArgs &a)
    {
        const int rank = a.plan.cluster > 1 ? int(blockIdx.x) % a.plan.cluster : 0;
        first = rank * a.plan.block_cols;
        n = min(a.plan.block_cols, a.dim - first);
        tpr = a.plan.tpr;
        t = a.plan.teams > 1 ? threadIdx.x & (tpr - 1) : threadIdx.x;
    }
    __device__ __forceinline__ int col(int e) const
    {
        return first + (ALIGNED ? t * kColsPerThread + e : e * tpr + t);
    }
    __device__ __forceinline__ bool has(int e) const
    {
        return ALIGNED ? t * kColsPerThread < n : e * tpr + t < n;
    }
};

template <bool ALIGNED, typename T>
__device__ __forceinline__ void load_row(const T *row, const Cols<ALIGNED> &c, bool active,
                                         float (&v)[8])
{
    if constexpr (ALIGNED) {
        Raw8<T> r{};
        if (active && c.has(0)) r = ld8_stream(row + c.col(0));
        unpack8<T>(r, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = active && c.has(e) ? to_f32(row[c.col(e)]) : 0.0f;
    }
}

template <bool ALIGNED, typename T>
__device__ __forceinline__ void store_row(T *row, const Cols<ALIGNED> &c, bool active,
                                          const float (&v)[8])
{
    if constexpr (ALIGNED) {
        if (active && c.has(0)) st8(row + c.col(0), pack8<T>(v));
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (active && c.has(e)) row[c.col(e)] = from_f32<T>(v[e]);
    }
}

template <typename T>
__device__ __forceinline__ float load_param1(const void *p, long long i)
{
    return to_f32(static_cast<const T *>(p)[i]);
}

__device__ __forceinline__ float param_at(const ParamPtr &p, int group, int col)
{
    const long long i = group * p.stride + col;
    return p.type == GBSSIM_F32    ? load_param1<float>(p.p, i)
           : p.type == GBSSIM_BF16 ? load_param1<bf16>(p.p, i)
                                   : load_param1<f16>(p.p, i);
}

// The thread's eight values of a parameter plus `offset`; `missing` where it is null.
template <bool ALIGNED>
__device__ __forceinline__ void load_param(const ParamPtr &p, int group, const Cols<ALIGNED> &c,
                                           float offset, float missing,
                                           float (&v)[8])
{
#pragma unroll
    for (int e = 0; e < 8; ++e)
        v[e] = !p.p ? missing : (c.has(e) ? param_at(p, group, c.col(e)) + offset : 0.0f);
}

// Element offset of row r of a tensor.
__device__ __forceinline__ long long row_offset(const RowPtr &p, int b, int t)
{
    return b * p.sb + t * p.st;
}

// Sums over a team.  All teams of a block call together.
struct TeamSum {
    float2 (*slots)[16];         // [2][16]: one per warp
    float2 (*cluster_slots)[4];  // [2][4]: one per block of the cluster
    int parity, tpr, warps, cluster;

    __device__ __forceinline__ float2 operator()(float2 v)
    {
        if (tpr < 32) {
            for (int o = tpr >> 1; o > 0; o >>= 1) {
                v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
                v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
            }
            return v;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        }
        if (warps == 1) return v;
        // one barrier a sum: the slots alternate, and a thread that writes a
        // slot again has passed the barrier of the sum in between, which every
        // thread reaches only after it has read this one
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0) slots[parity][warp] = v;
        __syncthreads();
        v = (lane & 15) < warps ? slots[parity][lane & 15] : make_float2(0.0f, 0.0f);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        }
        if (cluster > 1) {
            namespace cg = cooperative_groups;
            cg::cluster_group cl = cg::this_cluster();
            if (int(threadIdx.x) < cluster)
                cl.map_shared_rank(&cluster_slots[parity][0], threadIdx.x)[cl.block_rank()] = v;
            cl.sync();
            v = make_float2(0.0f, 0.0f);
            for (int r = 0; r < cluster; ++r) {
                v.x += cluster_slots[parity][r].x;
                v.y += cluster_slots[parity][r].y;
            }
        }
        parity ^= 1;
        return v;
    }
};

// The rows of this block (or cluster): of group `group`, rows [r0, r1).
struct BlockRows {
    int group, r0, r1;
    __device__ __forceinline__ BlockRows(const RowPlan &p)
    {
        const int item = int(blockIdx.x) / p.cluster;
        group = item / p.splits;
        const long long s = item - group * p.splits;
        r0 = group * p.group_rows + int(s * p.group_rows / p.splits);
        r1 = group * p.group_rows + int((s + 1) * p.group_rows / p.splits);
    }
};

#endif

}  // namespace gbssim
