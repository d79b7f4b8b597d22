// Shared parts of the residual-norm kernels: the norms before and after a
// residual block with its gate and residual scale, forward and backward.
//
//   y^ = (y - m1) r1,  z = y^ (w1 + o) + b1,  x' = s x + g z,
//   x^ = (x' - m2) r2, u = x^ (w2 + o) + b2,
// per row of D columns; m, r the row's mean (zero for the root-mean-square
// norm) and 1 / sqrt(mean((. - m)^2) + eps).
#pragma once

#include <algorithm>

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
    const void *end;   // past the last row's last element
    int row_bytes;     // from one row to the next, where one stride reaches all rows
};

struct ParamPtr {
    const void *p;
    int type, per_sample;
    long long stride;  // elements between samples; 0: one for all
};

// How rows and columns fall onto blocks.  A group is group_rows consecutive rows:
// those that share the per-sample parameters, or all rows.  Dense rows of D
// columns start D mod 8 elements further past a 16-byte boundary (of eight
// elements) from one to the next; a block takes only rows of one such class
// (row number mod `classes`), whose columns its threads cut alike, so that eight
// columns of a thread are whole aligned words in every row.  `splits` blocks (or
// clusters) share a class of a group.
struct RowPlan {
    int aligned;       // rows start on 16-byte boundaries in every tensor
    int classes;       // 8 / gcd(8, D); 1 also where a group has too few rows to part
    int stages;        // rows of each thread in flight
    int cluster;       // blocks of a cluster (1, 2, 4)
    int block_cols;    // columns of a block: a multiple of 8 (counted from the shift)
    int tpr;           // threads of a team in a block
    int teams;         // teams of a block
    int groups, group_rows, splits;
    int threads;
    unsigned grid;     // groups * classes * splits * cluster
};

struct ResidualNormArgs {
    RowPtr x, y, gate_rows;
    ParamPtr gate, w1, b1, w2, b2;
    int tokens, dim;   // tokens: 0 where one stride reaches every row of every tensor
    int post, pre;     // gbssim_row_norm
    float scale, offset, eps, inv_dim;
    RowPlan plan;
    // forward
    void *x_out, *u;
    float4 *stats;     // (m1, r1, m2, r2) of each row
    // backward
    RowPtr gx, gu;
    void *dx, *dy, *dgate_rows;
    float *partials;   // [groups * classes * splits][sums][dim]
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

// The rows of this block (or cluster): first + i * step, i < count, of one class
// of group `group`.
struct BlockRows {
    int group, first, count, step;
    int shift;  // columns that the class's rows start past a multiple of eight elements
    __device__ __forceinline__ BlockRows(const ResidualNormArgs &a)
    {
        const RowPlan &p = a.plan;
        const int item = int(blockIdx.x) / p.cluster;
        const int cls = item / p.splits, split = item - cls * p.splits;
        group = cls / p.classes;
        const int k = cls - group * p.classes;
        const int begin = group * p.group_rows;
        const int skip = (k - begin) & (p.classes - 1);
        const long long n = skip < p.group_rows ? (p.group_rows - skip + p.classes - 1) / p.classes : 0;
        const int i0 = int(split * n / p.splits);
        count = int((split + 1) * n / p.splits) - i0;
        step = p.classes;
        first = begin + skip + i0 * step;
        shift = p.classes > 1 ? (k * (a.dim & 7)) & 7 : 0;
    }
};

// The eight neighbouring columns of this thread; first may be negative, and the
// row has those from `from` up to `upto`.  ALIGNED: all eight or none.
template <bool ALIGNED>
struct Cols {
    int first, from, upto;
    int t;  // place in the team
    __device__ __forceinline__ Cols(const ResidualNormArgs &a, int shift)
    {
        const int rank = a.plan.cluster > 1 ? int(blockIdx.x) % a.plan.cluster : 0;
        t = a.plan.teams > 1 ? threadIdx.x & (a.plan.tpr - 1) : threadIdx.x;
        first = rank * a.plan.block_cols + t * kColsPerThread - (ALIGNED ? 0 : shift);
        from = max(0, -first);
        upto = t * kColsPerThread < a.plan.block_cols ? max(0, min(kColsPerThread, a.dim - first)) : 0;
    }
    __device__ __forceinline__ bool any() const { return from < upto; }
    __device__ __forceinline__ bool all() const { return ALIGNED ? upto > 0 : upto - from == 8; }
    __device__ __forceinline__ bool has(int e) const
    {
        return ALIGNED ? upto > 0 : e >= from && e < upto;
    }
};

// Column `col` of row r of a tensor.
template <typename T>
__device__ __forceinline__ const unsigned char *row_at(const RowPtr &p, int tokens, int r, int col)
{
    const unsigned char *base = static_cast<const unsigned char *>(p.p) + col * int(sizeof(T));
    if (tokens == 0) return base + (long long)r * p.row_bytes;
    const int b = r / tokens, t = r - b * tokens;
    return base + (b * p.sb + t * p.st) * int(sizeof(T));
}

// Rows on their way through shared memory: every thread copies its own columns
// of a row some rows ahead (cp.async) and reads them back itself, so the copies
// need no barrier.  A stage holds, per tensor, 16-byte words [word][thread].
//
// Where a tensor's rows are not aligned as the block's columns are, a thread
// copies the aligned words that its columns lie in -- one more than they fill --
// and shifts.  A word that reaches over the tensor's first or last element is
// put together from single elements.
template <typename T, bool ALIGNED>
struct Staged {
    static constexpr int kUnits = (sizeof(T) == 4 ? 2 : 1) + (ALIGNED ? 0 : 1);

    // at: the thread's first column; slot: its first word, `pitch` bytes from word to word.
    static __device__ __forceinline__ void fetch(const RowPtr &p, const unsigned char *at,
                                                 const Cols<ALIGNED> &c, unsigned slot, int pitch)
    {
        if constexpr (ALIGNED) {
#pragma unroll
            for (int u = 0; u < kUnits; ++u) copy16_async<false>(slot + u * pitch, at + u * 16);
        } else {
            const unsigned char *from = at + c.from * int(sizeof(T));
            const unsigned char *stop = at + c.upto * int(sizeof(T));
            const unsigned char *word = at - (reinterpret_cast<uintptr_t>(at) & 15);
#pragma unroll
            for (int u = 0; u < kUnits; ++u, word += 16, slot += pitch) {
                if (word >= stop || word + 16 <= from) continue;
                if (word >= p.p && word + 16 <= p.end) {
                    copy16_async<true>(slot, word);
                } else {
                    T *to = static_cast<T *>(__cvta_shared_to_generic(slot));
#pragma unroll 1
                    for (int i = 0; i < 16; i += int(sizeof(T)))
                        if (word + i >= from && word + i < stop)
                            to[i / int(sizeof(T))] = *reinterpret_cast<const T *>(word + i);
                }
            }
        }
    }

    // The thread's columns of a row, zero where the row has none.
    static __device__ __forceinline__ void read(const RowPtr &p, int tokens, int row,
                                                const Cols<ALIGNED> &c, bool active, unsigned slot,
                                                int pitch, f32x2 (&v)[4])
    {
        Raw8<T> r{};
        if constexpr (ALIGNED) {
            if (active && c.any()) {
#pragma unroll
                for (int u = 0; u < kUnits; ++u) r.w[u] = ld_shared16(slot + u * pitch);
            }
            unpack8<T>(r, v);
        } else {
            if (active && c.any()) {
                const int s = int(reinterpret_cast<uintptr_t>(row_at<T>(p, tokens, row, c.first)) & 15) /
                              int(sizeof(T));
                if (s == 0) {
#pragma unroll
                    for (int u = 0; u < kUnits - 1; ++u) r.w[u] = ld_shared16(slot + u * pitch);
                } else {
                    Wide8<T> w;
#pragma unroll
                    for (int u = 0; u < kUnits; ++u) {
                        const uint4 q = ld_shared16(slot + u * pitch);
                        w.w[4 * u] = q.x; w.w[4 * u + 1] = q.y;
                        w.w[4 * u + 2] = q.z; w.w[4 * u + 3] = q.w;
                    }
                    r = shift_down<T>(w, s);
                }
            }
            float f[8];
            unpack8<T>(r, f);
            if (!c.all()) {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = c.has(e) ? f[e] : 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = pair(f[2 * e], f[2 * e + 1]);
        }
    }
};

__device__ __forceinline__ void staged_commit()
{
    asm volatile("cp.async.commit_group;" ::: "memory");
}

// Waits until at most stages - 1 of this thread's latest groups are in flight.
__device__ __forceinline__ void staged_wait(int stages)
{
    if (stages >= 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
    else if (stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
    else if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Stores the thread's columns of a row, the first at `to`: in whole words where
// it has all eight and they are aligned, one by one at a row's ends.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void store_cols(T *to, const Cols<ALIGNED> &c, bool active,
                                           const f32x2 (&v)[4])
{
    if constexpr (ALIGNED) {
        if (active && c.any()) st8(to, pack8<T>(v));
    } else {
        if (!active) return;
        if (c.all() && (reinterpret_cast<uintptr_t>(to) & 15) == 0) {
            st8(to, pack8<T>(v));
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 h = halves(v[e / 2]);
                if (c.has(e)) to[e] = from_f32<T>(e & 1 ? h.y : h.x);
            }
        }
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
                                           float offset, float missing, f32x2 (&v)[4])
{
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        f[e] = !p.p ? missing : (c.has(e) ? param_at(p, group, c.first + e) + offset : 0.0f);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = pair(f[2 * e], f[2 * e + 1]);
}

// Sums over a team, of one value or of two.  All threads of a block call together.
struct TeamSum {
    float2 (*slots)[16];         // [2][warp]
    float2 (*cluster_slots)[4];  // [2][block of the cluster]
    int parity, tpr, warps, cluster;

    template <int N>
    __device__ __forceinline__ void operator()(float (&v)[N])
    {
        if (tpr < 32) {
#pragma unroll 1
            for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
                for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
            return;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        if (warps == 1) return;
        // one barrier a sum: the slots alternate, and a thread that writes a
        // slot again has passed the barrier of the sum in between, which every
        // thread reaches only after it has read this one
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        float2 *const mine = slots[parity];
        if (lane == 0) {
            mine[warp].x = v[0];
            if (N == 2) mine[warp].y = v[N - 1];
        }
        __syncthreads();
        float2 got = make_float2(0.0f, 0.0f);
        if ((lane & 15) < warps) got = mine[lane & 15];
        v[0] = got.x;
        if (N == 2) v[N - 1] = got.y;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        if (cluster > 1) {
            namespace cg = cooperative_groups;
            cg::cluster_group cl = cg::this_cluster();
            if (int(threadIdx.x) < cluster)
                cl.map_shared_rank(&cluster_slots[parity][0], threadIdx.x)[cl.block_rank()] =
                    make_float2(v[0], v[N - 1]);
            cl.sync();
            v[0] = v[N - 1] = 0.0f;
            for (int r = 0; r < cluster; ++r) {
                const float2 c = cluster_slots[parity][r];
                v[0] += c.x;
                if (N == 2) v[N - 1] += c.y;
            }
        }
        parity ^= 1;
    }

    __device__ __forceinline__ float one(float v)
    {
        float a[1] = {v};
        (*this)(a);
        return a[0];
    }
};

// Launches a kernel with its ring of staged rows: as many stages as leave
// `per_sm` blocks of the largest team (or as many threads of smaller ones) room
// on an SM, one at least.
template <class Kernel>
cudaError_t launch_staged(Kernel kernel, ResidualNormArgs &a, int units, int per_sm, cudaStream_t s)
{
    constexpr int kSmemPerSm = 200 * 1024, kMaxStages = 4, kMaxBlockSmem = 220 * 1024;
    const int stage = units * 16 * a.plan.threads;
    const int blocks = per_sm * kMaxTeamThreads / a.plan.threads;
    a.plan.stages = std::max(1, std::min(kMaxStages, kSmemPerSm / (stage * blocks)));
    const int smem = a.plan.stages * stage;
    if (smem > 40 * 1024) {  // with the static arrays: above what needs no asking for
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kMaxBlockSmem);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.plan.grid);
    cfg.blockDim = dim3(unsigned(a.plan.threads));
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(a.plan.cluster);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.plan.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

#endif

}  // namespace gbssim
