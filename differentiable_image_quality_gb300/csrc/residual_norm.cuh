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
    int aligned;       // every thread's columns lie on 16-byte boundaries in every row
    int stages;        // rows of each thread in flight
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

// The eight neighbouring columns of this thread.
template <bool ALIGNED>
struct Cols {
    int first;  // of the thread
    int count;  // how many of the eight the row has; all or none where ALIGNED
    int t;      // place in the team
    bool last;  // the thread whose right neighbour has no column of the row
    __device__ __forceinline__ Cols(const ResidualNormArgs &a)
    {
        const int rank = a.plan.cluster > 1 ? int(blockIdx.x) % a.plan.cluster : 0;
        t = a.plan.teams > 1 ? threadIdx.x & (a.plan.tpr - 1) : threadIdx.x;
        first = rank * a.plan.block_cols + t * kColsPerThread;
        const int end = min(a.dim, (rank + 1) * a.plan.block_cols);
        count = max(0, min(kColsPerThread, end - first));
        last = count > 0 && first + kColsPerThread >= end;
    }
    __device__ __forceinline__ bool has(int e) const { return ALIGNED ? count > 0 : e < count; }
};

// Rows on their way through shared memory: every thread copies its own columns
// of a row some rows ahead (cp.async) and reads them back itself, so the copies
// need no barrier.  A stage holds, per tensor, 16-byte words [word][thread].
//
// Where rows do not start on 16-byte boundaries a thread copies the aligned
// words that its columns lie in -- one more than they fill -- and shifts.  A word
// that reaches over the tensor's first or last element is put together from
// single elements.
template <typename T, bool ALIGNED>
struct Staged {
    static constexpr int kUnits = (sizeof(T) == 4 ? 2 : 1) + (ALIGNED ? 0 : 1);

    // Of a row whose first column is at `row`; slot: the thread's first word.
    static __device__ __forceinline__ void fetch(const RowPtr &p, const T *row, int first,
                                                 int count, uint4 *slot, int threads)
    {
        const unsigned char *at = reinterpret_cast<const unsigned char *>(row + first);
        if constexpr (ALIGNED) {
#pragma unroll
            for (int u = 0; u < kUnits; ++u) copy16_async(slot + u * threads, at + u * 16, false);
        } else {
            const unsigned char *stop = at + count * sizeof(T);
            const unsigned char *word = at - (reinterpret_cast<uintptr_t>(at) & 15);
#pragma unroll
            for (int u = 0; u < kUnits; ++u, word += 16) {
                if (word >= stop) continue;
                if (word >= p.p && word + 16 <= p.end) {
                    copy16_async(slot + u * threads, word, true);
                } else {
                    const T *from = reinterpret_cast<const T *>(word);
                    T *to = reinterpret_cast<T *>(slot + u * threads);
                    for (int i = 0; i < int(16 / sizeof(T)); ++i)
                        if (reinterpret_cast<const unsigned char *>(from + i) >= at &&
                            reinterpret_cast<const unsigned char *>(from + i) < stop)
                            to[i] = from[i];
                }
            }
        }
    }

    static __device__ __forceinline__ void read(const T *row, const Cols<ALIGNED> &c, bool active,
                                                const uint4 *slot, int threads, float (&v)[8])
    {
        if (!active || c.count == 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.0f;
            return;
        }
        if constexpr (ALIGNED) {
            Raw8<T> r;
#pragma unroll
            for (int u = 0; u < kUnits; ++u) r.w[u] = slot[u * threads];
            unpack8<T>(r, v);
        } else {
            Wide8<T> w;
#pragma unroll
            for (int u = 0; u < kUnits; ++u)
                reinterpret_cast<uint4 *>(w.w)[u] = slot[u * threads];
            const int s = int(reinterpret_cast<uintptr_t>(row + c.first) & 15) / int(sizeof(T));
            unpack8<T>(shift_down<T>(w, s), v);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = c.has(e) ? v[e] : 0.0f;
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

// Stores the thread's columns of a row.  Where the row does not start on a
// 16-byte boundary, a thread takes the last `s` elements of its left neighbour
// (by shuffle) in front of its own first 8 - s and stores those as whole words;
// the first lane of a run stores its own first elements, the last its own last
// ones, one by one.  All lanes of a warp call together.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void store_row(T *row, const Cols<ALIGNED> &c, bool active,
                                          const float (&v)[8])
{
    T *at = row + c.first;
    if constexpr (ALIGNED) {
        if (active && c.count > 0) st8(at, pack8<T>(v));
    } else {
        const Raw8<T> own = pack8<T>(v);
        const uint32_t *ow = reinterpret_cast<const uint32_t *>(&own);
        constexpr int W = 2 * sizeof(T);                 // words of eight elements
        constexpr int P = sizeof(T) == 4 ? 4 : 4;        // words of the neighbour that may be needed
        constexpr int G = 16 / int(sizeof(T));           // elements of a 16-byte word
        Wide8<T> both;                                   // neighbour's last word, then own
#pragma unroll
        for (int i = 0; i < P; ++i) both.w[i] = __shfl_up_sync(0xffffffffu, ow[W - P + i], 1);
#pragma unroll
        for (int i = 0; i < W; ++i) both.w[P + i] = ow[i];
        if (!active || c.count == 0) return;
        const int s = int(reinterpret_cast<uintptr_t>(at) & 15) / int(sizeof(T));
        const bool head = c.t == 0 || (threadIdx.x & 31) == 0;
        const bool tail = c.last || (threadIdx.x & 31) == 31;
        if (s == 0 ? c.count == 8 : (!head && c.count >= 8 - s)) {
            // elements [-s, 8 - s): from element G - s of `both`; s = 0 is own, unshifted
            st8(at - s, s == 0 ? own : shift_down<T>(both, G - s));
            if (s == 0 || !tail) return;
#pragma unroll
            for (int e = 1; e < 8; ++e)
                if (e >= 8 - s && e < c.count) at[e] = from_f32<T>(v[e]);
            return;
        }
        // the left neighbour's last elements, unless the neighbour stores them itself
        if (s > 0 && !head) {
            const T *left = reinterpret_cast<const T *>(both.w);
#pragma unroll
            for (int i = 1; i < G; ++i)
                if (i >= G - s) at[i - G] = left[i];
        }
        // own elements: the right neighbour stores those from 8 - s on, unless this is a run's end
        const int stop = s == 0 || tail ? c.count : min(c.count, 8 - s);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < stop) at[e] = from_f32<T>(v[e]);
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
        v[e] = !p.p ? missing : (c.has(e) ? param_at(p, group, c.first + e) + offset : 0.0f);
}

// Row r of a tensor.
template <typename T>
__device__ __forceinline__ const T *row_of(const RowPtr &p, int tokens, int r)
{
    const int b = r / tokens, t = r - b * tokens;
    return static_cast<const T *>(p.p) + (b * p.sb + t * p.st);
}

// Sums of N values over a team.  All threads of a block call together.
struct TeamSum {
    float (*slots)[2][16];         // [2][N][warp]
    float (*cluster_slots)[2][4];  // [2][N][block of the cluster]
    int parity, tpr, warps, cluster;

    template <int N>
    __device__ __forceinline__ void operator()(float (&v)[N])
    {
        if (tpr < 32) {
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
#pragma unroll
        for (int k = 0; k < N; ++k)
            if (lane == k) slots[parity][k][warp] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k)
            v[k] = (lane & 15) < warps ? slots[parity][k][lane & 15] : 0.0f;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        if (cluster > 1) {
            namespace cg = cooperative_groups;
            cg::cluster_group cl = cg::this_cluster();
            if (int(threadIdx.x) < cluster) {
#pragma unroll
                for (int k = 0; k < N; ++k)
                    cl.map_shared_rank(&cluster_slots[parity][k][0], threadIdx.x)[cl.block_rank()] = v[k];
            }
            cl.sync();
#pragma unroll
            for (int k = 0; k < N; ++k) {
                v[k] = 0.0f;
                for (int r = 0; r < cluster; ++r) v[k] += cluster_slots[parity][k][r];
            }
        }
        parity ^= 1;
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
    // one attribute for all sizes: every launch of the kernel sets the same
    const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kMaxBlockSmem);
    if (e != cudaSuccess) return e;
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
