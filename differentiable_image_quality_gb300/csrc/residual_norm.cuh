// Shared parts of the residual-norm kernels: the norms before and after a
// residual block with its gate and residual scale, forward and backward.
//
//   y^ = (y - m1) r1,  z = y^ (w1 + o) + b1,  x' = s x + g z,
//   x^ = (x' - m2) r2, u = x^ (w2 + o) + b2,
// per row of D columns; m, r the row's mean (zero for the root-mean-square
// norm) and 1 / sqrt(mean((. - m)^2) + eps).
#pragma once

#include <algorithm>
#include <atomic>

#include <cooperative_groups.h>

#include "gbssim.h"
#include "common.cuh"
#include "dtypes.cuh"

namespace gbssim {

// Every thread owns eight columns of a row for the whole kernel, so that the
// parameters of its columns and their gradients' sums stay in registers.  A row
// belongs to a team: `tpr` lanes of a warp (a power of two) for rows of up to
// 256 columns, else a block, and a cluster of blocks for rows that are wider than
// a block's threads (64 registers each in the forward, 128 in the backward).
constexpr int kColsPerThread = 8;
constexpr int kFwdThreads = 1024, kBwdThreads = 512;  // of a block, at most
constexpr int kSmallBlock = 128;  // threads of a block that holds several teams
// Threads an SM holds of the backward's kernel that needs fewest registers (96).
constexpr int kBwdResidentPlain = 640;
constexpr int kMaxDim = 16384;    // 2 forward or 4 backward blocks

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
    int uneven;        // a tensor's rows change their alignment within a block
    int even_out;      // a block's columns of an output are aligned in groups of eight
    int classes;       // 8 / gcd(8, D); 1 also where a group has too few rows to part
    int cluster;       // blocks of a cluster (1, 2, 4)
    int block_cols;    // columns of a block: a multiple of 8 (counted from the shift)
    int tpr;           // threads of a team in a block
    int teams;         // teams of a block
    int groups, group_rows, splits;
    int threads;
    unsigned grid;     // groups * classes * splits * cluster
    int device;
};

struct ResidualNormArgs {
    RowPtr x, y, gate_rows;
    ParamPtr gate, w1, b1, w2, b2;
    int tokens, dim;   // tokens: 0 where one stride reaches every row of every tensor
    int post, pre;     // gbssim_row_norm
    float scale, offset, eps, inv_dim;
    RowPlan plan;
    unsigned exchange_extra;  // test hook: see TeamSum
    // forward
    void *x_out, *u;
    float4 *stats;     // (m1, r1, m2, r2) of each row
    // backward
    RowPtr gx, gu;
    void *dx, *dy, *dgate_rows;
    float *partials;   // [groups * classes * splits][sums][dim], then what is folded of them
    int sum_a, sum_f, sum_c, sum_e, sums;  // places of the column sums, -1: not wanted
};

// The gradients that many samples share, where others are per sample.  Partials are
// first folded, kFoldedPartials into one set of the five gradients, where more groups
// have factors of their own than a column has threads, and where there are more than
// kMostUnfolded: backward, bfloat16, folded and not, 1000 x 8 x 1024 52 and 44 us, 8000 x 2 x
// 1024 221 and 201, 16000 x 2 x 256 186 and 200.  8, 16, 32 and 64 in a set: 31, 33, 38 and
// 47 us at 512 x 8 x 1024, 427, 402, 393 and 390 at 8000 x 16 x 306.
constexpr int kFinishLanes = 64;  // threads of a column that add its partials
constexpr int kMostUnfolded = 8192, kFoldedPartials = 16;

// Outputs of the parameters' gradients.
struct ParamGrad {
    void *p;
    int type, per_sample;
};
struct ParamGrads {
    ParamGrad gate, w1, b1, w2, b2;
};

// How many clusters of 2 and of 4 blocks the current device holds at one block an SM.
struct ClusterRoom {
    int of2, of4;
};
cudaError_t residual_norm_cluster_room(ClusterRoom *room);

cudaError_t residual_norm_fwd_launch(const ResidualNormArgs &a, int res, int blk, cudaStream_t s);
cudaError_t residual_norm_bwd_launch(const ResidualNormArgs &a, int res, int blk,
                                     const ParamGrads &g, cudaStream_t s);
// Which of the backward's kernels a call takes.
inline int residual_norm_bwd_norms(const ResidualNormArgs &a)
{
    if (a.b1.p || a.sum_f >= 0) return 2;
    return a.post == GBSSIM_ROW_LAYER || a.pre == GBSSIM_ROW_LAYER || a.sum_e >= 0 ? 1 : 0;
}
inline bool residual_norm_bwd_any(const ResidualNormArgs &a)
{
    return !a.y.p || !a.gx.p || !a.gu.p || !a.dx || !a.dy || a.tokens != 0 || a.plan.uneven;
}
inline bool residual_norm_bwd_plain(const ResidualNormArgs &a)
{
    return !a.gate_rows.p && !residual_norm_bwd_any(a) && a.plan.cluster == 1 &&
           residual_norm_bwd_norms(a) == 0;
}

cudaError_t residual_norm_bwd_f32_launch(const ResidualNormArgs &a, int blk, cudaStream_t s);
cudaError_t residual_norm_bwd_16_launch(const ResidualNormArgs &a, int blk, cudaStream_t s);
// Kernel-side failures on the current device since the last call that cleared them.
cudaError_t residual_norm_fwd_status(unsigned *flags, bool clear);
cudaError_t residual_norm_bwd_f32_status(unsigned *flags, bool clear);
cudaError_t residual_norm_bwd_16_status(unsigned *flags, bool clear);

#ifdef __CUDACC__

// The rows of this block (or cluster): first + i * step, i < count, of one class
// of group `group`.
struct BlockRows {
    int group, first, count, step;
    int shift;  // columns that the class's rows start past a multiple of eight elements
    __device__ __forceinline__ BlockRows(const ResidualNormArgs &a, int cluster)
    {
        const RowPlan &p = a.plan;
        const int item = int(blockIdx.x) / cluster;
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
    int t;            // place in the team
    int lane, lanes;  // and in its lanes of this warp
    int words;        // 16-byte words of float32 that those lanes have of a row (ALIGNED)
    bool whole;       // all eight, and outputs' groups of eight are aligned
    __device__ __forceinline__ Cols(const ResidualNormArgs &a, int cluster, int shift)
    {
        const int rank = int(blockIdx.x) % cluster;
        t = a.plan.teams > 1 ? threadIdx.x & (a.plan.tpr - 1) : threadIdx.x;
        first = rank * a.plan.block_cols + t * kColsPerThread - (ALIGNED ? 0 : shift);
        from = max(0, -first);
        upto = t * kColsPerThread < a.plan.block_cols ? max(0, min(kColsPerThread, a.dim - first)) : 0;
        whole = upto - from == kColsPerThread && a.plan.even_out;
        lanes = min(a.plan.tpr, 32);
        lane = t & (lanes - 1);
        const int group = (t - lane) * kColsPerThread;  // columns of the block ahead of these lanes
        words = max(0, min(a.plan.block_cols - group, a.dim - (first - lane * kColsPerThread))) / 4;
    }
    __device__ __forceinline__ bool any() const { return from < upto; }
    __device__ __forceinline__ bool all() const { return ALIGNED ? upto > 0 : upto - from == 8; }
    __device__ __forceinline__ bool has(int e) const
    {
        return ALIGNED ? upto > 0 : e >= from && e < upto;
    }
};

// Column `col` of row r of a tensor; ANY: of one whose rows may need two strides.
template <typename T, bool ANY>
__device__ __forceinline__ const unsigned char *row_at(const RowPtr &p, int tokens, int r, int col)
{
    const unsigned char *base = static_cast<const unsigned char *>(p.p) + col * int(sizeof(T));
    if (!ANY || tokens == 0) return base + (long long)r * p.row_bytes;
    const int b = r / tokens, t = r - b * tokens;
    return base + (b * p.sb + t * p.st) * int(sizeof(T));
}

// Rows on their way through shared memory: every thread copies its own columns
// of a row some rows ahead (cp.async) and reads them back itself, so the copies
// need no barrier.  A stage holds, per tensor, 16-byte words [word][thread].
//
// Eight float32 columns are two words.  Aligned rows: the lanes of a team in a warp
// copy one another's, so that a copy of the warp covers whole lines: lane g takes
// words g and g + lanes, word w being the (w % 2)th of lane w / 2.  (Each lane its
// own two words, 32 bytes apart, would ask L2 for every sector twice.)
//
// Where a tensor's rows are not aligned as the block's columns are, a thread
// copies the aligned words that its columns lie in -- one more than they fill --
// and shifts.  Near the tensor's first and last element the words are put
// together from single elements instead: nothing outside the tensor is read.
template <typename T, bool ALIGNED, bool ANY>
struct Staged {
    static constexpr int kUnits = (sizeof(T) == 4 ? 2 : 1) + (ALIGNED ? 0 : 1);

    // at: the thread's first column; slot: its first word, `pitch` bytes from word to word.
    static __device__ __forceinline__ void fetch(const RowPtr &p, const unsigned char *at,
                                                 const Cols<ALIGNED> &c, unsigned slot, int pitch)
    {
        if constexpr (ALIGNED && sizeof(T) == 4) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int w = c.lane + u * c.lanes, other = w / 2 - c.lane;
                if (w < c.words)
                    copy16_async<false>(slot + other * 16 + (w & 1) * pitch,
                                        at + (w - 2 * c.lane) * 16);
            }
        } else if constexpr (ALIGNED) {
            if (c.any()) copy16_async<false>(slot, at);
        } else {
            if (!c.any()) return;
            const unsigned char *word = at - (reinterpret_cast<uintptr_t>(at) & 15);
            if (c.all() && word == at) {
#pragma unroll
                for (int u = 0; u < kUnits - 1; ++u) copy16_async<false>(slot + u * pitch, at + u * 16);
            } else if (word >= p.p && word + 16 * kUnits <= p.end) {
                // the ends of the row before and after, where they come along, are not looked at
#pragma unroll
                for (int u = 0; u < kUnits; ++u) copy16_async<true>(slot + u * pitch, word + u * 16);
            } else {
                const unsigned char *from = at + c.from * int(sizeof(T));
                const unsigned char *stop = at + c.upto * int(sizeof(T));
#pragma unroll 1
                for (int u = 0; u < kUnits; ++u, word += 16, slot += pitch) {
                    T *to = static_cast<T *>(__cvta_shared_to_generic(slot));
#pragma unroll 1
                    for (int i = 0; i < 16; i += int(sizeof(T)))
                        if (word + i >= from && word + i < stop)
                            to[i / int(sizeof(T))] = *reinterpret_cast<const T *>(word + i);
                }
            }
        }
    }

    // By how many elements a block's columns of a row (`from` is the first) lie past
    // a 16-byte boundary; the same for all its threads.
    static __device__ __forceinline__ int shift_of(const RowPtr &p, int tokens, int row, int from)
    {
        if (ALIGNED || !p.p) return 0;
        return int(reinterpret_cast<uintptr_t>(row_at<T, ANY>(p, tokens, row, from)) & 15) /
               int(sizeof(T));
    }

    // The thread's columns of a row, zero where the row has none.  known: the shift,
    // where that is the same in all rows of a block (it is unless ANY).
    static __device__ __forceinline__ void read(const RowPtr &p, int tokens, int row, int known,
                                                const Cols<ALIGNED> &c, bool active, unsigned slot,
                                                int pitch, f32x2 (&v)[4])
    {
        Raw8<T> r;
        const bool wanted = active && c.any();
        if constexpr (ALIGNED) {
#pragma unroll
            for (int u = 0; u < kUnits; ++u) r.w[u] = ld_shared16(slot + u * pitch, wanted);
            unpack8<T>(r, v);
        } else {
            const int s = ANY ? shift_of(p, tokens, row, c.first) : known;
            if (s == 0) {
#pragma unroll
                for (int u = 0; u < kUnits - 1; ++u) r.w[u] = ld_shared16(slot + u * pitch, wanted);
            } else {
                Wide8<T> w;
#pragma unroll
                for (int u = 0; u < kUnits; ++u) {
                    const uint4 q = ld_shared16(slot + u * pitch, wanted);
                    w.w[4 * u] = q.x; w.w[4 * u + 1] = q.y;
                    w.w[4 * u + 2] = q.z; w.w[4 * u + 3] = q.w;
                }
                r = shift_down<T>(w, s);
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

// Waits until at most PENDING of this thread's latest groups are in flight.
template <int PENDING>
__device__ __forceinline__ void staged_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

// Stores the thread's columns of a row, the first at `to`: whole where it has all
// eight and they are aligned, one by one at a row's ends.
template <typename T, bool ALIGNED>
__device__ __forceinline__ void store_cols(T *to, const Cols<ALIGNED> &c, bool active,
                                           const f32x2 (&v)[4])
{
    if constexpr (ALIGNED) {
        if (active && c.any()) st8_whole(to, pack8<T>(v));
    } else {
        if (active && c.whole) {
            st8_whole(to, pack8<T>(v));
        } else if (active) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float2 h = halves(v[e / 2]);
                if (c.has(e)) to[e] = from_f32<T>(e & 1 ? h.y : h.x);
            }
        }
    }
}

// The thread's eight values of a parameter as they lie in memory.  A block asks for
// all its parameters before it converts the first: one after the other, each
// waited about a microsecond, which is what a call of a few rows then took.
struct RawParam {
    uint32_t w[8];  // two 16-bit values a word (the first four words), or one value a word
    bool packed;
};

template <bool ALIGNED>
__device__ __forceinline__ RawParam fetch_param(const ParamPtr &p, int group, const Cols<ALIGNED> &c)
{
    RawParam r;
    r.packed = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) r.w[e] = 0u;
    if (!p.p) return r;
    const bool wide = p.type == GBSSIM_F32;
    const unsigned char *at =
        static_cast<const unsigned char *>(p.p) + (group * p.stride + c.first) * (wide ? 4 : 2);
    if (c.all() && (reinterpret_cast<uintptr_t>(at) & 15) == 0) {
        const uint4 lo = __ldg(reinterpret_cast<const uint4 *>(at));
        r.w[0] = lo.x; r.w[1] = lo.y; r.w[2] = lo.z; r.w[3] = lo.w;
        r.packed = !wide;
        if (wide) {
            const uint4 hi = __ldg(reinterpret_cast<const uint4 *>(at) + 1);
            r.w[4] = hi.x; r.w[5] = hi.y; r.w[6] = hi.z; r.w[7] = hi.w;
        }
    } else if (wide) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c.has(e)) r.w[e] = __ldg(reinterpret_cast<const uint32_t *>(at) + e);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c.has(e)) r.w[e] = __ldg(reinterpret_cast<const unsigned short *>(at) + e);
    }
    return r;
}

// The values plus `offset`; `missing` where the parameter is null.  Either way zero in
// columns that the row does not have: a mean puts something into y^ and x^ there, and
// this factor keeps it out of the row's sums.
template <bool ALIGNED>
__device__ __forceinline__ void param_values(const ParamPtr &p, const RawParam &r,
                                             const Cols<ALIGNED> &c, float offset, float missing,
                                             f32x2 (&v)[4])
{
    if (!p.p) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = both(missing);
    } else if (p.type == GBSSIM_F32) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = pair(__uint_as_float(r.w[2 * e]), __uint_as_float(r.w[2 * e + 1]));
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t w = r.packed ? r.w[e] : r.w[2 * e] | r.w[2 * e + 1] << 16;
            const float2 h = p.type == GBSSIM_BF16 ? unpack2<bf16>(w) : unpack2<f16>(w);
            v[e] = pair(h.x, h.y);
        }
    }
    if (p.p && offset != 0.0f) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = add2(v[e], both(offset));
    }
    if (!c.all()) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 h = halves(v[e]);
            v[e] = pair(c.has(2 * e) ? h.x : 0.0f, c.has(2 * e + 1) ? h.y : 0.0f);
        }
    }
}

// ------------------------------------------------------ sums over a team

__device__ __forceinline__ unsigned peer_address(unsigned shared, int rank)
{
    unsigned r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(shared), "r"(rank));
    return r;
}

// Writes four floats to a block of the cluster and counts them on its barrier.
__device__ __forceinline__ void send16(unsigned to, float4 v, unsigned bar)
{
    asm volatile(
        "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
        "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
        : "memory");
}

// What the warps of a block tell one another, and the blocks of a cluster: every
// block sends its sums to all, as bytes that the receiver's barrier counts.  (A
// cluster-wide barrier would first wait for the rows that the blocks have just
// stored.)
struct TeamSlots {
    float warps[2][4][32];     // [parity][value][warp]
    float4 blocks[2][4];       // [parity][block]
    uint64_t arrived[2];
    float2 columns[32];        // of each warp: how many, and 1 / that
    float2 block_columns[4];   // of each block
};

// About a second: an exchange that takes longer has failed.
constexpr long long kExchangeCycles = 2000000000ll;

// Kernel-side failures of this file's kernels (bit 1: an exchange ran out of time).
static __device__ unsigned g_exchange_status;

// Sums over a team, of one value or of two.  All threads of a block call together.
// CLUSTER: a row may be shared by blocks of a cluster.
template <bool CLUSTER>
struct TeamSum {
    TeamSlots &slots;
    int parity, tpr, warps, cluster;
    unsigned phases;      // of arrived[0] and arrived[1], one bit each
    unsigned extra;       // test hook: bytes announced beyond those sent (0)
    bool dead;            // an exchange ran out of time: wait for no other
    float inv_columns;    // 1 / columns of the team's lanes in this warp (count_columns)
    float inv_block;      // 1 / columns of the block

    __device__ __forceinline__ TeamSum(TeamSlots &s, const ResidualNormArgs &a)
        : slots(s), parity(0), tpr(a.plan.tpr), warps(a.plan.teams > 1 ? 1 : a.plan.threads / 32),
          cluster(CLUSTER ? a.plan.cluster : 1), phases(0), extra(a.exchange_extra), dead(false),
          inv_columns(0.0f), inv_block(0.0f)
    {
        if (cluster == 1) return;
        if (threadIdx.x == 0) {
            mbar_init(&slots.arrived[0], 1);
            mbar_init(&slots.arrived[1], 1);
            mbar_init_fence();
        }
        cooperative_groups::this_cluster().sync();  // before anyone sends
    }

    // Sum over the team's lanes of this warp.
    __device__ __forceinline__ float lanes(float v) const
    {
        if (tpr < 32) {
#pragma unroll 1
            for (int o = tpr >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            return v;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }

    // Sum over the lanes that hold the warps' values: all, or each half alike.
    __device__ __forceinline__ float over_warps(float v) const
    {
        if (warps > 16) v += __shfl_xor_sync(0xffffffffu, v, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }

    // The warp whose value this lane takes.
    __device__ __forceinline__ int my_warp() const
    {
        return threadIdx.x & (warps > 16 ? 31 : 15);
    }

    // The warps' values, one warp to each lane of a warp or of a half.  One barrier: the
    // slots alternate, and a thread that writes a slot again has passed the
    // barrier of the sum in between, which every thread reaches only after it has
    // read this one.
    template <int N>
    __device__ __forceinline__ void of_warps(float (&v)[N])
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0) {
#pragma unroll
            for (int k = 0; k < N; ++k) slots.warps[parity][k][warp] = v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k)
            v[k] = my_warp() < warps ? slots.warps[parity][k][my_warp()] : 0.0f;
    }

    // A row whose sums did not arrive has no result.
    __device__ __forceinline__ float or_nan(float v) const
    {
        return dead ? __uint_as_float(0x7fffffffu) : v;
    }

    // This block's values to all blocks, and all blocks' into slots.blocks.  A
    // block sends its next values only after its threads have read all of these,
    // and nobody gets further than one exchange ahead of the others: two sets of
    // slots are enough.
    __device__ __forceinline__ void exchange(float4 v)
    {
        if (!dead) {
            uint64_t *bar = &slots.arrived[parity];
            if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, unsigned(cluster) * 16u + extra);
            if (int(threadIdx.x) < cluster) {
                const int rank = int(cooperative_groups::this_cluster().block_rank());
                send16(peer_address(smem_u32(&slots.blocks[parity][rank]), threadIdx.x), v,
                       peer_address(smem_u32(bar), threadIdx.x));
            }
            // once a wait has run out, nothing arrives here again: the barrier's
            // phase is still open, and takes no second arrival
            if (!mbar_wait_bounded(bar, (phases >> parity) & 1u, kExchangeCycles)) {
                dead = true;
                atomicOr(&g_exchange_status, 2u);
            }
        }
        phases ^= 1u << parity;
    }

    template <int N>
    __device__ __forceinline__ void operator()(float (&v)[N])
    {
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = lanes(v[k]);
        if (warps == 1 && cluster == 1) return;
        of_warps(v);
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = over_warps(v[k]);
        if (cluster > 1) {
            exchange(make_float4(v[0], v[N > 1 ? 1 : 0], v[N > 2 ? 2 : 0], v[N > 3 ? 3 : 0]));
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = 0.0f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float4 b = r < cluster ? slots.blocks[parity][r] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                v[0] += b.x;
                if (N > 1) v[N > 1 ? 1 : 0] += b.y;
                if (N > 2) v[N > 2 ? 2 : 0] += b.z;
                if (N > 3) v[N > 3 ? 3 : 0] += b.w;
            }
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] = or_nan(v[k]);
        }
        parity ^= 1;
    }

    __device__ __forceinline__ float one(float v)
    {
        float a[1] = {v};
        (*this)(a);
        return a[0];
    }

    static __device__ __forceinline__ float2 with_inverse(float n)
    {
        return make_float2(n, n > 0.0f ? 1.0f / n : 0.0f);
    }

    // Once, before join_squares: how many columns the lanes, warps and blocks have.
    __device__ __forceinline__ void count_columns(int mine)
    {
        const float n = lanes(float(max(0, mine)));
        inv_columns = with_inverse(n).y;
        if (warps == 1 && cluster == 1) return;
        const int lane = threadIdx.x & 31;
        float w[1] = {n};
        of_warps(w);
        if (threadIdx.x < 32) slots.columns[lane] = with_inverse(w[0]);
        const float block = over_warps(w[0]);
        inv_block = with_inverse(block).y;
        if (cluster > 1) {
            exchange(make_float4(block, 0.0f, 0.0f, 0.0f));
            if (threadIdx.x < 4)
                slots.block_columns[lane] =
                    lane < cluster ? with_inverse(slots.blocks[parity][lane].x) : make_float2(0.0f, 0.0f);
        }
        parity ^= 1;
        __syncthreads();
    }

    // From the sum s of the team's columns in this warp and the sum q of their
    // squares about their own mean: the row's sum, and its squares about its mean.
    // With n columns of mean m = s / n apiece, q joins as q + n (m - row mean)^2.
    __device__ __forceinline__ float2 join_squares(float s, float q, float inv_dim)
    {
        if (warps == 1 && cluster == 1) return make_float2(s, q);
        float w[2] = {s, q};
        of_warps(w);
        const float2 n = slots.columns[my_warp()];
        const float block = over_warps(w[0]);
        const float d = fmaf(w[0], n.y, -block * inv_block);
        float2 r = make_float2(block, over_warps(fmaf(n.x * d, d, w[1])));
        if (cluster > 1) {
            exchange(make_float4(r.x, r.y, 0.0f, 0.0f));
            float2 v[4], c[4];
            float total = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                c[k] = slots.block_columns[k];
                const float4 b = k < cluster ? slots.blocks[parity][k] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                v[k] = make_float2(b.x, b.y);
                total += b.x;
            }
            const float row = total * inv_dim;
            r = make_float2(total, 0.0f);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float dk = fmaf(v[k].x, c[k].y, -row);
                r.y += fmaf(c[k].x * dk, dk, v[k].y);
            }
            r.y = or_nan(r.y);
        }
        parity ^= 1;
        return r;
    }

    // No block leaves while another might still send to it.
    __device__ __forceinline__ void finish()
    {
        if (cluster > 1) cooperative_groups::this_cluster().sync();
    }
};

// The flags of this file's kernels on the current device; clear: and zero them.
inline cudaError_t exchange_status(unsigned *flags, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(flags, g_exchange_status, sizeof(unsigned));
    if (e == cudaSuccess && clear && *flags) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_exchange_status, &zero, sizeof(unsigned));
    }
    return e;
}

// Shared memory of an SM that rings of staged rows share.
constexpr int kStagedSmem = 200 * 1024, kStagedBlock = 220 * 1024;

// The stages of a ring of staged rows, of `units` 16-byte words a thread each: two
// where they leave room for `per_sm` blocks of 512 threads, or as many threads of
// smaller ones, on an SM.  More rows in flight made the widest forward slower:
// 65536 x 4096 bfloat16 took 332 us with two stages, 346 with three, 372 with four.
constexpr int stages_of(int units, int per_sm)
{
    const int fit = kStagedSmem / (units * 16 * 512 * per_sm);
    return fit < 1 ? 1 : fit > 2 ? 2 : fit;
}

// asked: of this kernel alone, one bit for each device on which it may use more
// shared memory than it may without asking.
template <class Kernel>
cudaError_t launch_staged(Kernel kernel, std::atomic<unsigned long long> &asked,
                          const ResidualNormArgs &a, int units, int stages, cudaStream_t s)
{
    const int smem = stages * units * 16 * a.plan.threads;
    const unsigned long long bit = a.plan.device < 64 ? 1ull << a.plan.device : 0ull;
    // (with the static arrays, 40 KB are below what needs no asking for)
    if (smem > 40 * 1024 && !(asked.load(std::memory_order_relaxed) & bit)) {
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kStagedBlock);
        if (e != cudaSuccess) return e;
        asked.fetch_or(bit, std::memory_order_relaxed);
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
