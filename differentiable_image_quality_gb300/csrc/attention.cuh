// What the attention kernels share: the shape of a call, where a block's queries
// and keys lie, bounded waits.
#pragma once

#include <cuda.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "dtypes.cuh"
#include "packed.cuh"
#include "tensor_core.cuh"

namespace gbssim {

constexpr int kAttnMaxDim = 128;
constexpr int kAttnBlocks = 152;  // that run at once: one to an SM

struct AttnShape {
    int sequences;           // samples, or sequences of a packed batch
    int q_tokens, k_tokens;  // of a sample, or rows of the packed tensors
    int heads, kv_heads, group, dim;
    int causal, packed;
    const int *kv_lengths, *q_offsets, *k_offsets;
};

// Where a block's queries and keys lie.
struct AttnPlace {
    int sequence;       // packed: as many as there are where it is the rows behind them
    int batch;          // outermost coordinate of the tensors
    int q_row, k_row;   // of the sequence's first query and key
    int queries, keys;  // of the sequence
    int shift;          // causal: query i sees keys up to i + shift
    int tile;           // which tile of the sequence
    int q_tiles_before; // of the queries of the sequences before it, in tiles of 128
};

// Where the last search of a packed batch ended: ahead of sequence `base` there are
// `before` tiles of the keys or the queries.  A block's items lie close to one another, so
// one search goes on from the last one (from the first sequence each time, 4096 of 128
// tokens, 8 heads of 64, took 8.5 ms forward and 22 ms backward, for 1.16 and 3.2; with
// the heads' items of a tile next to one another 0.72 and 2.65).  Kept in shared
// memory: registers are short where the searching warp's code is.
struct AttnCursor {
    int base, before, q_before, by_keys;
};

// The sequence and tile of `index`, tiles of `rows` rows of the queries or (BY_KEYS)
// the keys, all of a sequence's before the next one's; false behind the last.  By
// a whole warp; `kept` is that warp's alone, zero before its first search.
template <bool BY_KEYS>
__device__ __forceinline__ bool find_place(const AttnShape &s, int index, int rows, AttnPlace &p, AttnCursor &kept)
{
    if (!s.packed) {
        const int most = BY_KEYS ? s.k_tokens : s.q_tokens;
        const int tiles = (most + rows - 1) / rows;
        p.sequence = p.batch = index / tiles;
        p.tile = index - p.batch * tiles;
        p.q_tiles_before = p.batch * ((s.q_tokens + kAttnTile - 1) / kAttnTile);
        p.q_row = p.k_row = 0;
        p.queries = s.q_tokens;
        p.keys = s.kv_lengths ? min(max(__ldg(s.kv_lengths + p.batch), 0), s.k_tokens) : s.k_tokens;
        p.shift = s.k_tokens - s.q_tokens;
        return p.batch < s.sequences;
    }
    const int lane = threadIdx.x % 32;
    AttnCursor c{0, 0, 0, BY_KEYS};
    if (kept.by_keys == BY_KEYS && index >= kept.before / 2) c = kept;
    bool found = false;
    bool back = index < c.before;
    if (back) c.base -= 32;
    while (!found && c.base <= s.sequences) {
        const int base = c.base;
        int q_first = 0, queries = 0, k_first = 0, keys = 0;
        if (base + lane <= s.sequences) {
            packed_span(s.q_offsets, s.sequences, s.q_tokens, base + lane, q_first, queries);
            packed_span(s.k_offsets, s.sequences, s.k_tokens, base + lane, k_first, keys);
        }
        const int tiles = ((BY_KEYS ? keys : queries) + rows - 1) / rows;
        const int q_tiles = (queries + kAttnTile - 1) / kAttnTile;
        int sum = tiles, q_sum = q_tiles;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
            const int up = __shfl_up_sync(0xffffffffu, sum, d);
            const int q_up = __shfl_up_sync(0xffffffffu, q_sum, d);
            if (lane >= d) {
                sum += up;
                q_sum += q_up;
            }
        }
        const int all = __shfl_sync(0xffffffffu, sum, 31), q_all = __shfl_sync(0xffffffffu, q_sum, 31);
        if (back) {
            c.before -= all;
            c.q_before = max(c.q_before - q_all, 0);
            back = index < c.before && base > 0;
            if (back) {
                c.base -= 32;
                continue;
            }
        }
        const unsigned past = __ballot_sync(0xffffffffu, c.before + sum > index);
        if (past) {
            const int l = __ffs(past) - 1;
            p.tile = index - c.before - __shfl_sync(0xffffffffu, sum - tiles, l);
            p.q_tiles_before = c.q_before + __shfl_sync(0xffffffffu, q_sum - q_tiles, l);
            p.batch = 0;
            p.sequence = base + l;
            p.q_row = __shfl_sync(0xffffffffu, q_first, l);
            p.k_row = __shfl_sync(0xffffffffu, k_first, l);
            p.queries = __shfl_sync(0xffffffffu, queries, l);
            p.keys = __shfl_sync(0xffffffffu, keys, l);
            // the rows behind the last sequences have no partners
            if (base + l == s.sequences) (BY_KEYS ? p.queries : p.keys) = 0;
            p.shift = p.keys - p.queries;
            found = true;
        } else {
            c.base += 32;
            c.before += all;
            c.q_before = add_tiles(c.q_before, q_all);
        }
    }
    __syncwarp();
    if (lane == 0) kept = c;
    __syncwarp();
    return found;
}

// Most tiles of `rows` rows that a call can have.
inline long long most_tiles(const AttnShape &s, int tokens, int rows)
{
    if (s.packed) return (long long)tokens / rows + s.sequences + 1;
    return (long long)s.sequences * ((tokens + rows - 1) / rows);
}

// Waits of at most about a second each.  A wait that runs out marks the block:
// every other wait of the block then ends too, its roles leave their loops, and what
// they have in flight is waited for before tensor memory is freed.
constexpr long long kAttnWaitCycles = 2'000'000'000LL;
constexpr long long kAttnDrainCycles = 500'000'000LL;

__device__ __forceinline__ bool attn_wait_slow(uint64_t *bar, unsigned parity, volatile unsigned *failed)
{
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (*failed) return false;
        if (clock64() - t0 > kAttnWaitCycles) {
            *failed = 1;
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ bool attn_wait(uint64_t *bar, unsigned parity, volatile unsigned *failed)
{
    return mbar_try_wait(bar, parity) || attn_wait_slow(bar, parity, failed);
}

// A place in a ring of N buffers and the parity of its round, without divisions.
template <int N>
struct RingAt {
    int slot = 0;
    unsigned parity = 0;
    __device__ __forceinline__ void next()
    {
        if (++slot == N) {
            slot = 0;
            parity ^= 1;
        }
    }
};

// By a whole warp, which then goes one way.
__device__ __forceinline__ bool attn_wait_warp(uint64_t *bar, unsigned parity, volatile unsigned *failed)
{
    return __all_sync(0xffffffffu, attn_wait(bar, parity, failed));
}

// A value that all lanes have, where the compiler knows that they do.
__device__ __forceinline__ unsigned uniform(unsigned v) { return __shfl_sync(0xffffffffu, v, 0); }

// A kernel's shared memory, asked for once on each device (1.5 us a call otherwise).
// `registers`: what its warpgroups' threads have after they have shared them out anew, one
// of each of `groups`; more than the kernel is launched with would be waited for without
// end, so such a build is refused.
template <typename Kernel>
inline cudaError_t allow_smem(Kernel kernel, std::atomic<unsigned long long> &done, size_t bytes, int registers = 0,
                              int groups = 1)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kernel);
    if (e == cudaSuccess && (attr.numRegs + 7) / 8 * 8 * groups < registers) e = cudaErrorLaunchOutOfResources;
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// A launch whose blocks may start while the kernel ahead on the stream ends; they wait
// for it (pdl_wait) before they touch what it wrote.
// `kernel_ahead`: what is ahead is one; behind a copy or a fill nothing starts early.
template <typename Args>
inline cudaError_t launch_after(void (*kernel)(Args), dim3 grid, unsigned threads, size_t smem,
                                cudaStream_t stream, const Args &a, bool kernel_ahead = true)
{
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &early;
    cfg.numAttrs = kernel_ahead;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// ------------------------------------------------------------------- forward

struct AttnFwdArgs {
    CUtensorMap q, k, v;
    AttnShape s;
    float scale_log2;
    int tile_heads;   // heads of a tile: 1, or the group's where all its rows fit one tile
    int tile_tokens;  // tokens of a tile
    int splits;       // parts of the keys
    int tiles;        // of q_tokens (batch form), or the most there can be (packed)
    unsigned items;   // of all blocks
    unsigned *counter;  // of items taken, or null: dealt out beforehand
    int ragged;       // keys may end before the tensor does
    unsigned extra;   // test hook, see gbssim_tune_attention
    void *out;
    float *lse;       // or null
    float *part_out, *part_lse;  // of each part, where there are several
};

cudaError_t attention_fwd_launch(const AttnFwdArgs &a, int dtype, int q_tiles, cudaStream_t stream);
cudaError_t attention_fwd_status(unsigned *flags, bool clear);
cudaError_t attention_join_launch(const AttnFwdArgs &a, int dtype, cudaStream_t stream);

// ------------------------------------------------------------------ backward

struct AttnBwdArgs {
    CUtensorMap q, k, v, g;  // g: the output's gradient
    AttnShape s;
    float scale, scale_log2;
    int q_tiles, k_tiles;  // in all samples, or the most there can be (packed)
    unsigned key_items, items;  // of all blocks: tiles of keys, and with those of queries
    int key_parts;              // that the query heads of a key head are parted into
    float *parts;               // [key_parts][dv, dk] float32, where there are several
    int queries_wanted;
    int ragged;
    unsigned extra;  // test hook, see gbssim_tune_attention
    // for the row sums
    const void *out, *g_data, *v_data, *q_data, *k_data;
    long long o_batch, o_token, o_head;  // strides, elements
    long long g_batch, g_token, g_head, v_batch, v_token, v_head;
    long long q_batch, q_token, q_head, k_batch, k_token, k_head;
    const float *lse;
    void *dq, *dk, *dv;      // each may be null
    float *stats;            // [heads][q_tiles][2][128]
    unsigned *largest;       // [sequences + 1][kv_heads][2]: |g|, |v|, as bits (float16)
    unsigned *counter;       // of items taken
};

cudaError_t attention_bwd_launch(const AttnBwdArgs &a, int dtype, cudaStream_t stream);
cudaError_t attention_bwd_status(unsigned *flags, bool clear);

}  // namespace gbssim
