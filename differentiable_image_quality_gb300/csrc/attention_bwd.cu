// Attention backward.  From the output's gradient g, with D_i = g_i . o_i:
//   p_ij = exp(s_ij - lse_i),  dp_ij = g_i . v_j,  ds_ij = p_ij (dp_ij - D_i),
//   dv_j = sum_i p_ij g_i,  dk_j = scale sum_i ds_ij q_i,  dq_i = scale sum_j ds_ij k_j.
//
// Blocks of two kinds in one launch: those of 128 keys go over the queries and sum
// dk and dv, those of 128 queries over the keys and sum dq.  Both form p and ds
// again, seven products instead of five, and every sum stays in one block: no
// partial gradients in memory, no atomics, results that repeat bit for bit.
//
// Bound by the tensor cores for heads of 128 (8192 tokens, 8 heads: 538 us, 1.28
// PFLOP/s of the five products, 1.79 of the seven; a tile of keys takes 2048 cycles of
// products, one of queries 1536, and what the warps do between them 1500 and 1100).
// Heads of 64 (330 us) wait for the exchange between the warps and the products, which
// the tensor cores take at two thirds of their rate where they are 64 columns wide.
#include <climits>

#include "attention.cuh"

namespace gbssim {
namespace {

using namespace tc;

__device__ unsigned g_attention_status;

template <int DP>
constexpr int tile_bytes()
{
    return DP / kSlabCols * kSlabBytes;
}

// float16 leaves little room below: probabilities go into their product times 2^14,
// and ds times a power of two for each key head of a sequence, chosen from the largest
// |g| and |v| there so that no product of them overflows.  bfloat16 needs neither.
constexpr int kProbBits = 14;
template <typename T>
constexpr bool kScaled = std::is_same<T, f16>::value;

__device__ __forceinline__ unsigned *largest_at(const AttnBwdArgs &a, int sequence, int kv_head)
{
    return a.largest + 2 * ((long long)sequence * a.s.kv_heads + kv_head);
}

// What an item's power of two comes from is asked for at its start, and looked at when its
// first dp is here: waited for by the copying warp before the others know of the item, it
// cost 24 packed images (16 heads of 64, 235 us) 8 us.
template <typename T>
__device__ __forceinline__ uint2 ask_largest(const AttnBwdArgs &a, int sequence, int kv_head)
{
    uint2 m{0, 0};
    if constexpr (kScaled<T>)
        asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(m.x), "=r"(m.y) : "l"(largest_at(a, sequence, kv_head)));
    return m;
}

__device__ __forceinline__ int scale_bits(const uint2 &largest, int dim)
{
    const auto value = [](unsigned bits) { return __half2float(__ushort_as_half(static_cast<unsigned short>(bits))); };
    // |dp - D| <= 2 dim |g| |v|, since o is a mean of v; above 2^-44 where it is not zero
    const float most = 2.0f * dim * value(largest.x) * value(largest.y);
    return most > 0.0f ? 14 + 127 - (__float_as_int(most) >> 23) : 0;
}

// 2^bits, from -126 to 127.
__device__ __forceinline__ float power_of_two(int bits) { return __int_as_float((bits + 127) << 23); }

// ------------------------------------------------------------------- row sums

// Per row -log2(e) lse (plus the bits that float16 probabilities are moved by) and -D,
// in tiles of 128 queries; rows that the sequence does not have, and those that see
// no key, have -infinity: their probabilities are zero.
constexpr int kSumThreads = 256;

// The largest magnitude, as float16's bits, of finite elements: what others make of theirs
// is not finite whatever the scale.  Bits of magnitudes order as the magnitudes do; moved
// up by 0x400 those of infinities and NaN are negative.
__device__ __forceinline__ unsigned largest8(const uint4 &w)
{
    unsigned m = 0x04000400u;
    for (uint32_t x : {w.x, w.y, w.z, w.w}) m = __vmaxs2(m, (x & 0x7fff7fffu) + 0x04000400u);
    return max(m >> 16, m & 0xffffu) - 0x400u;
}

// A block has 32 tokens and up to 64 heads, whose rows lie one behind the other in
// memory; LANES read a row, eight columns each, and a thread asks for four rows
// together.  (A block to a tile of one head, rows far apart: 14000 x 16 rows of 64 took
// 79 us.)  The sums go to the tiles through shared memory.
constexpr int kSumTokens = 32, kSumHeads = 64, kSumRows = 4;
constexpr int kShareSequences = 128;  // four steps of the search

// Over few keys the output's rounding is a good part of dp - D: there D = sum_j p_ij dp_ij
// in float32 instead, whose dots cost little.  By a whole warp, LANES to a row of `g`, two
// keys at a time: halves of the lanes add up one key's dots each, half of those s, the
// others dp (each dot in all lanes: the sums of 4096 sequences of 16 tokens, 8 heads of 64,
// took 357 us for 276).
constexpr int kFewKeys = 16;

// Eight columns as pairs, and their dot with others.
template <typename T>
__device__ __forceinline__ void load_pairs(const T *p, f32x2 (&v)[4])
{
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 x = unpack2<T>(words[e]);
        v[e] = pair(x.x, x.y);
    }
}

template <typename T>
__device__ __forceinline__ float dot8(const T *p, const f32x2 (&v)[4])
{
    f32x2 u[4], sum = 0;
    load_pairs<T>(p, u);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum = fma2(u[e], v[e], sum);
    return sum2(sum);
}

template <typename T, int LANES>
__device__ __forceinline__ float sum_of_few(const AttnBwdArgs &a, const AttnPlace &pl, int query, int head, bool some,
                                            const T *g_row)
{
    const AttnShape &s = a.s;
    const int lane = threadIdx.x % LANES, col = lane * 8, kv_head = head / s.group;
    const int seen = !some ? 0 : s.causal ? min(pl.keys, query + 1 + pl.shift) : pl.keys;
    const int mine = col < s.dim ? seen : 0;  // keys that this lane has columns of
    f32x2 g[4] = {}, q[4] = {};
    float lse = 0.0f, sum = 0.0f;
    if (mine > 0) {
        load_pairs<T>(static_cast<const T *>(a.q_data) + pl.batch * a.q_batch + (long long)(pl.q_row + query) * a.q_token +
                          head * a.q_head + col,
                      q);
        load_pairs<T>(g_row, g);
    }
    if (seen > 0)
        lse = a.lse[((long long)pl.batch * s.heads + head) * s.q_tokens + pl.q_row + query] * 1.4426950408889634f;
    const T *k = static_cast<const T *>(a.k_data) + pl.batch * a.k_batch + pl.k_row * a.k_token + kv_head * a.k_head + col;
    const T *v = static_cast<const T *>(a.v_data) + pl.batch * a.v_batch + pl.k_row * a.v_token + kv_head * a.v_head + col;
    const int second = lane & 1;
    const bool is_dp = lane & 2;
    for (int j = 0; j < pl.keys; j += 2) {
        float x[2], y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[i] = j + i < mine ? dot8<T>(k, q) : 0.0f;
            y[i] = j + i < mine ? dot8<T>(v, g) : 0.0f;
            k += a.k_token;
            v += a.v_token;
        }
        __syncwarp();
        const float xs = (second ? x[1] : x[0]) + __shfl_xor_sync(0xffffffffu, second ? x[0] : x[1], 1);
        const float ys = (second ? y[1] : y[0]) + __shfl_xor_sync(0xffffffffu, second ? y[0] : y[1], 1);
        float z = (is_dp ? ys : xs) + __shfl_xor_sync(0xffffffffu, is_dp ? xs : ys, 2);
#pragma unroll
        for (int d = 4; d < LANES; d *= 2) z += __shfl_xor_sync(0xffffffffu, z, d);
        const float dp = __shfl_xor_sync(0xffffffffu, z, 2);
        if (!is_dp && j + second < seen) sum = fmaf(exp2_fast(fmaf(z, a.scale_log2, -lse)), dp, sum);
    }
    __syncwarp();
    return sum + __shfl_xor_sync(0xffffffffu, sum, 1);  // in the first two lanes
}

// Where the search of a block of row sums starts: each warp counts the tiles of its share
// of the sequences, and the shares ahead of the one with `index` are passed at once
// (4096 sequences of 128 tokens, 8 heads of 64: 2644 -> 2117 us, the whole backward).
// By the whole block.
__device__ __forceinline__ void skip_shares(const AttnShape &s, bool by_keys, int index, AttnCursor &c)
{
    constexpr int kShares = kSumThreads / 32;
    __shared__ int tiles[kShares], q_tiles[kShares];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int share = (s.sequences / 32 + kShares) / kShares * 32;  // of sequences + 1
    int sum = 0, q_sum = 0;
#pragma unroll 4
    for (int i = lane; i < share; i += 32) {
        const int n = warp * share + i;
        if (n > s.sequences) continue;
        int first, queries, keys;
        packed_span(s.q_offsets, s.sequences, s.q_tokens, n, first, queries);
        packed_span(s.k_offsets, s.sequences, s.k_tokens, n, first, keys);
        sum = add_tiles(sum, ((by_keys ? keys : queries) + kSumTokens - 1) / kSumTokens);
        q_sum = add_tiles(q_sum, (queries + kAttnTile - 1) / kAttnTile);
    }
#pragma unroll
    for (int d = 16; d; d /= 2) {
        sum = add_tiles(sum, __shfl_xor_sync(0xffffffffu, sum, d));
        q_sum = add_tiles(q_sum, __shfl_xor_sync(0xffffffffu, q_sum, d));
    }
    if (lane == 0) {
        tiles[warp] = sum;
        q_tiles[warp] = q_sum;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 0; w < kShares && c.before + tiles[w] <= index; ++w) {
            c.base += share;
            c.before += tiles[w];
            c.q_before = add_tiles(c.q_before, q_tiles[w]);
        }
    }
    __syncthreads();
}

template <typename T, int LANES>
__global__ void __launch_bounds__(kSumThreads, 4) attention_sums_kernel(const AttnBwdArgs a, const unsigned q_blocks)
{
    constexpr int kTeams = kSumThreads / LANES;
    __shared__ AttnPlace place;
    __shared__ int there;
    __shared__ float sums[kSumHeads][kSumTokens + 1];
    __shared__ unsigned most[kSumHeads];  // the largest of each head, as bits (float16)
    const AttnShape &s = a.s;
    const bool values = blockIdx.x >= q_blocks;  // the largest |v| (float16)
    const int from = blockIdx.y * kSumHeads, heads = min(kSumHeads, (values ? s.kv_heads : s.heads) - from);
    pdl_trigger();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.counter = 0;  // of the blocks' items
    if (heads <= 0) return;
    const int index = values ? blockIdx.x - q_blocks : blockIdx.x;
    __shared__ AttnCursor start;
    if (threadIdx.x == 0) start = {0, 0, 0, values};
    if (s.packed && s.sequences >= kShareSequences) skip_shares(s, values, index, start);
    if (threadIdx.x < 32) {
        __syncwarp();
        AttnPlace p;
        const bool ok = values ? find_place<true>(s, index, kSumTokens, p, start)
                               : find_place<false>(s, index, kSumTokens, p, start);
        if (threadIdx.x == 0) {
            place = p;
            there = ok;
        }
    } else if (threadIdx.x - 32 < kSumHeads) {
        most[threadIdx.x - 32] = 0;
    }
    __syncthreads();
    if (!there) return;
    const AttnPlace pl = place;
    const int lane = threadIdx.x % LANES, team = threadIdx.x / LANES;
    const bool mine = lane * 8 < s.dim;
    const int first = pl.tile * kSumTokens, rows = values ? pl.keys : pl.queries;
    const int count = max(0, min(kSumTokens, rows - first));
    const T *const x = values ? static_cast<const T *>(a.v_data) + pl.batch * a.v_batch +
                                    (long long)(pl.k_row + first) * a.v_token + from * a.v_head + lane * 8
                              : static_cast<const T *>(a.g_data) + pl.batch * a.g_batch +
                                    (long long)(pl.q_row + first) * a.g_token + from * a.g_head + lane * 8;
    const long long x_token = values ? a.v_token : a.g_token, x_head = values ? a.v_head : a.g_head;
    const T *const o = static_cast<const T *>(a.out) + pl.batch * a.o_batch +
                       (long long)(pl.q_row + first) * a.o_token + from * a.o_head + lane * 8;
    // rows that count for the largest: of a query that sees a key, of a key that has queries
    const int counted = values ? (pl.queries > 0 ? 0 : INT_MAX)
                        : pl.keys == 0 ? INT_MAX : s.causal ? -pl.shift - first : 0;
    const int all = count * heads;
    const bool few = !values && pl.keys <= kFewKeys;
    for (int base = 0; (kScaled<T> || !few) && base < all; base += kTeams * kSumRows) {  // all threads alike: they shuffle
        Raw8<T> rx[kSumRows], ro[kSumRows];
#pragma unroll
        for (int i = 0; i < kSumRows; ++i) {
            const int r = base + i * kTeams + team, t = r / heads, h = r - t * heads;
            rx[i].w[0] = ro[i].w[0] = make_uint4(0, 0, 0, 0);
            if (!mine || r >= all) continue;
            rx[i].w[0] = *reinterpret_cast<const uint4 *>(x + t * x_token + h * x_head);
            if (!values) ro[i].w[0] = *reinterpret_cast<const uint4 *>(o + t * a.o_token + h * a.o_head);
        }
#pragma unroll
        for (int i = 0; i < kSumRows; ++i) {
            const int r = base + i * kTeams + team, t = r / heads, h = r - t * heads;
            if (!values) {
                float u[8], v[8], sum = 0.0f;
                unpack8<T>(rx[i], u);
                unpack8<T>(ro[i], v);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fmaf(u[e], v[e], sum);
                __syncwarp();
#pragma unroll
                for (int d = LANES / 2; d; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
                if (lane == 0 && r < all) sums[h][t] = sum;
            }
            if constexpr (kScaled<T>) {
                unsigned m = t < counted ? 0 : largest8(rx[i].w[0]);
                __syncwarp();
#pragma unroll
                for (int d = LANES / 2; d; d /= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
                if (lane == 0 && r < all) atomicMax(&most[h], m);
            }
        }
    }
    // a loop of its own, so that the other's registers are enough; float16's sums are written
    // anew by the threads that wrote them
    for (int base = 0; few && base < all; base += kTeams) {
        const int r = base + team, t = r / heads, h = r - t * heads;
        const float sum =
            sum_of_few<T, LANES>(a, pl, first + t, from + h, r < all, x + t * x_token + h * x_head);
        if (lane == 0 && r < all) sums[h][t] = sum;
    }
    __syncthreads();
    if constexpr (kScaled<T>) {
        // hardly a block has more than the others had: most need no atomic in memory
        const int h = threadIdx.x;
        if (h < heads) {
            unsigned *const to = largest_at(a, pl.sequence, values ? from + h : (from + h) / s.group) + values;
            if (most[h] > __ldcg(to)) atomicMax(to, most[h]);
        }
    }
    if (values) return;
    // the sequence's last block also has the rows that its last tile does not have
    const int tiles = tiles_within(a.q_tiles, pl.q_tiles_before, (rows + kAttnTile - 1) / kAttnTile);
    const int end = first + kSumTokens >= rows ? tiles * kAttnTile : min(first + kSumTokens, tiles * kAttnTile);
    const int width = end - first;
    for (int i = threadIdx.x; i < heads * width; i += kSumThreads) {
        const int h = i / width, r = i - h * width, t = first + r, head = from + h;
        float l = -INFINITY, sum = 0.0f;
        if (r < count) {
            const float lse = a.lse[((long long)pl.batch * s.heads + head) * s.q_tokens + pl.q_row + t];
            if (lse != -INFINITY) l = (kScaled<T> ? float(kProbBits) : 0.0f) - lse * 1.4426950408889634f;
            sum = sums[h][r];
        }
        float *const stats =
            a.stats + ((long long)head * a.q_tiles + pl.q_tiles_before + t / kAttnTile) * 2 * kAttnTile;
        stats[t % kAttnTile] = l;
        stats[kAttnTile + t % kAttnTile] = -sum;
    }
}

// ------------------------------------------------------------------ gradients

// Sixteen warps on the tiles, four beside one another on a tile's columns, so that each
// SM partition has four to hide their waits in (with two, 8192 x 8 heads of 64 took
// 370 us); then one warp that copies and one that issues products.
constexpr int kWarps = 16, kColumns = 32;  // columns of a warp's part of a tile
constexpr int kBwdThreads = (kWarps + 2) * 32;

// Barriers of one of the two kinds of work.  Each goes from item to item with its
// phases running on.
struct BwdBarriers {
    uint64_t own_full, own_empty, full[8], empty[8], s_full[2], p_full[2], dp_full, ds_full, done, patched;
};

constexpr int kItemSlots = 4;

// An item: a tile of keys of a key head, or of queries of a head, and what goes over it.
// (Sixteen words: with seventeen, 4096 packed sequences of 128 tokens took 2 % longer.)
struct BwdItem {
    AttnPlace pl;
    int head, part;    // part of the query heads that share a key head
    int from, all;     // keys: tiles of queries, from the first that sees the first key
    int q_head;        // keys: the first query head
    int total;         // tiles that the block goes over
    unsigned u;        // its number
};

struct BwdShared {
    BwdBarriers keys, queries;
    uint64_t item_full[kItemSlots], item_empty[kItemSlots];
    uint64_t keys_stored, drained;
    BwdItem item[kItemSlots], none;  // none: after the last
    AttnCursor cursor;
    unsigned tmem, failed;
};

// Which item comes next: blocks take them from a counter, the longest first, so that
// they end together whatever the lengths (dealt out beforehand, 4 x 4096 queries
// against 2333, 1000, 400 and 1800 keys took 600 us).  The warp that copies asks and
// tells the others of the block what it is through a ring.  In a
// block that failed it takes what is left, for the others to write NaN.
__device__ __forceinline__ bool wait_item(BwdShared &sh, uint64_t *bar, unsigned parity)
{
    return attn_wait_warp(bar, parity, &sh.failed) ||
           __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, kAttnDrainCycles));
}

// By a whole warp.  Causal: falling work, that of the first keys and of the last queries
// before the others; else a head's items one after another, which share its tiles in
// L2, or packed a tile's heads, so that the search has a short way (200 sequences of up
// to 600 tokens, 24 heads of 64: 904 -> 817 us).
template <bool KEYS>
__device__ __forceinline__ void find_item(const AttnBwdArgs &a, unsigned u, BwdItem &w, AttnCursor &cursor)
{
    const AttnShape &s = a.s;
    if (!KEYS) u -= a.key_items;
    w.part = KEYS ? u % a.key_parts : 0;
    if (KEYS) u /= a.key_parts;
    const int all = KEYS ? a.k_tiles : a.q_tiles;
    int index;
    if (s.causal || s.packed) {
        const int heads = KEYS ? s.kv_heads : s.heads;
        w.head = u % heads;
        const int i = u / heads;
        if (s.packed) {
            index = KEYS || !s.causal ? i : all - 1 - i;
        } else {
            const int tiles = all / s.sequences;
            const int tile = KEYS ? i / s.sequences : tiles - 1 - i / s.sequences;
            index = i % s.sequences * tiles + tile;
        }
    } else {
        w.head = u / all;
        index = u % all;
    }
    // packed: fewer tiles than there could be, then without rows
    if (!find_place<KEYS>(s, index, kAttnTile, w.pl, cursor)) w.pl = {};
    const AttnPlace &pl = w.pl;
    if (KEYS) {
        const int per = (s.group + a.key_parts - 1) / a.key_parts, first = pl.tile * kAttnTile;
        w.q_head = w.head * s.group + w.part * per;
        w.all = tiles_within(a.q_tiles, pl.q_tiles_before, (pl.queries + kAttnTile - 1) / kAttnTile);
        w.from = s.causal ? min(max(first - pl.shift, 0) / kAttnTile, w.all) : 0;
        w.total = first < pl.keys ? (w.all - w.from) * max(0, min(per, s.group - w.part * per)) : 0;
    } else {
        int seen = pl.keys;
        if (s.causal) seen = min(seen, min((pl.tile + 1) * kAttnTile, pl.queries) + pl.shift);
        w.total = seen <= 0 ? 0 : (seen + kAttnTile - 1) / kAttnTile;
    }
}

// The copying warp's n-th item; one that is as many as there are or more ends the work.  It
// asks when it has asked for all tiles of the last one, a few before the others have
// gone over them: an item that waited in a block any longer would keep another block
// idle at the end (asked for an item ahead, 8192 x 8 heads of 64 took 375 us for 333).
__device__ __forceinline__ BwdItem publish_item(const AttnBwdArgs &a, BwdShared &sh, unsigned &n)
{
    const unsigned slot = n % kItemSlots;
    BwdItem w{};
    if (threadIdx.x % 32 == 0) w.u = atomicAdd(a.counter, 1u);
    w.u = uniform(w.u);
    if (w.u < a.key_items)
        find_item<true>(a, w.u, w, sh.cursor);
    else if (w.u < a.items)
        find_item<false>(a, w.u, w, sh.cursor);
    if (n >= kItemSlots && !wait_item(sh, &sh.item_empty[slot], (n / kItemSlots - 1) & 1)) return sh.none;
    ++n;
    if (threadIdx.x % 32 == 0) {
        sh.item[slot] = w;
        mbar_arrive(&sh.item_full[slot]);
    }
    return w;
}

// The others' n-th.
__device__ __forceinline__ BwdItem take_item(BwdShared &sh, unsigned &n)
{
    const unsigned slot = n % kItemSlots;
    if (!wait_item(sh, &sh.item_full[slot], (n / kItemSlots) & 1)) return sh.none;
    ++n;
    const BwdItem w = sh.item[slot];
    __syncwarp();
    if (threadIdx.x % 32 == 0) mbar_arrive(&sh.item_empty[slot]);
    return w;
}


template <int DP>
constexpr int key_stages()  // pairs of a query tile and its gradient
{
    return DP == 64 ? 4 : 2;
}
// Rings of keys and of values: a tile of values is free after its product, one of keys
// only after the sums that ds goes into, so they do not wait for one another (in one
// ring of five, heads of 128, values came late: 8192 x 8 heads took 604 us for 538).
template <int DP>
constexpr int key_slots()
{
    return DP == 64 ? 4 : 3;
}
template <int DP>
constexpr int value_slots()
{
    return DP == 64 ? 4 : 2;
}

constexpr int kStatsBytes = 2 * kAttnTile * 4;

template <int DP>
constexpr size_t bwd_smem()
{
    constexpr size_t by_keys = size_t(2 + 2 * key_stages<DP>()) * tile_bytes<DP>() + key_stages<DP>() * kStatsBytes;
    constexpr size_t by_queries = size_t(2 + key_slots<DP>() + value_slots<DP>()) * tile_bytes<DP>();
    return (by_keys > by_queries ? by_keys : by_queries) + sizeof(BwdShared) + 1024;
}

__device__ __forceinline__ void bulk_load(void *dst, const void *src, unsigned bytes, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar))
        : "memory");
}

template <int DP>
__device__ __forceinline__ void load_tile(char *dst, const CUtensorMap *map, int head, int token, int batch,
                                          uint64_t *bar)
{
#pragma unroll
    for (int c = 0; c < DP / kSlabCols; ++c)
        tma_load_4d(dst + c * kSlabBytes, map, c * kSlabCols, head, token, batch, bar);
}

// Zeros in the rows from `rows` on, by a warp.
template <int DP>
__device__ __forceinline__ void zero_rows(char *tile, int rows)
{
    for (int i = rows * 8 + int(threadIdx.x % 32); i < kAttnTile * 8; i += 32)
#pragma unroll
        for (int c = 0; c < DP / kSlabCols; ++c)
            reinterpret_cast<uint4 *>(tile + c * kSlabBytes)[i] = make_uint4(0, 0, 0, 0);
}

// A warp's 32 values of a row as 16 columns of the A operand.
template <typename T>
__device__ __forceinline__ void store_part(unsigned at, const float (&v)[kColumns])
{
    uint32_t w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e] = pack2<T>(v[2 * e], v[2 * e + 1]);
    st16(at, w);
}

// A thread's row of an accumulator, columns [from, to), times `scale` to memory; zeros
// where `none`, NaN where the block failed.
template <typename T>
__device__ __forceinline__ void store_row(unsigned at, int from, int to, float scale, bool none, bool ok, bool mine,
                                          T *out)
{
    for (int i = from; i < to; i += 16) {
        uint32_t r[16];
        __syncwarp();
        ld16(at + i, r);
        wait_ld();
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = !ok ? NAN : none ? 0.0f : __uint_as_float(r[e]) * scale;
#pragma unroll
        for (int h = 0; h < 16; h += 8) {
            if (!mine || i + h >= to) continue;
            float (&q)[8] = *reinterpret_cast<float (*)[8]>(v + h);
            st8<T>(out + i + h, pack8<T>(q));
        }
    }
}

// Adds up the parts of dv and dk, eight columns a thread.
constexpr int kJoinThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) attention_join_keys_kernel(const AttnBwdArgs a)
{
    const AttnShape &s = a.s;
    const long long all = (long long)(s.packed ? 1 : s.sequences) * s.k_tokens * s.kv_heads * s.dim;
    const long long i = ((long long)blockIdx.x * kJoinThreads + threadIdx.x) * 8;
    T *const out = static_cast<T *>(blockIdx.y ? a.dk : a.dv);
    pdl_wait();
    if (i >= all || !out) return;
    float v[8] = {};
    for (int p = 0; p < a.key_parts; ++p) {
        const float4 *const x = reinterpret_cast<const float4 *>(a.parts + (2LL * p + blockIdx.y) * all + i);
        const float4 lo = x[0], hi = x[1];
        v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
        v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
    }
    st8<T>(out + i, pack8<T>(v));
}

// 128 keys of a key head against all queries that see them.  Lanes are keys, columns
// queries.  Tensor memory: scores, then p in their place; dp; dv; dk.  Heads of more than
// 64 columns: ds in dp's place; while the warps form p of a tile, the products of ds of
// the last one run; while they form ds, those of p and the next scores.  Narrower
// heads leave room for two tiles of scores, and beside p for ds: the next scores are
// there when they are wanted, and the next dp waits for nothing but that the last one
// has been read.  A warp may then be a tile ahead of another with p, so that p has a
// barrier for each of the two.
template <typename T, int DP>
__device__ __forceinline__ void by_keys(const AttnBwdArgs &a, char *base, BwdShared &sh, int warp, unsigned tmem,
                                        unsigned &n, BwdItem &w, bool &ok)
{
    constexpr int kTile = tile_bytes<DP>();
    constexpr int kStages = key_stages<DP>();
    const AttnShape &s = a.s;
    BwdBarriers &bar = sh.keys;
    volatile unsigned *const failed = &sh.failed;
    constexpr bool kTwo = DP == 64;
    const unsigned s_at = tmem, dp_at = tmem + (kTwo ? 256 : 128), dv_at = dp_at + 128, dk_at = dv_at + DP;
    char *const ring = base + 2 * kTile;
    char *const ring_stats = ring + 2 * kStages * kTile;
    const int lane = threadIdx.x % 32;

    if (warp == kWarps) {
        int it = 0;
        unsigned uses = 0, patches = 0;
        for (; w.u < a.key_items; w = publish_item(a, sh, n)) {
            if (!ok) continue;
            const AttnPlace pl = w.pl;
            const int kv_head = w.head, q_head = w.q_head, from = w.from, all = w.all, total = w.total;
            const int first = pl.tile * kAttnTile;
            for (int i = 0, g = 0, t = from; ok && i < total; ++i, ++it) {
                // the ring runs on while the last item's keys are still in use; they are
                // asked for before the ring would wait for their products
                if (i == min(kStages - 1, total - 1)) {
                    if (uses > 0) ok = attn_wait_warp(&bar.own_empty, (uses - 1) & 1, failed);
                    if (!ok) break;
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&bar.own_full, 2 * kTile + a.extra);
                        load_tile<DP>(base, &a.k, kv_head, pl.k_row + first, pl.batch, &bar.own_full);
                        load_tile<DP>(base + kTile, &a.v, kv_head, pl.k_row + first, pl.batch, &bar.own_full);
                    }
                    ++uses;
                }
                const int stage = it % kStages, head = q_head + g;
                if (it >= kStages) ok = attn_wait_warp(&bar.empty[stage], (it / kStages - 1) & 1, failed);
                if (!ok) break;
                // rows behind the sequence's are another's: zeros in their place
                const int rows = pl.queries - t * kAttnTile;
                const bool patch = s.packed && rows < kAttnTile;
                char *const tile = ring + 2 * stage * kTile;
                if (lane == 0) {
                    uint64_t *const to = patch ? &bar.patched : &bar.full[stage];
                    mbar_arrive_expect_tx(to, 2 * kTile + kStatsBytes);
                    load_tile<DP>(tile, &a.q, head, pl.q_row + t * kAttnTile, pl.batch, to);
                    load_tile<DP>(tile + kTile, &a.g, head, pl.q_row + t * kAttnTile, pl.batch, to);
                    bulk_load(ring_stats + stage * kStatsBytes,
                              a.stats + ((long long)head * a.q_tiles + pl.q_tiles_before + t) * 2 * kAttnTile,
                              kStatsBytes, to);
                }
                if (patch) {
                    ok = attn_wait_warp(&bar.patched, patches++ & 1, failed);
                    zero_rows<DP>(tile, rows);
                    zero_rows<DP>(tile + kTile, rows);
                    fence_proxy();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.full[stage]);
                }
                if (++t == all) {
                    t = from;
                    ++g;
                }
            }
        }
        if (!ok || !a.queries_wanted) {  // what is in flight lands before the block ends
            if (uses > 0) mbar_wait_bounded(&bar.own_full, (uses - 1) & 1, kAttnDrainCycles);
            for (int i = max(0, it - kStages); i < it; ++i)
                mbar_wait_bounded(&bar.full[i % kStages], (i / kStages) & 1, kAttnDrainCycles);
        } else if (uses > 0) {
            // the other kind's tiles take the place of these
            ok = attn_wait_warp(&bar.own_empty, (uses - 1) & 1, failed);
        }
    } else if (warp == kWarps + 1) {
        const unsigned leader = elect_leader();
        const int steps = (s.dim + 15) / 16;
        const unsigned id_s = instr_desc<T>(kAttnTile, false), id_d = instr_desc<T>(steps * 16, true);
        const unsigned s_full = smem_u32(bar.s_full), dp_full = smem_u32(&bar.dp_full), empty = smem_u32(bar.empty);
        const Desc k_tile = desc_k(smem_u32(base)), v_tile = advance(k_tile, kTile);
        const Desc ring_k = desc_k(smem_u32(ring)), ring_mn = desc_mn(smem_u32(ring));
        // places in the ring: of the next tile of queries for scores, for dp, and of the one
        // that p and ds are waiting for
        RingAt<kStages> at, dp_of, sum_of;
        unsigned uses = 0, phase = 0, scored = 0, tiles = 0;
        const auto scores = [&] {
            if (!attn_wait_warp(&bar.full[at.slot], at.parity, failed)) return false;
            const unsigned buf = kTwo ? scored & 1 : 0;
            product_k<DP / 16>(s_at + buf * 128, k_tile, advance(ring_k, 2 * at.slot * kTile), steps, id_s, leader);
            commit(s_full + 8 * buf, leader);
            ++scored;
            at.next();
            return true;
        };
        const auto products = [&] {  // of a tile that has its scores: it is here
            product_k<DP / 16>(dp_at, v_tile, advance(ring_k, (2 * dp_of.slot + 1) * kTile), steps, id_s, leader);
            commit(dp_full, leader);
            dp_of.next();
        };
        for (; uniform(w.u) < a.key_items; w = take_item(sh, n)) {
            const int total = uniform(w.total);
            if (!ok || total == 0) continue;
            ok = attn_wait_warp(&bar.own_full, uses++ & 1, failed);
            if (!ok) continue;
            fence_after();
            if (!(ok = scores())) continue;
            products();
            if (kTwo && total > 1 && !(ok = scores())) continue;
            for (int it = 0; it < total; ++it, phase ^= 1) {
                const Desc tile = advance(ring_mn, 2 * sum_of.slot * kTile);
                const unsigned p_at = s_at + (kTwo ? phase * 128 : 0), ds_at = kTwo ? p_at + 16 : dp_at;
                const bool more = it + 1 < total;
                if (!(ok = attn_wait_warp(&bar.p_full[kTwo ? phase : 0], kTwo ? tiles >> 1 & 1 : phase, failed))) break;
                ++tiles;
                fence_after();
                product_parts(dv_at, p_at, advance(tile, kTile), id_d, it > 0, leader);
                if (!kTwo && more && !(ok = scores())) break;
                if (!(ok = attn_wait_warp(&bar.ds_full, phase, failed))) break;
                fence_after();
                if (kTwo && more) products();
                product_parts(dk_at, ds_at, tile, id_d, it > 0, leader);
                commit(empty + 8 * sum_of.slot, leader);
                sum_of.next();
                if (!kTwo && more) products();
                if (kTwo && it + 2 < total && !(ok = scores())) break;
            }
            if (!ok) continue;
            commit(smem_u32(&bar.done), leader);
            commit(smem_u32(&bar.own_empty), leader);
        }
    } else {
        const int part = warp / 4, row = threadIdx.x % 128;
        const unsigned lanes = unsigned(warp % 4) << 21;
        const unsigned my_dp = dp_at + lanes + part * kColumns;
        const f32x2 c2 = both(a.scale_log2);
        RingAt<kStages> at;
        unsigned uses = 0, phase = 0, tiles = 0;
        for (; w.u < a.key_items; w = take_item(sh, n)) {
            const int total = w.total;
            const uint2 largest = ask_largest<T>(a, w.pl.sequence, w.head);
            int bits = 0;  // ds times 2^bits (float16)
            // columns before hidden0 - 128 t are queries of tile t that do not see this key
            const int key0 = w.pl.tile * kAttnTile + row;
            const int hidden0 = key0 >= w.pl.keys ? INT_MAX
                                : s.causal         ? max(key0 - w.pl.shift - part * kColumns, 0)
                                                   : 0;
            // a query that sees one key has p = 1 and ds = 0, exactly: all of a sequence with
            // one key, or the first that sees any, which sees the first key
            const int alone = w.pl.keys == 1 ? kAttnTile : s.causal && key0 == 0 && w.pl.shift <= 0 ? 1 : 0;
            for (int it = 0, t = w.from; ok && it < total; ++it, phase ^= 1) {
                const float *const stats =
                    reinterpret_cast<const float *>(ring_stats + at.slot * kStatsBytes) + part * kColumns;
                const int hidden = hidden0 == INT_MAX ? kColumns : hidden0 - t * kAttnTile;
                // its column among these, or those of all its tiles
                const int blank = alone > 1 ? kColumns : alone ? 1 - w.pl.shift - part * kColumns - t * kAttnTile : hidden;
                const bool masked = __any_sync(0xffffffffu, max(hidden, blank) > 0);
                const unsigned my_s = s_at + lanes + (kTwo ? phase * 128 : 0) + part * kColumns;
                ok = attn_wait_warp(&bar.full[at.slot], at.parity, failed) &&
                     attn_wait_warp(&bar.s_full[kTwo ? phase : 0], kTwo ? tiles >> 1 & 1 : phase, failed);
                if (!ok) break;
                ++tiles;
                at.next();
                fence_after();
                float p[kColumns];
                ld32(my_s, reinterpret_cast<uint32_t *>(p));
                wait_ld();
#pragma unroll
                for (int i = 0; i < kColumns; i += 4) {
                    const float4 l = *reinterpret_cast<const float4 *>(stats + i);
                    const float2 x = halves(fma2(pair(p[i], p[i + 1]), c2, pair(l.x, l.y)));
                    const float2 y = halves(fma2(pair(p[i + 2], p[i + 3]), c2, pair(l.z, l.w)));
                    p[i] = exp2_fast(x.x);
                    p[i + 1] = exp2_fast(x.y);
                    p[i + 2] = exp2_fast(y.x);
                    p[i + 3] = exp2_fast(y.y);
                }
                if (masked) {
#pragma unroll
                    for (int i = 0; i < kColumns; ++i) p[i] = i < hidden ? 0.0f : p[i];
                }
                store_part<T>(my_s, p);
                wait_st();
                fence_before();
                mbar_arrive(&bar.p_full[kTwo ? phase : 0]);
                ok = attn_wait_warp(&bar.dp_full, phase, failed);
                if (!ok) break;
                fence_after();
                if (kScaled<T> && it == 0) bits = scale_bits(largest, s.dim);
                const f32x2 up2 = both(power_of_two(bits - kProbBits));  // p is there times 2^kProbBits
                float d[kColumns];
                ld32(my_dp, reinterpret_cast<uint32_t *>(d));
                wait_ld();
#pragma unroll
                for (int i = 0; i < kColumns; i += 4) {
                    const float4 m = *reinterpret_cast<const float4 *>(stats + kAttnTile + i);
                    f32x2 x = add2(pair(d[i], d[i + 1]), pair(m.x, m.y));
                    f32x2 y = add2(pair(d[i + 2], d[i + 3]), pair(m.z, m.w));
                    if constexpr (kScaled<T>) {
                        x = mul2(x, up2);
                        y = mul2(y, up2);
                    }
                    const float2 e = halves(mul2(x, pair(p[i], p[i + 1])));
                    const float2 f = halves(mul2(y, pair(p[i + 2], p[i + 3])));
                    d[i] = e.x;
                    d[i + 1] = e.y;
                    d[i + 2] = f.x;
                    d[i + 3] = f.y;
                }
                if (masked) {
#pragma unroll
                    for (int i = 0; i < kColumns; ++i) d[i] = i < blank ? 0.0f : d[i];
                }
                store_part<T>(kTwo ? my_s + 16 : my_dp, d);
                wait_st();
                fence_before();
                mbar_arrive(&bar.ds_full);
                if (++t == w.all) t = w.from;
            }
            if (total > 0 && ok) ok = attn_wait_warp(&bar.done, uses & 1, failed);
            uses += total > 0;
            fence_after();
            const AttnPlace pl = w.pl;
            const int key = pl.tile * kAttnTile + row, count = s.packed ? pl.keys : s.k_tokens;
            const bool mine = key < count, none = total == 0 || key >= pl.keys;
            const long long out_at = ((long long)pl.batch * s.k_tokens + pl.k_row + key) * s.kv_heads + w.head;
            // two parts store dv, two dk, half of the columns each
            const bool is_dk = part >= 2;
            const int cut = min(s.dim, (s.dim / 2 + 15) / 16 * 16);
            const unsigned at_sum = (is_dk ? dk_at : dv_at) + lanes;
            const int c0 = part & 1 ? cut : 0, c1 = part & 1 ? s.dim : cut;
            float scale = is_dk ? a.scale : 1.0f;
            if constexpr (kScaled<T>) scale *= power_of_two(is_dk ? -bits : -kProbBits);
            if (a.key_parts == 1) {
                T *const out = static_cast<T *>(is_dk ? a.dk : a.dv);
                store_row<T>(at_sum, c0, c1, scale, none, ok, mine && out, out + out_at * s.dim);
            } else {
                const long long all = (long long)(s.packed ? 1 : s.sequences) * s.k_tokens * s.kv_heads;
                float *const out = a.parts + ((2LL * w.part + is_dk) * all + out_at) * s.dim;
                store_row<float>(at_sum, c0, c1, scale, none, ok, mine, out);
            }
        }
        // the sums are read: tensor memory is the other kind's
        fence_before();
        mbar_arrive(&sh.keys_stored);
    }
}

// 128 queries of a head against all keys that they see.  Lanes are queries, columns
// keys.  Tensor memory: two tiles of scores, so that the next one's are there when
// they are wanted, then ds in their place, so that the next dp waits for nothing but
// that the last one has been read; dp; dq.
template <typename T, int DP>
__device__ __forceinline__ void by_queries(const AttnBwdArgs &a, char *base, BwdShared &sh, int warp, unsigned tmem,
                                           unsigned &n, BwdItem &w, bool &ok)
{
    constexpr int kTile = tile_bytes<DP>();
    constexpr int kKeys = key_slots<DP>(), kValues = value_slots<DP>();
    const AttnShape &s = a.s;
    BwdBarriers &bar = sh.queries;
    volatile unsigned *const failed = &sh.failed;
    const unsigned s_at = tmem, dp_at = tmem + 256, dq_at = tmem + 384;
    char *const k_ring = base + 2 * kTile, *const v_ring = k_ring + kKeys * kTile;
    uint64_t *const k_full = bar.full, *const v_full = bar.full + kKeys;
    uint64_t *const k_empty = bar.empty, *const v_empty = bar.empty + kKeys;
    const int lane = threadIdx.x % 32;

    if (warp == kWarps) {
        RingAt<kKeys> k_at;
        RingAt<kValues> v_at;
        int issued = 0;  // pairs
        unsigned uses = 0, patches = 0;
        for (; w.u < a.items; w = publish_item(a, sh, n)) {
            if (!ok) continue;
            const AttnPlace pl = w.pl;
            const int total = w.total, head = w.head, kv_head = head / s.group;
            for (int j = 0; ok && j < total; ++j) {
                if (j == min(1, total - 1)) {  // as above
                    if (uses > 0) ok = attn_wait_warp(&bar.own_empty, (uses - 1) & 1, failed);
                    if (!ok) break;
                    if (lane == 0) {
                        const int row = pl.q_row + pl.tile * kAttnTile;
                        mbar_arrive_expect_tx(&bar.own_full, 2 * kTile + a.extra);
                        load_tile<DP>(base, &a.q, head, row, pl.batch, &bar.own_full);
                        load_tile<DP>(base + kTile, &a.g, head, row, pl.batch, &bar.own_full);
                    }
                    ++uses;
                }
                if (issued >= kKeys) ok = attn_wait_warp(&k_empty[k_at.slot], k_at.parity ^ 1, failed);
                if (!ok) break;
                // keys behind the last one may be anything: zeros in their place
                const int rows = pl.keys - j * kAttnTile, row = pl.k_row + j * kAttnTile;
                const bool patch = a.ragged && rows < kAttnTile;
                char *const tile = k_ring + k_at.slot * kTile;
                if (lane == 0) {
                    uint64_t *const to = patch ? &bar.patched : &k_full[k_at.slot];
                    mbar_arrive_expect_tx(to, kTile);
                    load_tile<DP>(tile, &a.k, kv_head, row, pl.batch, to);
                }
                if (patch) {
                    ok = attn_wait_warp(&bar.patched, patches++ & 1, failed);
                    zero_rows<DP>(tile, rows);
                    fence_proxy();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&k_full[k_at.slot]);
                }
                ++issued;
                k_at.next();
                if (ok && issued > kValues) ok = attn_wait_warp(&v_empty[v_at.slot], v_at.parity ^ 1, failed);
                if (lane == 0) {  // also after a failure: both rings have as many on their way
                    mbar_arrive_expect_tx(&v_full[v_at.slot], kTile);
                    load_tile<DP>(v_ring + v_at.slot * kTile, &a.v, kv_head, row, pl.batch, &v_full[v_at.slot]);
                }
                v_at.next();
            }
        }
        // what is in flight lands before the block ends
        if (uses > 0) mbar_wait_bounded(&bar.own_full, (uses - 1) & 1, kAttnDrainCycles);
        for (int i = max(0, issued - kKeys); i < issued; ++i)
            mbar_wait_bounded(&k_full[i % kKeys], (i / kKeys) & 1, kAttnDrainCycles);
        for (int i = max(0, issued - kValues); i < issued; ++i)
            mbar_wait_bounded(&v_full[i % kValues], (i / kValues) & 1, kAttnDrainCycles);
    } else if (warp == kWarps + 1) {
        const unsigned leader = elect_leader();
        const int steps = (s.dim + 15) / 16;
        const unsigned id_s = instr_desc<T>(kAttnTile, false), id_d = instr_desc<T>(steps * 16, true);
        const unsigned s_full = smem_u32(bar.s_full), dp_full = smem_u32(&bar.dp_full);
        const Desc q_tile = desc_k(smem_u32(base)), g_tile = advance(q_tile, kTile);
        const Desc keys_k = desc_k(smem_u32(k_ring)), keys_mn = desc_mn(smem_u32(k_ring));
        const Desc values_k = desc_k(smem_u32(v_ring));
        // the next keys and values, and the keys that ds is waiting for
        RingAt<kKeys> k_at, sum_of;
        RingAt<kValues> v_at;
        unsigned uses = 0, phase = 0, scored = 0;
        const auto scores = [&] {
            if (!attn_wait_warp(&k_full[k_at.slot], k_at.parity, failed)) return false;
            product_k<DP / 16>(s_at + (scored & 1) * 128, q_tile, advance(keys_k, k_at.slot * kTile), steps, id_s,
                               leader);
            commit(s_full + 8 * (scored & 1), leader);
            ++scored;
            k_at.next();
            return true;
        };
        const auto products = [&] {
            if (!attn_wait_warp(&v_full[v_at.slot], v_at.parity, failed)) return false;
            product_k<DP / 16>(dp_at, g_tile, advance(values_k, v_at.slot * kTile), steps, id_s, leader);
            commit(dp_full, leader);
            commit(smem_u32(&v_empty[v_at.slot]), leader);
            v_at.next();
            return true;
        };
        ok = ok && attn_wait_warp(&sh.keys_stored, 0, failed);
        for (; uniform(w.u) < a.items; w = take_item(sh, n)) {
            const int total = uniform(w.total);
            if (!ok || total == 0) continue;
            ok = attn_wait_warp(&bar.own_full, uses++ & 1, failed);
            if (!ok) continue;
            fence_after();
            ok = scores() && products();
            if (ok && total > 1) ok = scores();
            for (int j = 0; ok && j < total; ++j, phase ^= 1) {
                if (!(ok = attn_wait_warp(&bar.ds_full, phase, failed))) break;
                fence_after();
                if (j + 1 < total && !(ok = products())) break;
                product_parts(dq_at, s_at + phase * 128, advance(keys_mn, sum_of.slot * kTile), id_d, j > 0,
                                 leader);
                commit(smem_u32(&k_empty[sum_of.slot]), leader);
                sum_of.next();
                if (j + 2 < total) ok = scores();
            }
            if (!ok) continue;
            commit(smem_u32(&bar.done), leader);
            commit(smem_u32(&bar.own_empty), leader);
        }
    } else {
        const int part = warp / 4, row = threadIdx.x % 128;
        const unsigned lanes = unsigned(warp % 4) << 21;
        const f32x2 c2 = both(a.scale_log2);
        unsigned uses = 0, tiles = 0;
        for (; w.u < a.items; w = take_item(sh, n)) {
            const int total = w.total;
            const float *const stats =
                a.stats + ((long long)w.head * a.q_tiles + w.pl.q_tiles_before + w.pl.tile) * 2 * kAttnTile;
            const f32x2 l2 = both(stats[row]);
            const float less = stats[kAttnTile + row];
            const uint2 largest = ask_largest<T>(a, w.pl.sequence, w.head / s.group);
            int bits = 0;  // as above
            int end = s.causal ? min(w.pl.keys, w.pl.tile * kAttnTile + row + 1 + w.pl.shift) : w.pl.keys;
            if (end == 1) end = 0;  // ds = 0, as above
            for (int j = 0; ok && j < total; ++j, ++tiles) {
                const unsigned my_s = s_at + lanes + (tiles & 1) * 128 + part * kColumns;
                const unsigned my_dp = dp_at + lanes + part * kColumns;
                const int left = end - j * kAttnTile - part * kColumns;
                const bool masked = __any_sync(0xffffffffu, left < kColumns);
                ok = attn_wait_warp(&bar.s_full[tiles & 1], (tiles >> 1) & 1, failed);
                if (!ok) break;
                fence_after();
                float p[kColumns], d[kColumns];
                ld32(my_s, reinterpret_cast<uint32_t *>(p));
                wait_ld();
#pragma unroll
                for (int i = 0; i < kColumns; i += 2) {
                    const float2 x = halves(fma2(pair(p[i], p[i + 1]), c2, l2));
                    p[i] = exp2_fast(x.x);
                    p[i + 1] = exp2_fast(x.y);
                }
                ok = attn_wait_warp(&bar.dp_full, tiles & 1, failed);
                if (!ok) break;
                fence_after();
                if (kScaled<T> && j == 0) bits = scale_bits(largest, s.dim);
                const float up = kScaled<T> ? power_of_two(bits - kProbBits) : 1.0f;
                const f32x2 n2 = both(less * up);
                ld32(my_dp, reinterpret_cast<uint32_t *>(d));
                wait_ld();
#pragma unroll
                for (int i = 0; i < kColumns; i += 2) {
                    f32x2 x = pair(d[i], d[i + 1]);
                    x = kScaled<T> ? fma2(x, both(up), n2) : add2(x, n2);
                    const float2 e = halves(mul2(x, pair(p[i], p[i + 1])));
                    d[i] = e.x;
                    d[i + 1] = e.y;
                }
                if (masked) {
#pragma unroll
                    for (int i = 0; i < kColumns; ++i) d[i] = i < left ? d[i] : 0.0f;
                }
                store_part<T>(my_s, d);
                wait_st();
                fence_before();
                mbar_arrive(&bar.ds_full);
            }
            if (ok && total > 0) ok = attn_wait_warp(&bar.done, uses & 1, failed);
            uses += total > 0;
            fence_after();
            const AttnPlace pl = w.pl;
            const int query = pl.tile * kAttnTile + row;
            const long long out_at = ((long long)pl.batch * s.q_tokens + pl.q_row + query) * s.heads + w.head;
            const float scale = kScaled<T> ? a.scale * power_of_two(-bits) : a.scale;
            store_row<T>(dq_at + lanes, min(s.dim, part * 32), min(s.dim, part * 32 + 32), scale, total == 0, ok,
                         query < pl.queries, static_cast<T *>(a.dq) + out_at * s.dim);
        }
    }
}

template <typename T, int DP>
__global__ void __launch_bounds__(kBwdThreads, 1) attention_bwd_kernel(const __grid_constant__ AttnBwdArgs a)
{
    extern __shared__ char raw[];
    char *const base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    BwdShared &sh = *reinterpret_cast<BwdShared *>(base + bwd_smem<DP>() - 1024 - sizeof(BwdShared));
    const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    if (warp == kWarps && lane == 0) {
        for (const CUtensorMap *m : {&a.q, &a.k, &a.v, &a.g}) prefetch_map(m);
        sh.failed = 0;
        sh.none = {};
        sh.cursor = {};
        sh.none.u = UINT_MAX;
        for (BwdBarriers *b : {&sh.keys, &sh.queries}) {
            for (uint64_t *x : {&b->own_full, &b->own_empty, &b->s_full[0], &b->s_full[1], &b->dp_full, &b->done,
                                &b->patched})
                mbar_init(x, 1);
            for (int i = 0; i < 8; ++i) {
                mbar_init(&b->full[i], 1);
                mbar_init(&b->empty[i], 1);
            }
            mbar_init(&b->p_full[0], kWarps * 32);
            mbar_init(&b->p_full[1], kWarps * 32);
            mbar_init(&b->ds_full, kWarps * 32);
        }
        for (int i = 0; i < kItemSlots; ++i) {
            mbar_init(&sh.item_full[i], 1);
            mbar_init(&sh.item_empty[i], kWarps + 1);
        }
        mbar_init(&sh.keys_stored, kWarps * 32);
        mbar_init(&sh.drained, 1);
        mbar_init_fence();
    }
    if (warp == kWarps + 1) alloc_all(&sh.tmem);
    fence_before();
    __syncthreads();
    fence_after();
    const unsigned tmem = uniform(sh.tmem);
    pdl_wait();  // the row sums
    pdl_trigger();  // what adds up the parts waits for the end of this kernel
    bool ok = true;
    unsigned n = 0;
    BwdItem w = warp == kWarps ? publish_item(a, sh, n) : take_item(sh, n);
    by_keys<T, DP>(a, base, sh, warp, tmem, n, w, ok);
    by_queries<T, DP>(a, base, sh, warp, tmem, n, w, ok);
    if (!ok && warp == kWarps + 1) {
        commit(smem_u32(&sh.drained), elect_leader());
        mbar_wait_bounded(&sh.drained, 0, kAttnDrainCycles);
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    // here, since a wait may have run out in any warp, and after the others had nothing to
    // wait for any more
    if (threadIdx.x == 0 && *static_cast<volatile unsigned *>(&sh.failed)) atomicOr(&g_attention_status, 4u);
    if (warp == kWarps + 1) {
        fence_after();
        free_all(tmem);
    }
}

template <typename T, int DP>
cudaError_t launch(const AttnBwdArgs &a, cudaStream_t stream)
{
    constexpr size_t smem = bwd_smem<DP>();
    static_assert(smem <= 232448, "a block's shared memory");
    static std::atomic<unsigned long long> done{0};
    cudaError_t e = allow_smem(attention_bwd_kernel<T, DP>, done, smem);
    if (e != cudaSuccess) return e;
    if (kScaled<T> && a.largest) {
        e = cudaMemsetAsync(a.largest, 0, size_t(2) * (a.s.sequences + 1) * a.s.kv_heads * sizeof(unsigned), stream);
        if (e != cudaSuccess) return e;
    }
    if (a.q_tiles > 0) {
        const unsigned q_blocks = unsigned(most_tiles(a.s, a.s.q_tokens, kSumTokens));
        const unsigned v_blocks = kScaled<T> ? unsigned(most_tiles(a.s, a.s.k_tokens, kSumTokens)) : 0;
        const dim3 grid(q_blocks + v_blocks, unsigned((a.s.heads + kSumHeads - 1) / kSumHeads));
        const auto kernel = a.s.dim <= 32   ? attention_sums_kernel<T, 4>
                            : a.s.dim <= 64 ? attention_sums_kernel<T, 8>
                                            : attention_sums_kernel<T, 16>;
        kernel<<<grid, kSumThreads, 0, stream>>>(a, q_blocks);
    } else {
        e = cudaMemsetAsync(a.counter, 0, sizeof(unsigned), stream);
        if (e != cudaSuccess) return e;
    }
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (a.items == 0) return cudaSuccess;
    e = launch_after(attention_bwd_kernel<T, DP>, dim3(std::min(a.items, unsigned(kAttnBlocks))), kBwdThreads, smem,
                     stream, a, a.q_tiles > 0);
    if (e != cudaSuccess || a.key_parts == 1) return e;
    const long long n = (long long)(a.s.packed ? 1 : a.s.sequences) * a.s.k_tokens * a.s.kv_heads * a.s.dim / 8;
    return launch_after(attention_join_keys_kernel<T>, dim3(unsigned((n + kJoinThreads - 1) / kJoinThreads), 2),
                        kJoinThreads, 0, stream, a);
}

}  // namespace

cudaError_t attention_bwd_launch(const AttnBwdArgs &a, int dtype, cudaStream_t stream)
{
    if (dtype == GBSSIM_BF16) return a.s.dim <= 64 ? launch<bf16, 64>(a, stream) : launch<bf16, 128>(a, stream);
    return a.s.dim <= 64 ? launch<f16, 64>(a, stream) : launch<f16, 128>(a, stream);
}

cudaError_t attention_bwd_status(unsigned *flags, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(flags, g_attention_status, sizeof(unsigned));
    if (e == cudaSuccess && clear && *flags) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_attention_status, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace gbssim
