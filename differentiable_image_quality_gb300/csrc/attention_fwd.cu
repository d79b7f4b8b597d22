// Attention forward: s = scale q k^T, p = softmax over the keys that a query sees,
// o = p v, and each row's log-sum for the backward.
//
// One pass over the keys in tiles of 128 with each row's running maximum and sum, so
// that scores never leave the SM.  Per tile of 128 queries and 128 keys of 128 columns
// the tensor cores take 1024 cycles for the two products, an SM partition's exponential
// unit 512 and its issue slots about 400 for the softmax, which depends on the first
// product and feeds the second: so a block has two tiles of queries, one's softmax
// beside the other's products, the sums in tensor memory, keys and values in a ring of
// tiles that the copy unit runs ahead in.  16384 causal tokens, 16 heads of 128: 568 us,
// 1.94 PFLOP/s, bound by the tensor cores (642 in long runs, by power); heads of 64 (8192, 16 heads: 282 us) by both
// units at about half; one token over 65536 keys (268 MB) 45 us, bound by memory.
#include <climits>

#include "attention.cuh"

namespace gbssim {
namespace {

__device__ unsigned g_attention_status;

constexpr int kStages64 = 8, kStages128 = 5;

template <int DP>
constexpr int stages()
{
    return DP == 64 ? kStages64 : kStages128;
}

template <int DP>
constexpr int tile_bytes()
{
    return DP / tc::kSlabCols * tc::kSlabBytes;
}

// One block's share of the work: a tile (or two) of queries of a head, against some of
// the keys.
template <int QT>
struct FwdItem {
    AttnPlace pl;
    int head, kv_head, split;
    int first;           // query
    int j0, j1[QT], end; // key tiles: from j0, per tile of queries to j1
    unsigned u;          // its number
};

constexpr int kItemSlots = 4;

template <int QT>
struct FwdShared {
    uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][2], o_full[2];
    uint64_t kv_full[8], kv_empty[8], patched, drained;
    uint64_t item_full[kItemSlots], item_empty[kItemSlots];
    FwdItem<QT> item[kItemSlots], none;  // none: after the last
    AttnCursor cursor;
    unsigned tmem, failed;
};

template <int DP, int QT>
constexpr size_t fwd_smem()
{
    return size_t(QT + stages<DP>()) * tile_bytes<DP>() + sizeof(FwdShared<QT>) + 1024;
}

// The rescaling of a row's accumulator is put off until its maximum has grown by
// kLate (of the exponent, base 2), so that after the first tiles hardly any row needs it:
// probabilities stay below 2^kLate, which float32 sums and bfloat16 hold without loss.
// float16 has room for little below 2^-14: there they go into their product times 2^kUp,
// up to 2^15 together, so that what is 2^-25 of a row's largest keeps all its digits and
// the least step is 2^-35 of it.  (8 x 1024, 16 heads of 72: 50.5 us with 8 and 7, 50.5
// so, 51.8 with 3 and 12, 57.4 with 2 and 13; 8192, 16 heads of 64, scores of standard
// deviation 3: 275, 290, 293, 297.)
template <typename T>
constexpr float kLate = std::is_same<T, f16>::value ? 4.0f : 8.0f;
template <typename T>
constexpr float kUp = std::is_same<T, f16>::value ? 11.0f : 0.0f;

// The index-th of the call's, by a whole warp.  Those of one head follow one another,
// so that its keys stay in L2; causal ones by falling work instead, the longest first.
// Packed, a tile's heads follow one another, so that the search has a short way (24
// sequences of up to 1500 tokens, 16 heads of 64: 95 -> 91 us; 200 of up to 600, 24 heads
// of 64: 318 -> 276).
template <int QT>
__device__ __forceinline__ void find_item(const AttnFwdArgs &a, unsigned u, FwdItem<QT> &w, AttnCursor &cursor)
{
    const AttnShape &s = a.s;
    const int head_blocks = s.heads / a.tile_heads;
    const int batches = s.packed ? 1 : s.sequences;
    w.split = u % a.splits;
    u /= a.splits;
    int tile, batch;
    if (s.causal) {
        w.head = u % head_blocks;
        u /= head_blocks;
        batch = u % batches;
        tile = a.tiles - 1 - u / batches;
    } else if (s.packed) {
        w.head = u % head_blocks;
        tile = u / head_blocks;
        batch = 0;
    } else {
        tile = u % a.tiles;
        u /= a.tiles;
        w.head = u % head_blocks;
        batch = u / head_blocks;
    }
    w.kv_head = a.tile_heads > 1 ? w.head : w.head / s.group;
    if (!find_place<false>(s, batch * a.tiles + tile, a.tile_tokens * QT, w.pl, cursor)) {
        w.pl = {};  // packed: fewer tiles than there could be
    }
    w.first = w.pl.tile * a.tile_tokens * QT;
    int most = 0;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int from = w.first + t * a.tile_tokens;
        const int rows = min(a.tile_tokens, w.pl.queries - from);
        int seen = w.pl.keys;
        if (s.causal) seen = min(seen, from + rows + w.pl.shift);
        w.j1[t] = rows <= 0 || seen <= 0 ? 0 : (seen + kAttnTile - 1) / kAttnTile;
        most = max(most, w.j1[t]);
    }
    const int per = (most + a.splits - 1) / a.splits;
    w.j0 = w.split * per;
    w.end = w.j0;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        w.j1[t] = max(w.j0, min(w.j1[t], w.j0 + per));
        w.end = max(w.end, w.j1[t]);
    }
}

// A block's n-th item: to and fro, so that falling work evens out between the blocks.
__device__ __forceinline__ unsigned item_of(unsigned n)
{
    return n * gridDim.x + (n & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

template <int QT>
__device__ __forceinline__ bool wait_item(FwdShared<QT> &sh, uint64_t *bar, unsigned parity)
{
    return attn_wait_warp(bar, parity, &sh.failed) ||
           __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, kAttnDrainCycles));
}

// The copying warp's n-th item, told to the others of the block through a ring: dealt out
// beforehand, or where lengths differ taken from a counter, so that the blocks end
// together (24 sequences of up to 1500 tokens, 16 heads of 64: 115 us dealt out, 96 taken;
// setting the counter costs 2 us).  One that is as many as there are or more ends the
// work.  A block that failed takes what is left, for its rows to become NaN.
template <int QT>
__device__ __forceinline__ FwdItem<QT> publish_item(const AttnFwdArgs &a, FwdShared<QT> &sh, unsigned &n)
{
    const unsigned slot = n % kItemSlots;
    FwdItem<QT> w{};
    if (a.counter) {
        if (threadIdx.x % 32 == 0) w.u = atomicAdd(a.counter, 1u);
        w.u = uniform(w.u);
    } else {
        w.u = item_of(n);
    }
    if (w.u < a.items) find_item(a, w.u, w, sh.cursor);
    if (n >= kItemSlots && !wait_item(sh, &sh.item_empty[slot], (n / kItemSlots - 1) & 1)) return sh.none;
    ++n;
    if (threadIdx.x % 32 == 0) {
        sh.item[slot] = w;
        tc::mbar_arrive(&sh.item_full[slot]);
    }
    return w;
}

// The others' n-th.
template <int QT>
__device__ __forceinline__ FwdItem<QT> take_item(FwdShared<QT> &sh, unsigned &n)
{
    const unsigned slot = n % kItemSlots;
    if (!wait_item(sh, &sh.item_full[slot], (n / kItemSlots) & 1)) return sh.none;
    ++n;
    const FwdItem<QT> w = sh.item[slot];
    __syncwarp();
    if (threadIdx.x % 32 == 0) tc::mbar_arrive(&sh.item_empty[slot]);
    return w;
}

// Threads: four warps for each tile of queries, then a warp that copies, one that issues
// products and, beside two tiles, two that only give their registers up.
template <int QT>
constexpr int fwd_threads()
{
    return QT * 128 + (QT == 2 ? 128 : 64);
}
// Registers of a thread at the launch (168), and after the warps without tiles have
// given some up: 2 x 208 + 88 = 3 x 168.
constexpr int kTileRegisters = 208, kOtherRegisters = 88;

template <typename T, int DP, int QT>
__global__ void __launch_bounds__(fwd_threads<QT>(), 1) attention_fwd_kernel(const __grid_constant__ AttnFwdArgs a)
{
    using namespace tc;
    constexpr int kStages = stages<DP>();
    constexpr int kTile = tile_bytes<DP>();
    constexpr int kSlabs = DP / kSlabCols;
    constexpr int kCopy = QT * 4, kIssue = QT * 4 + 1;  // warps
    extern __shared__ char raw[];
    char *const base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    char *const ring = base + QT * kTile;
    FwdShared<QT> &sh = *reinterpret_cast<FwdShared<QT> *>(ring + kStages * kTile);

    const int warp = uniform(threadIdx.x / 32), lane = threadIdx.x % 32;
    const AttnShape &s = a.s;
    if (warp == kCopy && lane == 0) {
        for (const CUtensorMap *m : {&a.q, &a.k, &a.v}) prefetch_map(m);
        sh.failed = 0;
        for (int i = 0; i < QT; ++i) {
            mbar_init(&sh.q_full[i], 1);
            mbar_init(&sh.q_empty[i], 1);
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_full[i][0], 128);
            mbar_init(&sh.p_full[i][1], 128);
            mbar_init(&sh.o_full[i], 1);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.kv_full[i], 1);
            mbar_init(&sh.kv_empty[i], 1);
        }
        for (int i = 0; i < kItemSlots; ++i) {
            mbar_init(&sh.item_full[i], 1);
            mbar_init(&sh.item_empty[i], QT * 4 + 1);
        }
        sh.none = {};
        sh.cursor = {};
        sh.none.u = UINT_MAX;
        mbar_init(&sh.patched, 1);
        mbar_init(&sh.drained, 1);
        mbar_init_fence();
    }
    if (warp == kIssue) alloc_all(&sh.tmem);
    fence_before();
    __syncthreads();
    fence_after();
    volatile unsigned *const failed = &sh.failed;
    const unsigned tmem = uniform(sh.tmem);
    pdl_trigger();  // the parts' join waits for the end of this kernel by itself

    if (warp == kCopy) {
        // ---- copies: queries, then keys and values in turn
        if constexpr (QT == 2) release_registers<kOtherRegisters>();
        const unsigned box = unsigned(kSlabs * kRowBytes) * a.tile_heads * a.tile_tokens;
        int it = 0, patches = 0, uses[QT] = {};
        bool ok = true;
        unsigned n = 0;
        for (FwdItem<QT> w = publish_item(a, sh, n); w.u < a.items; w = publish_item(a, sh, n)) {
            if (!ok) continue;
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                if (!ok || w.j1[t] <= w.j0) continue;
                if (uses[t] > 0) ok = attn_wait_warp(&sh.q_empty[t], (uses[t] - 1) & 1, failed);
                if (!ok) continue;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&sh.q_full[t], box + (t == 0 ? a.extra : 0));
                    for (int c = 0; c < kSlabs; ++c)
                        tma_load_4d(base + t * kTile + c * kSlabBytes, &a.q, c * kSlabCols, w.head * a.tile_heads,
                                    w.pl.q_row + w.first + t * a.tile_tokens, w.pl.batch, &sh.q_full[t]);
                }
                ++uses[t];
            }
            for (int i = 2 * w.j0; ok && i < 2 * w.end; ++i) {
                const int slot = it % kStages, j = i / 2;
                const bool value = i & 1;
                // values behind the last key may be anything: a tile that holds some has them
                // zeroed before it is used, since 0 times an infinity or NaN is not 0
                const bool patch = value && a.ragged && (j + 1) * kAttnTile > w.pl.keys;
                if (it >= kStages) ok = attn_wait_warp(&sh.kv_empty[slot], (it / kStages - 1) & 1, failed);
                if (!ok) break;
                char *const dst = ring + slot * kTile;
                if (lane == 0) {
                    uint64_t *const bar = patch ? &sh.patched : &sh.kv_full[slot];
                    mbar_arrive_expect_tx(bar, kTile);
                    for (int c = 0; c < kSlabs; ++c)
                        tma_load_4d(dst + c * kSlabBytes, value ? &a.v : &a.k, c * kSlabCols, w.kv_head,
                                    w.pl.k_row + j * kAttnTile, w.pl.batch, bar);
                }
                if (patch) {
                    ok = attn_wait_warp(&sh.patched, patches++ & 1, failed);
                    const int rows = w.pl.keys - j * kAttnTile;  // the last tile: one at least
                    for (int e = rows * 8 + lane; e < kAttnTile * 8; e += 32)
                        for (int c = 0; c < kSlabs; ++c)
                            reinterpret_cast<uint4 *>(dst + c * kSlabBytes)[e] = make_uint4(0, 0, 0, 0);
                    fence_proxy();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.kv_full[slot]);
                }
                ++it;
            }
        }
        if (lane == 0) {
            // what is still in flight lands before the block ends
            for (int i = max(0, it - kStages); i < it; ++i)
                mbar_wait_bounded(&sh.kv_full[i % kStages], (i / kStages) & 1, kAttnDrainCycles);
            for (int t = 0; t < QT; ++t)
                if (uses[t] > 0) mbar_wait_bounded(&sh.q_full[t], (uses[t] - 1) & 1, kAttnDrainCycles);
        }
    } else if (warp == kIssue) {
        // ---- products
        if constexpr (QT == 2) release_registers<kOtherRegisters>();
        const unsigned leader = elect_leader();
        const int k_steps = (s.dim + 15) / 16;
        const unsigned id_s = instr_desc<T>(kAttnTile, false);
        const unsigned id_o = instr_desc<T>(k_steps * 16, true);
        const Desc k_ring = desc_k(smem_u32(ring)), v_ring = desc_mn(smem_u32(ring));
        const Desc q_tiles = desc_k(smem_u32(base));
        const unsigned full = smem_u32(sh.kv_full), empty = smem_u32(sh.kv_empty);
        const unsigned q_empty = smem_u32(sh.q_empty), s_full = smem_u32(sh.s_full), o_full = smem_u32(sh.o_full);
        const auto scores = [&](int t, int slot) {
            product_k<DP / 16>(tmem + t * kAttnTile, advance(q_tiles, t * kTile), advance(k_ring, slot * kTile),
                               k_steps, id_s, leader);
            commit(s_full + 8 * t, leader);
        };
        RingAt<kStages> at;
        unsigned uses[QT] = {}, phase[QT] = {};
        bool ok = true;
        const auto keys_here = [&] { return attn_wait_warp(&sh.kv_full[at.slot], at.parity, failed); };
        unsigned n = 0;
        for (FwdItem<QT> w = take_item(sh, n); w.u < a.items; w = take_item(sh, n)) {
            // known to be the same in all lanes
            w.j0 = uniform(w.j0);
            w.end = uniform(w.end);
#pragma unroll
            for (int t = 0; t < QT; ++t) w.j1[t] = uniform(w.j1[t]);
            if (!ok || w.end <= w.j0) continue;
            ok = keys_here();
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                if (!ok || w.j1[t] <= w.j0) continue;
                ok = attn_wait_warp(&sh.q_full[t], uses[t] & 1, failed);
                if (!ok) continue;
                ++uses[t];
                fence_after();
                scores(t, at.slot);
                if (w.j1[t] == w.j0 + 1) commit(q_empty + 8 * t, leader);
            }
            if (ok) commit(empty + 8 * at.slot, leader);
            at.next();
            ok = ok && keys_here();
            for (int j = w.j0; ok && j < w.end; ++j) {
                const int v_slot = at.slot;
                const Desc v_tile = advance(v_ring, v_slot * kTile);
                at.next();
                const bool more = j + 1 < w.end;
                bool here = !more;  // the next keys
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    if (j >= w.j1[t]) continue;
                    const unsigned o_at = tmem + QT * kAttnTile + t * DP, p_at = tmem + t * kAttnTile;
                    // the first half of the probabilities goes ahead of the second; its
                    // threads have read the last item's sums before
                    if (!(ok = ok && attn_wait_warp(&sh.p_full[t][0], phase[t], failed))) continue;
                    fence_after();
                    product_half(o_at, p_at, v_tile, id_o, j > w.j0, leader);
                    if (!(ok = attn_wait_warp(&sh.p_full[t][1], phase[t], failed))) continue;
                    fence_after();
                    product_half(o_at, p_at + 32, advance(v_tile, step_mn(4)), id_o, true, leader);
                    phase[t] ^= 1;
                    if (!here) here = ok = keys_here();
                    if (!ok) continue;
                    if (j + 1 < w.j1[t]) {
                        scores(t, at.slot);
                        if (j + 2 == w.j1[t]) commit(q_empty + 8 * t, leader);
                    } else {
                        commit(o_full + 8 * t, leader);
                    }
                }
                if (!ok) break;
                commit(empty + 8 * v_slot, leader);
                if (more) {
                    commit(empty + 8 * at.slot, leader);
                    at.next();
                    ok = keys_here();
                }
            }
        }
        if (!ok) {
            commit(smem_u32(&sh.drained), leader);
            mbar_wait_bounded(&sh.drained, 0, kAttnDrainCycles);
        }
    } else if (warp < kCopy) {
        // ---- softmax: a thread has a row
        if constexpr (QT == 2) take_registers<kTileRegisters>();
        const int t = warp / 4, row = threadIdx.x % 128;
        const unsigned lanes = unsigned(warp % 4) << 21;
        const unsigned s_at = tmem + lanes + t * kAttnTile;
        const unsigned o_at = tmem + lanes + QT * kAttnTile + t * DP;
        const float c = a.scale_log2;
        const long long rows = (long long)(s.packed ? 1 : s.sequences) * s.q_tokens * s.heads;
        int tiles = 0, uses = 0;
        bool ok = true;
        unsigned n = 0;
        for (FwdItem<QT> w = take_item(sh, n); w.u < a.items; w = take_item(sh, n)) {
            const int token = w.first + t * a.tile_tokens + row / a.tile_heads;
            const int row_head = w.head * a.tile_heads + row % a.tile_heads;
            const bool mine = row < a.tile_tokens * a.tile_heads && token < w.pl.queries;
            const int seen = s.causal ? min(w.pl.keys, token + 1 + w.pl.shift) : w.pl.keys;
            const int end = QT == 1 || t == 0 ? w.j1[0] : w.j1[QT - 1];
            float top = -INFINITY, sum = 0.0f;
            for (int j = w.j0; ok && j < end; ++j) {
                ok = attn_wait_warp(&sh.s_full[t], tiles & 1, failed);
                if (!ok) break;
                fence_after();
                uint32_t r[128];
                float *const v = reinterpret_cast<float *>(r);
#pragma unroll
                for (int i = 0; i < 4; ++i) ld32(s_at + 32 * i, r + 32 * i);
                wait_ld();
                const int left = seen - j * kAttnTile;
                if (__any_sync(0xffffffffu, left < kAttnTile)) {
#pragma unroll
                    for (int i = 0; i < 128; ++i) v[i] = i < left ? v[i] : -INFINITY;
                }
                float m[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
                for (int i = 4; i < 128; i += 2) m[i / 2 % 4] = fmaxf(fmaxf(m[i / 2 % 4], v[i]), v[i + 1]);
                const float now = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * c;
                if (__any_sync(0xffffffffu, now > top + kLate<T>)) {
                    // each row by itself: what else is in the tile (rows that are no query
                    // among them) changes no bit of it
                    const float next = now > top + kLate<T> ? now : top;
                    const float f = next == -INFINITY ? 1.0f : exp2_fast(top - next);
                    top = next;
                    sum *= f;
                    if (j > w.j0) {
                        for (int i = 0; i < DP; i += 16) {
                            uint32_t o[16];
                            ld16(o_at + i, o);
                            wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                            st16(o_at + i, o);
                        }
                    }
                }
                const float off = top == -INFINITY ? 0.0f : kUp<T> - top;
                const f32x2 c2 = both(c), off2 = both(off);
                f32x2 part[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < 128; i += 32) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 x = halves(fma2(pair(v[i + 2 * e], v[i + 2 * e + 1]), c2, off2));
                        const float y = exp2_fast(x.x), z = exp2_fast(x.y);
                        part[e % 2] = add2(part[e % 2], pair(y, z));
                        p[e] = pack2<T>(y, z);
                    }
                    st16(s_at + i / 2, p);
                    if (i % 64 == 32) {
                        wait_st();
                        fence_before();
                        mbar_arrive(&sh.p_full[t][i / 64]);
                    }
                }
                sum += sum2(add2(part[0], part[1]));
                ++tiles;
            }
            const bool some = end > w.j0;
            if (some && ok) ok = attn_wait_warp(&sh.o_full[t], uses & 1, failed);
            uses += some;
            fence_after();
            const float scale = ok ? (sum == 0.0f ? 0.0f : 1.0f / sum) : NAN;
            const float lse =
                !ok ? NAN : sum == 0.0f ? -INFINITY : (top + (log2f(sum) - kUp<T>)) * 0.69314718055994531f;
            // dense rows [batch, token, head], of all parts where the keys are split
            const long long at =
                ((long long)w.pl.batch * s.q_tokens + w.pl.q_row + token) * s.heads + row_head;
            const long long lse_at =
                ((long long)w.pl.batch * s.heads + row_head) * s.q_tokens + w.pl.q_row + token;
            T *const out = static_cast<T *>(a.out) + at * s.dim;
            float *const part = a.part_out + (w.split * rows + at) * s.dim;
            for (int i = 0; i < s.dim; i += 32) {
                uint32_t o[32];
                __syncwarp();
                if (some) {
                    ld32(o_at + i, o);
                    wait_ld();
                }
                float v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    v[e] = some && sum != 0.0f ? __uint_as_float(o[e]) * scale : (ok ? 0.0f : NAN);
#pragma unroll
                for (int h = 0; h < 32; h += 8) {
                    if (!mine || i + h >= s.dim) continue;
                    float (&q)[8] = *reinterpret_cast<float (*)[8]>(v + h);
                    if (a.splits > 1)
                        st8<float>(part + i + h, pack8<float>(q));
                    else
                        st8<T>(out + i + h, pack8<T>(q));
                }
            }
            if (mine && a.splits > 1)
                a.part_lse[w.split * rows + lse_at] = lse;
            else if (mine && a.lse)
                a.lse[lse_at] = lse;
        }
    } else {
        if constexpr (QT == 2) release_registers<kOtherRegisters>();
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    // here, since a wait may have run out in any warp, and after the others had nothing to
    // wait for any more
    if (threadIdx.x == 0 && *failed) atomicOr(&g_attention_status, 4u);
    if (warp == kIssue) {
        fence_after();
        free_all(tmem);
    }
}

// Joins the parts of the keys: weights exp(lse of the part - lse of the row).  A block
// has a row; its threads ask for all parts together, eight columns each, and add up
// in shared memory (a thread to a row's columns, one part after the other: 15 us for
// 32 rows of 19 parts).
constexpr int kJoinThreads = 128, kMostSplits = 152;

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) attention_join_kernel(const AttnFwdArgs a)
{
    __shared__ float weight[kMostSplits];
    __shared__ float sums[kJoinThreads][9];
    const AttnShape &s = a.s;
    const int chunks = s.dim / 8, teams = kJoinThreads / chunks;
    const long long rows = (long long)s.sequences * s.q_tokens * s.heads;  // (a packed batch has no parts)
    const long long row = blockIdx.x;
    const int head = int(row % s.heads);
    const long long token = row / s.heads;
    const long long lse_at = (token / s.q_tokens * s.heads + head) * s.q_tokens + token % s.q_tokens;
    pdl_wait();
    const int team = threadIdx.x / chunks, col = (threadIdx.x - team * chunks) * 8;
    // the first warp: the row's log-sum, and what each part counts
    if (threadIdx.x < 32) {
        float top = -INFINITY, sum = 0.0f;
        for (int p = threadIdx.x; p < a.splits; p += 32) top = fmaxf(top, a.part_lse[p * rows + lse_at]);
#pragma unroll
        for (int d = 16; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        for (int p = threadIdx.x; p < a.splits; p += 32) {
            const float l = a.part_lse[p * rows + lse_at], f = l == -INFINITY ? 0.0f : expf(l - top);
            weight[p] = f;
            sum += f;
        }
#pragma unroll
        for (int d = 16; d; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const float scale = sum == 0.0f ? 0.0f : 1.0f / sum;
        for (int p = threadIdx.x; p < a.splits; p += 32) weight[p] *= scale;
        if (a.lse && threadIdx.x == 0) a.lse[lse_at] = sum == 0.0f ? -INFINITY : top + logf(sum);
    }
    __syncthreads();
    float v[8] = {};
    if (team < teams) {
#pragma unroll 4
        for (int p = team; p < a.splits; p += teams) {
            const float f = weight[p];
            const float4 *const o = reinterpret_cast<const float4 *>(a.part_out + (p * rows + row) * s.dim + col);
            const float4 x = o[0], y = o[1];
            if (f == 0.0f) continue;  // a part without keys
            v[0] += f * x.x; v[1] += f * x.y; v[2] += f * x.z; v[3] += f * x.w;
            v[4] += f * y.x; v[5] += f * y.y; v[6] += f * y.z; v[7] += f * y.w;
        }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[threadIdx.x][e] = v[e];
    __syncthreads();
    if (team > 0) return;
    for (int t = 1; t < teams; ++t)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += sums[t * chunks + threadIdx.x][e];
    st8<T>(static_cast<T *>(a.out) + row * s.dim + col, pack8<T>(v));
}

template <typename T, int DP, int QT>
cudaError_t launch(const AttnFwdArgs &a, cudaStream_t stream)
{
    constexpr size_t smem = fwd_smem<DP, QT>();
    static_assert(smem <= 232448, "a block's shared memory");
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = allow_smem(attention_fwd_kernel<T, DP, QT>, done, smem,
                                     QT == 2 ? 2 * kTileRegisters + kOtherRegisters : 0, 3);
    if (e != cudaSuccess) return e;
    const unsigned grid = std::min(a.items, unsigned(kAttnBlocks));
    attention_fwd_kernel<T, DP, QT><<<grid, fwd_threads<QT>(), smem, stream>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_of(const AttnFwdArgs &a, int q_tiles, cudaStream_t stream)
{
    if (a.s.dim <= 64) return q_tiles == 1 ? launch<T, 64, 1>(a, stream) : launch<T, 64, 2>(a, stream);
    return q_tiles == 1 ? launch<T, 128, 1>(a, stream) : launch<T, 128, 2>(a, stream);
}

}  // namespace

cudaError_t attention_fwd_launch(const AttnFwdArgs &a, int dtype, int q_tiles, cudaStream_t stream)
{
    return dtype == GBSSIM_BF16 ? launch_of<bf16>(a, q_tiles, stream) : launch_of<f16>(a, q_tiles, stream);
}

cudaError_t attention_join_launch(const AttnFwdArgs &a, int dtype, cudaStream_t stream)
{
    const unsigned grid = unsigned((long long)a.s.sequences * a.s.q_tokens * a.s.heads);
    if (dtype == GBSSIM_BF16)
        return launch_after(attention_join_kernel<bf16>, grid, kJoinThreads, 0, stream, a);
    return launch_after(attention_join_kernel<f16>, grid, kJoinThreads, 0, stream, a);
}

cudaError_t attention_fwd_status(unsigned *flags, bool clear)
{
    cudaError_t e = cudaMemcpyFromSymbol(flags, g_attention_status, sizeof(unsigned));
    if (e == cudaSuccess && clear && *flags) {
        const unsigned zero = 0;
        e = cudaMemcpyToSymbol(g_attention_status, &zero, sizeof(unsigned));
    }
    return e;
}

}  // namespace gbssim
