// Entry points of attention: argument checks and launch planning.
#include <climits>
#include <cmath>

#include "api_host.cuh"
#include "attention.cuh"
#include "tensor_map.cuh"

using namespace gbssim;

namespace {

struct Extent {
    const void *p;
    size_t bytes;
};

bool meet(const Extent &a, const Extent &b)
{
    return a.bytes && b.bytes && overlaps(a.p, a.bytes, b.p, b.bytes);
}

bool is_packed(const gbssim_attention &d) { return d.q_offsets != nullptr; }
int samples(const gbssim_attention &d) { return is_packed(d) ? 1 : d.sequences; }

long long q_rows(const gbssim_attention &d) { return (long long)samples(d) * d.q_tokens; }
long long k_rows(const gbssim_attention &d) { return (long long)samples(d) * d.k_tokens; }

Extent heads_extent(const gbssim_attention &d, const gbssim_heads &t, int tokens, int heads)
{
    const int n = samples(d);
    if (!t.data || n == 0 || tokens == 0) return {nullptr, 0};
    const long long last = (n - 1) * t.batch_stride + (tokens - 1) * t.token_stride +
                           (heads - 1) * t.head_stride + d.dim;
    return {t.data, size_t(last) * 2};
}

Extent dense_extent(const gbssim_attention &d, const void *p, long long rows, int heads)
{
    return {p, p ? size_t(rows) * heads * d.dim * 2 : 0};
}

Extent floats(const gbssim_attention &d, const float *p)
{
    return {p, p ? size_t(q_rows(d)) * d.heads * 4 : 0};
}

Extent ints(const int *p, int n) { return {p, p ? size_t(n) * 4 : 0}; }

bool multiple16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Strides of extents above one: positive multiples of 16 bytes, below 2^40 bytes.
int check_stride(long long stride, int extent)
{
    if (extent < 2) return GBSSIM_OK;
    if (stride < 1) return GBSSIM_EINVAL;
    if (stride >= (1LL << 39)) return GBSSIM_ESHAPE;
    return stride % 8 ? GBSSIM_EALIGN : GBSSIM_OK;
}

int check_heads(const gbssim_attention &d, const gbssim_heads &t, int tokens, int heads)
{
    const int n = samples(d);
    if (n == 0 || tokens == 0) return GBSSIM_OK;
    if (!t.data) return GBSSIM_EINVAL;
    if (!multiple16(t.data)) return GBSSIM_EALIGN;
    int rc;
    if ((rc = check_stride(t.batch_stride, n)) || (rc = check_stride(t.token_stride, tokens)) ||
        (rc = check_stride(t.head_stride, heads)))
        return rc;
    return GBSSIM_OK;
}

int check_desc(const gbssim_attention *d)
{
    if (!d) return GBSSIM_EINVAL;
    if (d->dtype != GBSSIM_BF16 && d->dtype != GBSSIM_F16) return GBSSIM_EINVAL;
    if (!(d->scale > 0.0f) || !std::isfinite(d->scale)) return GBSSIM_EINVAL;
    if ((d->q_offsets != nullptr) != (d->k_offsets != nullptr)) return GBSSIM_EINVAL;
    if (d->q_offsets && d->kv_lengths) return GBSSIM_EINVAL;
    if (d->sequences < 0 || d->q_tokens < 0 || d->k_tokens < 0) return GBSSIM_ESHAPE;
    if (d->dim < 8 || d->dim > kAttnMaxDim || d->dim % 8) return GBSSIM_ESHAPE;
    if (d->kv_heads < 1 || d->heads < d->kv_heads || d->heads % d->kv_heads) return GBSSIM_ESHAPE;
    if (d->q_tokens > INT_MAX / 4 || d->k_tokens > INT_MAX / 4 || d->sequences > INT_MAX / 4 ||
        d->heads > 65535)
        return GBSSIM_ESHAPE;
    for (const int *p : {d->kv_lengths, d->q_offsets, d->k_offsets})
        if (reinterpret_cast<uintptr_t>(p) % 4) return GBSSIM_EALIGN;
    int rc;
    if ((rc = check_heads(*d, d->q, d->q_tokens, d->heads)) ||
        (rc = check_heads(*d, d->k, d->k_tokens, d->kv_heads)) ||
        (rc = check_heads(*d, d->v, d->k_tokens, d->kv_heads)))
        return rc;
    return GBSSIM_OK;
}

AttnShape shape_of(const gbssim_attention &d)
{
    return {d.sequences, d.q_tokens, d.k_tokens, d.heads, d.kv_heads, d.heads / d.kv_heads, d.dim,
            d.causal != 0, is_packed(d), d.kv_lengths, d.q_offsets, d.k_offsets};
}

// A stride that nothing is read along has to be a valid one all the same.
long long any_stride(long long stride, int extent) { return extent > 1 ? stride : 8; }

bool encode(CUtensorMap &m, const gbssim_attention &d, const gbssim_heads &t, int tokens, int heads,
            int box_heads, int box_tokens)
{
    const int n = samples(d);
    // without a token nothing is read, but the map is a valid one
    const bool none = tokens == 0;
    const void *const some = d.q_tokens ? d.q.data : d.k.data;
    return encode_heads_map(m, none ? some : t.data, d.dtype == GBSSIM_BF16, d.dim, heads,
                            std::max(tokens, 1), n, any_stride(t.head_stride, none ? 1 : heads),
                            any_stride(t.token_stride, tokens), any_stride(t.batch_stride, none ? 1 : n),
                            box_heads, box_tokens);
}

struct FwdPlan {
    int tile_heads, tile_tokens, q_tiles, splits;
    long long tiles, items;
    bool counted;  // items are taken from a counter
};

FwdPlan plan_fwd(const gbssim_attention &d)
{
    const AttnShape s = shape_of(d);
    FwdPlan p{1, kAttnTile, 1, 1, 0, 0, false};
    // a sample whose queries of all the heads of a group fit one tile reads its keys once
    // for the group
    if (!s.packed && s.group > 1 && (long long)s.q_tokens * s.group <= kAttnTile) {
        p.tile_heads = s.group;
        p.tile_tokens = s.q_tokens;
    }
    const long long heads = s.heads / p.tile_heads;
    if (p.tile_heads == 1 && s.q_tokens > kAttnTile &&
        most_tiles(s, s.q_tokens, 2 * kAttnTile) * heads >= kAttnBlocks)
        p.q_tiles = 2;
    const int rows = p.tile_tokens * p.q_tiles;
    p.tiles = s.packed ? most_tiles(s, s.q_tokens, rows) : (s.q_tokens + rows - 1) / rows;
    const long long blocks = p.tiles * samples(d) * heads;
    const long long key_tiles = (s.k_tokens + kAttnTile - 1) / kAttnTile;
    // Few blocks and many keys: parts of two tiles at least, which a tile's 1.1 us and
    // the join's 4 us make worth it from eight tiles on.
    if (!s.packed && blocks > 0 && 2 * blocks <= kAttnBlocks && key_tiles >= 8)
        p.splits = int(std::min<long long>(kAttnBlocks / blocks, key_tiles / 2));
    p.items = blocks * p.splits;
    p.counted = (s.packed || s.kv_lengths) && p.items > 2 * kAttnBlocks;
    return p;
}

size_t fwd_bytes(const gbssim_attention &d, const FwdPlan &p)
{
    if (p.counted) return 16;
    return p.splits == 1 ? 0 : size_t(p.splits) * q_rows(d) * d.heads * (d.dim + 1) * sizeof(float);
}

// An item of keys goes over the queries of all heads that share them: with few key heads
// a few items are long, and the others' blocks wait.  Then several blocks take some of
// the heads each, and their sums are added after them: where the longest item is above
// the average block's work and the parts save more than the 4 us of adding them (a tile
// takes 0.8 us or more; 5 sequences of up to 600 tokens, 24 heads on 3 of 96: 70 us,
// parted 56; 2048 tokens, 32 heads on 4 of 128: 227, 187).
int key_parts(const gbssim_attention &d)
{
    const AttnShape s = shape_of(d);
    if (s.group == 1 || d.q_tokens == 0 || d.k_tokens == 0) return 1;
    const long long n = s.packed ? std::max(1, d.sequences) : 1;  // lengths are not known here
    const auto tiles = [&](int tokens) { return (tokens / n + kAttnTile - 1) / kAttnTile; };
    const long long q = tiles(d.q_tokens), k = tiles(d.k_tokens);
    const long long work = std::max(1, d.sequences) * q * k * (d.kv_heads * s.group + d.heads) / kAttnBlocks;
    const long long longest = q * s.group, most = std::max<long long>(work, 1);
    const int parts = int(std::min<long long>(s.group, (longest + most - 1) / most));
    return parts > 1 && longest - longest / parts >= 6 ? parts : 1;
}

// Of each sequence's key heads, and of the rows behind the last one: the largest |g| and
// |v|, which float16 takes its scales from.
size_t largest_words(const gbssim_attention &d)
{
    return d.dtype == GBSSIM_F16 ? size_t(2) * (d.sequences + 1) * d.kv_heads : 0;
}

// The backward's row sums, in tiles of 128 queries, those, and the counter of items; then
// the parts of dv and dk.
size_t sums_bytes(const gbssim_attention &d)
{
    const long long tiles = d.q_tokens ? most_tiles(shape_of(d), d.q_tokens, kAttnTile) : 0;
    const size_t n = size_t(d.heads) * tiles * 2 * kAttnTile * sizeof(float) +
                     (largest_words(d) + 1) * sizeof(unsigned);
    return (n + 15) / 16 * 16;
}

size_t bwd_bytes(const gbssim_attention &d)
{
    const int parts = key_parts(d);
    return sums_bytes(d) + (parts > 1 ? size_t(2) * parts * k_rows(d) * d.kv_heads * d.dim * sizeof(float) : 0);
}

unsigned g_extra = 0;  // test hook, see gbssim_tune_attention

}  // namespace

extern "C" size_t gbssim_attention_workspace_bytes(const gbssim_attention *d, int backward)
{
    if (check_desc(d) != GBSSIM_OK) return 0;
    if (backward) return q_rows(*d) || k_rows(*d) ? bwd_bytes(*d) : 0;
    if (q_rows(*d) == 0) return 0;
    return fwd_bytes(*d, plan_fwd(*d));
}

extern "C" int gbssim_attention_fwd(const gbssim_attention *d, void *out, float *lse_or_null,
                                    void *workspace, size_t workspace_bytes, void *stream)
{
    const CallRange range("gbssim_attention_fwd");
    int rc = check_desc(d);
    if (rc != GBSSIM_OK) return rc;
    if (q_rows(*d) == 0) return GBSSIM_OK;
    if (!out) return GBSSIM_EINVAL;
    if (!multiple16(out) || reinterpret_cast<uintptr_t>(lse_or_null) % 4) return GBSSIM_EALIGN;
    const FwdPlan p = plan_fwd(*d);
    const size_t need = fwd_bytes(*d, p);
    if (need && (!workspace || !multiple16(workspace) || workspace_bytes < need)) return GBSSIM_EWORKSPACE;
    const Extent in[6] = {heads_extent(*d, d->q, d->q_tokens, d->heads),
                          heads_extent(*d, d->k, d->k_tokens, d->kv_heads),
                          heads_extent(*d, d->v, d->k_tokens, d->kv_heads),
                          ints(d->kv_lengths, d->sequences),
                          ints(d->q_offsets, d->sequences + 1),
                          ints(d->k_offsets, d->sequences + 1)};
    const Extent outs[3] = {dense_extent(*d, out, q_rows(*d), d->heads), floats(*d, lse_or_null),
                            {workspace, need}};
    for (int i = 0; i < 3; ++i) {
        for (const Extent &e : in)
            if (meet(outs[i], e)) return GBSSIM_EINVAL;
        for (int j = 0; j < i; ++j)
            if (meet(outs[i], outs[j])) return GBSSIM_EINVAL;
    }
    const AttnShape s = shape_of(*d);
    if (p.items > INT_MAX || q_rows(*d) * d->heads * (d->dim / 8) / 128 >= INT_MAX) return GBSSIM_ESHAPE;
    AttnFwdArgs a{};
    if (!encode(a.q, *d, d->q, d->q_tokens, d->heads, p.tile_heads, p.tile_tokens) ||
        !encode(a.k, *d, d->k, d->k_tokens, d->kv_heads, 1, kAttnTile) ||
        !encode(a.v, *d, d->v, d->k_tokens, d->kv_heads, 1, kAttnTile))
        return cuda_fail(cudaErrorInvalidValue);
    a.s = s;
    a.scale_log2 = float(double(d->scale) * 1.4426950408889634);
    a.tile_heads = p.tile_heads;
    a.tile_tokens = p.tile_tokens;
    a.splits = p.splits;
    a.tiles = int(p.tiles);
    a.items = unsigned(p.items);
    a.counter = p.counted ? static_cast<unsigned *>(workspace) : nullptr;
    a.ragged = s.packed || s.kv_lengths;
    a.extra = g_extra;
    a.out = out;
    a.lse = lse_or_null;
    a.part_out = static_cast<float *>(workspace);
    a.part_lse = p.splits > 1 ? a.part_out + size_t(p.splits) * q_rows(*d) * d->heads * d->dim : nullptr;
    cudaError_t e = cudaSuccess;
    if (p.counted) e = cudaMemsetAsync(workspace, 0, sizeof(unsigned), static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e);
    e = attention_fwd_launch(a, d->dtype, p.q_tiles, static_cast<cudaStream_t>(stream));
    if (e == cudaSuccess && p.splits > 1)
        e = attention_join_launch(a, d->dtype, static_cast<cudaStream_t>(stream));
    return cuda_fail(e);
}

extern "C" int gbssim_attention_bwd(const gbssim_attention *d, const gbssim_heads *grad_out, const gbssim_heads *out,
                                    const float *lse, void *grad_q_or_null, void *grad_k_or_null,
                                    void *grad_v_or_null, void *workspace, size_t workspace_bytes, void *stream)
{
    const CallRange range("gbssim_attention_bwd");
    int rc = check_desc(d);
    if (rc != GBSSIM_OK) return rc;
    const bool queries = q_rows(*d) > 0, keys = k_rows(*d) > 0;
    if (!queries && !keys) return GBSSIM_OK;
    if (!grad_out || !out || (queries && !lse)) return GBSSIM_EINVAL;
    if ((rc = check_heads(*d, *grad_out, d->q_tokens, d->heads)) ||
        (rc = check_heads(*d, *out, d->q_tokens, d->heads)))
        return rc;
    for (const void *p : {grad_q_or_null, grad_k_or_null, grad_v_or_null})
        if (!multiple16(p)) return GBSSIM_EALIGN;
    if (reinterpret_cast<uintptr_t>(lse) % 4) return GBSSIM_EALIGN;
    const size_t need = bwd_bytes(*d);
    if (need && (!workspace || !multiple16(workspace) || workspace_bytes < need)) return GBSSIM_EWORKSPACE;
    const Extent in[9] = {heads_extent(*d, d->q, d->q_tokens, d->heads),
                          heads_extent(*d, d->k, d->k_tokens, d->kv_heads),
                          heads_extent(*d, d->v, d->k_tokens, d->kv_heads),
                          ints(d->kv_lengths, d->sequences),
                          ints(d->q_offsets, d->sequences + 1),
                          ints(d->k_offsets, d->sequences + 1),
                          heads_extent(*d, *grad_out, d->q_tokens, d->heads),
                          heads_extent(*d, *out, d->q_tokens, d->heads), floats(*d, lse)};
    const Extent outs[4] = {dense_extent(*d, grad_q_or_null, q_rows(*d), d->heads),
                            dense_extent(*d, grad_k_or_null, k_rows(*d), d->kv_heads),
                            dense_extent(*d, grad_v_or_null, k_rows(*d), d->kv_heads),
                            {workspace, need}};
    for (int i = 0; i < 4; ++i) {
        for (const Extent &e : in)
            if (meet(outs[i], e)) return GBSSIM_EINVAL;
        for (int j = 0; j < i; ++j)
            if (meet(outs[i], outs[j])) return GBSSIM_EINVAL;
    }
    const AttnShape s = shape_of(*d);
    const long long q_tiles = queries ? most_tiles(s, d->q_tokens, kAttnTile) : 0;
    const long long k_tiles = keys ? most_tiles(s, d->k_tokens, kAttnTile) : 0;
    if (q_tiles * d->heads + k_tiles * d->heads > INT_MAX || k_rows(*d) * d->kv_heads > INT_MAX || q_tiles + k_tiles > INT_MAX) return GBSSIM_ESHAPE;
    AttnBwdArgs a{};
    if (!encode(a.q, *d, d->q, d->q_tokens, d->heads, 1, kAttnTile) ||
        !encode(a.k, *d, d->k, d->k_tokens, d->kv_heads, 1, kAttnTile) ||
        !encode(a.v, *d, d->v, d->k_tokens, d->kv_heads, 1, kAttnTile) ||
        !encode(a.g, *d, *grad_out, d->q_tokens, d->heads, 1, kAttnTile))
        return cuda_fail(cudaErrorInvalidValue);
    a.s = s;
    a.scale = d->scale;
    a.scale_log2 = float(double(d->scale) * 1.4426950408889634);
    a.q_tiles = int(q_tiles);
    a.k_tiles = int(k_tiles);
    a.ragged = s.packed || s.kv_lengths;
    a.extra = g_extra;
    a.out = out->data;
    a.o_batch = out->batch_stride;
    a.o_token = out->token_stride;
    a.o_head = out->head_stride;
    a.g_data = grad_out->data;
    a.g_batch = grad_out->batch_stride;
    a.g_token = grad_out->token_stride;
    a.g_head = grad_out->head_stride;
    a.v_data = d->v.data;
    a.v_batch = d->v.batch_stride;
    a.v_token = d->v.token_stride;
    a.v_head = d->v.head_stride;
    a.q_data = d->q.data;
    a.q_batch = d->q.batch_stride;
    a.q_token = d->q.token_stride;
    a.q_head = d->q.head_stride;
    a.k_data = d->k.data;
    a.k_batch = d->k.batch_stride;
    a.k_token = d->k.token_stride;
    a.k_head = d->k.head_stride;
    a.lse = lse;
    a.dq = queries ? grad_q_or_null : nullptr;
    a.dk = keys ? grad_k_or_null : nullptr;
    a.dv = keys ? grad_v_or_null : nullptr;
    a.key_parts = queries ? key_parts(*d) : 1;
    a.parts = reinterpret_cast<float *>(static_cast<char *>(workspace) + sums_bytes(*d));
    a.key_items = a.dk || a.dv ? unsigned(k_tiles * d->kv_heads * a.key_parts) : 0;
    if (!a.key_items) a.key_parts = 1;
    a.queries_wanted = a.dq != nullptr;
    a.items = a.key_items + (a.dq ? unsigned(q_tiles * d->heads) : 0);
    a.stats = static_cast<float *>(workspace);
    unsigned *const words = reinterpret_cast<unsigned *>(a.stats + size_t(d->heads) * q_tiles * 2 * kAttnTile);
    a.largest = words;
    a.counter = words + largest_words(*d);
    return cuda_fail(attention_bwd_launch(a, d->dtype, static_cast<cudaStream_t>(stream)));
}

#ifdef GBSSIM_TEST_HOOKS
// ---- test build only (csrc/gbssim_test_hooks.h)
extern "C" void gbssim_tune_attention(int extra_bytes)
{
    g_extra = extra_bytes > 0 ? unsigned(extra_bytes) : 0u;
}
#endif
