// Attention forward: s = scale q k^T, p = softmax over the keys that a query sees,
// o = p v, and each row's log-sum for the backward.
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

struct FwdShared {
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2];
    uint64_t kv_full[8], kv_empty[8], patched, drained;
    AttnPlace place;
    int there;
    unsigned tmem, failed;
};

template <int DP, int QT>
constexpr size_t fwd_smem()
{
    return size_t(QT + stages<DP>()) * tile_bytes<DP>() + sizeof(FwdShared) + 1024;
}

// The rescaling of a row's accumulator is put off until its maximum has grown by
// this much (of the exponent, base 2): probabilities stay below 2^8, which float32
// sums and either 16-bit type hold without loss, and after the first tiles hardly
// any row needs it.
constexpr float kLateMax = 8.0f;

template <typename T, int DP, int QT>
__global__ void __launch_bounds__(QT * 128 + 64, 1) attention_fwd_kernel(const __grid_constant__ AttnFwdArgs a)
{
    using namespace tc;
    constexpr int kStages = stages<DP>();
    constexpr int kTile = tile_bytes<DP>();
    constexpr int kSlabs = DP / kSlabCols;
    extern __shared__ char raw[];
    char *const base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    char *const ring = base + QT * kTile;
    FwdShared &sh = *reinterpret_cast<FwdShared *>(ring + kStages * kTile);

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const AttnShape &s = a.s;
    const int head_blocks = s.heads / a.tile_heads;
    const int tiles = a.tiles, batches = s.packed ? 1 : s.sequences;

    // Blocks of one head follow one another, so that its keys stay in L2; causal ones
    // by falling work instead, the longest first.
    unsigned u = blockIdx.x;
    const int split = u % a.splits;
    u /= a.splits;
    int tile, head, batch;
    if (s.causal) {
        head = u % head_blocks;
        u /= head_blocks;
        batch = u % batches;
        tile = tiles - 1 - u / batches;
    } else {
        tile = u % tiles;
        u /= tiles;
        head = u % head_blocks;
        batch = u / head_blocks;
    }
    const int kv_head = a.tile_heads > 1 ? head : head / s.group;

    if (warp == QT * 4) {
        AttnPlace place;
        const bool there = find_place<false>(s, batch * tiles + tile, a.tile_tokens * QT, place);
        if (lane == 0) {
            sh.place = place;
            sh.there = there;
            sh.failed = 0;
            for (int i = 0; i < QT; ++i) {
                mbar_init(&sh.q_full[i], 1);
                mbar_init(&sh.s_full[i], 1);
                mbar_init(&sh.p_full[i], 128);
                mbar_init(&sh.o_full[i], 1);
            }
            for (int i = 0; i < kStages; ++i) {
                mbar_init(&sh.kv_full[i], 1);
                mbar_init(&sh.kv_empty[i], 1);
            }
            mbar_init(&sh.patched, 1);
            mbar_init(&sh.drained, 1);
            mbar_init_fence();
        }
    }
    if (warp == QT * 4 + 1) alloc_all(&sh.tmem);
    fence_before();
    __syncthreads();
    fence_after();
    const AttnPlace pl = sh.place;
    volatile unsigned *const failed = &sh.failed;
    const unsigned tmem = sh.tmem;

    // this block's key tiles: from j0, per tile of queries to j1[w]
    const int first = pl.tile * a.tile_tokens * QT;
    int j1[QT], last = 0;
    int most = 0;
#pragma unroll
    for (int w = 0; w < QT; ++w) {
        const int rows = min(a.tile_tokens, pl.queries - first - w * a.tile_tokens);
        int seen = pl.keys;
        if (s.causal) seen = min(seen, first + w * a.tile_tokens + rows + pl.shift);
        j1[w] = !sh.there || rows <= 0 || seen <= 0 ? 0 : (seen + kAttnTile - 1) / kAttnTile;
        most = max(most, j1[w]);
    }
    const int per = (most + a.splits - 1) / a.splits, j0 = split * per;
#pragma unroll
    for (int w = 0; w < QT; ++w) {
        j1[w] = max(j0, min(j1[w], j0 + per));
        last = max(last, j1[w]);
    }

    if (warp == QT * 4) {
        // ---- copies: queries, then keys and values in turn
        const unsigned box = unsigned(kSlabs * kRowBytes) * a.tile_heads * a.tile_tokens;
        int issued = 0;
        if (lane == 0 && last > j0) {
            for (int w = 0; w < QT; ++w) {
                if (j1[w] <= j0) continue;
                mbar_arrive_expect_tx(&sh.q_full[w], box + (w == 0 ? a.extra : 0));
                for (int c = 0; c < kSlabs; ++c)
                    tma_load_4d(base + w * kTile + c * kSlabBytes, &a.q, c * kSlabCols,
                                head * a.tile_heads, pl.q_row + first + w * a.tile_tokens, pl.batch,
                                &sh.q_full[w]);
            }
        }
        const int n = 2 * (last - j0);
        bool ok = true;
        for (int it = 0; ok && it < n; ++it) {
            const int slot = it % kStages, j = j0 + it / 2;
            const bool value = it & 1;
            // values behind the last key may be anything: a tile that holds some has them
            // zeroed before it is used, since 0 times an infinity or NaN is not 0
            const bool patch = value && a.ragged && (j + 1) * kAttnTile > pl.keys;
            if (it >= kStages) ok = attn_wait_warp(&sh.kv_empty[slot], (it / kStages - 1) & 1, failed);
            if (!ok) break;
            char *const dst = ring + slot * kTile;
            if (lane == 0) {
                uint64_t *const bar = patch ? &sh.patched : &sh.kv_full[slot];
                mbar_arrive_expect_tx(bar, kTile);
                for (int c = 0; c < kSlabs; ++c)
                    tma_load_4d(dst + c * kSlabBytes, value ? &a.v : &a.k, c * kSlabCols, kv_head,
                                pl.k_row + j * kAttnTile, pl.batch, bar);
            }
            issued = it + 1;
            if (patch) {
                ok = attn_wait_warp(&sh.patched, 0, failed);
                const int rows = pl.keys - j * kAttnTile;  // the last tile: one at least
                for (int i = rows * 8 + lane; i < kAttnTile * 8; i += 32)
                    for (int c = 0; c < kSlabs; ++c)
                        reinterpret_cast<uint4 *>(dst + c * kSlabBytes)[i] = make_uint4(0, 0, 0, 0);
                fence_proxy();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.kv_full[slot]);
            }
        }
        if (*failed && lane == 0) {
            // what is still in flight lands first
            for (int it = max(0, issued - kStages); it < issued; ++it)
                mbar_wait_bounded(&sh.kv_full[it % kStages], (it / kStages) & 1, kAttnDrainCycles);
            atomicOr(&g_attention_status, 4u);
        }
    } else if (warp == QT * 4 + 1) {
        // ---- products
        if (lane == 0 && last > j0) {
            const int k_steps = (s.dim + 15) / 16;
            const unsigned id_s = instr_desc<T>(kAttnTile, false);
            const unsigned id_o = instr_desc<T>(k_steps * 16, true);
            const unsigned ring_u = smem_u32(ring), q_u = smem_u32(base);
            const auto scores = [&](int w, int slot) {
                const unsigned k_tile = ring_u + slot * kTile, q_tile = q_u + w * kTile;
                for (int i = 0; i < k_steps; ++i) {
                    const unsigned at = (i / 4) * kSlabBytes + (i % 4) * kStepK;
                    mma(tmem + w * kAttnTile, desc_k(q_tile + at), desc_k(k_tile + at), id_s, i > 0);
                }
                commit(&sh.s_full[w]);
            };
            bool ok = attn_wait(&sh.kv_full[0], 0, failed);
#pragma unroll
            for (int w = 0; w < QT; ++w) {
                if (!ok || j1[w] <= j0) continue;
                ok = attn_wait(&sh.q_full[w], 0, failed);
                if (ok) scores(w, 0);
            }
            if (ok) commit(&sh.kv_empty[0]);
            for (int j = j0; ok && j < last; ++j) {
                const int it = 2 * (j - j0) + 1, v_slot = it % kStages, k_slot = (it + 1) % kStages;
                const bool more = j + 1 < last;
                ok = attn_wait(&sh.kv_full[v_slot], (it / kStages) & 1, failed);
                if (ok && more) ok = attn_wait(&sh.kv_full[k_slot], ((it + 1) / kStages) & 1, failed);
                const uint64_t v_desc = desc_mn(ring_u + v_slot * kTile, kSlabBytes);
#pragma unroll
                for (int w = 0; w < QT; ++w) {
                    if (!ok || j >= j1[w]) continue;
                    ok = attn_wait(&sh.p_full[w], (j - j0) & 1, failed);
                    if (!ok) continue;
                    fence_after();
                    for (int i = 0; i < kAttnTile / 16; ++i)
                        mma_ta(tmem + QT * kAttnTile + w * DP, tmem + w * kAttnTile + i * 8,
                               advance(v_desc, i * kStepMn), id_o, j > j0 || i > 0);
                    if (j + 1 < j1[w])
                        scores(w, k_slot);
                    else
                        commit(&sh.o_full[w]);
                }
                if (ok) {
                    commit(&sh.kv_empty[v_slot]);
                    if (more) commit(&sh.kv_empty[k_slot]);
                }
            }
            if (!ok) {
                commit(&sh.drained);
                mbar_wait_bounded(&sh.drained, 0, kAttnDrainCycles);
            }
        }
    } else if (sh.there) {
        // ---- softmax: a thread has a row
        const int w = warp / 4, row = threadIdx.x % 128;
        const unsigned lanes = unsigned(warp % 4) << 21;
        const unsigned s_at = tmem + lanes + w * kAttnTile;
        const unsigned o_at = tmem + lanes + QT * kAttnTile + w * DP;
        const int token = first + w * a.tile_tokens + row / a.tile_heads;
        const int row_head = head * a.tile_heads + row % a.tile_heads;
        const bool mine = row < a.tile_tokens * a.tile_heads && token < pl.queries;
        const int seen = s.causal ? min(pl.keys, token + 1 + pl.shift) : pl.keys;
        const int end = QT == 1 || w == 0 ? j1[0] : j1[QT - 1];
        const float c = a.scale_log2;
        float top = -INFINITY, sum = 0.0f;
        bool ok = true;
        for (int j = j0; j < end; ++j) {
            ok = attn_wait_warp(&sh.s_full[w], (j - j0) & 1, failed);
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
            for (int i = 4; i < 128; ++i) m[i % 4] = fmaxf(m[i % 4], v[i]);
            const float now = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * c;
            if (__any_sync(0xffffffffu, now > top + kLateMax)) {
                const float next = fmaxf(top, now);
                const float f = next == -INFINITY ? 1.0f : exp2_fast(top - next);
                top = next;
                sum *= f;
                if (j > j0) {
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
            const float off = top == -INFINITY ? 0.0f : -top;
            float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < 128; i += 32) {
                uint32_t p[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float x = exp2_fast(fmaf(v[i + 2 * e], c, off));
                    const float y = exp2_fast(fmaf(v[i + 2 * e + 1], c, off));
                    part[2 * (e % 2)] += x;
                    part[2 * (e % 2) + 1] += y;
                    p[e] = pack2<T>(x, y);
                }
                st16(s_at + i / 2, p);
            }
            sum += (part[0] + part[1]) + (part[2] + part[3]);
            wait_st();
            fence_before();
            mbar_arrive(&sh.p_full[w]);
        }
        if (ok && end > j0) ok = attn_wait_warp(&sh.o_full[w], 0, failed);
        fence_after();
        const float scale = ok ? (sum == 0.0f ? 0.0f : 1.0f / sum) : NAN;
        const float lse = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
        // dense rows [batch, token, head], of all parts where the keys are split
        const long long at = ((long long)pl.batch * s.q_tokens + pl.q_row + token) * s.heads + row_head;
        const long long rows = (long long)batches * s.q_tokens * s.heads;
        const long long lse_at =
            ((long long)pl.batch * s.heads + row_head) * s.q_tokens + pl.q_row + token;
        T *const out = static_cast<T *>(a.out) + at * s.dim;
        float *const part = a.part_out + (split * rows + at) * s.dim;
        for (int i = 0; i < s.dim; i += 16) {
            uint32_t o[16];
            __syncwarp();
            if (end > j0) {
                ld16(o_at + i, o);
                wait_ld();
            }
            float v[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = end > j0 && sum != 0.0f ? __uint_as_float(o[e]) * scale : (ok ? 0.0f : NAN);
#pragma unroll
            for (int h = 0; h < 16; h += 8) {
                if (!mine || i + h >= s.dim) continue;
                float (&q)[8] = *reinterpret_cast<float (*)[8]>(v + h);
                if (a.splits > 1)
                    st8<float>(part + i + h, pack8<float>(q));
                else
                    st8<T>(out + i + h, pack8<T>(q));
            }
        }
        if (mine && a.splits > 1)
            a.part_lse[split * rows + lse_at] = lse;
        else if (mine && a.lse)
            a.lse[lse_at] = lse;
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    if (warp == QT * 4 + 1) {
        fence_after();
        free_all(tmem);
    }
}

// Joins the parts of the keys: weights exp(lse of the part - lse of the row).  A
// thread has eight columns of a row.
template <typename T>
__global__ void attention_join_kernel(const AttnFwdArgs a)
{
    const AttnShape &s = a.s;
    const int chunks = s.dim / 8;
    const long long rows = (long long)(s.packed ? 1 : s.sequences) * s.q_tokens * s.heads;
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= rows * chunks) return;
    const long long row = i / chunks;
    const int col = int(i - row * chunks) * 8;
    const int head = int(row % s.heads);
    const long long token = row / s.heads;
    const long long lse_at = (token / s.q_tokens * s.heads + head) * s.q_tokens + token % s.q_tokens;
    float top = -INFINITY;
    for (int p = 0; p < a.splits; ++p) top = fmaxf(top, a.part_lse[p * rows + lse_at]);
    float sum = 0.0f, v[8] = {};
    for (int p = 0; p < a.splits; ++p) {
        const float l = a.part_lse[p * rows + lse_at];
        if (l == -INFINITY) continue;
        const float f = expf(l - top);
        const float4 *const o = reinterpret_cast<const float4 *>(a.part_out + (p * rows + row) * s.dim + col);
        const float4 x = o[0], y = o[1];
        sum += f;
        v[0] += f * x.x; v[1] += f * x.y; v[2] += f * x.z; v[3] += f * x.w;
        v[4] += f * y.x; v[5] += f * y.y; v[6] += f * y.z; v[7] += f * y.w;
    }
    const float scale = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= scale;
    st8<T>(static_cast<T *>(a.out) + row * s.dim + col, pack8<T>(v));
    if (a.lse && col == 0) a.lse[lse_at] = sum == 0.0f ? -INFINITY : top + logf(sum);
}

template <typename T, int DP, int QT>
cudaError_t launch(const AttnFwdArgs &a, cudaStream_t stream)
{
    constexpr size_t smem = fwd_smem<DP, QT>();
    static_assert(smem <= 232448, "a block's shared memory");
    static std::atomic<unsigned long long> done{0};
    const cudaError_t e = allow_smem(attention_fwd_kernel<T, DP, QT>, done, smem);
    if (e != cudaSuccess) return e;
    const long long grid = (long long)a.splits * a.tiles * (a.s.packed ? 1 : a.s.sequences) *
                           (a.s.heads / a.tile_heads);
    attention_fwd_kernel<T, DP, QT><<<unsigned(grid), QT * 128 + 64, smem, stream>>>(a);
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
    const long long n = (long long)(a.s.packed ? 1 : a.s.sequences) * a.s.q_tokens * a.s.heads * (a.s.dim / 8);
    const unsigned grid = unsigned((n + 127) / 128);
    if (dtype == GBSSIM_BF16)
        attention_join_kernel<bf16><<<grid, 128, 0, stream>>>(a);
    else
        attention_join_kernel<f16><<<grid, 128, 0, stream>>>(a);
    return cudaGetLastError();
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
