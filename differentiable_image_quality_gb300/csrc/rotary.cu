// Rotary positions with several axes: pair p of a head belongs to an axis and has a
// frequency; at a token whose position on that axis is x the pair (u, v) becomes
// (u cos a - v sin a, u sin a + v cos a), a = x f_p; with -a for the inverse, which is
// also the gradient.
//
// Angles are taken modulo a turn in fixed point: f / (2 pi) as a fraction of 2^64,
// times the position, wraps by itself, so far positions lose nothing; sine and
// cosine then see at most half a turn, in float32.
//
// Bound by memory: every element is read and written once.  A block forms the
// sines and cosines of some tokens once, in shared memory, for all their heads of
// both tensors; a thread keeps those of its eight columns in registers for four
// heads at a time, whose loads are under way together.
#include <algorithm>
#include <climits>
#include <mutex>

#include "api_host.cuh"
#include "dtypes.cuh"

namespace gbssim {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 256, kMaxRotaryDim = 512;
constexpr int kHeadsAtOnce = 4;
constexpr int kNoAngle = 255;  // in an axis's place: the frequency is NaN or infinite

struct RotaryTensor {
    const void *in;
    void *out;
    long long batch, token, head;  // strides of the input, elements
    int heads;
};

struct RotaryArgs {
    RotaryTensor t[2];
    const void *positions;
    const double *frequencies;
    long long pos_batch, pos_token;
    int pos_type, axes, ends[GBSSIM_ROTARY_AXES];  // pairs up to and with each axis
    int batch, tokens, dim, pairs, adjacent;
    float sign;
    int block_tokens;
};

// How a thread's eight columns find their partners.
enum Mode {
    kHalves,     // a chunk of the first half and one of the second, n a multiple of 8
    kAdjacent,   // neighbours: within the chunk
    kWindow,     // eight columns anywhere else in the row, at any offset
    kSingle      // a column a thread: any alignment
};

// The fraction of a turn that a unit of position is, times 2^64.
__device__ __forceinline__ unsigned long long turn_fraction(double f)
{
    double t = f * 0.15915494309189535;  // 1 / (2 pi)
    t -= floor(t);
    return t < 1.0 ? (unsigned long long)(t * 18446744073709551616.0) : 0ull;
}

// cos and sin of position x fraction.
__device__ __forceinline__ float2 turn_of(const RotaryArgs &a, const void *pos, long long at, unsigned long long f)
{
    unsigned long long phase;
    if (a.pos_type == GBSSIM_POS_I32) {
        phase = (unsigned long long)(long long)static_cast<const int *>(pos)[at] * f;
    } else if (a.pos_type == GBSSIM_POS_I64) {
        phase = (unsigned long long)static_cast<const long long *>(pos)[at] * f;
    } else {
        const float x = static_cast<const float *>(pos)[at];
        if (!(fabsf(x) < 9.0e18f)) return make_float2(NAN, NAN);
        // the fraction of |x| has no bit that float32 does not hold; below 2^-32 of a
        // unit it is cut
        const float whole = floorf(fabsf(x));
        const unsigned part = unsigned((fabsf(x) - whole) * 4294967296.0f);
        phase = (unsigned long long)(long long)whole * f + __umul64hi(f, (unsigned long long)part << 32);
        if (x < 0.0f) phase = 0ull - phase;
    }
    float s, c;
    sincospif(float(int(unsigned(phase >> 32))) * 4.656612873077393e-10f, &s, &c);  // 2^-31 half turns
    return make_float2(c, s * a.sign);
}

template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T *p)
{
    Raw8<T> r;
    const uint4 *const w = reinterpret_cast<const uint4 *>(p);
#pragma unroll
    for (int i = 0; i < int(sizeof(r.w) / 16); ++i) r.w[i] = ld_stream16(w + i);
    return r;
}

// Eight columns of a row from `first` on, which may be any; those outside read zeros.
template <typename T>
__device__ __forceinline__ Raw8<T> load_window(const T *row, int first, int dim)
{
    constexpr int kWord = 16 / int(sizeof(T));
    const int w0 = first >= 0 ? first / kWord : -((-first + kWord - 1) / kWord);
    Wide8<T> wide;
#pragma unroll
    for (int i = 0; i < Wide8<T>::kUnits; ++i) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (w0 + i >= 0 && (w0 + i) * kWord < dim) w = reinterpret_cast<const uint4 *>(row)[w0 + i];
        wide.w[4 * i] = w.x;
        wide.w[4 * i + 1] = w.y;
        wide.w[4 * i + 2] = w.z;
        wide.w[4 * i + 3] = w.w;
    }
    return shift_down<T>(wide, first - w0 * kWord);
}

// Table of a token in shared memory: per column the factor of its own value and that
// of its partner's, [2][dim] (kHalves, kAdjacent: per pair, [2][dim / 2 or pairs]).
template <Mode M>
__device__ __forceinline__ int table_width(const RotaryArgs &a)
{
    return M == kWindow ? a.dim : M == kAdjacent ? a.dim / 2 : a.pairs;
}

template <typename T, Mode M>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a)
{
    extern __shared__ __align__(16) float table[];
    __shared__ unsigned long long fraction[kMaxPairs];
    __shared__ unsigned char axis_of[kMaxPairs];
    const int n = a.pairs, width = table_width<M>(a);
    for (int i = threadIdx.x; i < n; i += kThreads) {
        int axis = 0;
        while (i >= a.ends[axis]) ++axis;
        const double f = a.frequencies[i];
        axis_of[i] = static_cast<unsigned char>(isfinite(f) ? axis : kNoAngle);
        fraction[i] = turn_fraction(f);
    }
    const long long rows = (long long)a.batch * a.tokens;
    // lanes of a head: chunks of eight columns (kHalves: of both halves), or columns
    const int lanes = M == kHalves ? n / 8 + (a.dim - 2 * n) / 8 : M == kSingle ? a.dim - n : a.dim / 8;
    const int teams = kThreads / min(lanes, kThreads);
    const int team = threadIdx.x / lanes, lane0 = threadIdx.x - team * lanes;
    const int heads = a.t[0].heads + a.t[1].heads;
    const int groups = (heads + kHeadsAtOnce - 1) / kHeadsAtOnce;

    for (long long base = (long long)blockIdx.x * a.block_tokens; base < rows;
         base += (long long)gridDim.x * a.block_tokens) {
        const int count = int(min((long long)a.block_tokens, rows - base));
        __syncthreads();
        for (int i = threadIdx.x; i < count * n; i += kThreads) {
            const int t = i / n, p = i - t * n;
            const long long row = base + t, b = row / a.tokens;
            const int axis = axis_of[p];
            float2 cs = make_float2(NAN, NAN);
            if (axis != kNoAngle)
                cs = turn_of(a, a.positions, b * a.pos_batch + (row - b * a.tokens) * a.pos_token + axis,
                             fraction[p]);
            float *const own = table + 2 * t * width, *const other = own + width;
            if constexpr (M == kWindow) {
                own[p] = own[p + n] = cs.x;
                other[p] = -cs.y;
                other[p + n] = cs.y;
            } else {
                own[p] = cs.x;
                other[p] = cs.y;
            }
        }
        if constexpr (M == kWindow || M == kAdjacent) {  // columns without a position
            const int turned = M == kWindow ? 2 * n : n, rest = width - turned;
            for (int i = threadIdx.x; i < count * rest; i += kThreads) {
                float *const own = table + 2 * (i / rest) * width + turned + i % rest;
                own[0] = 1.0f;
                own[width] = 0.0f;
            }
        }
        __syncthreads();
        if (team >= teams) continue;
        for (int item = team; item < count * groups; item += teams) {
            const int t = item / groups, first = (item - t * groups) * kHeadsAtOnce;
            const long long row = base + t, b = row / a.tokens, token = row - b * a.tokens;
            const float *const own = table + 2 * t * width, *const other = own + width;
            const auto in = [&](int h) {
                const RotaryTensor &x = h < a.t[0].heads ? a.t[0] : a.t[1];
                return static_cast<const T *>(x.in) + b * x.batch + token * x.token +
                       (h < a.t[0].heads ? h : h - a.t[0].heads) * x.head;
            };
            const auto out = [&](int h) {
                const RotaryTensor &x = h < a.t[0].heads ? a.t[0] : a.t[1];
                return static_cast<T *>(x.out) +
                       (row * x.heads + (h < a.t[0].heads ? h : h - a.t[0].heads)) * a.dim;
            };
            if constexpr (M == kSingle) {
                for (int lane = lane0; lane < a.dim - n; lane += kThreads) {
                    const bool turned = lane < n;
                    const int u = !turned ? lane + n : a.adjacent ? 2 * lane : lane;
                    const int v = a.adjacent ? u + 1 : u + n;
                    const float c = turned ? own[lane] : 1.0f, s = turned ? other[lane] : 0.0f;
                    for (int h = first; h < min(first + kHeadsAtOnce, heads); ++h) {
                        const T *const x = in(h);
                        T *const y = out(h);
                        if (!turned) {
                            y[u] = x[u];
                            continue;
                        }
                        const float xu = to_f32(x[u]), xv = to_f32(x[v]);
                        y[u] = from_f32<T>(xu * c - xv * s);
                        y[v] = from_f32<T>(xu * s + xv * c);
                    }
                }
                continue;
            }
            const int lane = lane0;
            if constexpr (M == kHalves) {
                const int chunks = n / 8;
                if (lane >= chunks) {  // columns without a position
                    const int at = 2 * n + (lane - chunks) * 8;
#pragma unroll
                    for (int i = 0; i < kHeadsAtOnce; ++i)
                        if (first + i < heads) st8<T>(out(first + i) + at, load8<T>(in(first + i) + at));
                    continue;
                }
                float c[8], s[8];
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(own + lane * 8 + e);
                    const float4 y = *reinterpret_cast<const float4 *>(other + lane * 8 + e);
                    c[e] = x.x; c[e + 1] = x.y; c[e + 2] = x.z; c[e + 3] = x.w;
                    s[e] = y.x; s[e + 1] = y.y; s[e + 2] = y.z; s[e + 3] = y.w;
                }
                Raw8<T> u[kHeadsAtOnce], v[kHeadsAtOnce];
#pragma unroll
                for (int i = 0; i < kHeadsAtOnce; ++i)
                    if (first + i < heads) {
                        u[i] = load8<T>(in(first + i) + lane * 8);
                        v[i] = load8<T>(in(first + i) + n + lane * 8);
                    }
#pragma unroll
                for (int i = 0; i < kHeadsAtOnce; ++i)
                    if (first + i < heads) {
                        float x[8], y[8], p[8], q[8];
                        unpack8<T>(u[i], x);
                        unpack8<T>(v[i], y);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            p[e] = x[e] * c[e] - y[e] * s[e];
                            q[e] = x[e] * s[e] + y[e] * c[e];
                        }
                        T *const to = out(first + i) + lane * 8;
                        st8<T>(to, pack8<T>(p));
                        st8<T>(to + n, pack8<T>(q));
                    }
            } else if constexpr (M == kAdjacent) {
                const float4 c = *reinterpret_cast<const float4 *>(own + lane * 4);
                const float4 s = *reinterpret_cast<const float4 *>(other + lane * 4);
                const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
                Raw8<T> u[kHeadsAtOnce];
#pragma unroll
                for (int i = 0; i < kHeadsAtOnce; ++i)
                    if (first + i < heads) u[i] = load8<T>(in(first + i) + lane * 8);
#pragma unroll
                for (int i = 0; i < kHeadsAtOnce; ++i)
                    if (first + i < heads) {
                        float x[8], p[8];
                        unpack8<T>(u[i], x);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            p[2 * e] = x[2 * e] * cc[e] - x[2 * e + 1] * ss[e];
                            p[2 * e + 1] = x[2 * e] * ss[e] + x[2 * e + 1] * cc[e];
                        }
                        st8<T>(out(first + i) + lane * 8, pack8<T>(p));
                    }
            } else if constexpr (M == kWindow) {
                const int at = lane * 8;
                float c[8], s[8];
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(own + at + e);
                    const float4 y = *reinterpret_cast<const float4 *>(other + at + e);
                    c[e] = x.x; c[e + 1] = x.y; c[e + 2] = x.z; c[e + 3] = x.w;
                    s[e] = y.x; s[e + 1] = y.y; s[e + 2] = y.z; s[e + 3] = y.w;
                }
                const bool up = at < n, down = at + 8 > n && at < 2 * n;
                for (int h = first; h < min(first + kHeadsAtOnce, heads); ++h) {
                    const T *const row_in = in(h);
                    float x[8], y[8], z[8];
                    unpack8<T>(load8<T>(row_in + at), x);
                    if (up) unpack8<T>(load_window<T>(row_in, at + n, a.dim), y);
                    if (down) unpack8<T>(load_window<T>(row_in, at - n, a.dim), z);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int j = at + e;
                        // a column without a position keeps its value, whatever lies beside it
                        if (j < 2 * n) x[e] = x[e] * c[e] + (j < n ? y[e] : z[e]) * s[e];
                    }
                    st8<T>(out(h) + at, pack8<T>(x));
                }
            }
        }
    }
}

template <typename T, Mode M>
cudaError_t launch(RotaryArgs a, cudaStream_t stream)
{
    const int width = M == kWindow ? a.dim : M == kAdjacent ? a.dim / 2 : a.pairs;
    const long long rows = (long long)a.batch * a.tokens;
    // enough blocks for eight on each SM before a block takes more than a token
    constexpr int kMostTokens = 16, kBlocks = 152 * 8;
    a.block_tokens = int(std::min<long long>({kMostTokens, std::max<long long>(1, rows / kBlocks),
                                              std::max(1, 4096 / width)}));
    const long long blocks = std::min<long long>(ceil_div(rows, a.block_tokens), kBlocks);
    const size_t smem = size_t(2) * a.block_tokens * width * sizeof(float);
    rotary_kernel<T, M><<<unsigned(blocks), kThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_mode(const RotaryArgs &a, Mode m, cudaStream_t stream)
{
    switch (m) {
    case kHalves: return launch<T, kHalves>(a, stream);
    case kAdjacent: return launch<T, kAdjacent>(a, stream);
    case kWindow: return launch<T, kWindow>(a, stream);
    default: return launch<T, kSingle>(a, stream);
    }
}

struct Extent {
    const void *p;
    size_t bytes;
};

bool meet(const Extent &a, const Extent &b)
{
    return a.bytes && b.bytes && overlaps(a.p, a.bytes, b.p, b.bytes);
}

Extent heads_extent(const gbssim_rotary &d, const gbssim_heads &t, int heads)
{
    if (!heads) return {nullptr, 0};
    const long long last = (d.batch - 1) * t.batch_stride + (d.tokens - 1) * t.token_stride +
                           (heads - 1) * t.head_stride + d.dim;
    return {t.data, size_t(last) * dtype_bytes(d.dtype)};
}

int check_heads(const gbssim_rotary &d, const gbssim_heads &t, int heads)
{
    if (!heads) return GBSSIM_OK;
    if (!t.data) return GBSSIM_EINVAL;
    if (t.batch_stride < 0 || t.token_stride < 0 || t.head_stride < 0) return GBSSIM_EINVAL;
    return reinterpret_cast<uintptr_t>(t.data) % dtype_bytes(d.dtype) ? GBSSIM_EALIGN : GBSSIM_OK;
}

bool whole_words(const gbssim_rotary &d, const gbssim_heads &t, const void *out, int heads)
{
    if (!heads) return true;
    const int word = 16 / dtype_bytes(d.dtype);
    return reinterpret_cast<uintptr_t>(t.data) % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0 &&
           (d.batch < 2 || t.batch_stride % word == 0) && (d.tokens < 2 || t.token_stride % word == 0) &&
           (heads < 2 || t.head_stride % word == 0);
}

}  // namespace
}  // namespace gbssim

using namespace gbssim;

extern "C" int gbssim_rotary_turn(const gbssim_rotary *d, void *q_out, void *k_out, void *stream)
{
    const CallRange range("gbssim_rotary_turn");
    if (!d || !dtype_ok(d->dtype)) return GBSSIM_EINVAL;
    if (d->pos_type < GBSSIM_POS_I32 || d->pos_type > GBSSIM_POS_F32) return GBSSIM_EINVAL;
    if (d->layout < GBSSIM_ROTARY_HALF || d->layout > GBSSIM_ROTARY_ADJACENT) return GBSSIM_EINVAL;
    if (d->batch < 0 || d->tokens < 0 || d->q_heads < 0 || d->k_heads < 0) return GBSSIM_ESHAPE;
    if (d->q_heads > 65535 || d->k_heads > 65535) return GBSSIM_ESHAPE;
    if (d->axes < 1 || d->axes > GBSSIM_ROTARY_AXES) return GBSSIM_ESHAPE;
    if (d->dim < 2 || d->dim > kMaxRotaryDim) return GBSSIM_ESHAPE;
    RotaryArgs a{};
    for (int i = 0; i < d->axes; ++i) {
        if (d->pairs[i] < 1 || d->pairs[i] > kMaxPairs) return GBSSIM_ESHAPE;
        a.pairs += d->pairs[i];
        a.ends[i] = a.pairs;
    }
    if (2 * a.pairs > d->dim) return GBSSIM_ESHAPE;
    const long long rows = (long long)d->batch * d->tokens;
    if (rows == 0 || d->q_heads + d->k_heads == 0) return GBSSIM_OK;
    if (!d->positions || !d->frequencies) return GBSSIM_EINVAL;
    if (d->pos_batch_stride < 0 || d->pos_token_stride < 0) return GBSSIM_EINVAL;
    const int pos_bytes = d->pos_type == GBSSIM_POS_I64 ? 8 : 4;
    if (reinterpret_cast<uintptr_t>(d->positions) % pos_bytes || reinterpret_cast<uintptr_t>(d->frequencies) % 8)
        return GBSSIM_EALIGN;
    int rc;
    if ((rc = check_heads(*d, d->q, d->q_heads)) || (rc = check_heads(*d, d->k, d->k_heads))) return rc;
    if ((d->q_heads && !q_out) || (d->k_heads && !k_out)) return GBSSIM_EINVAL;
    const int size = dtype_bytes(d->dtype);
    if (reinterpret_cast<uintptr_t>(q_out) % size || reinterpret_cast<uintptr_t>(k_out) % size) return GBSSIM_EALIGN;
    const long long pos_last = (d->batch - 1) * d->pos_batch_stride + (d->tokens - 1) * d->pos_token_stride + d->axes;
    const Extent in[4] = {heads_extent(*d, d->q, d->q_heads), heads_extent(*d, d->k, d->k_heads),
                          {d->positions, size_t(pos_last) * pos_bytes}, {d->frequencies, size_t(a.pairs) * 8}};
    const Extent out[2] = {{q_out, size_t(rows) * d->q_heads * d->dim * size},
                           {k_out, size_t(rows) * d->k_heads * d->dim * size}};
    for (const Extent &o : out)
        for (const Extent &i : in)
            if (meet(o, i)) return GBSSIM_EINVAL;
    if (meet(out[0], out[1])) return GBSSIM_EINVAL;

    a.t[0] = {d->q.data, q_out, d->q.batch_stride, d->q.token_stride, d->q.head_stride, d->q_heads};
    a.t[1] = {d->k.data, k_out, d->k.batch_stride, d->k.token_stride, d->k.head_stride, d->k_heads};
    a.positions = d->positions;
    a.frequencies = d->frequencies;
    a.pos_batch = d->pos_batch_stride;
    a.pos_token = d->pos_token_stride;
    a.pos_type = d->pos_type;
    a.axes = d->axes;
    a.batch = d->batch;
    a.tokens = d->tokens;
    a.dim = d->dim;
    a.adjacent = d->layout == GBSSIM_ROTARY_ADJACENT;
    a.sign = d->inverse ? -1.0f : 1.0f;
    Mode m = kSingle;
    if (d->dim % 8 == 0 && whole_words(*d, d->q, q_out, d->q_heads) && whole_words(*d, d->k, k_out, d->k_heads))
        m = a.adjacent ? kAdjacent : a.pairs % 8 == 0 ? kHalves : kWindow;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_fail(d->dtype == GBSSIM_F32    ? launch_mode<float>(a, m, st)
                     : d->dtype == GBSSIM_BF16 ? launch_mode<bf16>(a, m, st)
                                               : launch_mode<f16>(a, m, st));
}
