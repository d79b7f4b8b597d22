// Rotary positions with several axes: pair p of a head belongs to an axis and has a
// frequency; at a token whose position on that axis is x the pair (u, v) becomes
// (u cos a - v sin a, u sin a + v cos a), a = x f_p; with -a for the inverse, which is
// also the gradient.
//
// Angles are taken modulo a turn in fixed point: f / (2 pi) as a fraction of 2^64,
// times the position, wraps by itself, so far positions lose nothing but that quotient's
// rounding; sine and cosine then see at most half a turn, in float32.
//
// Bound by memory: every element is read and written once.  A thread has eight columns
// of a token (in the layout of halves, four of each half) and goes over the token's
// heads with their sines and cosines in registers, two heads' loads under way while it
// turns the last two, and the first ones before it knows the angles.  Nothing but the
// frequencies' turns is in shared memory, so that no thread waits for another.
// 65536 tokens, 20 heads of 128, bfloat16 (671 MB): 127 us, 5.3 TB/s; 32400 tokens, 24
// heads of 88, float32 (547 MB): 108 us; 512 tokens: 6.4 us.
#include <algorithm>
#include <climits>

#include "api_host.cuh"
#include "dtypes.cuh"
#include "rotary_angle.cuh"

namespace gbssim {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxPairs = 256, kMaxRotaryDim = 512;
constexpr int kHeadsAtOnce = 2;
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
};

// How a thread's columns find their partners.
enum Mode {
    kHalves,    // V columns of the first half and V of the second
    kAdjacent,  // neighbours, within eight columns
    kSingle     // a pair or a column a thread: any alignment
};

// A pair's axis, and a flag where its frequency is below zero.
constexpr int kNegative = 64;

// cos and sin of position x frequency.  Where results are rounded to 16 bits (2^-8, 2^-11)
// the hardware's approximations do, which are within 2^-21 over a turn; they take a
// tenth of the instructions of the exact functions.
template <bool EXACT>
__device__ __forceinline__ float2 turn_of(const RotaryArgs &a, long long at, turns64 fraction, const turns64 &whole,
                                          bool negative)
{
    turns64 phase;
    if (a.pos_type == GBSSIM_POS_I32) {
        phase = turn_phase((long long)static_cast<const int *>(a.positions)[at], fraction);
    } else if (a.pos_type == GBSSIM_POS_I64) {
        phase = turn_phase(static_cast<const long long *>(a.positions)[at], fraction);
    } else {
        const float x = static_cast<const float *>(a.positions)[at];
        if (!(fabsf(x) < 9.0e18f)) return make_float2(NAN, NAN);
        phase = turn_phase(x, fraction, whole, negative);
    }
    const float turned = float(int(unsigned(phase >> 32)));  // 2^-31 half turns
    float s, c;
    if constexpr (EXACT)
        sincospif(turned * 4.656612873077393e-10f, &s, &c);
    else
        __sincosf(turned * 1.4629180792671596e-9f, &s, &c);
    return make_float2(c, s * a.sign);
}

// V consecutive elements as they lie in memory: 4 to 32 bytes.
template <typename T, int V>
struct Words {
    static constexpr int kWords = V * int(sizeof(T)) / 4;
    uint32_t w[kWords];
};

template <typename T, int V>
__device__ __forceinline__ Words<T, V> load(const T *p)
{
    Words<T, V> r;
    if constexpr (r.kWords >= 4) {
#pragma unroll
        for (int i = 0; i < r.kWords; i += 4) {
            const uint4 x = ld_stream16(reinterpret_cast<const uint32_t *>(p) + i);
            r.w[i] = x.x;
            r.w[i + 1] = x.y;
            r.w[i + 2] = x.z;
            r.w[i + 3] = x.w;
        }
    } else if constexpr (r.kWords == 2) {
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(p));
        r.w[0] = x.x;
        r.w[1] = x.y;
    } else {
        r.w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
    }
    return r;
}

template <typename T, int V>
__device__ __forceinline__ void store(T *p, const Words<T, V> &r)
{
    if constexpr (r.kWords >= 4) {
#pragma unroll
        for (int i = 0; i < r.kWords; i += 4)
            reinterpret_cast<uint4 *>(p)[i / 4] = make_uint4(r.w[i], r.w[i + 1], r.w[i + 2], r.w[i + 3]);
    } else if constexpr (r.kWords == 2) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(r.w[0], r.w[1]);
    } else {
        *reinterpret_cast<uint32_t *>(p) = r.w[0];
    }
}

template <typename T, int V>
__device__ __forceinline__ void unpack(const Words<T, V> &r, float (&v)[V])
{
#pragma unroll
    for (int i = 0; i < V; i += 2) {
        if constexpr (sizeof(T) == 4) {
            v[i] = __uint_as_float(r.w[i]);
            v[i + 1] = __uint_as_float(r.w[i + 1]);
        } else {
            const float2 x = unpack2<T>(r.w[i / 2]);
            v[i] = x.x;
            v[i + 1] = x.y;
        }
    }
}

template <typename T, int V>
__device__ __forceinline__ Words<T, V> pack(const float (&v)[V])
{
    Words<T, V> r;
#pragma unroll
    for (int i = 0; i < V; i += 2) {
        if constexpr (sizeof(T) == 4) {
            r.w[i] = __float_as_uint(v[i]);
            r.w[i + 1] = __float_as_uint(v[i + 1]);
        } else {
            r.w[i / 2] = pack2<T>(v[i], v[i + 1]);
        }
    }
    return r;
}

// How the work is cut: a head's columns go to `lanes` threads, its token's heads in
// turn to `parts` of them, so that neighbouring threads read neighbouring heads.
struct Cut {
    int lanes, parts;
};

template <typename T, Mode M, int V>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a, const Cut cut)
{
    __shared__ turns64 fraction[kMaxPairs], whole[kMaxPairs];
    __shared__ unsigned char axis_of[kMaxPairs];
    const int n = a.pairs;
    for (int i = threadIdx.x; i < n; i += kThreads) {
        int axis = 0;
        while (i >= a.ends[axis]) ++axis;
        const double f = a.frequencies[i];
        const bool some = isfinite(f);
        axis_of[i] = static_cast<unsigned char>(!some ? kNoAngle : f < 0.0 ? axis + kNegative : axis);
        fraction[i] = some ? turn_fraction(f) : 0;
        // (for other positions as well: 1 % of a long call's time)
        whole[i] = some && a.pos_type == GBSSIM_POS_F32 ? whole_turns(f) : 0;
    }
    __syncthreads();
    const int end = a.t[0].heads + a.t[1].heads, step = cut.parts;
    const long long items = (long long)a.batch * a.tokens * cut.parts * cut.lanes;
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < items; i += (long long)gridDim.x * kThreads) {
        long long row, b;
        int lane, first;
        if (items <= 0xffffffffLL) {  // divisions of 32 bits take a fifth of the time
            const unsigned team = unsigned(i) / unsigned(cut.lanes), r = team / unsigned(cut.parts);
            lane = int(unsigned(i) - team * cut.lanes);
            first = int(team - r * cut.parts);
            row = r;
            b = r / unsigned(a.tokens);
        } else {
            const long long team = i / cut.lanes;
            row = team / cut.parts;
            lane = int(i - team * cut.lanes);
            first = int(team - row * cut.parts);
            b = row / a.tokens;
        }
        const long long token = row - b * a.tokens;
        const long long pos = b * a.pos_batch + token * a.pos_token;
        const auto turn = [&](int p) {
            const int axis = axis_of[p];
            if (axis == kNoAngle) return make_float2(NAN, NAN);
            return turn_of<sizeof(T) == 4>(a, pos + axis % kNegative, fraction[p], whole[p], axis >= kNegative);
        };
        // the rows of this token's heads: the first tensor's, then the second's
        const T *const in0 = static_cast<const T *>(a.t[0].in) + b * a.t[0].batch + token * a.t[0].token;
        const T *const in1 = static_cast<const T *>(a.t[1].in) + b * a.t[1].batch + token * a.t[1].token;
        T *const out0 = static_cast<T *>(a.t[0].out) + row * a.t[0].heads * a.dim;
        T *const out1 = static_cast<T *>(a.t[1].out) + row * a.t[1].heads * a.dim;
        const auto in = [&](int h) {
            return h < a.t[0].heads ? in0 + h * a.t[0].head : in1 + (h - a.t[0].heads) * a.t[1].head;
        };
        const auto out = [&](int h) {
            return h < a.t[0].heads ? out0 + h * a.dim : out1 + (h - a.t[0].heads) * a.dim;
        };

        if constexpr (M == kSingle) {
            const bool turned = lane < n;
            const int u = !turned ? lane + n : a.adjacent ? 2 * lane : lane;
            const int v = a.adjacent ? u + 1 : u + n;
            const float2 cs = turned ? turn(lane) : make_float2(1.0f, 0.0f);
            constexpr int kGroup = 8;
            for (int g = first; g < end; g += kGroup * step) {
                T xu[kGroup], xv[kGroup];
#pragma unroll
                for (int e = 0; e < kGroup; ++e) {
                    const int h = g + e * step;
                    if (h >= end) continue;
                    const T *const x = in(h);
                    xu[e] = x[u];
                    if (turned) xv[e] = x[v];
                }
#pragma unroll
                for (int e = 0; e < kGroup; ++e) {
                    const int h = g + e * step;
                    if (h >= end) continue;
                    T *const y = out(h);
                    if (turned) {
                        const float p = to_f32(xu[e]), q = to_f32(xv[e]);
                        y[u] = from_f32<T>(p * cs.x - q * cs.y);
                        y[v] = from_f32<T>(p * cs.y + q * cs.x);
                    } else {
                        y[u] = xu[e];
                    }
                }
            }
        } else if constexpr (M == kHalves) {
            const int chunks = n / V;
            if (lane >= chunks) {  // columns without a position
                const int at = 2 * n + (lane - chunks) * V;
#pragma unroll 4
                for (int h = first; h < end; h += step) store<T, V>(out(h) + at, load<T, V>(in(h) + at));
                continue;
            }
            // two buffers, so that a group's loads are under way while the last one is turned
            Words<T, V> u[2][kHeadsAtOnce], v[2][kHeadsAtOnce];
            const auto fetch = [&](int h, int buf) {
#pragma unroll
                for (int e = 0; e < kHeadsAtOnce; ++e)
                    if (h + e * step < end) {
                        const T *const x = in(h + e * step) + lane * V;
                        u[buf][e] = load<T, V>(x);
                        v[buf][e] = load<T, V>(x + n);
                    }
            };
            float c[V], s[V];
            const auto turn_heads = [&](int h, int buf) {
#pragma unroll
                for (int e = 0; e < kHeadsAtOnce; ++e)
                    if (h + e * step < end) {
                        float x[V], y[V], p[V], q[V];
                        unpack<T, V>(u[buf][e], x);
                        unpack<T, V>(v[buf][e], y);
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            p[j] = x[j] * c[j] - y[j] * s[j];
                            q[j] = x[j] * s[j] + y[j] * c[j];
                        }
                        T *const to = out(h + e * step) + lane * V;
                        store<T, V>(to, pack<T, V>(p));
                        store<T, V>(to + n, pack<T, V>(q));
                    }
            };
            fetch(first, 0);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float2 cs = turn(lane * V + e);
                c[e] = cs.x;
                s[e] = cs.y;
            }
            const int group = kHeadsAtOnce * step;
            for (int h = first; h < end; h += 2 * group) {
                fetch(h + group, 1);
                turn_heads(h, 0);
                fetch(h + 2 * group, 0);
                turn_heads(h + group, 1);
            }
        } else {
            Words<T, 8> u[2][kHeadsAtOnce];
            const auto fetch = [&](int h, int buf) {
#pragma unroll
                for (int e = 0; e < kHeadsAtOnce; ++e)
                    if (h + e * step < end) u[buf][e] = load<T, 8>(in(h + e * step) + lane * 8);
            };
            float c[4], s[4];
            // a pair without a position is turned by nothing; it has to keep a NaN to itself
            const int here = min(max(n - lane * 4, 0), 4);
            const auto turn_heads = [&](int h, int buf) {
#pragma unroll
                for (int e = 0; e < kHeadsAtOnce; ++e)
                    if (h + e * step < end) {
                        float x[8], p[8];
                        unpack<T, 8>(u[buf][e], x);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            p[2 * j] = j < here ? x[2 * j] * c[j] - x[2 * j + 1] * s[j] : x[2 * j];
                            p[2 * j + 1] = j < here ? x[2 * j] * s[j] + x[2 * j + 1] * c[j] : x[2 * j + 1];
                        }
                        store<T, 8>(out(h + e * step) + lane * 8, pack<T, 8>(p));
                    }
            };
            fetch(first, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 cs = e < here ? turn(lane * 4 + e) : make_float2(1.0f, 0.0f);
                c[e] = cs.x;
                s[e] = cs.y;
            }
            const int group = kHeadsAtOnce * step;
            for (int h = first; h < end; h += 2 * group) {
                fetch(h + group, 1);
                turn_heads(h, 0);
                fetch(h + 2 * group, 0);
                turn_heads(h + group, 1);
            }
        }
    }
}

template <typename T, Mode M, int V>
cudaError_t launch(const RotaryArgs &a, cudaStream_t stream)
{
    const long long rows = (long long)a.batch * a.tokens;
    const int heads = a.t[0].heads + a.t[1].heads;
    Cut cut;
    cut.lanes = M == kHalves ? a.pairs / V + (a.dim - 2 * a.pairs) / V : M == kSingle ? a.dim - a.pairs : a.dim / V;
    // Few tokens: threads share a token's heads, four each at least, until they fill the
    // GPU.  Many: one thread for all of them, which forms their sines and cosines once
    // (65536 x 20 heads of 128, bfloat16: one thread 129 us, two 136, four 152), but two
    // in float32, whose rows are twice as long (32400 x 24 heads of 88: 121, 108).
    constexpr long long kRoom = 152LL * 1024;
    const long long most = std::max(1, heads / 4), wanted = ceil_div(kRoom, rows * cut.lanes);
    cut.parts = int(std::min(most, std::max<long long>(wanted, sizeof(T) == 4 ? 2 : 1)));
    const long long items = rows * cut.lanes * cut.parts;
    const long long blocks = std::min<long long>(ceil_div(items, kThreads), 1 << 20);
    rotary_kernel<T, M, V><<<unsigned(blocks), kThreads, 0, stream>>>(a, cut);
    return cudaGetLastError();
}

// v: columns that a thread may take at once.
template <typename T>
cudaError_t launch_mode(const RotaryArgs &a, int v, cudaStream_t stream)
{
    if (a.adjacent) return v == 8 ? launch<T, kAdjacent, 8>(a, stream) : launch<T, kSingle, 1>(a, stream);
    switch (v) {
    case 4: return launch<T, kHalves, 4>(a, stream);
    case 2: return launch<T, kHalves, 2>(a, stream);
    default: return launch<T, kSingle, 1>(a, stream);
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

// Whether every row of the tensor and of its output starts on a multiple of `bytes`.
bool aligned(const gbssim_rotary &d, const gbssim_heads &t, const void *out, int heads, int bytes)
{
    if (!heads) return true;
    const int size = dtype_bytes(d.dtype);
    const auto on = [&](long long n) { return n * size % bytes == 0; };
    return reinterpret_cast<uintptr_t>(t.data) % bytes == 0 && reinterpret_cast<uintptr_t>(out) % bytes == 0 &&
           on(d.dim) && (d.batch < 2 || on(t.batch_stride)) && (d.tokens < 2 || on(t.token_stride)) &&
           (heads < 2 || on(t.head_stride));
}

// How many columns a thread can take at once: as many as both halves, the rest of a row
// and the alignment of every row allow.
int columns(const gbssim_rotary &d, int pairs, const void *q_out, const void *k_out)
{
    const bool adjacent = d.layout == GBSSIM_ROTARY_ADJACENT;
    for (int v = adjacent ? 8 : 4; v > 1; v /= 2) {
        const int bytes = std::min(16, v * dtype_bytes(d.dtype));
        if (d.dim % v || (!adjacent && (pairs % v || (d.dim - 2 * pairs) % v))) continue;
        if (aligned(d, d.q, q_out, d.q_heads, bytes) && aligned(d, d.k, k_out, d.k_heads, bytes)) return v;
    }
    return 1;
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
    const int v = columns(*d, a.pairs, q_out, k_out);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_fail(d->dtype == GBSSIM_F32    ? launch_mode<float>(a, v, st)
                     : d->dtype == GBSSIM_BF16 ? launch_mode<bf16>(a, v, st)
                                               : launch_mode<f16>(a, v, st));
}
