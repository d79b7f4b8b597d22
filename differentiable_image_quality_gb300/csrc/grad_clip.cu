// The global norm of many gradient tensors, and clipping by it.
//
//   S = sum over every element of every tensor of g^2 (or |g|, or max |g|),
//   norm = sqrt(S) (or S),   c = min(1, max_norm / (norm + 1e-6)),   out = c g.
//
// Both kernels are bound by memory: the norm reads every gradient once, the
// scaling reads it again (from L2 as far as it is still there) and writes the
// output.  All tensors go through one launch: their addresses and lengths
// travel in the kernel's parameters, so a call copies no table to the device
// and can be captured in a CUDA graph.  Tensors are cut into chunks of 32 KB; a
// block takes a contiguous run of chunks, whatever tensors they belong to, so
// the work is even for any mix of sizes, and the order of every sum depends on
// the sizes, the alignments and the device alone: the same inputs give the same
// bits.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "gbssim.h"
#include "api_host.cuh"
#include "common.cuh"
#include "dtypes.cuh"

namespace gbssim {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 8;        // the norm of 1.0 G bfloat16: 290 us, 4 302, 5 308, 6 323
constexpr int kMaxBlocks = 2048;       // of one norm launch: sizes the workspace
constexpr int kVecs = 8;               // 16-byte words a thread holds of a norm chunk
constexpr int kChunkWords = kThreads * kVecs;  // 32 KB
constexpr int kScaleElems = 8192;      // elements of a scaling chunk: 32 a thread
constexpr float kClipEps = 1e-6f;

// Tensors of one launch, in the kernel's parameters (at most 32764 bytes).
// first[i] is the number of chunks ahead of tensor i; first[n] all of them.
template <int CAP>
struct NormTable {
    const void *g[CAP];
    long long count[CAP];
    unsigned first[CAP + 1];
    unsigned char type[CAP];
    int n;
    unsigned slot0;  // partial sums written by earlier launches of this call
    int last;        // this launch finishes the call
    double *partials;
    unsigned *counter;
    float *norm;     // out
    float *coef;     // out, or null
    float max_norm;
};

template <int CAP>
struct ScaleTable {
    const void *g[CAP];
    void *out[CAP];
    long long count[CAP];
    unsigned first[CAP + 1];
    unsigned char type[CAP], out_type[CAP];
    unsigned char pad[CAP];  // elements by which chunks are shifted, and kApart
    int n;
    int in_place;  // every output is its gradient
    const float *coef;
};

constexpr unsigned char kApart = 8;  // gradient and output are not aligned alike
// Two sizes of tables, as a launch copies all of its parameters: 26 tensors, time
// on the host, norm 21.5 us with the small one, 24.5 with the large, clip 27.0 and 31.2.
constexpr int kCapSmall = 32, kCapLarge = 1024;
static_assert(sizeof(ScaleTable<kCapLarge>) <= 32764, "kernel parameter space");
static_assert(sizeof(NormTable<kCapLarge>) <= 32764, "kernel parameter space");

// The tensor that chunk c belongs to.
template <class Table>
__device__ __forceinline__ int tensor_of(const Table &t, unsigned c)
{
    int lo = 0, hi = t.n;  // first[lo] <= c < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.first[mid] <= c) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The contiguous run of chunks [c0, c1) of this block.
__device__ __forceinline__ void block_run(unsigned chunks, unsigned &c0, unsigned &c1)
{
    const unsigned long long b = blockIdx.x, nb = gridDim.x;
    c0 = unsigned(b * chunks / nb);
    c1 = unsigned((b + 1) * chunks / nb);
}

// ------------------------------------------------------------------ the norm

// 16-byte word w (counted from the 16-byte boundary at or before the tensor's
// first element) of a tensor, zero outside it.
template <typename T>
__device__ __forceinline__ uint4 load_word(const unsigned char *base, long long w, int pad,
                                           long long n)
{
    constexpr int V = 16 / sizeof(T);
    const long long e = w * V - pad;  // first element of the word
    if (e >= 0 && e + V <= n) return ld_stream16(base + w * 16);
    alignas(16) T v[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        v[i] = (e + i >= 0 && e + i < n) ? reinterpret_cast<const T *>(base)[w * V + i]
                                         : from_f32<T>(0.0f);
    return *reinterpret_cast<const uint4 *>(v);
}

template <typename T>
__device__ __forceinline__ float2 word_pair(uint32_t a)
{
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(a), 0.0f);
    else return unpack2<T>(a);
}

// Sum over the thread's words of a chunk in double, read once more: for values
// whose squares (or sum) leave float32's range.
template <int P, typename T>
__device__ __noinline__ double sum_wide(const unsigned char *base, long long w0, int pad,
                                        long long n)
{
    double s = 0.0;
    for (int i = 0; i < kVecs; ++i) {
        const uint4 r = load_word<T>(base, w0 + i * kThreads, pad, n);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
        for (int k = 0; k < 4; ++k) {
            const float2 v = word_pair<T>(w[k]);
            const double a = v.x, b = v.y;
            s += P == 2 ? a * a + b * b : fabs(a) + fabs(b);
        }
    }
    return s;
}

// One chunk's contribution of this thread.  Squares are summed in float32 over
// the thread's 32 or 64 values, then in double.  A float32 sum that overflowed,
// or lies so low that squares may have been lost below float32's range, is
// taken again in double: the norm is right wherever the gradients are finite.
// P = 0 keeps the largest |g| as its bits: they order as the values do, and a
// NaN's lie above infinity's.
template <int P, typename T>
__device__ __forceinline__ void add_chunk(const void *g, long long n, unsigned k, double &sum,
                                          uint32_t &top)
{
    const unsigned long long addr = reinterpret_cast<unsigned long long>(g);
    const unsigned char *base = reinterpret_cast<const unsigned char *>(addr & ~15ull);
    const int pad = int(addr & 15) / int(sizeof(T));
    const long long w0 = (long long)k * kChunkWords + threadIdx.x;
    uint4 r[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) r[i] = load_word<T>(base, w0 + i * kThreads, pad, n);
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
        const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = word_pair<T>(w[j]);
            if (P == 0) {
                top = max(top, max(__float_as_uint(fabsf(v.x)), __float_as_uint(fabsf(v.y))));
            } else if (P == 1) {
                s0 += fabsf(v.x);
                s1 += fabsf(v.y);
            } else {
                s0 = fmaf(v.x, v.x, s0);
                s1 = fmaf(v.y, v.y, s1);
            }
        }
    }
    if (P != 0) {
        const float s = s0 + s1;
        if (s == 0.0f || (s >= 0x1p-80f && s <= 0x1p126f)) {
            // s == 0: nothing but zeros, or every square was lost
            uint32_t any = 0;
            if (P == 2 && s == 0.0f) {
#pragma unroll
                for (int i = 0; i < kVecs; ++i) any |= r[i].x | r[i].y | r[i].z | r[i].w;
            }
            if (any & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu)) sum += sum_wide<P, T>(base, w0, pad, n);
            else sum += double(s);
        } else {
            sum += sum_wide<P, T>(base, w0, pad, n);
        }
    }
}

template <int P>
__device__ __forceinline__ double join(double a, double b)
{
    // P = 0: bit patterns held as whole numbers, never NaN themselves
    return P == 0 ? fmax(a, b) : a + b;
}

// Joins one value per thread over the block in a fixed order, for thread 0.
template <int P>
__device__ __forceinline__ double block_join(double d, double *scratch)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) d = join<P>(d, __shfl_down_sync(0xffffffffu, d, o));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    if (lane == 0) scratch[warp] = d;
    __syncthreads();
    double t = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < kThreads / 32; ++w) t = join<P>(t, scratch[w]);
    return t;
}

template <int P, int CAP>
__global__ void __launch_bounds__(kThreads)
    grad_norm_kernel(const __grid_constant__ NormTable<CAP> t)
{
    __shared__ double scratch[kThreads / 32];
    if (t.coef && t.first[t.n]) pdl_trigger();  // only the scaling kernel starts early
    unsigned c0, c1;
    block_run(t.first[t.n], c0, c1);
    double sum = 0.0;
    uint32_t top = 0;
    if (c0 < c1) {
        int i = tensor_of(t, c0);
        for (unsigned c = c0; c < c1; ++c) {
            while (t.first[i + 1] <= c) ++i;
            const unsigned k = c - t.first[i];
            if (t.type[i] == GBSSIM_F32) add_chunk<P, float>(t.g[i], t.count[i], k, sum, top);
            else if (t.type[i] == GBSSIM_BF16) add_chunk<P, bf16>(t.g[i], t.count[i], k, sum, top);
            else add_chunk<P, f16>(t.g[i], t.count[i], k, sum, top);
        }
    }
    const double b = block_join<P>(P == 0 ? double(top) : sum, scratch);
    if (threadIdx.x == 0) t.partials[t.slot0 + blockIdx.x] = b;
    if (!t.last || !finish_ticket<kThreads>(t.counter)) return;
    const unsigned total = t.slot0 + gridDim.x;
    double s = 0.0;
    for (unsigned j = threadIdx.x; j < total; j += kThreads) s = join<P>(s, __ldcg(t.partials + j));
    s = block_join<P>(s, scratch);
    if (threadIdx.x == 0) {
        const float norm = P == 0 ? __uint_as_float(uint32_t(s)) : float(P == 2 ? sqrt(s) : s);
        *t.norm = norm;
        if (t.coef) {
            const float c = t.max_norm / (norm + kClipEps);
            // no limit, no clipping, also where that is inf / inf; a norm's NaN stays
            *t.coef = c > 1.0f || (isinf(t.max_norm) && !isnan(norm)) ? 1.0f : c;
        }
        *t.counter = 0u;
    }
}

// ------------------------------------------------------------------ the scaling

// Groups of V consecutive elements: 8 where both types have 16 bits, else 4, so
// that a lane's access is at most 16 bytes and a warp's whole lines.
template <typename T, typename O>
constexpr int kGroup = sizeof(T) == 2 && sizeof(O) == 2 ? 8 : 4;

template <typename T, int V>
struct Group {
    static constexpr int kWords = V * int(sizeof(T)) / 4;
    uint32_t w[kWords];
};

template <typename T, int V>
__device__ __forceinline__ Group<T, V> load_group(const T *p)
{
    Group<T, V> g;
    if constexpr (Group<T, V>::kWords == 4) {
        const uint4 q = ld_stream16(p);
        g.w[0] = q.x; g.w[1] = q.y; g.w[2] = q.z; g.w[3] = q.w;
    } else {
        asm volatile("ld.global.L1::no_allocate.v2.u32 {%0, %1}, [%2];"
                     : "=r"(g.w[0]), "=r"(g.w[1])
                     : "l"(p));
    }
    return g;
}

template <typename T, int V>
__device__ __forceinline__ void unpack_group(const Group<T, V> &g, float (&v)[V])
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = __uint_as_float(g.w[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 h = unpack2<T>(g.w[i]);
            v[2 * i] = h.x;
            v[2 * i + 1] = h.y;
        }
    }
}

template <typename O, int V>
__device__ __forceinline__ void store_group(O *p, const float (&v)[V])
{
    uint32_t w[V * int(sizeof(O)) / 4];
    if constexpr (sizeof(O) == 4) {
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] = __float_as_uint(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) w[i] = pack2<O>(v[2 * i], v[2 * i + 1]);
    }
    if constexpr (V * sizeof(O) == 16) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
}

// Chunk k: elements [k E - pad, (k + 1) E - pad) of the tensor, E = kScaleElems.
// Whole chunks whose groups are aligned in both tensors take one access a group.
// Where gradients and their output reach a group's boundary at different elements
// (apart), the gradients' own aligned words go through shared memory and come out
// again as the output's groups.  The first and last chunk of a tensor take one
// element a lane.
template <typename T, typename O>
__device__ __noinline__ void scale_chunk(const void *gv, void *ov, long long n, unsigned k,
                                         int pad, bool apart, float c, uint4 *stage)
{
    constexpr int kEach = kScaleElems / kThreads, V = kGroup<T, O>;
    const T *g = static_cast<const T *>(gv);
    O *o = static_cast<O *>(ov);
    long long e0 = (long long)k * kScaleElems - pad;
    if (apart && e0 >= 8 && e0 + kScaleElems + 8 <= n) {
        constexpr int kWords = kScaleElems * int(sizeof(T)) / 16;
        const uintptr_t at = reinterpret_cast<uintptr_t>(g + e0);
        const uint4 *word = reinterpret_cast<const uint4 *>(at & ~uintptr_t(15));
        uint4 r[kWords / kThreads];
#pragma unroll
        for (int j = 0; j < kWords / kThreads; ++j) r[j] = ld_stream16(word + threadIdx.x + j * kThreads);
        __syncthreads();  // the chunk before has been read out
#pragma unroll
        for (int j = 0; j < kWords / kThreads; ++j) stage[threadIdx.x + j * kThreads] = r[j];
        if (threadIdx.x == 0) stage[kWords] = ld_stream16(word + kWords);
        __syncthreads();
        const T *in = reinterpret_cast<const T *>(stage) + int(at & 15) / int(sizeof(T)) + threadIdx.x * V;
        o += e0 + threadIdx.x * V;
#pragma unroll
        for (int j = 0; j < kEach / V; ++j) {
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = to_f32(in[j * (kThreads * V) + i]) * c;
            store_group<O, V>(o + j * (kThreads * V), v);
        }
        return;
    }
    if (!apart && e0 >= 0 && e0 + kScaleElems <= n) {
        g += e0 + threadIdx.x * V;
        o += e0 + threadIdx.x * V;
        Group<T, V> r[kEach / V];
#pragma unroll
        for (int j = 0; j < kEach / V; ++j) r[j] = load_group<T, V>(g + j * (kThreads * V));
#pragma unroll
        for (int j = 0; j < kEach / V; ++j) {
            float v[V];
            unpack_group<T, V>(r[j], v);
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] *= c;
            store_group<O, V>(o + j * (kThreads * V), v);
        }
        return;
    }
    const long long end = min(n, e0 + kScaleElems);
    if (e0 < 0) e0 = 0;
    const int len = int(end - e0);
    constexpr int kBatch = 8;
    g += e0;
    o += e0;
#pragma unroll 1
    for (int e = threadIdx.x; e < len; e += kBatch * kThreads) {
        T v[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (e + j * kThreads < len) v[j] = g[e + j * kThreads];
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
            if (e + j * kThreads < len) o[e + j * kThreads] = from_f32<O>(to_f32(v[j]) * c);
    }
}

template <typename T>
__device__ __forceinline__ void scale_chunk_to(int out_type, const void *g, void *o, long long n,
                                               unsigned k, int pad, bool apart, float c,
                                               uint4 *stage)
{
    if (out_type == GBSSIM_F32) scale_chunk<T, float>(g, o, n, k, pad, apart, c, stage);
    else if (out_type == GBSSIM_BF16) scale_chunk<T, bf16>(g, o, n, k, pad, apart, c, stage);
    else scale_chunk<T, f16>(g, o, n, k, pad, apart, c, stage);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, 4)
    grad_scale_kernel(const __grid_constant__ ScaleTable<CAP> t)
{
    __shared__ uint4 stage[kScaleElems * 4 / 16 + 1];
    pdl_wait();
    const float c = __ldcg(t.coef);
    if (t.in_place && c == 1.0f) return;  // 1 * g is g, to the bit
    const unsigned chunks = t.first[t.n];
    // neighbouring chunks by neighbouring blocks: reading and writing at once,
    // blocks in runs of their own took 142 us for 59 M float32, these 116.  From
    // the end, which the norm read last.
    for (unsigned done = blockIdx.x; done < chunks; done += gridDim.x) {
        const unsigned q = chunks - 1 - done;
        const int i = tensor_of(t, q);
        const unsigned k = q - t.first[i];
        const int pad = t.pad[i] & 7;
        const bool apart = t.pad[i] & kApart;
        if (t.type[i] == GBSSIM_F32)
            scale_chunk_to<float>(t.out_type[i], t.g[i], t.out[i], t.count[i], k, pad, apart, c, stage);
        else if (t.type[i] == GBSSIM_BF16)
            scale_chunk_to<bf16>(t.out_type[i], t.g[i], t.out[i], t.count[i], k, pad, apart, c, stage);
        else
            scale_chunk_to<f16>(t.out_type[i], t.g[i], t.out[i], t.count[i], k, pad, apart, c, stage);
    }
}

// ------------------------------------------------------------------ host side

constexpr size_t kCoefOffset = 256, kPartialOffset = 512;

struct List {
    const void *const *g;
    void *const *out;  // null: the norm alone
    const long long *count;
    const unsigned char *type, *out_type;
    int n;
};

// Chunks of one norm launch or scaling launch are counted in 32 bits.
constexpr long long kMaxChunks = 0x7fffffffll;

long long norm_chunks(const void *g, long long count, int type)
{
    if (count == 0) return 0;
    const long long v = 16 / dtype_bytes(type);
    const long long pad = (reinterpret_cast<uintptr_t>(g) & 15) / dtype_bytes(type);
    return ceil_div(ceil_div(count + pad, v), kChunkWords);
}

// The shift of a tensor's chunks that aligns the groups of its output, and whether
// it leaves those of its gradient unaligned.
unsigned char chunk_pad(const void *g, int type, const void *o, int out_type)
{
    const int group = type != GBSSIM_F32 && out_type != GBSSIM_F32 ? 8 : 4;
    const auto lead = [&](const void *p, int t) {
        return int(reinterpret_cast<uintptr_t>(p) / dtype_bytes(t) % group);
    };
    const int pad = lead(o, out_type);
    return (unsigned char)(lead(g, type) == pad ? pad : pad | kApart);
}

unsigned grid_for(long long chunks, int sm_count)
{
    const long long most = std::min<long long>((long long)sm_count * kBlocksPerSm, kMaxBlocks);
    return unsigned(std::max<long long>(1, std::min(chunks, most)));
}

template <int P, int CAP>
cudaError_t launch_norm(const List &l, int i0, int n, bool last, int sm_count, unsigned &slot,
                        unsigned char *ws, float *norm, float *coef, float max_norm, cudaStream_t s)
{
    NormTable<CAP> t;
    long long chunks = 0;
    t.n = n;
    for (int i = 0; i < n; ++i) {
        t.g[i] = l.g[i0 + i];
        t.count[i] = l.count[i0 + i];
        t.type[i] = l.type[i0 + i];
        t.first[i] = unsigned(chunks);
        chunks += norm_chunks(t.g[i], t.count[i], t.type[i]);
    }
    t.first[n] = unsigned(chunks);
    t.slot0 = slot;
    t.last = last;
    t.counter = reinterpret_cast<unsigned *>(ws);
    t.coef = coef;
    t.partials = reinterpret_cast<double *>(ws + kPartialOffset);
    t.norm = norm;
    t.max_norm = max_norm;
    const unsigned grid = grid_for(chunks, sm_count);
    slot += grid;
    grad_norm_kernel<P, CAP><<<grid, kThreads, 0, s>>>(t);
    return cudaGetLastError();
}

template <int CAP>
cudaError_t launch_norm_type(int p, const List &l, int i0, int n, bool last, int sm_count,
                             unsigned &slot, unsigned char *ws, float *norm, float *coef,
                             float max_norm, cudaStream_t s)
{
    if (p == GBSSIM_NORM_2)
        return launch_norm<2, CAP>(l, i0, n, last, sm_count, slot, ws, norm, coef, max_norm, s);
    if (p == GBSSIM_NORM_1)
        return launch_norm<1, CAP>(l, i0, n, last, sm_count, slot, ws, norm, coef, max_norm, s);
    return launch_norm<0, CAP>(l, i0, n, last, sm_count, slot, ws, norm, coef, max_norm, s);
}

// The scaling kernel starts while the norm kernel ends (programmatic dependent
// launch); it waits for its results before it reads the coefficient.
template <int CAP>
cudaError_t launch_scale(const List &l, int i0, int n, bool in_place, int sm_count,
                         const float *coef, cudaStream_t s)
{
    ScaleTable<CAP> t;
    long long chunks = 0;
    t.n = n;
    for (int i = 0; i < n; ++i) {
        t.g[i] = l.g[i0 + i];
        t.out[i] = l.out[i0 + i];
        t.count[i] = l.count[i0 + i];
        t.type[i] = l.type[i0 + i];
        t.out_type[i] = l.out_type[i0 + i];
        t.pad[i] = chunk_pad(t.g[i], t.type[i], t.out[i], t.out_type[i]);
        t.first[i] = unsigned(chunks);
        if (t.count[i] > 0)
            chunks += ceil_div(t.count[i] + (t.pad[i] & 7), kScaleElems);
    }
    t.first[n] = unsigned(chunks);
    t.in_place = in_place;
    t.coef = coef;
    if (chunks == 0) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid_for(chunks, sm_count));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, grad_scale_kernel<CAP>, t);
}

int check_list(const List &l)
{
    if (l.n < 0) return GBSSIM_EINVAL;
    if (l.n == 0) return GBSSIM_OK;
    if (!l.g || !l.count || !l.type) return GBSSIM_EINVAL;
    long long chunks = 0;
    for (int i = 0; i < l.n; ++i) {
        if (!dtype_ok(l.type[i])) return GBSSIM_EINVAL;
        if (l.count[i] < 0 || l.count[i] / kScaleElems > kMaxChunks) return GBSSIM_ESHAPE;
        chunks += l.count[i] / kScaleElems + 2;  // at least the tensor's chunks of either kernel
        if (chunks > kMaxChunks) return GBSSIM_ESHAPE;
        if (l.count[i] > 0 && !l.g[i]) return GBSSIM_EINVAL;
        if (reinterpret_cast<uintptr_t>(l.g[i]) % dtype_bytes(l.type[i])) return GBSSIM_EALIGN;
    }
    return GBSSIM_OK;
}

struct Range {
    uintptr_t at, end;
    bool out;
};

// Outputs may not overlap one another, nor any gradient but their own in place.
int check_outputs(const List &l, bool &in_place)
{
    in_place = true;
    if (l.n == 0) return GBSSIM_OK;
    if (!l.out || !l.out_type) return GBSSIM_EINVAL;
    Range *r = new (std::nothrow) Range[size_t(l.n) * 2];
    if (!r) return GBSSIM_EINVAL;
    int m = 0, rc = GBSSIM_OK;
    for (int i = 0; i < l.n && rc == GBSSIM_OK; ++i) {
        const uintptr_t o = reinterpret_cast<uintptr_t>(l.out[i]);
        if (!dtype_ok(l.out_type[i]) || (l.count[i] > 0 && !o)) rc = GBSSIM_EINVAL;
        else if (o % dtype_bytes(l.out_type[i])) rc = GBSSIM_EALIGN;
        else if (l.count[i] > 0) {
            const uintptr_t g = reinterpret_cast<uintptr_t>(l.g[i]);
            const bool own = o == g && l.out_type[i] == l.type[i];
            r[m++] = {o, o + uintptr_t(l.count[i]) * dtype_bytes(l.out_type[i]), true};
            if (!own) {
                in_place = false;
                r[m++] = {g, g + uintptr_t(l.count[i]) * dtype_bytes(l.type[i]), false};
            }
        }
    }
    if (rc == GBSSIM_OK) {
        std::sort(r, r + m, [](const Range &a, const Range &b) { return a.at < b.at; });
        uintptr_t any = 0, outs = 0;  // furthest ends so far
        for (int i = 0; i < m; ++i) {
            if (r[i].at < (r[i].out ? any : outs)) rc = GBSSIM_EINVAL;
            any = std::max(any, r[i].end);
            if (r[i].out) outs = std::max(outs, r[i].end);
        }
    }
    delete[] r;
    return rc;
}

size_t workspace_need(int n)
{
    return kPartialOffset + size_t(std::max<long long>(1, ceil_div(n, kCapLarge))) * kMaxBlocks * 8;
}

int check_common(const List &l, int norm_type, const float *out_norm, const void *workspace,
                 size_t workspace_bytes)
{
    const int rc = check_list(l);
    if (rc != GBSSIM_OK) return rc;
    if (norm_type < GBSSIM_NORM_INF || norm_type > GBSSIM_NORM_2 || !out_norm) return GBSSIM_EINVAL;
    if (reinterpret_cast<uintptr_t>(out_norm) % 4) return GBSSIM_EALIGN;
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 ||
        workspace_bytes < workspace_need(l.n))
        return GBSSIM_EWORKSPACE;
    return GBSSIM_OK;
}

// The norm's launches; the coefficient too where coef is not null.
int run_norm(const List &l, int norm_type, float *out_norm, float *coef, float max_norm,
             void *workspace, int sm_count, cudaStream_t s)
{
    unsigned slot = 0;
    int i0 = 0;
    do {
        const int n = std::min(l.n - i0, kCapLarge);
        const bool last = i0 + n == l.n;
        unsigned char *ws = static_cast<unsigned char *>(workspace);
        const cudaError_t e =
            n <= kCapSmall ? launch_norm_type<kCapSmall>(norm_type, l, i0, n, last, sm_count, slot,
                                                         ws, out_norm, coef, max_norm, s)
                           : launch_norm_type<kCapLarge>(norm_type, l, i0, n, last, sm_count, slot,
                                                         ws, out_norm, coef, max_norm, s);
        if (e != cudaSuccess) return cuda_fail(e);
        i0 += n;
    } while (i0 < l.n);
    return GBSSIM_OK;
}

}  // namespace
}  // namespace gbssim

using namespace gbssim;

extern "C" size_t gbssim_grad_workspace_bytes(int n) { return n < 0 ? 0 : workspace_need(n); }

extern "C" int gbssim_grad_norm(const void *const *grads, const long long *counts,
                                const unsigned char *dtypes, int n, int norm_type, float *out_norm,
                                void *workspace, size_t workspace_bytes, void *stream)
{
    const CallRange range("gbssim_grad_norm");
    const List l{grads, nullptr, counts, dtypes, nullptr, n};
    const int rc = check_common(l, norm_type, out_norm, workspace, workspace_bytes);
    if (rc != GBSSIM_OK) return rc;
    int sm_count = 0;
    const cudaError_t e = current_sm_count(&sm_count);
    if (e != cudaSuccess) return cuda_fail(e);
    return run_norm(l, norm_type, out_norm, nullptr, 0.0f, workspace, sm_count,
                    static_cast<cudaStream_t>(stream));
}

extern "C" int gbssim_grad_clip(const void *const *grads, void *const *outs,
                                const long long *counts, const unsigned char *dtypes,
                                const unsigned char *out_dtypes, int n, int norm_type,
                                float max_norm, float *out_norm, void *workspace,
                                size_t workspace_bytes, void *stream)
{
    const CallRange range("gbssim_grad_clip");
    const List l{grads, outs, counts, dtypes, out_dtypes, n};
    int rc = check_common(l, norm_type, out_norm, workspace, workspace_bytes);
    if (rc != GBSSIM_OK) return rc;
    if (!(max_norm >= 0.0f)) return GBSSIM_EINVAL;
    bool in_place = false;
    if ((rc = check_outputs(l, in_place))) return rc;
    int sm_count = 0;
    cudaError_t e = current_sm_count(&sm_count);
    if (e != cudaSuccess) return cuda_fail(e);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    float *coef = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + kCoefOffset);
    if ((rc = run_norm(l, norm_type, out_norm, coef, max_norm, workspace, sm_count, s))) return rc;
    for (int i0 = 0; i0 < n; i0 += kCapLarge) {
        const int m = std::min(n - i0, kCapLarge);
        e = m <= kCapSmall ? launch_scale<kCapSmall>(l, i0, m, in_place, sm_count, coef, s)
                           : launch_scale<kCapLarge>(l, i0, m, in_place, sm_count, coef, s);
        if (e != cudaSuccess) return cuda_fail(e);
    }
    return GBSSIM_OK;
}
