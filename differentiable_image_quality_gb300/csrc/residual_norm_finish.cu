// The second part of the residual norm's backward: the parameters' gradients from
// the blocks' column sums.  Its reads are the partials, some megabytes in most
// calls; what it costs there is the time of a few dependent loads, so a column's
// partials go to 16 to 64 threads, and a thread asks for all that it reads at once (8 x
// 2000 x 256 with a gate per sample 23 us one after the other, 18 so).  Calls of many
// samples with parameters of their own have many groups of few partials instead:
// there a thread takes a column of a group, and what all groups share is folded 16
// partials at a time first (16000 rows of 1001 columns in 8000 samples: 7.1 ms
// without that, 0.31 with).  Four blocks an SM in those: 8000 x 16 x 1001 940 us, 962
// with the two that the registers would leave.
#include <climits>

#include "residual_norm.cuh"

namespace gbssim {
namespace {

constexpr int kFinishCols = 8;
// Gradients that groups have of their own: from this many on a thread takes one, its
// partials one after the other, where 64 threads a column would make a long grid
// (backward, bfloat16, all parameters per sample: 4 x 400 x 4096 39 us, 32 so;
// 24 x 300 x 1024 41, 27; below, 8 x 1024 x 1152 33, 35 so, 2 x 400 x 4096 26, 31).
constexpr int kManyOwn = 12288;
constexpr int kGroupThreads = 256;

__device__ __forceinline__ void store_param(const ParamGrad &g, int group, int dim, int col, float v)
{
    if (!g.p) return;
    const long long i = (g.per_sample ? (long long)group * dim : 0) + col;
    if (g.type == GBSSIM_F32) static_cast<float *>(g.p)[i] = v;
    else if (g.type == GBSSIM_BF16) static_cast<bf16 *>(g.p)[i] = from_f32<bf16>(v);
    else static_cast<f16 *>(g.p)[i] = from_f32<f16>(v);
}

__device__ __forceinline__ const ParamGrad &output(const ParamGrads &g, int k)
{
    return k == 0 ? g.gate : k == 1 ? g.w1 : k == 2 ? g.b1 : k == 3 ? g.w2 : g.b2;
}

// A parameter's value at a column as it lies in memory: all are asked for before
// the first is converted.
__device__ __forceinline__ uint32_t ask(const ParamPtr &p, int group, int col)
{
    if (!p.p) return 0;
    const long long i = group * p.stride + col;
    return p.type == GBSSIM_F32 ? __ldg(static_cast<const uint32_t *>(p.p) + i)
                                : __ldg(static_cast<const unsigned short *>(p.p) + i);
}

__device__ __forceinline__ float told(const ParamPtr &p, uint32_t v)
{
    return p.type == GBSSIM_F32    ? __uint_as_float(v)
           : p.type == GBSSIM_BF16 ? __uint_as_float(v << 16)
                                   : __half2float(__ushort_as_half((unsigned short)v));
}

// What turns A and F into the gradients of a group's gate, w1 and b1.
struct Factors {
    uint32_t gate, w, b;
    __device__ __forceinline__ void fetch(const ResidualNormArgs &a, int group, int col)
    {
        gate = a.gate_rows.p ? 0 : ask(a.gate, group, col);
        w = ask(a.w1, group, col);
        b = ask(a.b1, group, col);
    }
};

// The column sums of a thread's partials, and the gradients they make.
struct ColumnSums {
    float A = 0.0f, F = 0.0f, C = 0.0f, E = 0.0f;

    __device__ __forceinline__ ColumnSums operator+(const ColumnSums &o) const
    {
        ColumnSums s;
        s.A = A + o.A, s.F = F + o.F, s.C = C + o.C, s.E = E + o.E;
        return s;
    }
    // adds to the gradients of gate, w1, b1, w2, b2
    __device__ __forceinline__ void add_to(float (&v)[5], const ResidualNormArgs &a, const Factors &f) const
    {
        const float gate = a.gate.p && !a.gate_rows.p ? told(a.gate, f.gate) : 1.0f;
        const float w = a.w1.p ? told(a.w1, f.w) + a.offset : 1.0f;
        v[0] += fmaf(w, A, told(a.b1, f.b) * F);
        v[1] = fmaf(gate, A, v[1]);
        v[2] = fmaf(gate, F, v[2]);
        v[3] += C;
        v[4] += E;
    }
};

// Reads partials: only the sums that the outputs of one kind (per sample or shared)
// are made of.
struct Reader {
    const float *p;
    long long step;         // from a partial to the next
    long long a, f, c, e;   // -1: not wanted
    __device__ __forceinline__ Reader(const ResidualNormArgs &n, const ParamGrads &g, bool shared, int col)
        : p(n.partials + col), step((long long)n.sums * n.dim)
    {
        const bool first = wants(g.gate, shared) || wants(g.w1, shared) || wants(g.b1, shared);
        a = first && n.sum_a >= 0 ? (long long)n.sum_a * n.dim : -1;
        f = first && n.sum_f >= 0 ? (long long)n.sum_f * n.dim : -1;
        c = wants(g.w2, shared) ? (long long)n.sum_c * n.dim : -1;
        e = wants(g.b2, shared) ? (long long)n.sum_e * n.dim : -1;
    }
    static __device__ __forceinline__ bool wants(const ParamGrad &g, bool shared)
    {
        return g.p && bool(g.per_sample) != shared;
    }
    __device__ __forceinline__ ColumnSums at(long long i, bool there) const
    {
        const float *q = p + i * step;
        ColumnSums s;
        if (there && a >= 0) s.A = __ldcg(q + a);
        if (there && f >= 0) s.F = __ldcg(q + f);
        if (there && c >= 0) s.C = __ldcg(q + c);
        if (there && e >= 0) s.E = __ldcg(q + e);
        return s;
    }
    // partials begin, begin + by, ... below end, four of them at a time
    __device__ __forceinline__ ColumnSums over(long long begin, long long end, int by) const
    {
        ColumnSums s;
        for (long long i = begin; i < end; i += 4 * by) {
            ColumnSums t[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k] = at(i + k * by, i + k * by < end);
            s = s + ((t[0] + t[1]) + (t[2] + t[3]));
        }
        return s;
    }
};

// Whether groups have different factors.
__host__ __device__ inline bool factors_vary(const ResidualNormArgs &a)
{
    return a.gate.stride || a.w1.stride || a.b1.stride;
}

// Adds v over the block's LANES threads of each of its COLS columns, in a fixed order,
// and stores the outputs that are per sample, or those that are not.
template <int COLS, int LANES>
__device__ __forceinline__ void finish_columns(float (&v)[5], const ResidualNormArgs &a,
                                               const ParamGrads &g, int first, int group, bool shared)
{
    constexpr int kWarps = COLS * LANES / 32;
    __shared__ float part[5][kWarps][COLS];
#pragma unroll
    for (int k = 0; k < 5; ++k) {
#pragma unroll
        for (int off = COLS; off < 32; off *= 2) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
        if ((threadIdx.x & 31) < COLS) part[k][threadIdx.x / 32][threadIdx.x & 31] = v[k];
    }
    __syncthreads();
    if (threadIdx.x < 5 * COLS) {
        const int k = threadIdx.x / COLS, to = first + threadIdx.x % COLS;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += part[k][w][threadIdx.x % COLS];
        const ParamGrad &out = output(g, k);
        if (to < a.dim && bool(out.per_sample) != shared) store_param(out, group, a.dim, to, s);
    }
}

// A block takes COLS columns (whole sectors of each partial), LANES threads of a
// column every LANES-th partial each.  Part y < groups of the grid makes the gradients
// that each group has of its own, the last those shared by all: where groups have
// factors of their own (at most LANES groups then), a thread's partials are of one.
template <int COLS, int LANES>
__global__ void __launch_bounds__(COLS * LANES)
    residual_norm_finish_kernel(const __grid_constant__ ResidualNormArgs a,
                                const __grid_constant__ ParamGrads g, int shared_part)
{
    const int lane = threadIdx.x / COLS;
    const int across = (a.dim + COLS - 1) / COLS;  // blocks of a part
    const int y = int(blockIdx.x) / across, first = (int(blockIdx.x) - y * across) * COLS;
    const int col = min(first + int(threadIdx.x) % COLS, a.dim - 1);
    const bool shared = y == shared_part;
    const int each = a.plan.classes * a.plan.splits;  // partials of a group
    const bool vary = shared && each > 0 && factors_vary(a);
    const int by = vary ? LANES / a.plan.groups : LANES;
    const int group = !shared ? y : vary ? min(lane / by, a.plan.groups - 1) : 0;
    const long long p0 = (long long)group * each;
    const long long p1 = shared && !vary ? (long long)a.plan.groups * each : p0 + each;
    Factors f{};
    if (a.plan.groups > 0) f.fetch(a, group, col);
    const Reader r(a, g, shared, col);
    float v[5] = {};
    pdl_wait();
    // (threads past the last group's have no partials)
    r.over(vary && lane >= by * a.plan.groups ? p1 : p0 + (vary ? lane % by : lane), p1, by).add_to(v, a, f);
    finish_columns<COLS, LANES>(v, a, g, first, y, shared);
}

// The gradients that groups have of their own, a thread for a column of a group.
__global__ void __launch_bounds__(kGroupThreads, 4)
    residual_norm_groups_kernel(const __grid_constant__ ResidualNormArgs a,
                                const __grid_constant__ ParamGrads g)
{
    const int across = (a.dim + kGroupThreads - 1) / kGroupThreads;
    const int group = int(blockIdx.x) / across;
    const int at = (int(blockIdx.x) - group * across) * kGroupThreads + threadIdx.x;
    const int col = min(at, a.dim - 1), each = a.plan.classes * a.plan.splits;
    Factors f;
    f.fetch(a, group, col);
    const Reader r(a, g, false, col);
    float v[5] = {};
    pdl_trigger();
    pdl_wait();
    r.over((long long)group * each, ((long long)group + 1) * each, 1).add_to(v, a, f);
#pragma unroll
    for (int k = 0; k < 5; ++k)
        if (at < a.dim && output(g, k).per_sample) store_param(output(g, k), group, a.dim, at, v[k]);
}

// kFoldedPartials partials of all groups into one set of the five gradients.
__global__ void __launch_bounds__(kGroupThreads, 4)
    residual_norm_fold_kernel(const __grid_constant__ ResidualNormArgs a,
                              const __grid_constant__ ParamGrads g, float *folded, int partials)
{
    const int across = (a.dim + kGroupThreads - 1) / kGroupThreads;
    const int chunk = int(blockIdx.x) / across;
    const int at = (int(blockIdx.x) - chunk * across) * kGroupThreads + threadIdx.x;
    const int col = min(at, a.dim - 1), each = a.plan.classes * a.plan.splits;
    const int p0 = chunk * kFoldedPartials, count = min(kFoldedPartials, partials - p0);
    const Reader r(a, g, true, col);
    float v[5] = {};
    pdl_trigger();
    pdl_wait();
    if (factors_vary(a)) {
        for (int i = 0; i < count; i += 4) {
            Factors f[4];
            ColumnSums t[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                f[k].fetch(a, (p0 + min(i + k, count - 1)) / each, col);
                t[k] = r.at(p0 + i + k, i + k < count);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) t[k].add_to(v, a, f[k]);
        }
    } else {
        Factors f;
        f.fetch(a, 0, col);
        r.over(p0, (long long)p0 + count, 1).add_to(v, a, f);
    }
    if (at >= a.dim) return;
#pragma unroll
    for (int k = 0; k < 5; ++k) folded[((long long)chunk * 5 + k) * a.dim + at] = v[k];
}

// The gradients shared by all groups, from the folded ones.
__global__ void __launch_bounds__(kFinishCols * kFinishLanes)
    residual_norm_finish_folded_kernel(const __grid_constant__ ResidualNormArgs a,
                                       const __grid_constant__ ParamGrads g, const float *folded,
                                       int chunks)
{
    const int first = int(blockIdx.x) * kFinishCols, col = first + threadIdx.x % kFinishCols;
    float v[5] = {};
    pdl_wait();
    if (col < a.dim) {
#pragma unroll 4
        for (int c = threadIdx.x / kFinishCols; c < chunks; c += kFinishLanes)
#pragma unroll
            for (int k = 0; k < 5; ++k) v[k] += __ldcg(folded + ((long long)c * 5 + k) * a.dim + col);
    }
    finish_columns<kFinishCols, kFinishLanes>(v, a, g, first, 0, true);
}

// Each of these kernels may start while the one ahead of it ends.
template <class... Params, class... Args>
cudaError_t launch_next(void (*kernel)(Params...), long long blocks, int threads, cudaStream_t s,
                        const Args &...args)
{
    if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

long long up(long long a, long long b) { return (a + b - 1) / b; }

}  // namespace

cudaError_t residual_norm_bwd_launch(const ResidualNormArgs &a, int res, int blk,
                                     const ParamGrads &g, cudaStream_t s)
{
    cudaError_t e = cudaSuccess;
    if (a.plan.grid > 0) {
        e = res == GBSSIM_F32 ? residual_norm_bwd_f32_launch(a, blk, s)
                              : residual_norm_bwd_16_launch(a, blk, s);
    }
    if (e != cudaSuccess || a.sums == 0) return e;
    bool own = false, shared = false;
    for (const ParamGrad *p : {&g.gate, &g.w1, &g.b1, &g.w2, &g.b2})
        if (p->p) (p->per_sample ? own : shared) = true;
    const int each = a.plan.classes * a.plan.splits;
    const long long partials = (long long)a.plan.groups * each;
    // (without rows there are no partials, and all gradients are zero)
    const bool many_own = own && (long long)a.plan.groups * a.dim >= kManyOwn && partials > 0;
    const bool many = shared && partials > 0 && a.plan.groups > kFinishLanes &&
                      (factors_vary(a) || partials > kMostUnfolded);
    if (many_own) {
        e = launch_next(residual_norm_groups_kernel, a.plan.groups * up(a.dim, kGroupThreads),
                        kGroupThreads, s, a, g);
        own = false;
    }
    if (e == cudaSuccess && many) {
        float *folded = a.partials + partials * a.sums * a.dim;
        const int n = int(partials), chunks = int(up(partials, kFoldedPartials));
        e = launch_next(residual_norm_fold_kernel, chunks * up(a.dim, kGroupThreads), kGroupThreads, s,
                        a, g, folded, n);
        if (e == cudaSuccess)
            e = launch_next(residual_norm_finish_folded_kernel, up(a.dim, kFinishCols),
                            kFinishCols * kFinishLanes, s, a, g,
                            static_cast<const float *>(folded), chunks);
        shared = false;
    }
    if (e != cudaSuccess || !(own || shared)) return e;
    // Blocks that all run at once: 64 threads a column, for the shortest chain of loads.
    // Otherwise fewer of them, by how many partials there are, and more columns a
    // block.  Backward, bfloat16, a gate per sample, with 8 columns of 64, 16 of 32 and
    // 16 of 16: 3000 x 1024 (256 blocks of the first) 18, 21, 23 us; 4000 x 2048 (512) 32,
    // 30, 30; 3000 x 4096 47, 45, 43; 1000 x 8192 49, 42, 40; 32 x 200 x 306 31, 29, 34;
    // 8 x 600 x 1024 29, 25, 26.
    constexpr int kLongGrid = 304, kFewPartials = 160;
    const int shared_part = own ? a.plan.groups : 0, parts = shared_part + (shared ? 1 : 0);
    if (parts == 0) return cudaSuccess;  // no samples: their own gradients are empty
    const int most_groups = shared && factors_vary(a) ? a.plan.groups : 0;
    if (parts * up(a.dim, kFinishCols) <= kLongGrid || most_groups > 32)
        return launch_next(residual_norm_finish_kernel<kFinishCols, kFinishLanes>,
                           parts * up(a.dim, kFinishCols), kFinishCols * kFinishLanes, s, a, g, shared_part);
    if (partials > kFewPartials || most_groups > 16)
        return launch_next(residual_norm_finish_kernel<16, 32>, parts * up(a.dim, 16), 512, s, a, g,
                           shared_part);
    return launch_next(residual_norm_finish_kernel<16, 16>, parts * up(a.dim, 16), 256, s, a, g, shared_part);
}

}  // namespace gbssim
