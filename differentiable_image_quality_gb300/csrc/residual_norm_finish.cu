// The second part of the residual norm's backward: the parameters' gradients from
// the blocks' column sums.  Its reads are the partials, some megabytes in most
// calls; what it costs there is the time of a few dependent loads, so a column's
// partials go to 64 threads.  Calls of thousands of samples with parameters of
// their own have many groups of few partials instead: there a thread takes a
// column of a group, and what all groups share is folded 64 partials at a time
// first (16000 rows of 1001 columns in 8000 samples: 7.1 ms without that).
#include <climits>

#include "residual_norm.cuh"

namespace gbssim {
namespace {

constexpr int kFinishCols = 8, kFinishLanes = 64;
// A group's partials go to one thread a column where they are fewer than this and
// the groups more: 64 lanes would idle and the grid be long (512 samples of 16 rows
// of 1001 columns: 96 us, 353 with 64 threads a column; 64 samples of 32: 37, 65).
constexpr int kFewPartials = 32;
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

// The gradients of gate, w1, b1, w2, b2 at one column, added up over partials.
struct ColumnGrads {
    float v[5] = {};
    // what turns A and F into the gradients, of one group
    float gate, w, b;
    __device__ __forceinline__ void factors(const ResidualNormArgs &a, int group, int col)
    {
        gate = a.gate.p && !a.gate_rows.p ? param_at(a.gate, group, col) : 1.0f;
        w = a.w1.p ? param_at(a.w1, group, col) + a.offset : 1.0f;
        b = a.b1.p ? param_at(a.b1, group, col) : 0.0f;
    }
    __device__ __forceinline__ void add(const ResidualNormArgs &a, long long p, int col)
    {
        const float *src = a.partials + p * a.sums * a.dim + col;
        const float A = a.sum_a >= 0 ? __ldcg(src + (long long)a.sum_a * a.dim) : 0.0f;
        const float F = a.sum_f >= 0 ? __ldcg(src + (long long)a.sum_f * a.dim) : 0.0f;
        const float C = a.sum_c >= 0 ? __ldcg(src + (long long)a.sum_c * a.dim) : 0.0f;
        const float E = a.sum_e >= 0 ? __ldcg(src + (long long)a.sum_e * a.dim) : 0.0f;
        v[0] += fmaf(w, A, b * F);
        v[1] = fmaf(gate, A, v[1]);
        v[2] = fmaf(gate, F, v[2]);
        v[3] += C;
        v[4] += E;
    }
};

// Whether groups have different factors.
__device__ __forceinline__ bool factors_vary(const ResidualNormArgs &a)
{
    return a.gate.stride || a.w1.stride || a.b1.stride;
}

// Adds v over the block's 64 threads of a column, in a fixed order, and stores the
// outputs that are per sample, or those that are not.
__device__ __forceinline__ void finish_columns(float (&v)[5], const ResidualNormArgs &a,
                                               const ParamGrads &g, int first, int group, bool shared)
{
    constexpr int kWarps = kFinishCols * kFinishLanes / 32;
    __shared__ float part[5][kWarps][kFinishCols];
    // a warp holds four threads of each column
#pragma unroll
    for (int k = 0; k < 5; ++k) {
        v[k] += __shfl_xor_sync(0xffffffffu, v[k], 8);
        v[k] += __shfl_xor_sync(0xffffffffu, v[k], 16);
        if ((threadIdx.x & 31) < kFinishCols) part[k][threadIdx.x / 32][threadIdx.x & 7] = v[k];
    }
    __syncthreads();
    if (threadIdx.x < 5 * kFinishCols) {
        const int k = threadIdx.x / kFinishCols, to = first + threadIdx.x % kFinishCols;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) s += part[k][w][threadIdx.x % kFinishCols];
        const ParamGrad &out = output(g, k);
        if (to < a.dim && bool(out.per_sample) != shared) store_param(out, group, a.dim, to, s);
    }
}

// A block takes 8 columns (one sector of each partial), 64 threads of a column
// every 64th partial each.  Part y < groups of the grid makes the gradients that
// each group has of its own, the last those shared by all.
__global__ void __launch_bounds__(kFinishCols * kFinishLanes)
    residual_norm_finish_kernel(const __grid_constant__ ResidualNormArgs a,
                                const __grid_constant__ ParamGrads g, int shared_part)
{
    const int lane = threadIdx.x / kFinishCols;
    const int across = (a.dim + kFinishCols - 1) / kFinishCols;  // blocks of a part
    const int y = int(blockIdx.x) / across, first = (int(blockIdx.x) - y * across) * kFinishCols;
    const int col = first + threadIdx.x % kFinishCols;
    const bool shared = y == shared_part;
    const int each = a.plan.classes * a.plan.splits;  // partials of a group
    const int p0 = shared ? 0 : y * each;
    const int p1 = shared ? a.plan.groups * each : p0 + each;
    ColumnGrads c;
    pdl_wait();
    if (col < a.dim && p0 < p1) {
        const bool vary = shared && factors_vary(a);
        if (!vary) c.factors(a, p0 / each, col);
#pragma unroll 4
        for (long long p = p0 + lane; p < p1; p += kFinishLanes) {
            if (vary) c.factors(a, int(p) / each, col);
            c.add(a, p, col);
        }
    }
    finish_columns(c.v, a, g, first, y, shared);
}

// The gradients that groups have of their own, a thread for a column of a group.
__global__ void __launch_bounds__(kGroupThreads)
    residual_norm_groups_kernel(const __grid_constant__ ResidualNormArgs a,
                                const __grid_constant__ ParamGrads g)
{
    const int across = (a.dim + kGroupThreads - 1) / kGroupThreads;
    const int group = int(blockIdx.x) / across;
    const int col = (int(blockIdx.x) - group * across) * kGroupThreads + threadIdx.x;
    const int each = a.plan.classes * a.plan.splits;
    pdl_wait();
    if (col >= a.dim) return;
    ColumnGrads c;
    c.factors(a, group, col);
#pragma unroll 4
    for (int p = 0; p < each; ++p) c.add(a, (long long)group * each + p, col);
#pragma unroll
    for (int k = 0; k < 5; ++k)
        if (output(g, k).per_sample) store_param(output(g, k), group, a.dim, col, c.v[k]);
}

// kFoldedPartials partials of all groups into one set of the five gradients.
__global__ void __launch_bounds__(kGroupThreads)
    residual_norm_fold_kernel(const __grid_constant__ ResidualNormArgs a, float *folded, int partials)
{
    const int across = (a.dim + kGroupThreads - 1) / kGroupThreads;
    const int chunk = int(blockIdx.x) / across;
    const int col = (int(blockIdx.x) - chunk * across) * kGroupThreads + threadIdx.x;
    const int each = a.plan.classes * a.plan.splits;
    pdl_wait();
    if (col >= a.dim) return;
    const int p0 = chunk * kFoldedPartials, count = min(kFoldedPartials, partials - p0);
    const bool vary = factors_vary(a);
    ColumnGrads c;
    c.factors(a, p0 / each, col);
#pragma unroll 4
    for (int i = 0; i < count; ++i) {
        if (vary && (p0 + i) % each == 0) c.factors(a, (p0 + i) / each, col);
        c.add(a, p0 + i, col);
    }
#pragma unroll
    for (int k = 0; k < 5; ++k) folded[((long long)chunk * 5 + k) * a.dim + col] = c.v[k];
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
    finish_columns(v, a, g, first, 0, true);
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
    const int threads = kFinishCols * kFinishLanes;
    const long long across = up(a.dim, kFinishCols);
    // (without rows there are no partials, and all gradients are zero)
    const bool few = own && each < kFewPartials && a.plan.groups > kFewPartials && partials > 0;
    const bool many = shared && partials > kMostUnfolded;
    if (few) {
        e = launch_next(residual_norm_groups_kernel, a.plan.groups * up(a.dim, kGroupThreads),
                        kGroupThreads, s, a, g);
        own = false;
    }
    if (e == cudaSuccess && many) {
        float *folded = a.partials + partials * a.sums * a.dim;
        const int n = int(partials), chunks = int(up(partials, kFoldedPartials));
        e = launch_next(residual_norm_fold_kernel, chunks * up(a.dim, kGroupThreads), kGroupThreads, s,
                        a, folded, n);
        if (e == cudaSuccess)
            e = launch_next(residual_norm_finish_folded_kernel, across, threads, s, a, g,
                            static_cast<const float *>(folded), chunks);
        shared = false;
    }
    if (e != cudaSuccess || !(own || shared)) return e;
    const int shared_part = own ? a.plan.groups : 0;
    return launch_next(residual_norm_finish_kernel, across * (shared_part + (shared ? 1 : 0)), threads,
                       s, a, g, shared_part);
}

}  // namespace gbssim
