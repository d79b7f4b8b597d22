// Entry points of the residual norm: argument checks and launch planning.
#include <algorithm>
#include <climits>
#include <mutex>

#include "api_host.cuh"
#include "residual_norm.cuh"

using namespace gbssim;

namespace {

struct Extent {
    const void *p;
    size_t bytes;
};

int check_param(const gbssim_param &p)
{
    if (!p.data) return GBSSIM_OK;
    if (!dtype_ok(p.dtype) || (p.per_sample && p.sample_stride < 0)) return GBSSIM_EINVAL;
    return reinterpret_cast<uintptr_t>(p.data) % dtype_bytes(p.dtype) ? GBSSIM_EALIGN : GBSSIM_OK;
}

int check_rows(const gbssim_rows &r, int dtype)
{
    if (!r.data) return GBSSIM_OK;
    if (r.batch_stride < 0 || r.token_stride < 0) return GBSSIM_EINVAL;
    return reinterpret_cast<uintptr_t>(r.data) % dtype_bytes(dtype) ? GBSSIM_EALIGN : GBSSIM_OK;
}

int check_out(const void *p, int dtype)
{
    return reinterpret_cast<uintptr_t>(p) % dtype_bytes(dtype) ? GBSSIM_EALIGN : GBSSIM_OK;
}

long long row_count(const gbssim_residual_norm &d) { return (long long)d.batch * d.tokens; }

Extent rows_extent(const gbssim_residual_norm &d, const gbssim_rows &r, int dtype)
{
    if (!r.data || row_count(d) == 0) return {nullptr, 0};
    const long long last = (d.batch - 1) * r.batch_stride + (d.tokens - 1) * r.token_stride + d.dim;
    return {r.data, size_t(last) * dtype_bytes(dtype)};
}

Extent param_extent(const gbssim_residual_norm &d, const gbssim_param &p)
{
    const long long last = (p.per_sample ? (d.batch - 1) * p.sample_stride : 0) + d.dim;
    return {p.data, p.data && d.batch > 0 ? size_t(last) * dtype_bytes(p.dtype) : 0};
}

// A parameter's gradient: dense.
Extent grad_extent(const gbssim_residual_norm &d, const void *p, const gbssim_param &of)
{
    return {p, size_t(of.per_sample ? d.batch : 1) * d.dim * dtype_bytes(of.dtype)};
}

Extent dense_extent(const gbssim_residual_norm &d, const void *p, int dtype)
{
    return {p, size_t(row_count(d)) * d.dim * dtype_bytes(dtype)};
}

bool meet(const Extent &a, const Extent &b)
{
    return a.bytes && b.bytes && overlaps(a.p, a.bytes, b.p, b.bytes);
}

int check_desc(const gbssim_residual_norm *d)
{
    if (!d) return GBSSIM_EINVAL;
    if (!dtype_ok(d->res_dtype) || !dtype_ok(d->blk_dtype) ||
        (d->res_dtype != d->blk_dtype && d->res_dtype != GBSSIM_F32))
        return GBSSIM_EINVAL;
    for (int kind : {d->post_norm, d->pre_norm})
        if (kind < GBSSIM_ROW_NONE || kind > GBSSIM_ROW_LAYER) return GBSSIM_EINVAL;
    if (!(d->eps >= 0.0f)) return GBSSIM_EINVAL;
    if (d->batch < 0 || d->tokens < 0 || d->dim < 1 || d->dim > kMaxDim) return GBSSIM_ESHAPE;
    if (row_count(*d) > INT_MAX - 65536) return GBSSIM_ESHAPE;
    const bool some = row_count(*d) > 0;
    if (some && !d->x.data) return GBSSIM_EINVAL;
    // without a block's output there is nothing to normalise or gate
    const bool post_params = d->post_weight.data || d->post_bias.data;
    if (some && !d->y.data &&
        (d->gate_rows.data || d->gate.data || post_params || d->post_norm != GBSSIM_ROW_NONE))
        return GBSSIM_EINVAL;
    if (d->gate_rows.data && d->gate.data) return GBSSIM_EINVAL;
    int rc;
    if ((rc = check_rows(d->x, d->res_dtype)) || (rc = check_rows(d->y, d->blk_dtype)) ||
        (rc = check_rows(d->gate_rows, d->blk_dtype)) || (rc = check_param(d->gate)) ||
        (rc = check_param(d->post_weight)) || (rc = check_param(d->post_bias)) ||
        (rc = check_param(d->pre_weight)) || (rc = check_param(d->pre_bias)))
        return rc;
    return GBSSIM_OK;
}

// The inputs as extents.
int inputs_of(const gbssim_residual_norm &d, Extent *e)
{
    int n = 0;
    e[n++] = rows_extent(d, d.x, d.res_dtype);
    e[n++] = rows_extent(d, d.y, d.blk_dtype);
    e[n++] = rows_extent(d, d.gate_rows, d.blk_dtype);
    for (const gbssim_param *p : {&d.gate, &d.post_weight, &d.post_bias, &d.pre_weight, &d.pre_bias})
        e[n++] = param_extent(d, *p);
    return n;
}

bool multiple16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Eight elements of an output are stored at once.
bool out_aligned(const void *p, int dtype)
{
    return reinterpret_cast<uintptr_t>(p) % (8 * dtype_bytes(dtype)) == 0;
}

bool rows_aligned(const gbssim_residual_norm &d, const gbssim_rows &r, int dtype)
{
    const int v = 16 / dtype_bytes(dtype);
    return multiple16(r.data) && (d.batch < 2 || r.batch_stride % v == 0) &&
           (d.tokens < 2 || r.token_stride % v == 0);
}

bool inputs_aligned(const gbssim_residual_norm &d)
{
    return d.dim % kColsPerThread == 0 && rows_aligned(d, d.x, d.res_dtype) &&
           rows_aligned(d, d.y, d.blk_dtype) && rows_aligned(d, d.gate_rows, d.blk_dtype);
}

// A plan counts on as many resident threads of an SM as a block has at most (64
// registers each in the forward, 128 in the backward), or on `resident`.

// SMs that a plan counts on at most: bounds the partial sums on any device.
constexpr int kMaxPlanSms = 256;

// What a plan has to know of the device.
struct Room {
    int sms, clusters2, clusters4;
    int device;
    bool most;  // not of a device: at least what any has
};

// Read once per device.
int device_room(Room *out)
{
    constexpr int kMost = 64;
    static std::mutex mutex;
    static Room known[kMost];
    int dev = 0, sms = 0;
    cudaError_t e = current_sm_count(&sms, &dev);
    if (e != cudaSuccess) return cuda_fail(e);
    std::lock_guard<std::mutex> lock(mutex);
    Room fresh{}, &r = dev < kMost ? known[dev] : fresh;
    if (r.sms == 0) {
        ClusterRoom c{};
        e = residual_norm_cluster_room(&c);
        if (e != cudaSuccess) return cuda_fail(e);
        if (c.of2 < 1 || c.of4 < 1) return cuda_fail(cudaErrorInvalidConfiguration);
        r = {std::min(sms, kMaxPlanSms), std::min(c.of2, kMaxPlanSms / 2), std::min(c.of4, kMaxPlanSms / 4), dev, false};
    }
    *out = r;
    return GBSSIM_OK;
}

// Rows of one class that a sample with parameters of its own must have for its rows
// to be parted into classes.  The forward gains from one on (8 rows a sample of 1001
// columns in 64 samples: 9.9 -> 6.2 us, 16 in 512: 68 -> 27).  The backward pays a
// set of partial sums per class: 16 rows of 1001 in 512 samples 90 us, parted 96, and
// in 8000 samples 1016, parted 1128; 32 in 64 samples 43, parted 37.  Without such
// parameters the classes always pay (24 rows: forward 7.2 -> 4.3, backward 10.4 -> 7.4).
constexpr int kFwdClassRows = 1, kBwdClassRows = 4;

// Into how many parts to split each item (a group's rows of one class) for `blocks`
// blocks that run at once.  A block works through its rows in a loop, so a few
// blocks too many would double the time: the number of rounds is chosen, and with
// it the most parts that fit.  A round takes its rows and some start.  One more part
// than fits one round, as against this rule (backward, bfloat16, gate per sample):
// 2 x 1464 x 6830 190 us against 118, 5 x 2000 x 1152 55 against 43, 100 x 100 x 4096
// 179 against 136; never more than one round: the last 169 us, 160 x 100 x 4096 326
// against 263.
constexpr int kMostRounds = 8, kRoundStart = 8;  // in rows

int splits_for(long long items, long long rows, long long blocks)
{
    const long long rounds = ceil_div(items, blocks);
    long long best = 1, least = LLONG_MAX;
    if (rounds > kMostRounds) return 1;
    for (long long w = rounds; w <= 2 * rounds; ++w) {
        const long long s = std::min(w * blocks / items, rows);
        const long long time = w * (ceil_div(rows, s) + kRoundStart);
        if (time < least) {
            least = time;
            best = s;
        }
    }
    return int(best);
}

// At least what splits_for gives for as many blocks or fewer.
int most_splits(long long items, long long rows, long long blocks)
{
    if (ceil_div(items, blocks) > kMostRounds) return 1;
    return int(std::min(rows, std::max(3LL, 2 * ceil_div(blocks, items))));
}

RowPlan make_plan(const gbssim_residual_norm &d, int most_threads, int resident, int class_rows,
                  const Room &room)
{
    RowPlan p{};
    p.device = room.device;
    bool own = false;
    for (const gbssim_param *q : {&d.gate, &d.post_weight, &d.post_bias, &d.pre_weight, &d.pre_bias})
        own = own || (q->data && q->per_sample);
    const long long rows = row_count(d);
    p.groups = own ? d.batch : 1;
    p.group_rows = own ? d.tokens : int(rows);
    // Samples with parameters of their own may have too few rows to part into
    // classes.  The widest rows fill a cluster's threads without a shift.
    p.classes = d.dim % 8 == 0 ? 1 : d.dim % 4 == 0 ? 2 : d.dim % 2 == 0 ? 4 : 8;
    if ((own && p.group_rows < class_rows * p.classes) || d.dim + 7 > kMaxDim) p.classes = 1;
    const int chunks = (d.dim + (p.classes > 1 ? 7 : 0) + kColsPerThread - 1) / kColsPerThread;
    // A cluster's blocks have 512 threads at most, so that the forward has two on an
    // SM: 4000 x 13000 took 152 us with four blocks a row, 185 with two.
    const int most_shared = std::min(most_threads, 512);
    p.cluster = chunks <= most_threads ? 1 : chunks <= 2 * most_shared ? 2 : 4;
    const int per = (chunks + p.cluster - 1) / p.cluster;
    p.block_cols = per * kColsPerThread;
    if (per <= 32) {
        p.tpr = 1;
        while (p.tpr < per) p.tpr *= 2;
        p.threads = kSmallBlock;
        p.teams = kSmallBlock / p.tpr;
    } else {
        p.tpr = p.threads = (per + 31) / 32 * 32;
        p.teams = 1;
    }
    if (rows == 0) return p;
    const long long blocks =
        (long long)(p.cluster == 4 ? room.clusters4 : p.cluster == 2 ? room.clusters2 : room.sms) *
        (resident / p.threads);
    const long long items = (long long)p.groups * p.classes;
    const long long item_rows = ceil_div(ceil_div(p.group_rows, p.classes), p.teams);
    p.splits = room.most ? most_splits(items, item_rows, blocks) : splits_for(items, item_rows, blocks);
    p.grid = unsigned(items) * unsigned(p.splits) * unsigned(p.cluster);
    return p;
}

// Rows are addressed by batch and token, in one step where that is the same (and
// the step fits 32 bits).
bool one_stride(const gbssim_residual_norm &d, const gbssim_rows &r)
{
    return !r.data || ((d.batch < 2 || r.batch_stride == d.tokens * r.token_stride) &&
                       r.token_stride <= INT_MAX / 4);
}

// Whether a tensor's rows that a block meets, `classes` apart, all lie alike to a
// 16-byte boundary.
bool even(const RowPtr &p, const RowPlan &plan)
{
    return !p.p || (long long)p.row_bytes * plan.classes % 16 == 0;
}

bool dense(const gbssim_residual_norm &d, const gbssim_rows &r)
{
    return (d.tokens < 2 || r.token_stride == d.dim) &&
           (d.batch < 2 || r.batch_stride == (long long)d.tokens * d.dim);
}

RowPtr row_ptr(const gbssim_residual_norm &d, const gbssim_rows &r, int dtype)
{
    const Extent e = rows_extent(d, r, dtype);
    return {r.data, r.batch_stride, r.token_stride, static_cast<const char *>(e.p) + e.bytes,
            int(r.token_stride * dtype_bytes(dtype))};
}
ParamPtr param_ptr(const gbssim_param &p) { return {p.data, p.dtype, p.per_sample != 0, p.per_sample ? p.sample_stride : 0}; }

unsigned g_exchange_extra = 0;  // test hook, see gbssim_tune_exchange

ResidualNormArgs make_args(const gbssim_residual_norm &d)
{
    ResidualNormArgs a{};
    a.x = row_ptr(d, d.x, d.res_dtype);
    a.y = row_ptr(d, d.y, d.blk_dtype);
    a.gate_rows = row_ptr(d, d.gate_rows, d.blk_dtype);
    a.gate = param_ptr(d.gate);
    a.w1 = param_ptr(d.post_weight);
    a.b1 = param_ptr(d.post_bias);
    a.w2 = param_ptr(d.pre_weight);
    a.b2 = param_ptr(d.pre_bias);
    a.dim = d.dim;
    a.post = d.post_norm;
    a.pre = d.pre_norm;
    a.scale = d.residual_scale;
    a.offset = d.weight_offset;
    a.eps = d.eps;
    a.inv_dim = float(1.0 / d.dim);
    a.exchange_extra = g_exchange_extra;
    return a;
}

// Another plan's blocks for the same rows and columns.
void replan_blocks(RowPlan &p, const RowPlan &q)
{
    p.splits = q.splits;
    p.grid = q.grid;
}

bool grid_fits(const RowPlan &p)
{
    return (long long)p.groups * p.classes * p.splits * p.cluster <= INT_MAX;
}

// Which column sums the backward has to keep: A and F for the gate and the post
// norm, C and E for the pre norm.
int wanted_sums(const gbssim_residual_norm &d, const gbssim_residual_norm_grads &g,
                ResidualNormArgs &a)
{
    int n = 0;
    const bool gate = g.gate && !d.gate_rows.data;
    a.sum_a = gate || g.post_weight ? n++ : -1;
    a.sum_f = g.post_bias || (gate && d.post_bias.data) ? n++ : -1;
    a.sum_c = g.pre_weight ? n++ : -1;
    a.sum_e = g.pre_bias ? n++ : -1;
    return n;
}

constexpr int kMaxSums = 4;  // of a backward's partials

}  // namespace

extern "C" int gbssim_residual_norm_fwd(const gbssim_residual_norm *d, void *x_out_or_null,
                                        void *u_or_null, float *stats_or_null, void *stream)
{
    const CallRange range("gbssim_residual_norm_fwd");
    int rc = check_desc(d);
    if (rc != GBSSIM_OK) return rc;
    if (row_count(*d) == 0) return GBSSIM_OK;
    if ((d->y.data != nullptr) != (x_out_or_null != nullptr)) return GBSSIM_EINVAL;
    if (!x_out_or_null && !u_or_null) return GBSSIM_EINVAL;
    if ((rc = check_out(x_out_or_null, d->res_dtype)) || (rc = check_out(u_or_null, d->blk_dtype)))
        return rc;
    if (reinterpret_cast<uintptr_t>(stats_or_null) % 16) return GBSSIM_EALIGN;
    Extent in[8];
    const int n_in = inputs_of(*d, in);
    const Extent out[3] = {dense_extent(*d, x_out_or_null, d->res_dtype),
                           dense_extent(*d, u_or_null, d->blk_dtype),
                           {stats_or_null, stats_or_null ? size_t(row_count(*d)) * 16 : 0}};
    for (int i = 0; i < 3; ++i) {
        if (!out[i].p) continue;
        for (int j = 0; j < n_in; ++j) {
            // x' may take x's own place: every element is read before it is written
            const bool own = i == 0 && j == 0 && out[0].p == in[0].p && dense(*d, d->x);
            if (!own && meet(out[i], in[j])) return GBSSIM_EINVAL;
        }
        for (int j = 0; j < i; ++j)
            if (out[j].p && meet(out[i], out[j])) return GBSSIM_EINVAL;
    }
    Room room{};
    if ((rc = device_room(&room))) return rc;
    ResidualNormArgs a = make_args(*d);
    a.plan = make_plan(*d, kFwdThreads, kFwdThreads, kFwdClassRows, room);
    if (!grid_fits(a.plan)) return GBSSIM_ESHAPE;
    a.plan.aligned = inputs_aligned(*d) && out_aligned(x_out_or_null, d->res_dtype) &&
                     out_aligned(u_or_null, d->blk_dtype);
    a.tokens = one_stride(*d, d->x) && one_stride(*d, d->y) && one_stride(*d, d->gate_rows)
                   ? 0
                   : d->tokens;
    a.plan.uneven = !(even(a.x, a.plan) && even(a.y, a.plan));
    a.plan.even_out = d->dim * a.plan.classes % 8 == 0 && out_aligned(x_out_or_null, d->res_dtype) &&
                      out_aligned(u_or_null, d->blk_dtype);
    a.x_out = x_out_or_null;
    a.u = u_or_null;
    a.stats = reinterpret_cast<float4 *>(stats_or_null);
    return cuda_fail(residual_norm_fwd_launch(a, d->res_dtype, d->blk_dtype,
                                              static_cast<cudaStream_t>(stream)));
}

extern "C" size_t gbssim_residual_norm_workspace_bytes(const gbssim_residual_norm *d)
{
    if (check_desc(d) != GBSSIM_OK || row_count(*d) == 0) return 0;
    const RowPlan p = make_plan(*d, kBwdThreads, kBwdResidentPlain, kBwdClassRows,
                                {kMaxPlanSms, kMaxPlanSms / 2, kMaxPlanSms / 4, 0, true});
    const size_t partials = size_t(p.groups) * p.classes * p.splits;
    const size_t folded =
        p.groups > kFinishLanes ? (partials + kFoldedPartials - 1) / kFoldedPartials * 5 : 0;
    return (partials * kMaxSums + folded) * d->dim * sizeof(float);
}

extern "C" int gbssim_residual_norm_bwd(const gbssim_residual_norm *d,
                                        const gbssim_rows *grad_x_out_or_null,
                                        const gbssim_rows *grad_u_or_null, const float *stats,
                                        const gbssim_residual_norm_grads *grads, void *workspace,
                                        size_t workspace_bytes, void *stream)
{
    const CallRange range("gbssim_residual_norm_bwd");
    int rc = check_desc(d);
    if (rc != GBSSIM_OK) return rc;
    if (!grads) return GBSSIM_EINVAL;
    const gbssim_rows none{};
    const gbssim_rows gx = grad_x_out_or_null ? *grad_x_out_or_null : none;
    const gbssim_rows gu = grad_u_or_null ? *grad_u_or_null : none;
    const bool some = row_count(*d) > 0;
    if (some && (!stats || (!gx.data && !gu.data))) return GBSSIM_EINVAL;
    // a gradient is asked only of what is there
    if (some && ((grads->y && !d->y.data) || (grads->gate && !d->gate.data && !d->gate_rows.data) ||
                 (grads->post_weight && !d->post_weight.data) ||
                 (grads->post_bias && !d->post_bias.data) ||
                 (grads->pre_weight && !d->pre_weight.data) ||
                 (grads->pre_bias && !d->pre_bias.data)))
        return GBSSIM_EINVAL;
    const int gate_type = d->gate_rows.data ? d->blk_dtype : d->gate.dtype;
    if ((rc = check_rows(gx, d->res_dtype)) || (rc = check_rows(gu, d->blk_dtype)) ||
        (rc = check_out(grads->x, d->res_dtype)) || (rc = check_out(grads->y, d->blk_dtype)) ||
        (grads->gate && (rc = check_out(grads->gate, gate_type))) ||
        (grads->post_weight && (rc = check_out(grads->post_weight, d->post_weight.dtype))) ||
        (grads->post_bias && (rc = check_out(grads->post_bias, d->post_bias.dtype))) ||
        (grads->pre_weight && (rc = check_out(grads->pre_weight, d->pre_weight.dtype))) ||
        (grads->pre_bias && (rc = check_out(grads->pre_bias, d->pre_bias.dtype))))
        return rc;
    if (reinterpret_cast<uintptr_t>(stats) % 16) return GBSSIM_EALIGN;
    const size_t need = gbssim_residual_norm_workspace_bytes(d);
    if (need && (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 || workspace_bytes < need))
        return GBSSIM_EWORKSPACE;

    Extent in[11], out[8];
    int n_in = inputs_of(*d, in), n_out = 0;
    in[n_in++] = rows_extent(*d, gx, d->res_dtype);
    in[n_in++] = rows_extent(*d, gu, d->blk_dtype);
    in[n_in++] = {stats, size_t(row_count(*d)) * 16};
    const auto add_out = [&](const Extent &e) {
        if (e.p) out[n_out++] = e;
    };
    add_out(dense_extent(*d, grads->x, d->res_dtype));
    add_out(dense_extent(*d, grads->y, d->blk_dtype));
    if (d->gate_rows.data) add_out(dense_extent(*d, grads->gate, d->blk_dtype));
    else add_out(grad_extent(*d, grads->gate, d->gate));
    add_out(grad_extent(*d, grads->post_weight, d->post_weight));
    add_out(grad_extent(*d, grads->post_bias, d->post_bias));
    add_out(grad_extent(*d, grads->pre_weight, d->pre_weight));
    add_out(grad_extent(*d, grads->pre_bias, d->pre_bias));
    add_out({workspace, need});
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (in[j].p && meet(out[i], in[j])) return GBSSIM_EINVAL;
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return GBSSIM_EINVAL;
    }

    Room room{};
    if ((rc = device_room(&room))) return rc;
    ResidualNormArgs a = make_args(*d);
    a.gx = row_ptr(*d, gx, d->res_dtype);
    a.gu = row_ptr(*d, gu, d->blk_dtype);
    a.plan = make_plan(*d, kBwdThreads, kBwdThreads, kBwdClassRows, room);
    a.plan.aligned = inputs_aligned(*d) && rows_aligned(*d, gx, d->res_dtype) &&
                     rows_aligned(*d, gu, d->blk_dtype) && out_aligned(grads->x, d->res_dtype) &&
                     out_aligned(grads->y, d->blk_dtype) &&
                     (!d->gate_rows.data || out_aligned(grads->gate, d->blk_dtype));
    a.tokens = one_stride(*d, d->x) && one_stride(*d, d->y) && one_stride(*d, d->gate_rows) &&
                       one_stride(*d, gx) && one_stride(*d, gu)
                   ? 0
                   : d->tokens;
    a.plan.uneven = !(even(a.x, a.plan) && even(a.y, a.plan) && even(a.gate_rows, a.plan) &&
                      even(a.gx, a.plan) && even(a.gu, a.plan));
    a.plan.even_out = d->dim * a.plan.classes % 8 == 0 && out_aligned(grads->x, d->res_dtype) &&
                      out_aligned(grads->y, d->blk_dtype) &&
                      (!d->gate_rows.data || out_aligned(grads->gate, d->blk_dtype));
    a.stats = const_cast<float4 *>(reinterpret_cast<const float4 *>(stats));
    a.dx = grads->x;
    a.dy = grads->y;
    a.dgate_rows = d->gate_rows.data ? grads->gate : nullptr;
    a.partials = static_cast<float *>(workspace);
    a.sums = wanted_sums(*d, *grads, a);
    // the kernel for the plainest calls leaves room for more blocks: 71050 x 964
    // bfloat16 took 223 us with 512 threads an SM, 204 with 640
    if (residual_norm_bwd_plain(a) && (a.plan.aligned || d->blk_dtype != GBSSIM_F32))
        replan_blocks(a.plan, make_plan(*d, kBwdThreads, kBwdResidentPlain, kBwdClassRows, room));
    ParamGrads g{};
    if (!d->gate_rows.data) g.gate = {grads->gate, d->gate.dtype, a.gate.per_sample};
    g.w1 = {grads->post_weight, d->post_weight.dtype, a.w1.per_sample};
    g.b1 = {grads->post_bias, d->post_bias.dtype, a.b1.per_sample};
    g.w2 = {grads->pre_weight, d->pre_weight.dtype, a.w2.per_sample};
    g.b2 = {grads->pre_bias, d->pre_bias.dtype, a.b2.per_sample};
    if (!grid_fits(a.plan)) return GBSSIM_ESHAPE;
    return cuda_fail(residual_norm_bwd_launch(a, d->res_dtype, d->blk_dtype, g,
                                              static_cast<cudaStream_t>(stream)));
}

#ifdef GBSSIM_TEST_HOOKS
// ---- test build only (csrc/gbssim_test_hooks.h)
extern "C" void gbssim_tune_exchange(int extra_bytes)
{
    g_exchange_extra = extra_bytes > 0 ? unsigned(extra_bytes) : 0u;
}
#endif
