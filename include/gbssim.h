/*
 * gbssim.h -- C ABI of a fused, differentiable SSIM loss for NVIDIA GB300 (sm_103a).
 *
 * What is computed (per image n, channel c, output pixel p of the domain Omega):
 *   mu1, mu2, E[x^2], E[y^2], E[xy] under an 11x11 Gaussian window (sigma 1.5,
 *   weights normalised to sum to one) -- the five blurred quantities of the
 *   TriSSIM README, "How it works", with the fixed 11x11 window of the fused-ssim
 *   README introduction;
 *   S(p) = (2 mu1 mu2 + C1)(2 sigma12 + C2) / ((mu1^2 + mu2^2 + C1)(sigma11 + sigma22 + C2)),
 *   C1 = 0.01^2, C2 = 0.03^2 (images in [0, 1]: fused-ssim README, "Constraints");
 *   mean[n] = average of S over the channels and Omega of image n (fused-ssim
 *   README, "Usage", returns this mean).
 * The backward applies the adjoint of the blur (a "full" correlation) to the
 * upstream gradients of the statistics and combines them by the chain rule of
 * the TriSSIM README, "How it works":
 *   grad_img1 = B^T(g_mu1) + 2 img1 B^T(g_s11) + img2 B^T(g_s12), grad_img2 likewise.
 *
 * Padding (fused-ssim README, "Usage"):
 *   GBSSIM_VALID      Omega = (H-10) x (W-10): windows that lie inside the image.
 *                     Needs H, W >= 11 (and D >= 11 in 3D).
 *   GBSSIM_SAME_ZERO  Omega = H x W: the image is extended by zeros; border
 *                     windows are not renormalised.  Needs H, W >= 1.
 *
 * Conventions shared by every call below:
 *   - Images are contiguous float32, NCHW (2D) or NCDHW (3D), in DEVICE memory,
 *     4-byte aligned.  Values are expected in [0, 1] but are not checked; NaN
 *     propagates.
 *   - All pointers are caller-owned.  The library allocates no memory and keeps
 *     no state between calls except small per-device launch caches.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Every call
 *     is asynchronous on that stream.  Argument errors are returned before any
 *     launch; a failed launch returns GBSSIM_ECUDA.
 *   - Return value: GBSSIM_OK (0) or a negative status; nothing aborts.
 *   - Calls are deterministic: the same inputs give bit-identical outputs.
 *
 * Accuracy.  The arithmetic is float32 (the means are summed in double).  The
 * kernels evaluate an exactly equivalent form of the definition: values are
 * shifted by one pixel of their neighbourhood before they are squared (2D; a
 * constant 1/2 in 3D), the fourth blurred quantity is E[(x - y)^2] instead of
 * E[xy], and the chain rule is taken through x - y.  Against a double-precision
 * evaluation of the definition, for images in [0, 1], the test suite holds
 * per-image means to 1e-5, gradients to 1e-4 of their largest element, 2D SSIM
 * maps to 5e-6 and 3D maps to 3e-5, flat (constant) regions included.
 */
#ifndef GBSSIM_H
#define GBSSIM_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GBSSIM_ABI_VERSION 1

typedef enum { GBSSIM_VALID = 0, GBSSIM_SAME_ZERO = 1 } gbssim_padding;

enum {
    GBSSIM_OK = 0,
    GBSSIM_EINVAL = -1,     /* null pointer where one is required, bad enum, aliasing */
    GBSSIM_ESHAPE = -2,     /* N, C < 1, a spatial extent too small, or sizes too large */
    GBSSIM_EALIGN = -3,     /* a pointer not 4-byte aligned */
    GBSSIM_EWORKSPACE = -4, /* workspace or saved buffer missing or too small */
    GBSSIM_ECUDA = -5,      /* a CUDA runtime call or launch failed */
    GBSSIM_ETOOLARGE = -6   /* too large for the fixed scratch of ssim_fwd_noalloc */
};

/* ABI version of the loaded library (GBSSIM_ABI_VERSION at its build). */
int gbssim_abi_version(void);

/* A static, human-readable description of a status code. */
const char *gbssim_strerror(int status);

/* The eleven float32 taps the kernels use (host copy), w[0..10].  They are the
 * float32 roundings of exp(-(k-5)^2 / 4.5), k = 0..10, divided by their sum. */
void gbssim_window(float w[11]);

/* Kernel-side failures recorded on the current device since the previous call,
 * as bit flags in *flags_out, which this call then clears.
 *   bit 0 (GBSSIM_DEV_STAGING_TIMEOUT): a 2D kernel waited about a second for
 *   its staged input rows without them arriving; its blocks stopped early, so
 *   that call's gradients and map are not valid, and the mean of each image
 *   with a stopped block is NaN.
 *   bit 1 (GBSSIM_DEV_EXCHANGE_TIMEOUT): blocks of a residual norm that share a
 *   row (more than 4096 columns) waited about a second for one another's sums;
 *   that call's outputs are not valid.
 *   bit 2 (GBSSIM_DEV_ATTENTION_TIMEOUT): a block of an attention call waited about a
 *   second for a tile or a product; that call's outputs are not valid, rows that it had
 *   not written yet are NaN.
 * Synchronises the device: a diagnostic, not part of the hot path.  Returns
 * GBSSIM_OK, GBSSIM_EINVAL (null flags_out) or GBSSIM_ECUDA. */
#define GBSSIM_DEV_STAGING_TIMEOUT 1u
#define GBSSIM_DEV_EXCHANGE_TIMEOUT 2u
#define GBSSIM_DEV_ATTENTION_TIMEOUT 4u
int gbssim_device_status(unsigned *flags_out);

/* ------------------------------------------------------------------ 2D ----- */

/* Bytes of scratch that ssim_fwd needs for the given shape (per-block partial
 * sums and a completion counter).  Returns 0 if the shape is invalid.  The
 * buffer must be zero-filled once before its first use; every completed call
 * leaves it zero-filled again.  Two calls that run at the same time must not
 * share one workspace. */
size_t gbssim_workspace_bytes(int N, int C, int H, int W, int padding);

/* Bytes of the optional `saved` buffer of ssim_fwd: one float32 field the size
 * of the input for grad_img1, plus one more when want_grad2 != 0. */
size_t gbssim_saved_bytes(int N, int C, int H, int W, int want_grad2);

/* Forward.
 *   img1, img2       [N, C, H, W] float32, device.
 *   out_mean         [N] float32, device: mean SSIM of each image.
 *   out_map_or_null  [N, C, Ho, Wo] float32, device, or NULL: the SSIM map.
 *   saved_or_null    device buffer of saved_bytes >= gbssim_saved_bytes(..., want_grad2),
 *                    or NULL.  When given, the forward also computes, for each
 *                    image, the gradient of mean[n] itself (i.e. with dL = 1)
 *                    with respect to img1 (and img2 when want_grad2 != 0), so
 *                    that ssim_bwd is a single scaling pass.  NULL is the
 *                    inference mode ("train=False" of the fused-ssim README,
 *                    "Usage"): only the mean (and map) are computed.
 *   workspace        device buffer of workspace_bytes >= gbssim_workspace_bytes(...).
 */
int ssim_fwd(const float *img1, const float *img2, int N, int C, int H, int W, int padding,
             float *out_mean, float *out_map_or_null, float *saved_or_null, size_t saved_bytes,
             int want_grad2, void *workspace, size_t workspace_bytes, void *stream);

/* Backward of loss = sum_n dL[n] * mean[n] (dL = dLoss/dmean, [N] float32, device).
 *   saved_or_null    the buffer written by a matching ssim_fwd (same images, shape
 *                    and padding; want_grad2 set there if grad_img2 is wanted
 *                    here), or NULL to recompute everything from img1 and img2.
 *   grad_img1        [N, C, H, W] float32, device; overwritten (not accumulated).
 *   grad_img2_or_null  likewise, or NULL to skip it (fused-ssim README,
 *                    "Constraints": by default only img1 is differentiable).
 * Gradient buffers must not overlap img1, img2 or each other. */
int ssim_bwd(const float *dL, const float *img1, const float *img2, int N, int C, int H, int W,
             int padding, const float *saved_or_null, size_t saved_bytes, float *grad_img1,
             float *grad_img2_or_null, void *stream);

/* Forward and backward in one call, for a loss whose derivative with respect to
 * each image's mean SSIM is known before the forward -- the usual training loss
 * 1 - mean over the batch has dL[n] = -1/N.  One kernel pass computes the
 * means (and the map), the upstream gradients of the statistics, the adjoint
 * and the chain rule (TriSSIM README, "How it works"), so the statistics are
 * formed once and no intermediate field is written.  Arguments as in ssim_fwd
 * and ssim_bwd; dL is [N] float32 on the device, read by the kernel.  The
 * workspace is sized by gbssim_workspace_bytes. */
int ssim_fwd_bwd(const float *img1, const float *img2, int N, int C, int H, int W, int padding,
                 const float *dL, float *out_mean, float *out_map_or_null, float *grad_img1,
                 float *grad_img2_or_null, void *workspace, size_t workspace_bytes, void *stream);

/* Size of the device array behind ssim_fwd_noalloc (per GPU, for the process's life). */
#define GBSSIM_NOALLOC_SCRATCH_BYTES (1u << 20)

/* ssim_fwd for callers that cannot allocate device memory.  The pages describe
 * no such call; it exists for users of this library.  A plug-in running inside
 * an application that owns the device memory, or code on a latency-critical
 * path that must not call cudaMalloc (which can also synchronise the device),
 * cannot provide ssim_fwd's workspace.  This call takes the same arguments minus
 * the workspace and uses a fixed array that the library defines in device
 * memory instead: GBSSIM_NOALLOC_SCRATCH_BYTES on every GPU that loads the
 * library, held until the process exits.  It allocates nothing.
 *   - Shapes whose workspace (gbssim_workspace_bytes) would exceed that array
 *     return GBSSIM_ETOOLARGE; use ssim_fwd for them.  A 1 x 3 x 1080 x 1920
 *     pair needs about 35 KB of it.  This size check comes first: such a shape
 *     returns GBSSIM_ETOOLARGE whatever the other arguments are.  Any other
 *     argument error is reported as ssim_fwd reports it.
 *   - All calls on a device share the one array and it keeps the previous
 *     call's contents; the call clears the part that must start at zero, on
 *     `stream`, before its kernel.  Calls whose work overlaps on the GPU (other
 *     streams, other threads) race on it: order them on one stream.
 *   - Every call looks up the array's address on the current device (nothing
 *     is cached, so a device reset cannot leave a stale address).  The first
 *     call on each device also does the per-device set-up ssim_fwd does; make
 *     that first call before any stream capture.
 * Results are identical to ssim_fwd's. */
int ssim_fwd_noalloc(const float *img1, const float *img2, int N, int C, int H, int W,
                     int padding, float *out_mean, float *out_map_or_null, float *saved_or_null,
                     size_t saved_bytes, int want_grad2, void *stream);

/* ------------------------------------------------------- per-octave maps --- */
/* The per-octave stage of the ssimulacra2 hand-off page ("blur -> pointwise
 * sigma11 / sigma22 / sigma12 -> error maps", once per octave of a 2x pyramid),
 * with this library's 11x11 Gaussian window in place of that metric's
 * recursive blur and with SSIM's own three per-pixel maps as the error maps:
 *   l  = (2 mu1 mu2 + C1) / (mu1^2 + mu2^2 + C1)       luminance
 *   cs = (2 sigma12 + C2) / (sigma11 + sigma22 + C2)   contrast-structure
 *   S  = l * cs                                         SSIM (as ssim_fwd)
 * Octave 0 is the input pair; octave o + 1 is octave o downscaled 2x: each pixel
 * is the mean of the pixels of its 2x2 block that lie inside the image (so
 * ceil(H/2) x ceil(W/2); a ragged last row or column averages one or two
 * pixels).  The page gives no formula for the downscale or the error maps;
 * these are the plain readings.  Forward only; no gradients. */

/* Extents (H_o, W_o) of octave o: H_0 = H, H_{o+1} = ceil(H_o / 2). */

/* Workspace bytes of ssim_pyramid (0 if a shape or octave count is invalid:
 * octaves >= 1 and every octave extent must suit the padding, i.e. >= 11 for
 * valid).  Same zero-fill rule as gbssim_workspace_bytes.  It holds the
 * downscaled images of octaves 1 .. octaves-1 and the block partial sums. */
size_t gbssim_pyramid_workspace_bytes(int N, int C, int H, int W, int padding, int octaves);

/* Floats of the optional maps buffer: per octave o, three maps of
 * N*C*Ho_o*Wo_o floats (l, then cs, then S), octaves one after another.  0 if
 * invalid. */
size_t gbssim_pyramid_map_floats(int N, int C, int H, int W, int padding, int octaves);

/* Per-octave means and maps.
 *   img1, img2    [N, C, H, W] float32, device.
 *   octaves       number of octaves (>= 1).
 *   out_means     [octaves][3][N] float32, device: per octave the mean of l, of
 *                 cs and of S over the channels and output pixels of image n.
 *   maps_or_null  device buffer of gbssim_pyramid_map_floats(...) floats, or NULL.
 *   workspace     device buffer of gbssim_pyramid_workspace_bytes(...) bytes.
 * Octave 0's S mean equals ssim_fwd's mean. */
int ssim_pyramid(const float *img1, const float *img2, int N, int C, int H, int W, int padding,
                 int octaves, float *out_means, float *maps_or_null, void *workspace,
                 size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------ 3D ----- */
/* fused-ssim README, "3D data": the same statistics with an 11x11x11 window on
 * NCDHW volumes.  Arguments mean what they mean in 2D, with D added; both
 * paddings apply to all three axes (valid needs D, H, W >= 11).
 * The 3D calls keep two fields between their three kernels in the workspace:
 * the XY-blurred statistics of every slice and the Z-blurred derivatives of
 * SSIM, one float4 per (slice, output column) each; so ssim3d_bwd takes a
 * workspace too (it is only used when saved_or_null is NULL). */

/* Workspace bytes of ssim3d_fwd / ssim3d_bwd (0 for an invalid shape).  Same
 * zero-fill rule as gbssim_workspace_bytes. */
size_t gbssim3d_workspace_bytes(int N, int C, int D, int H, int W, int padding);

/* Bytes of the optional saved buffer (one field the size of the input per
 * wanted gradient). */
size_t gbssim3d_saved_bytes(int N, int C, int D, int H, int W, int want_grad2);

int ssim3d_fwd(const float *img1, const float *img2, int N, int C, int D, int H, int W,
               int padding, float *out_mean, float *out_map_or_null, float *saved_or_null,
               size_t saved_bytes, int want_grad2, void *workspace, size_t workspace_bytes,
               void *stream);

int ssim3d_bwd(const float *dL, const float *img1, const float *img2, int N, int C, int D,
               int H, int W, int padding, const float *saved_or_null, size_t saved_bytes,
               float *grad_img1, float *grad_img2_or_null, void *workspace,
               size_t workspace_bytes, void *stream);

/* The single-call forward + backward of ssim_fwd_bwd for volumes. */
int ssim3d_fwd_bwd(const float *img1, const float *img2, int N, int C, int D, int H, int W,
                   int padding, const float *dL, float *out_mean, float *out_map_or_null,
                   float *grad_img1, float *grad_img2_or_null, void *workspace,
                   size_t workspace_bytes, void *stream);

/* ------------------------------------- gradient norm and clipping --------- */
/* What a training step does between the loss's backward and the optimizer: the
 * global norm of all gradients, and clipping by it.  The tensors may be of
 * different types and lengths, each dense in memory (n, their order and their
 * shapes do not matter), aligned to its element size:
 *   S    = sum over all elements of g^2 (NORM_2) or |g| (NORM_1), max |g| (NORM_INF)
 *   norm = sqrt(S) (NORM_2), S (otherwise); 0 when there is no element
 *   c    = min(1, max_norm / (norm + 1e-6)),   out = g * c
 * Sums of squares are accumulated in float32 over at most 64 values, beyond
 * that in double; values whose squares leave float32's range are summed in
 * double throughout.  g * c is formed in float32 and rounded once.  A NaN
 * anywhere makes norm and c NaN; an infinity makes norm infinite and c zero
 * (so finite gradients become 0, infinite ones NaN), or 1 where max_norm is
 * infinite too (no limit, nothing is scaled): the caller decides, from the norm,
 * whether to skip the step. */

typedef enum { GBSSIM_F32 = 0, GBSSIM_BF16 = 1, GBSSIM_F16 = 2 } gbssim_dtype;
typedef enum { GBSSIM_NORM_INF = 0, GBSSIM_NORM_1 = 1, GBSSIM_NORM_2 = 2 } gbssim_norm_type;

/* Workspace bytes for n tensors.  Same zero-fill rule as gbssim_workspace_bytes;
 * 16-byte aligned.  A call's launches leave partial sums and c for one another in
 * it: calls that host threads make at the same time must not share one, not even
 * on one stream. */
size_t gbssim_grad_workspace_bytes(int n);

/* grads, counts, dtypes: HOST arrays of n device addresses, element counts and
 * gbssim_dtype codes (they are copied before the call returns).  out_norm: one
 * float32 on the device.  Up to 1024 tensors go through one launch. */
int gbssim_grad_norm(const void *const *grads, const long long *counts,
                     const unsigned char *dtypes, int n, int norm_type, float *out_norm,
                     void *workspace, size_t workspace_bytes, void *stream);

/* The norm, and every gradient scaled by c.  outs[i] may be grads[i] (in place,
 * same type) or another tensor of counts[i] elements of type out_dtypes[i], e.g.
 * a float32 main gradient of a 16-bit one.  Outputs must not overlap one another
 * or any other gradient.  max_norm: not negative. */
int gbssim_grad_clip(const void *const *grads, void *const *outs, const long long *counts,
                     const unsigned char *dtypes, const unsigned char *out_dtypes, int n,
                     int norm_type, float max_norm, float *out_norm, void *workspace,
                     size_t workspace_bytes, void *stream);

/* ---------------------------- the norms around a residual block, fused ---- */
/* One pass over what a transformer block does between its matrix products and
 * the residual stream: the norm after the block, its gate, the scaled residual
 * sum, and the norm before the next block.  Per row (one token) of dim columns,
 * x the residual stream and y the block's output:
 *   y^ = (y - m1) r1,   z = y^ (post_weight + o) + post_bias,
 *   x' = s x + gate z,
 *   x^ = (x' - m2) r2,  u = x^ (pre_weight + o) + pre_bias,
 * with m the row's mean (LAYER; zero for RMS) and r = 1 / sqrt(mean((. - m)^2) +
 * eps); ROW_NONE leaves a norm out (m = 0, r = 1).  A missing weight is 1
 * (without o), a missing bias 0, a missing gate 1.  s is residual_scale, o is
 * weight_offset, of both norms (1 for weights stored as a difference from one).
 *
 * Types: x and x' are res_dtype; y, u and a gate of its own per row blk_dtype;
 * res_dtype is blk_dtype or float32.  Each parameter has its own type.
 * Arithmetic is float32; each output is rounded once, and u is formed from x'
 * before x' is rounded.  Sums of a row's squares have to stay within float32's
 * range.  Rows that hold a NaN or an infinity affect no others.
 *
 * Shapes: batch x tokens rows, either of which may be 0 or 1; dim from 1 to
 * 16384.  Inputs may have any non-negative strides between rows (element
 * counts); the columns of a row are neighbours.  Outputs are dense. */

typedef enum { GBSSIM_ROW_NONE = 0, GBSSIM_ROW_RMS = 1, GBSSIM_ROW_LAYER = 2 } gbssim_row_norm;

/* A [batch, tokens, dim] tensor; data NULL: absent. */
typedef struct {
    const void *data;
    long long batch_stride, token_stride;
} gbssim_rows;

/* A [dim] parameter, or with per_sample != 0 a [batch, dim] one whose samples lie
 * sample_stride elements apart (>= 0); data NULL: absent. */
typedef struct {
    const void *data;
    int dtype, per_sample;
    long long sample_stride;
} gbssim_param;

typedef struct {
    int batch, tokens, dim;
    int res_dtype, blk_dtype;     /* gbssim_dtype */
    int post_norm, pre_norm;      /* gbssim_row_norm */
    float residual_scale, weight_offset, eps;
    gbssim_rows x, y;             /* y absent: x' = x, and only the pre norm is taken */
    gbssim_rows gate_rows;        /* a gate per row, or */
    gbssim_param gate;            /* a gate per column */
    gbssim_param post_weight, post_bias, pre_weight, pre_bias;
} gbssim_residual_norm;

/* Forward.
 *   x_out  [batch, tokens, dim] of res_dtype, given if and only if y is; may be x
 *          itself where x is dense.
 *   u      [batch, tokens, dim] of blk_dtype, or NULL: x' alone.
 *   stats  [batch * tokens][4] float32, 16-byte aligned, or NULL: m1, r1, m2, r2 of
 *          each row, which the backward needs.
 * One launch; no workspace. */
int gbssim_residual_norm_fwd(const gbssim_residual_norm *desc, void *x_out_or_null,
                             void *u_or_null, float *stats_or_null, void *stream);

/* Where the backward writes; NULL: not wanted.  x, y and the gradient of a gate per
 * row are dense [batch, tokens, dim] of their tensors' types; parameters' gradients
 * have their parameters' types and shapes, dense (summed over the rows that share
 * them). */
typedef struct {
    void *x, *y, *gate, *post_weight, *post_bias, *pre_weight, *pre_bias;
} gbssim_residual_norm_grads;

/* Workspace bytes of the backward (0 without rows, or for an invalid description);
 * 16-byte aligned, contents arbitrary.  As for gbssim_grad_workspace_bytes, calls
 * made at the same time must not share one, not even on one stream. */
size_t gbssim_residual_norm_workspace_bytes(const gbssim_residual_norm *desc);

/* Backward from the gradients of x' (res_dtype) and u (blk_dtype); either may be NULL
 * (zero).  desc is the forward's, stats what it wrote.  Outputs are overwritten, and
 * must not overlap any input or one another.  Without rows, the parameters'
 * gradients are zero. */
int gbssim_residual_norm_bwd(const gbssim_residual_norm *desc,
                             const gbssim_rows *grad_x_out_or_null,
                             const gbssim_rows *grad_u_or_null, const float *stats,
                             const gbssim_residual_norm_grads *grads, void *workspace,
                             size_t workspace_bytes, void *stream);

/* ------------------------------------------------------- rotary positions --- */
/* A [batch, tokens, heads, dim] tensor, strides in elements (the batch's is unused in
 * the packed form). */
typedef struct {
    const void *data;
    long long batch_stride, token_stride, head_stride;
} gbssim_heads;

/* Positions as rotations: the head's columns form pairs, pair p of axis a(p) turns by
 * the angle x f_p, x the token's position on that axis (a patch's row or column, a
 * frame's time, a voxel's coordinates) and f_p its frequency:
 *   (u, v) -> (u cos - v sin, u sin + v cos),   with inverse != 0 by the negative angle,
 * which undoes it and is its gradient.  The pairs of the axes follow one another: n =
 * pairs[0] + ... in all, 2 n <= dim; GBSSIM_ROTARY_HALF pairs columns p and p + n,
 * GBSSIM_ROTARY_ADJACENT 2 p and 2 p + 1.  Columns from 2 n on are copied.
 *
 * Angles are taken modulo a turn in 64-bit fixed point: what they lose is the rounding of
 * f_p / (2 pi) to float64, times the position, and then float32's of less than half a turn.
 * Frequencies are finite numbers of any size and sign (others make their pair NaN).
 * A float32 position that is NaN, infinite or above 9e18 makes its token's turned
 * columns of that axis NaN.  Results are rounded once from float32.
 *
 * Shapes: batch x tokens tokens (0 and 1 included), dim from 2 to 512, up to 65535
 * heads in each of two tensors that share their positions (queries and keys; 0 heads:
 * absent), any non-negative strides, the columns of a head side by side.  Outputs are
 * dense [batch, tokens, heads, dim] and must not overlap any input. */
#define GBSSIM_ROTARY_AXES 4
typedef enum { GBSSIM_POS_I32 = 0, GBSSIM_POS_I64 = 1, GBSSIM_POS_F32 = 2 } gbssim_pos_type;
typedef enum { GBSSIM_ROTARY_HALF = 0, GBSSIM_ROTARY_ADJACENT = 1 } gbssim_rotary_layout;

typedef struct {
    int batch, tokens, q_heads, k_heads, dim;
    int dtype;                     /* gbssim_dtype */
    int layout, inverse;
    int axes, pairs[GBSSIM_ROTARY_AXES];
    int pos_type;
    gbssim_heads q, k;
    const void *positions;         /* device, [batch, tokens, axes], an axis after the other */
    long long pos_batch_stride, pos_token_stride; /* elements, >= 0 */
    const double *frequencies;     /* device, [n]: radians for one unit of position */
} gbssim_rotary;

/* One launch; no workspace. */
int gbssim_rotary_turn(const gbssim_rotary *desc, void *q_out, void *k_out, void *stream);

/* ------------------------------------------------------------ attention --- */
/* Attention between the tokens of a batch, per head:
 *   s_ij = scale q_i . k_j,   p_ij = exp(s_ij - lse_i),   o_i = sum_j p_ij v_j,
 *   lse_i = log(sum_j exp(s_ij)),
 * over the keys j that query i sees.  A query that sees none has o = 0 and lse =
 * -infinity.  heads is a multiple of kv_heads: query head h reads the keys and
 * values of head h / (heads / kv_heads).
 *
 * Batch form: q is [sequences, q_tokens, heads, dim], k and v [sequences, k_tokens,
 * kv_heads, dim].  kv_lengths (device, [sequences], or NULL) says how many keys of a
 * sample count, from 0 to k_tokens; what lies behind them is not used, whatever it
 * holds.
 * Packed form (q_offsets and k_offsets given, device, [sequences + 1], ascending
 * from 0): sequences of any lengths, zero included, one behind the other in q
 * [q_tokens, heads, dim] and in k and v [k_tokens, kv_heads, dim]; sequence s has
 * the rows offsets[s] to offsets[s + 1] - 1 and sees no other's.  Rows behind the
 * last sequence belong to none: their outputs and gradients are zeros.
 * Lengths and offsets out of their range are brought into it: the results are then
 * not specified, but nothing outside the tensors is touched.
 *
 * causal != 0: query i sees the keys up to i + (keys - queries), the last query all
 * of them; keys and queries are the counts of the shapes (batch form, whatever
 * kv_lengths says: for samples that are padded behind their tokens) or of the sequence
 * (packed: also for new tokens against caches of different lengths).
 * A hidden key has p = 0 exactly.  A NaN or an infinity among the keys and values of
 * a query's own sequence may reach its output although it does not see them, and one
 * among queries and gradients the gradients of its own sequence.
 *
 * Types: bfloat16 or float16, one for all tensors.  Scores, statistics and sums are
 * float32; p is rounded to the tensors' type for its product with v (in float16 times a
 * power of two: what is 2^-25 of a row's largest keeps all digits, the least step is
 * 2^-35 of it), each output once.  Shapes: any number of tokens, 0 and 1 included; dim a multiple of 8 up to
 * 128.  Inputs have any positive strides that are multiples of 16 bytes, the
 * elements of a head side by side, and start on 16 bytes; outputs are dense. */

typedef struct {
    int sequences, q_tokens, k_tokens;
    int heads, kv_heads, dim;
    int dtype;    /* GBSSIM_BF16 or GBSSIM_F16 */
    int causal;
    float scale;  /* positive */
    gbssim_heads q, k, v;
    const int *kv_lengths, *q_offsets, *k_offsets;
} gbssim_attention;

/* Workspace bytes of the forward, or with backward != 0 the backward (0 for an invalid
 * description); 16-byte aligned, contents arbitrary.  Calls made at the same time must
 * not share one, not even on one stream. */
size_t gbssim_attention_workspace_bytes(const gbssim_attention *desc, int backward);

/* Forward.
 *   out  dense, of q's shape.
 *   lse  [sequences, heads, q_tokens] (packed: [heads, q_tokens]) float32, or NULL. */
int gbssim_attention_fwd(const gbssim_attention *desc, void *out, float *lse_or_null,
                         void *workspace, size_t workspace_bytes, void *stream);

/* Backward from the gradient of out and out itself (any strides that q may have):
 *   p_ij as above, from lse;  D_i = grad_out_i . out_i;
 *   ds_ij = p_ij (grad_out_i . v_j - D_i),
 *   grad_q_i = scale sum_j ds_ij k_j,  grad_k_j = scale sum_i ds_ij q_i,
 *   grad_v_j = sum_i p_ij grad_out_i,
 * the last two over all query heads that share the key head.  desc is the forward's,
 * out and lse are what it wrote.  Outputs are dense, of q's, k's and v's shapes, and
 * overwritten; NULL: not wanted.  p and ds are rounded to the tensors' type for their
 * products (in float16 times powers of two that keep small gradients, one for each key
 * head of a sequence, from its own finite |grad_out| and |v|), sums are float32.  A
 * query that sees one key has a zero gradient, exactly. */
int gbssim_attention_bwd(const gbssim_attention *desc, const gbssim_heads *grad_out,
                         const gbssim_heads *out, const float *lse, void *grad_q_or_null, void *grad_k_or_null,
                         void *grad_v_or_null, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GBSSIM_H */
