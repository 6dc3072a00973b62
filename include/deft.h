/*
 * deft.h -- C ABI of the MI355X (gfx950) deformable 3x3 convolution library.
 *
 * The layer (DefT explainer page, "The argument in one glance", parts "What
 * people did" and "This paper's idea"; "Following a deformable layer through
 * DefT", step 1): an offset convolution over the input predicts, for every
 * filter tap at every output pixel, a fractional (dy, dx); each tap's sample
 * point (its grid position plus that offset) is bilinearly interpolated from
 * its four neighbouring input pixels into a deformed column buffer; the main
 * convolution is a dense GEMM over those columns.  The offset convolution and
 * the sampling run fused in one kernel so the offsets never leave the chip,
 * and the input tile plus a halo sized from the offset distribution is staged
 * in LDS (section "How DefT works", "The idea"; "Why it works").
 *
 * Conventions for every call:
 *  - Tensors are dense, row-major, on the device, owned by the caller.  The
 *    library allocates no device memory in forward/backward; all scratch lives
 *    in the caller's workspace.
 *  - x [N][Cin][H][W]; w_off [Oc][Cin][kh][kw] with Oc = 2*G*kh*kw, channel
 *    2*(g*kh*kw + k) is dy and 2*(g*kh*kw + k)+1 is dx of tap k = i*kw + j of
 *    offset group g (channels [g*Cin/G, (g+1)*Cin/G)); b_off [Oc];
 *    w [Cout][Cin][kh][kw]; b [Cout]; y [N][Cout][Ho][Wo];
 *    offsets [N][Oc][Ho][Wo] are always fp32.  x, weights, biases, y, dy and
 *    the gradients have the descriptor's dtype.
 *  - Ho = (H + 2*pad_h - dil_h*(kh-1) - 1)/stride_h + 1, likewise Wo.
 *  - Out-of-image corners read zero; a tap whose sample point is not inside
 *    -1 < py < H, -1 < px < W (or is NaN) reads zero and gets no gradient.
 *  - `stream` is a hipStream_t (NULL = the null stream).  Calls are
 *    asynchronous on that stream; nothing synchronises implicitly.
 *  - Return 0 on success or a negative DEFT_ERR_* code.  Every argument is
 *    validated before anything is launched; on error nothing is launched and
 *    no output is touched.  A plan with N = 0 makes deft_forward,
 *    deft_backward and deft_debug_sample no-ops that return 0 without
 *    checking the tensor pointers (an empty batch has none).
 */
#ifndef DEFT_H
#define DEFT_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum deft_dtype { DEFT_F32 = 0, DEFT_BF16 = 1 };

enum deft_status {
  DEFT_OK = 0,
  DEFT_ERR_BAD_DESC = -1,     /* non-positive size, kernel, stride or dilation; negative pad */
  DEFT_ERR_GROUPS = -2,       /* offset_groups < 1 or Cin not divisible by it */
  DEFT_ERR_SHAPE = -3,        /* Ho or Wo < 1 */
  DEFT_ERR_NULLPTR = -4,      /* a required pointer is NULL */
  DEFT_ERR_WORKSPACE = -5,    /* workspace NULL or smaller than deft_workspace_bytes */
  DEFT_ERR_DTYPE = -6,        /* dtype not DEFT_F32 / DEFT_BF16 */
  DEFT_ERR_ALIGN = -7,        /* a device pointer is not 16-byte aligned */
  DEFT_ERR_HIP = -8,          /* a HIP runtime call or launch failed */
  DEFT_ERR_PLAN = -9,         /* forced tile/halo/chunk outside the supported range */
  DEFT_ERR_UNSUPPORTED = -10, /* channels per offset group not a multiple of 16, or size limits */
  DEFT_ERR_SCRATCH = -11      /* deft_forward_noalloc: the plan's forward scratch exceeds
                                 DEFT_NOALLOC_SCRATCH_BYTES */
};

/* Size of the static device scratch of deft_forward_noalloc (per GPU). */
#define DEFT_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/* Layer descriptor.  Main-convolution groups are 1; offset_groups = G. */
typedef struct deft_desc {
  int n, c_in, h, w, c_out, kh, kw;
  int stride_h, stride_w, pad_h, pad_w, dil_h, dil_w;
  int offset_groups;
  int dtype; /* enum deft_dtype */
} deft_desc;

/* Execution plan (opaque): output tile, halo, channel chunk, launch shape. */
typedef struct deft_plan deft_plan;

typedef struct deft_plan_info {
  int tile_h, tile_w;     /* output pixels per workgroup tile of the fused kernel */
  int halo;               /* LDS halo in input pixels around the tile's footprint (LDS-halo
                             forward; unused by the direct gather) */
  int chunk;              /* channels staged per LDS pass */
  int groups_per_wg;      /* offset groups handled by one workgroup */
  int num_workgroups;     /* fused-kernel grid size */
  int ho, wo, oc;
  int lds_bytes;          /* fused-kernel LDS per workgroup */
  double est_miss_fraction; /* planner's estimate of the share of taps outside bwd_halo, which
                               take the backward's slow path (-1: forced plan) */
  size_t ws_forward, ws_training;
  size_t ws_cols_offset;  /* byte offset in the workspace of the deformed columns
                             [N*Ho*Wo][kh*kw][Cin] that deft_forward leaves there */
  int bwd_tile_h, bwd_tile_w; /* output tile of the sampling backward */
  int bwd_chunk;          /* its channel chunk; 0: this plan has no backward (LDS) */
  int gemm_direct;        /* 1: the three GEMMs stage operands with direct global-to-LDS
                             loads (bf16, Ho*Wo and c_out multiples of 8, operands under
                             2 GiB); 0: register-staged generic GEMM */
  int dw_splits;          /* pixel ranges the dW GEMM is split into (one fp32 partial each) */
  int gather_direct;      /* 1: the forward gathers corners from a channel-minor copy of x held
                             in the caches (no LDS halo; halo then bounds only the backward's
                             candidate window); 0: LDS tile + halo */
  int gather_gemm;        /* 1: the forward runs the offset conv, then one launch that gathers the
                             columns straight into the main GEMM's LDS tiles (y and the columns
                             written; the GEMM reads no columns from HBM) */
  int bwd_halo;           /* the sampling backward's candidate window: taps whose corner lies
                             within it of their grid position are scattered through LDS, the
                             others one by one with global atomics */
} deft_plan_info;

/* Checks the descriptor alone.  Pure host function. */
int deft_desc_validate(const deft_desc* d);

/* Builds a plan.  halo_hist (host memory, may be NULL) is the required-halo
 * histogram of deft_halo_histogram: hist[i] for i < hist_len-2 counts taps
 * whose corner (y0, x0) lies exactly i pixels (Chebyshev distance) from the
 * tap's grid position, hist[hist_len-2] counts taps at hist_len-2 or more,
 * hist[hist_len-1] counts fully outside taps.  The forward's LDS halo, tile
 * and chunk come from a cost estimate (columns written, input staged, taps
 * outside the halo read from the caches, LDS occupancy and launch shape);
 * the backward's halo is the smallest that leaves at most 1e-5 of the taps
 * outside it besides those in the open-ended bin hist[hist_len-2], at most
 * 16.  NULL: forward halo from default shares, backward halo 4.  (DefT
 * page, "How DefT works", "The idea": pad each tile by just enough margin
 * that most sampled pixels stay on chip; "What it costs": tile sizing
 * depends on platform and layer shape.)  A forced plan uses its halo for
 * both.  Pure host function. */
int deft_plan_create(const deft_desc* d, const uint32_t* halo_hist, int hist_len,
                     deft_plan** out);

/* Plan with a forced tile (tile_h*tile_w <= 64), halo (0..32) and channel
 * chunk (multiple of 16 dividing Cin/G, at most 64; 0 = largest that fits;
 * -1 = direct gather: the forward reads the corners from a channel-minor copy
 * of x instead of an LDS halo; Cin a multiple of 16, at most 9 taps, and
 * Cin/(vG) a power of two <= 256 with v = 8 (bf16) or 4 (fp32) channels per
 * 16 bytes; -2 = direct gather fused into the main GEMM (bf16), which also needs Cin/G and
 * Cin multiples of 32, Ho*Wo and c_out multiples of 8).
 * DEFT_ERR_PLAN if its LDS does not fit or the direct gather is unsupported; deft_backward returns DEFT_ERR_PLAN
 * for a forced plan whose backward tile does not fit even with 8 channels.
 * Forward results (offsets, columns, y) are bit-identical across plans; the
 * backward's atomically accumulated sums (dx, dw, dw_off) and the per-chunk
 * offset-gradient partials agree across plans within rounding. */
int deft_plan_create_forced(const deft_desc* d, int tile_h, int tile_w, int halo, int chunk,
                            deft_plan** out);

int deft_plan_get_info(const deft_plan* p, deft_plan_info* info);
void deft_plan_destroy(deft_plan* p);

/* Workspace bytes for deft_forward (training = 0) or for a forward whose
 * columns are kept for deft_backward (training = 1). */
size_t deft_workspace_bytes(const deft_plan* p, int training);

/* Forward of the layer (DefT explainer page, "Following a deformable layer
 * through DefT": the offset convolution predicts each tap's fractional
 * displacement, the four neighbours of every displaced tap are blended
 * bilinearly into the deformed columns, and the main convolution multiplies
 * them; "This paper's idea": the offset convolution and the interpolation run
 * as one kernel, so the offsets stay on chip).  x, w_off, w, y and workspace
 * are required; b_off and b may be NULL (zero bias).  offsets_out (fp32
 * [N][Oc][Ho][Wo]) may be NULL; when given, the fused kernel also writes the
 * offsets it computed there (needed by deft_backward).  The deformed columns
 * are left in the workspace.  DEFT_ERR_NULLPTR, DEFT_ERR_WORKSPACE (NULL or
 * smaller than deft_workspace_bytes(p, 0)), DEFT_ERR_ALIGN; checks run before
 * any launch. */
int deft_forward(const deft_plan* p, const void* x, const void* w_off, const void* b_off,
                 const void* w, const void* b, void* y, float* offsets_out, void* workspace,
                 size_t ws_bytes, void* stream);

/* deft_forward for callers that cannot allocate device memory (code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc):
 * same arguments, checks, kernels and results as deft_forward, but with no
 * workspace argument.  The scratch that deft_forward takes from the workspace
 * lives in a static device array of the library, DEFT_NOALLOC_SCRATCH_BYTES
 * (64 MiB) per GPU, which every GPU the library runs on holds until the
 * process ends.  The call allocates nothing: on the first call with a device
 * current it looks up that device's copy of the array (hipGetSymbolAddress)
 * and keeps the address.  `stream` must belong to the current device.
 * DEFT_ERR_SCRATCH, before anything is launched, when
 * deft_workspace_bytes(p, 0) exceeds DEFT_NOALLOC_SCRATCH_BYTES (at C = 256,
 * 56 x 56, bf16 that is about 16.4 MB per image: up to 3 images).  Every
 * call on one GPU shares that GPU's array and leaves its contents there
 * (the next call overwrites what it reads before reading it): calls that
 * overlap on one GPU, on different streams or threads, race and must be
 * serialised by the caller.  The columns it leaves in the array are not
 * available to deft_backward (inference only). */
int deft_forward_noalloc(const deft_plan* p, const void* x, const void* w_off, const void* b_off,
                         const void* w, const void* b, void* y, float* offsets_out, void* stream);

/* deft_forward that also observes the offset distribution: the fused
 * sampling launch adds the required-halo histogram of every tap it samples to
 * `hist` (device uint32 [hist_len], 3 <= hist_len <= 64; the same bins as
 * deft_halo_histogram).  The counts are ADDED: the caller zeroes the buffer
 * and may let several calls accumulate before re-planning with
 * deft_plan_create (DefT page, "What to keep in mind": the gains rest on the
 * offset distribution, which shifts as training goes on and differs per
 * layer).  Other outputs are those of deft_forward.  DEFT_ERR_BAD_DESC for
 * hist_len out of range, DEFT_ERR_NULLPTR for a NULL hist (N > 0),
 * DEFT_ERR_ALIGN if hist is not 4-byte aligned; checks run before any launch. */
int deft_forward_hist(const deft_plan* p, const void* x, const void* w_off, const void* b_off,
                      const void* w, const void* b, void* y, float* offsets_out, void* workspace,
                      size_t ws_bytes, uint32_t* hist, int hist_len, void* stream);

/* The same forward in the unfused three-operator form the DefT explainer page
 * compares against ("What people did before this paper", "The argument in one
 * glance"): an offset-convolution launch writes the offsets to HBM
 * (`offsets`, fp32 [N][Oc][Ho][Wo], required), a sampling launch reads them
 * back with the input and writes the deformed columns, then the GEMM.  Same
 * arguments, checks and error codes as deft_forward, plus DEFT_ERR_NULLPTR
 * when `offsets` is NULL.  y, offsets and the columns left in the workspace
 * are bit-identical to deft_forward's with the same plan (same arithmetic in
 * the same order), so deft_backward may follow it. */
int deft_forward_unfused(const deft_plan* p, const void* x, const void* w_off, const void* b_off,
                         const void* w, const void* b, void* y, float* offsets, void* workspace,
                         size_t ws_bytes, void* stream);

/* Backward of the layer.  The DefT explainer page speaks of training only
 * through its cost ("This paper's idea", "Why it works": the layer's share of
 * training time), so this is the exact derivative of deft_forward: dW and db
 * of the main convolution, dCol, the bilinear scatter of dCol into dX with the
 * offset gradient from the corner differences, and the offset convolution's
 * dW_off, db_off and its contribution to dX.  It belongs to the forward that
 * last ran on this workspace (sized with training = 1; that forward must have
 * written offsets_out, passed here as `offsets`).  dy [N][Cout][Ho][Wo].
 * Writes (overwrites) dx, dw_off, dw; db_off and db may be NULL.  Gradients
 * are accumulated in fp32 and rounded once to the dtype.  DEFT_ERR_NULLPTR,
 * DEFT_ERR_WORKSPACE, DEFT_ERR_ALIGN, DEFT_ERR_PLAN (a plan without a
 * backward: bwd_chunk 0); checks run before any launch. */
int deft_backward(const deft_plan* p, const void* x, const void* w_off, const void* w,
                  const float* offsets, const void* dy, void* workspace, size_t ws_bytes,
                  void* dx, void* dw_off, void* db_off, void* dw, void* db, void* stream);

/* The integer tap-index / corner-mask stage on its own (DefT explainer page,
 * "Following a deformable layer through DefT", step 1: every filter position
 * at every output location gets its own sampling point), from fp32 offsets:
 * for every (n, g, k, ho, wo), laid out [N][G][kh*kw][Ho][Wo]:
 * py = float(ho*s - p + i*d) + dy (one fp32 add), px likewise; fully outside
 * taps give y0 = x0 = 0, mask = 0; otherwise y0 = floor(py), x0 = floor(px)
 * and mask bit q (q = 0..3 for corners (y0,x0), (y0,x0+1), (y0+1,x0),
 * (y0+1,x0+1)) is set when that corner is in the image.  Same device code as
 * the fused kernel. */
int deft_debug_sample_index(const deft_desc* d, const float* offsets, int32_t* y0, int32_t* x0,
                            uint8_t* mask, void* stream);

/* The sampling stage alone from given fp32 offsets, as the separate
 * interpolation operator of the three-operator layer (DefT explainer page,
 * "What people did before this paper"), writing the deformed columns
 * [N][Ho*Wo][kh*kw][Cin] (tap-major, channel-minor) of the descriptor's dtype
 * to `cols`.  DEFT_ERR_NULLPTR, DEFT_ERR_ALIGN (x and cols 16-byte, offsets
 * 4-byte aligned), DEFT_ERR_PLAN; checks run before any launch. */
int deft_debug_sample(const deft_plan* p, const void* x, const float* offsets, void* cols,
                      void* stream);

/* Required-halo histogram (device uint32 [hist_len], hist_len >= 3,
 * overwritten) of fp32 offsets, as described at deft_plan_create. */
int deft_halo_histogram(const deft_desc* d, const float* offsets, uint32_t* hist, int hist_len,
                        void* stream);

/* Dilated depthwise 1-D convolution, the workload of the JAX issue page on
 * grouped and dilated convolutions (its reproduction script: depthwise
 * lax.conv_general_dilated with feature_group_count = channels, "NTC" input,
 * "TIO" kernel with one input feature per group, stride 1, VALID padding,
 * rhs_dilation = dilation).  fp32, device pointers:
 *   x [batch][steps + dilation*(ksize-1)][channels]  (channel-minor)
 *   w [ksize][channels]
 *   y [batch][steps][channels]  (written)
 *   y[b][t][c] = sum_k w[k][c] * x[b][t + k*dilation][c].
 * channels a multiple of 4, 1 <= ksize <= 256, dilation >= 1, all pointers
 * 16-byte aligned.  DEFT_ERR_BAD_DESC for sizes out of range (also when the
 * input length exceeds 2^31 - 1 steps), DEFT_ERR_NULLPTR, DEFT_ERR_ALIGN; checks
 * run before any launch.  batch = 0 or steps = 0 is a no-op.  Asynchronous on
 * `stream`; the caller owns every buffer. */
int deft_dwconv1d_forward(const float* x, const float* w, float* y, int batch, int steps, int channels,
                          int ksize, int dilation, void* stream);

/* The depthwise convolution above followed by a pointwise (1x1) convolution,
 * fused so that the depthwise result never reaches memory (the FCM abstract's
 * fused depthwise + pointwise module).  fp32, device pointers:
 *   x    [batch][steps + dilation*(ksize-1)][channels]
 *   w_dw [ksize][channels]
 *   w_pw [channels][out_channels]
 *   z    [batch][steps][out_channels]  (written)
 *   z[b][t][o] = sum_c w_pw[c][o] * sum_k w_dw[k][c] * x[b][t + k*dilation][c].
 * channels and out_channels multiples of 32, 1 <= ksize <= 256, dilation >= 1,
 * pointers 16-byte aligned; errors as for deft_dwconv1d_forward. */
int deft_dwpw1d_forward(const float* x, const float* w_dw, const float* w_pw, float* z, int batch, int steps,
                        int channels, int out_channels, int ksize, int dilation, void* stream);

/* ---- Group norm with an activation ----
 *
 * x is [n][c][s] (DEFT_CHANNELS_FIRST, as the convolution layer writes y) or
 * [n][s][c] (DEFT_CHANNELS_LAST, as the 1-D convolutions do); a group is c /
 * groups consecutive channels of one image.  Over each group's m = s * c /
 * groups elements
 *   mean = sum(x) / m,   rstd = 1 / sqrt(sum((x - mean)^2) / m + eps)
 *   h = (x - mean) * rstd,   z = gamma * h + beta,   y = act(z)
 * with act: none, relu max(z, 0), silu z / (1 + exp(-z)), gelu z * Phi(z) (Phi
 * the normal distribution function, not its tanh approximation).  Arithmetic is
 * fp32, with fp64 for sums beyond one thread forward; y is rounded once.  The
 * activations' own relative errors are at most (2 |z| + 8) 2^-24 for silu, and for
 * the gelu's tail Phi(-|z|) (2 z^2 + 8) 2^-24 and its fit's, 6e-6 in bf16 and 6e-7
 * in fp32: gelu's exponential, and silu's with its quotient in bf16, are the
 * hardware's, uncorrected.  A NaN or an
 * infinity in x makes its whole group's y NaN, and no other group's. */
enum deft_layout { DEFT_CHANNELS_FIRST = 0, DEFT_CHANNELS_LAST = 1 };
enum deft_act { DEFT_ACT_NONE = 0, DEFT_ACT_RELU = 1, DEFT_ACT_SILU = 2, DEFT_ACT_GELU = 3 };

typedef struct deft_norm_desc {
  int n, c, s;   /* images, channels, positions (h * w, or steps) */
  int groups;    /* divides c */
  int layout;    /* enum deft_layout */
  int act;       /* enum deft_act */
  int dtype;     /* enum deft_dtype of x, gamma, beta, y and the gradients */
  double eps;    /* >= 0 */
} deft_norm_desc;

/* DEFT_OK, or the code with which the calls below refuse the descriptor. */
int deft_norm_desc_validate(const deft_norm_desc* d);

/* Bytes of a workspace for deft_norm_forward (training = 0), or for it and
 * deft_norm_backward (training = 1); 0 for a descriptor that they refuse.  It
 * and the calls look at the current device, which must be the same for all.
 * Zero a workspace before its first call, use it for one descriptor, and order
 * the calls on it: workgroups that share a group count their calls in it.  Calls
 * that break this end all the same; groups whose sums they lose become NaN, and
 * dgamma and dbeta may be left unwritten. */
size_t deft_norm_workspace_bytes(const deft_norm_desc* d, int training);

/* How the forward (back = 0) or the backward (1) cuts a descriptor with
 * elements, on a device of `cus` compute units (0: those of the current one):
 * cut[8] = {form: 0 one workgroup a group, 1 several that exchange their sums, 2
 * read twice; elements per access; accesses per thread; threads per workgroup;
 * workgroups that share a group (a band of groups); workgroups; whether each of
 * them reads all exchanged words; cus}.  For tests.  Errors as for
 * deft_norm_desc_validate; DEFT_ERR_BAD_DESC for no elements. */
int deft_debug_norm_cut(const deft_norm_desc* d, int back, int cus, int* cut);

/* How long (ticks of 10 ns; 2 ms at first) a workgroup of either call waits
 * for the others that share its group, before it computes their sums itself;
 * the results are the same.  For tests; holds for all later calls. */
void deft_debug_norm_patience(uint32_t ticks);

/* y = act(group norm of x), and mean and rstd (fp32 [n][groups], written) as
 * deft_norm_backward takes them.  y must not overlap x.  n = 0 or s = 0 is a
 * no-op that checks no pointer and writes nothing.
 * DEFT_ERR_BAD_DESC (a negative size, c, eps or enum out of range; y over x),
 * DEFT_ERR_GROUPS (groups < 1 or not a divisor of c), DEFT_ERR_DTYPE,
 * DEFT_ERR_UNSUPPORTED (more than 2048 channels per group; over 2^31 - 1 groups;
 * a launch of 2^32 threads, which takes over 2^26 - 1 groups of 64 threads or
 * fewer of more), DEFT_ERR_NULLPTR, DEFT_ERR_ALIGN (every pointer 16 bytes),
 * DEFT_ERR_WORKSPACE; checks run before any launch. */
int deft_norm_forward(const deft_norm_desc* d, const void* x, const void* gamma, const void* beta, void* y,
                      float* mean, float* rstd, void* workspace, size_t ws_bytes, void* stream);

/* Gradients at dy, with mean and rstd as the forward left them:
 *   dz = dy * act'(z)     (relu: dy where z > 0, else 0)
 *   dbeta = sum dz,  dgamma = sum dz * h          (over images and positions)
 *   dx = rstd * (gamma dz - mean_group(gamma dz) - h * mean_group(gamma dz h))
 * dx, dgamma and dbeta are written, each rounded once; any of them may be NULL
 * and is not computed then.  All sums run in a fixed order: a call repeats its
 * bits.  dx must overlap neither x nor dy.  n = 0 or s = 0 writes zeros to
 * dgamma and dbeta.  Errors as for deft_norm_forward. */
int deft_norm_backward(const deft_norm_desc* d, const void* x, const void* gamma, const void* beta,
                       const float* mean, const float* rstd, const void* dy, void* dx, void* dgamma, void* dbeta,
                       void* workspace, size_t ws_bytes, void* stream);

/* ---- The end of a training step: gradient norm and AdamW over a list of tensors ----
 *
 * Both take a host array that lists device tensors (dense, any number of
 * elements, of one dtype); the list travels in the launches' arguments, so a
 * call copies nothing to the device, keeps nothing, and can be captured in a
 * HIP graph, which then replays on the same addresses.  count = 0 and tensors
 * of no elements (whose pointers are not looked at) are allowed. */

/* Elements that share one scale of an 8-bit state. */
#define DEFT_STATE_BLOCK 256
/* Bytes of the record of skipped steps. */
#define DEFT_SKIPS_BYTES 48

typedef struct deft_adamw_desc {
  int p_dtype, g_dtype; /* enum deft_dtype of the weights and of the gradients */
  int state_bits;       /* 32: m and v are fp32.  8: e4m3 codes with scales */
  int master;           /* 1 (bf16 weights only): fp32 masters are updated, the weights are their
                           rounded copies and are only written */
  int64_t step;         /* this step's number, from 1 */
  double lr, beta1, beta2, eps; /* lr, eps >= 0; 0 <= beta < 1 */
  uint32_t seed;        /* 8-bit states: a new one for each step */
  uint32_t* skipped;    /* device, DEFT_SKIPS_BYTES, zeroed before the first step; may be NULL.  The first
                           word is how many steps control has skipped; the rest is the calls' own */
} deft_adamw_desc;

typedef struct deft_adamw_tensor {
  void* p;              /* weights, updated */
  const void* g;        /* gradient */
  void* m;              /* first moment, updated: fp32, or e4m3 (OCP, 448 its largest value) codes */
  void* v;              /* second moment, updated: fp32, or e4m3 codes of its square root */
  float* m_scale;       /* 8-bit states: fp32 [ceil(n / DEFT_STATE_BLOCK)]; m = code * scale, */
  float* v_scale;       /*   sqrt(v) = code * scale of its block of consecutive elements */
  float* master;        /* fp32 master weights, updated (desc.master) */
  int64_t n;            /* elements */
  double weight_decay;  /* decoupled, >= 0 */
} deft_adamw_tensor;

/* One AdamW step over all listed tensors.  Per element, in fp32 with one
 * rounding per operation, in this order:
 *   g  = coef * grad                              (with control)
 *   m  = beta1 * m + (1 - beta1) * g
 *   v  = beta2 * v + (1 - beta2) * (g * g)
 *   p  = p * (1 - lr * weight_decay)
 *        - (m / (sqrt(v) / sqrt(1 - beta2^step) + eps)) * (lr / (1 - beta1^step))
 * and p is rounded once to its dtype.  8-bit states: the step computes on code
 * * scale; then scale = max|.| / 448 over each block, m is rounded to the
 * nearest code, sqrt(v) to one of its two neighbours at random (unbiased, from
 * a hash of seed, the tensor's number in the list and the element), and never
 * from above zero to zero.  A block with a NaN or an infinity in m or v
 * gets the scale NaN there.  Zeroed states (codes and scales) are a fresh
 * start in both forms.
 * control (device, may be NULL): what deft_grad_norm wrote.  Its factor
 * multiplies the gradients; if it says that they are not finite, the step
 * writes nothing, but adds 1 to desc.skipped.
 * desc.skipped: a step's number in 1 - beta^step is desc.step less this count, so
 * skipped steps leave no mark on later ones, without a copy to the host.  Keep
 * the betas while one record is in use.  Without it, or with a schedule, skipped
 * steps count as steps.
 * schedule (device, may be NULL): 4 doubles {lr, 1 - beta1^step, 1 -
 * beta2^step, seed} that replace the descriptor's, read when the kernels run:
 * for a captured step whose rates change from replay to replay.
 * DEFT_ERR_DTYPE; DEFT_ERR_BAD_DESC (a negative size, a rate out of range,
 * masters for fp32 weights); DEFT_ERR_UNSUPPORTED (over 2^24 - 1 workgroups of
 * 1024 elements in one tensor); DEFT_ERR_NULLPTR; DEFT_ERR_ALIGN (tensors 16
 * bytes, scales and control 4, schedule and skipped 8).  Checks run before any launch. */
int deft_adamw_step(const deft_adamw_desc* d, const deft_adamw_tensor* t, int count, const float* control,
                    const double* schedule, void* stream);

/* Norm of all listed gradients and the factor that clips them:
 *   norm = sqrt(sum of squares) * inv_scale      (sums in fp64, fixed order)
 *   factor = inv_scale * min(1, max_norm / (norm + 1e-6))
 * with inv_scale > 0 the inverse of the loss's scale and max_norm > 0
 * (infinity: no clipping).  Writes control (device, 4 floats): {norm, factor,
 * 1 if every gradient is finite else 0, 0}; the factor is 0 where they are
 * not.  No gradient is changed: deft_adamw_step applies the factor.
 * DEFT_ERR_DTYPE, DEFT_ERR_BAD_DESC, DEFT_ERR_UNSUPPORTED (over 2^44 elements),
 * DEFT_ERR_NULLPTR, DEFT_ERR_ALIGN (gradients, control and workspace 16 bytes),
 * DEFT_ERR_WORKSPACE; checks run before any launch. */
int deft_grad_norm(const void* const* g, const int64_t* n, int count, int g_dtype, double max_norm,
                   double inv_scale, float* control, void* workspace, size_t ws_bytes, void* stream);

/* Workspace bytes of deft_grad_norm for a list of `count` tensors.  Zero a
 * workspace before its first call, and order the calls on it: its workgroups
 * count themselves in it. */
size_t deft_grad_norm_workspace_bytes(int count);

/* ---- Muon over a list of matrices ----
 *
 * (K. Jordan and others, 2024, with their coefficients.)
 *
 * Momentum steps whose updates have their singular values brought near 1.  A
 * tensor is a matrix [rows][cols] (a convolution's weight: its output channels by
 * all the rest); per matrix, with g its gradient (times the factor in control),
 *   m = mu m + (1 - mu) g
 *   u = mu m + (1 - mu) g  with nesterov, else m
 *   X = u / max(|u|_F, eps), then `steps` times
 *       G = X X^T,  X = (a I + b G + c G^2) X     with a, b, c = 3.4445, -4.7750, 2.0315
 *   p = p (1 - lr weight_decay) - lr scale X
 * (G from the smaller side).  m and p take one fp32 rounding per operation in this
 * order, p is rounded once to its dtype.  X is computed with 22 bits for each
 * factor and sums in fp32, as near to the formula's value as steps in fp32 are:
 * 2e-6 of its root mean square for matrices of normal values, up to 5e-5 where most
 * singular values are small (their part of an error grows by up to 3.4 a step).
 * X is held in multiples of 2^-38, which five steps make 5e-10 of an element: where
 * |u| is under 1e-4 eps, and the update tiny, that is more than those parts of it.
 * A matrix's last bits may depend on the others of the list, whose sizes choose
 * tiles and splits for all.
 * A zero direction leaves X zero; a NaN or an infinity in u makes all of p's
 * matrix NaN, and no other's.  Calls repeat their bits. */
typedef struct deft_muon_desc {
  int p_dtype, g_dtype; /* enum deft_dtype of the weights and of the gradients */
  int master;           /* 1 (bf16 weights only): fp32 masters are updated, the weights are their
                           rounded copies and are only written */
  int nesterov;         /* 0 or 1 */
  int steps;            /* 1 to 32; 5 is usual */
  double lr, momentum, eps; /* lr >= 0, 0 <= momentum < 1, eps >= 1e-30 */
} deft_muon_desc;

typedef struct deft_muon_tensor {
  void* p;              /* weights, updated */
  const void* g;        /* gradient */
  float* m;             /* momentum, updated */
  float* master;        /* fp32 master weights, updated (desc.master) */
  int64_t rows, cols;
  double weight_decay;  /* decoupled, >= 0 */
  double scale;         /* of the update, such as sqrt(max(1, rows / cols)) */
} deft_muon_tensor;

/* Workspace bytes of deft_muon_step for this list (its shapes), on a device of as
 * many compute units as the current one; 0 for a list that it refuses.  Nothing is
 * kept in it from call to call. */
size_t deft_muon_workspace_bytes(const deft_muon_tensor* t, int count);

/* One step over all listed matrices.  Like deft_adamw_step it takes a host array,
 * copies nothing to the device and can be captured; control (device, may be NULL)
 * is what deft_grad_norm wrote: where it says that the gradients are not finite, the
 * step writes nothing but its workspace.  schedule (device, may be NULL): one
 * double, the lr that replaces the descriptor's, read when the kernels run.
 * count = 0 and matrices of no elements are allowed.  What a step writes, p, m and
 * master of every matrix and the workspace, must not overlap, nor any gradient (not
 * checked here).
 * DEFT_ERR_DTYPE; DEFT_ERR_BAD_DESC (a negative size, a rate out of range, masters
 * for fp32 weights); DEFT_ERR_UNSUPPORTED (a smaller side over 2^15, a larger one
 * over 2^22, over 2^32 elements); DEFT_ERR_NULLPTR; DEFT_ERR_ALIGN (tensors and workspace 16 bytes,
 * control 4, schedule 8); DEFT_ERR_WORKSPACE.  Checks run before any launch. */
int deft_muon_step(const deft_muon_desc* d, const deft_muon_tensor* t, int count, const float* control,
                   const double* schedule, void* workspace, size_t ws_bytes, void* stream);

/* ---- Pointwise (1x1) convolution in 8 bits, with its gradients ----
 *
 * x is [n][c_in][s] (DEFT_CHANNELS_FIRST) or [n][s][c_in] (DEFT_CHANNELS_LAST),
 * y and dy likewise with c_out; w is [c_out][c_in].  Over the rows r, the n * s
 * positions in their order,
 *   y[r][o]  = sum_k qx[r][k] qw[o][k] + b[o]
 *   dx[r][k] = sum_o qdy[r][o] qw[o][k]
 *   dw[o][k] = sum_r q'dy[r][o] q'x[r][k],   db[o] = sum_r dy[r][o]
 * where q stands for values of e4m3 (OCP, 448 its largest) times a power of two
 * that a block of values shares: qx and qdy in blocks of 128 consecutive channels
 * of a row, q'x and q'dy in blocks of 128 consecutive rows of a channel, qw in
 * blocks of 128 x 128 (all from the first channel or row on; the last blocks may
 * be smaller).  With most the largest magnitude of a block's finite values, its
 * power is 2^e with the least whole e >= -127 for which most <= 448 * 2^e, and
 * each value is rounded to the nearest multiple, ties to even.  A NaN or an
 * infinity makes NaN of the sums that it enters, and of no others.  Products are
 * exact, sums fp32 (sums under 2^-126 may be lost), results rounded once; calls
 * repeat their bits.  bf16: within each 8 consecutive terms, what lies under 2^-13 of
 * the largest is cut off before they are added (the 8-bit matrix instructions' sum):
 * 1.5e-5 of the results' root mean square for normal values, 4.6e-5 where channels
 * differ in size, where their rounding is 1.66e-3. */
#define DEFT_PW8_BLOCK 128

typedef struct deft_pw8_desc {
  int n, s;              /* images, positions (h * w, or steps) */
  int c_in, c_out;
  int layout;            /* enum deft_layout of x, y, dx and dy */
  int dtype;             /* enum deft_dtype of all tensors */
  int training;          /* 1: packed weights and forward are for deft_pw8_backward, too */
} deft_pw8_desc;

/* DEFT_OK, or the code with which the calls below refuse the descriptor:
 * DEFT_ERR_BAD_DESC (negative n or s, c_in or c_out < 1, layout or training out
 * of range), DEFT_ERR_DTYPE, DEFT_ERR_UNSUPPORTED (over 2^31 - 129 rows or 2^20
 * channels; launches of 2^32 threads).  The sizes below are 0 for it, then. */
int deft_pw8_desc_validate(const deft_pw8_desc* d);

/* Bytes of the packed weights, and of what a training forward saves. */
size_t deft_pw8_packed_bytes(const deft_pw8_desc* d);
size_t deft_pw8_saved_bytes(const deft_pw8_desc* d);
/* Bytes of a workspace for the calls below on this descriptor; it depends on the
 * current device's number of units.  Nothing is kept in it from call to call. */
size_t deft_pw8_workspace_bytes(const deft_pw8_desc* d);

/* Codes of w, once for all calls until it changes.  Every byte of `packed` that
 * the other calls read is written.  It serves every n, s and layout. */
int deft_pw8_pack(const deft_pw8_desc* d, const void* w, void* packed, void* stream);

/* y; bias may be NULL.  training: writes `saved`, what the backward needs of x.
 * n * s = 0 is a no-op.  Errors of all calls, besides the descriptor's:
 * DEFT_ERR_NULLPTR, DEFT_ERR_ALIGN (pointers 16 bytes), DEFT_ERR_WORKSPACE,
 * DEFT_ERR_BAD_DESC (something written, the workspace included, over anything else
 * that the call takes; a backward without training); checks run before any launch. */
int deft_pw8_forward(const deft_pw8_desc* d, const void* x, const void* packed, const void* bias, void* y, void* saved,
                     void* workspace, size_t ws_bytes, void* stream);

/* Gradients at dy, with `saved` as the forward left it and the packed weights
 * that it used; any of dx, dw and db may be NULL and is not computed then.  n * s
 * = 0 writes zeros to dw and db. */
int deft_pw8_backward(const deft_pw8_desc* d, const void* saved, const void* packed, const void* dy, void* dx, void* dw,
                      void* db, void* workspace, size_t ws_bytes, void* stream);

/* Per-kernel timing for benchmarks (host-side events only; no device memory).
 * deft_timing_start(capacity) creates `capacity` event pairs for the calling
 * thread; while active, each kernel that deft_forward / deft_backward /
 * deft_debug_sample launch on this thread is bracketed by two events recorded
 * on the call's stream (launches beyond capacity are not recorded).
 * deft_timing_stop() waits for the last recorded event, computes each
 * launch's duration and deactivates timing; deft_timing_count and
 * deft_timing_get(i, &name, &ms) then return the i-th launch's kernel name
 * (a static string) and milliseconds.  Errors: DEFT_ERR_BAD_DESC for a
 * capacity < 1 or an index out of range, DEFT_ERR_HIP for event failures. */
int deft_timing_start(int capacity);
int deft_timing_stop(void);
int deft_timing_count(void);
int deft_timing_get(int i, const char** name, float* ms);

/* Static description of an error code. */
const char* deft_error_string(int code);

/* Text of the last HIP error seen by this thread, or "" */
const char* deft_last_hip_error(void);

#ifdef __cplusplus
}
#endif
#endif /* DEFT_H */
