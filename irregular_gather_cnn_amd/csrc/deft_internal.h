// Host-side internals of the deformable convolution library: the plan and
// the launchers each kernel file exports to deft_host.cpp.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "deft.h"

struct deft_plan {
  deft_desc d;
  int cus = 256;               // compute units of the device the plan was made for
  int max_lds = 160 * 1024;    // its LDS bytes per workgroup
  int ho, wo, oc, taps, ck, cg;
  // fused sampling kernel
  int tile_h, tile_w, halo, chunk, chunk_a, gw, gsplit;
  int bhalo;                   // sampling backward's candidate window (input pixels)
  int tiles_h, tiles_w, num_tiles, num_wg, mblocks;
  int foot_h, foot_w;          // nominal tile footprint (input pixels)
  int reg_h, reg_w;            // largest halo region (input pixels)
  int pstr, pstr_a;            // LDS pixel strides (elements)
  int lds_region, lds_off, lds_info, lds_total;  // byte offsets / total
  int direct;                  // 1: corners gathered from a channel-minor copy of x (no LDS halo)
  int bwd_mf;                  // bf16 sampling backward with the scatter on the MFMA units
  int stage_d;                 // direct: footprint-staging loads per wave per channel chunk
  int oc_pad;                  // rows of the prepared offset-conv weight
  double est_miss;
  // workspace layout (byte offsets, 256-aligned)
  size_t ws_wt, ws_woff, ws_cols, ws_xh, ws_fwd_end;
  size_t ws_w2, ws_dcol, ws_dx32, ws_doff, ws_doff16, ws_wofft, ws_train_end;
  int kk_pad;                  // padded (o, tap) depth of the transposed offset conv
  // sampling backward: each workgroup owns a core tile of input pixels
  // (btile_h x btile_w) and the (output pixel, tap) pairs that touch it
  int btile_h, btile_w, btiles_h, btiles_w, num_btiles, list_cap;
  int chunk_b, lb_dx, lb_dc, lb_cnt, lb_total;
  int woff_bands;              // row bands of the offset-weight backward
  size_t ws_list, ws_lcount, ws_doffp, ws_maxbits, ws_dwpart, ws_dwoffpart, ws_biaspart;
  // bf16 GEMMs with direct global-to-LDS staging (else the generic kernel)
  int gemm_dl;
  int dw_splits, dw_kper;      // dW partials: pixel ranges of dw_kper (per image on the generic path)
  // forward with the gather fused into the main GEMM (deft_igemm.hip): the
  // offset conv writes the offsets (to the caller's buffer or ws_offs), then
  // one launch gathers, multiplies and stores y and the columns
  int igemm;
  size_t ws_offs;
};

namespace deft {

// The offset-weight backward's form with its dOffset operand in bf16 pieces
// (four workgroups per CU): bf16, at most 32 offset channels, output rows a
// multiple of 8 pixels.
inline bool woff_a16(int dtype, int oc, int wo) { return dtype == DEFT_BF16 && oc <= 32 && wo % 8 == 0; }

// Records a HIP error for deft_last_hip_error and returns DEFT_ERR_HIP.
int report_hip_error(hipError_t e);
// Of the current device; 256 where there is none.
int compute_units();

// Timing hook (deft_timing_start): brackets a launch with events when active.
void timing_before(hipStream_t s, const char* name);
void timing_after(hipStream_t s);

#define DEFT_LAUNCH(name, kernel, grid, block, lds, stream, ...)               \
  do {                                                                        \
    ::deft::timing_before((stream), (name));                                  \
    hipLaunchKernelGGL(kernel, grid, block, lds, stream, __VA_ARGS__);        \
    ::deft::timing_after((stream));                                           \
  } while (0)

struct SampleArgs {
  const void* x = nullptr;
  const void* woff_p = nullptr;   // prepared offset-conv weight [oc_pad][taps][Cin]
  const void* b_off = nullptr;    // nullable, dtype
  const float* off_in = nullptr;  // sampling alone: offsets to sample from
  float* off_out = nullptr;       // nullable
  void* cols = nullptr;           // [N*Ho*Wo][taps][Cin]
  void* xh = nullptr;             // direct gather: channel-minor copy of x (workspace)
  uint32_t* hist = nullptr;       // nullable: required-halo histogram accumulated by the launch
  int hist_len = 0;
};

hipError_t launch_prep_forward(const deft_plan& p, const void* w, const void* w_off, void* wt, void* woff_p,
                               const void* x, void* xh, hipStream_t s);
// What a sampling launch computes: the fused offset conv + sampling, the
// offset conv alone (offsets to off_out), or the sampling alone from off_in.
enum SampleMode { kFusedMode = 0, kOffsetsMode = 1, kSampleMode = 2 };
hipError_t launch_sample(const deft_plan& p, SampleMode mode, const SampleArgs& a, hipStream_t s);
hipError_t launch_sample_index(const deft_desc& d, int ho, int wo, const float* off, int32_t* y0,
                               int32_t* x0, uint8_t* mask, hipStream_t s);
hipError_t launch_halo_hist(const deft_desc& d, int ho, int wo, const float* off, uint32_t* hist,
                            int hist_len, hipStream_t s);

hipError_t launch_gemm_forward(const deft_plan& p, const void* wt, const void* cols, const void* b,
                               void* y, hipStream_t s);
// dilated depthwise 1-D convolution (deft_dwconv.hip)
hipError_t launch_dwconv1d(const float* x, const float* w, float* y, int B, int T, int C, int K, int d,
                           hipStream_t st);
// fused depthwise + pointwise 1-D convolution (deft_dwpw.hip)
hipError_t launch_dwpw1d(const float* x, const float* wdw, const float* wpw, float* z, int B, int T, int C, int O,
                         int K, int d, hipStream_t st);
// gather fused into the main GEMM (deft_igemm.hip)
bool igemm_supported(const deft_plan& p);
hipError_t launch_igemm(const deft_plan& p, const void* xh, const float* off, const void* wt, const void* b,
                        void* y, void* cols, hipStream_t st);
// direct-staging bf16 GEMMs (deft_gemm_dl.hip)
bool gemm_dl_supported(const deft_plan& p);
void gemm_dl_dw_split(const deft_plan& p, int* splits, int* kper);
hipError_t dl_gemm_forward(const deft_plan& p, const void* wt, const void* cols, const void* b, void* y,
                           hipStream_t st);
hipError_t dl_gemm_dcol(const deft_plan& p, const void* w2, const void* dy, void* dcol, uint32_t* maxbits,
                        hipStream_t st);
hipError_t dl_gemm_dw(const deft_plan& p, const void* dy, const void* cols, float* part, hipStream_t st);

struct BackwardArgs {
  const void* x;
  const void* w_off;
  const void* w;
  const float* offsets;
  const void* dy;
  void* dx;
  void* dw_off;
  void* db_off;
  void* dw;
  void* db;
  char* ws;
};
hipError_t launch_backward(const deft_plan& p, const BackwardArgs& a, hipStream_t s);

// AdamW and the gradient norm over lists of tensors (deft_optim.hip).  A launch
// carries its tensors in its arguments (under 4 KB), so a call copies nothing
// to the device and can be captured; longer lists take several launches.
constexpr int kStateBlock = DEFT_STATE_BLOCK;  // elements per scale of an 8-bit state
constexpr int kAdamwElems = 4 * kStateBlock;   // per workgroup
constexpr int kAdamwThreads = kAdamwElems / 4;
constexpr int kAdamwList = 50, kNormList = 64; // tensors per launch
struct AdamwTensor {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  float* master;
  int64_t n;
  double decay;    // 1 - lr wd, to be rounded to fp32; wd where the schedule has lr
};
struct AdamwArgs {
  AdamwTensor t[kAdamwList];
  uint32_t first[kAdamwList];  // first workgroup of each tensor
  uint32_t id[kAdamwList];     // its number in the call's list
  uint16_t count;
  uint16_t lead;           // the call's first launch, which counts a skipped step
  float b1, c1, b2, c2, eps, rate, low;
  uint32_t seed;
  const float* control;    // nullable
  const double* schedule;  // nullable
  struct AdamwSkips* skips;  // nullable; where steps were skipped, rate and low are made from it and from:
  double lr, log1, log2;     // log2 of beta1 and beta2
  int64_t step;
};
// The device's record of skipped steps.  Corrections take fp64 powers, which every thread's
// computing them made a third of a large step's operations (284 us against 255 of 77 M
// elements): one thread of each call computes the next call's, where the count is not 0.
struct AdamwSkips {
  uint32_t count, unused[3];
  struct Next {
    double inverse;  // 1 / (1 - beta1^taken)
    float low;       // 1 / sqrt(1 - beta2^taken)
    uint32_t taken;  // the number of the step that they are for, among those taken
  } next[2];         // of steps of even and of odd number: a call reads one and writes the other
};
static_assert(sizeof(AdamwSkips) == DEFT_SKIPS_BYTES, "include/deft.h");
static_assert(sizeof(AdamwArgs) <= 4096, "kernel arguments");
hipError_t launch_adamw(const AdamwArgs& a, uint32_t blocks, int p_dtype, int g_dtype, int bits, bool master,
                        bool once, hipStream_t st);
constexpr int kSquareThreads = 1024;
constexpr int kNormPiece = 32768;    // elements a workgroup sums at a time
constexpr uint32_t kNormGrid = 256;  // workgroups, and partial sums, per launch
struct GradNormArgs {
  const void* g[kNormList];
  int64_t n[kNormList];
  uint32_t first[kNormList];  // first piece of each tensor
  int count;
  uint32_t pieces;
  uint32_t sums, at;          // partial sums of the whole call, and the first of this launch
  double* partials;
  uint64_t* arrived;          // workgroups of the call that have stored theirs; 0 between calls
  double max_norm, inv_scale;
  float* control;
};
static_assert(sizeof(GradNormArgs) <= 4096, "kernel arguments");
hipError_t launch_grad_norm(const GradNormArgs& a, int g_dtype, uint32_t grid, hipStream_t st);

// Group norm with activation (deft_norm_fwd.hip, deft_norm_bwd.hip).  A group
// of an image, or a band of whole groups where channels come last, is cut into
// `slices` that one workgroup each holds in registers.  One slice, or several
// that the chip holds at once: statistics and result in one launch, in which
// the slices' workgroups join their sums.  More: partial statistics, their
// combination, and the result from a second read.
constexpr int kNormThreads = 512;   // 1024 where a kernel's registers allow it (kNormWide)
constexpr int kNormWide = 1024;
// Backward kernels that hold a group whole in 8 accesses a thread and 128 registers:
// they run with 1024 threads what would take 16 accesses and half as many waves.
constexpr bool norm_bwd_wide(bool fp32, bool last, bool keep) { return fp32 || !(last || keep); }
enum NormMode { kNormWhole = 0, kNormJoint = 1, kNormStats = 2, kNormApply = 3 };
struct NormArgs {
  const void* x;
  const void* dy;     // backward
  const void* gamma;
  const void* beta;
  void* out;          // y, or dx (nullable)
  float* mean;        // [n][g]: written forward, read backward
  float* rstd;
  float* part;        // partial sums, one block per slice: see each kernel
  float* sums;        // backward, several slices: [n][g][2] sums of gamma dz and of gamma dz h
  void* dgamma;       // backward, nullable; written by the main kernel where `arrivals` is set
  void* dbeta;
  uint64_t* arrivals; // [bands or groups]: workgroups that have written their sums, 0 between calls
  int n, c, s, g, per, act;
  float eps;
  int slices, rp;     // channels last: rows (positions) per slice; first: channels per slice
  int bands;          // channels last
  int ws, cp;         // channels first: slices along the positions, and positions in each
  int lt;             // channels first: log2 of the lanes that share a channel's positions
  // joint: per cluster a call counter, words of each slice and group, totals of each group
  uint64_t* counter;
  uint64_t* words;
  uint64_t* totals;
  int direct;         // every workgroup reads every slice's words; else totals are made and read
  uint32_t patience;  // ticks (10 ns) that a workgroup waits for its peers
};
struct NormPlan {     // how a call is cut
  int vec, u, threads;  // elements per access, accesses per thread, threads per workgroup
  uint32_t blocks;
  size_t lds;
};
hipError_t launch_norm_fwd(const NormArgs& a, const NormPlan& p, int layout, int dtype, int mode, hipStream_t st);
hipError_t launch_norm_bwd(const NormArgs& a, const NormPlan& p, int layout, int dtype, int mode, hipStream_t st);
hipError_t launch_norm_combine(const NormArgs& a, int layout, hipStream_t st);
hipError_t launch_norm_bwd_sums(const NormArgs& a, int layout, int dtype, hipStream_t st);
hipError_t launch_norm_params(const float* part, int rows, int c, void* dgamma, void* dbeta, int dtype,
                              hipStream_t st);

// Pointwise convolution in 8 bits (deft_pw8_quantise.hip, deft_pw8_gemm.hip,
// deft_pw8_few.hip).  A matrix of codes over `rows` and a depth, stored by half
// blocks: codes [blocks][2][rows][64], scales [blocks][pw8_scale_rows].
constexpr int kPw8Block = DEFT_PW8_BLOCK;
// Where the 64 codes of a row's half of a block start.
__host__ __device__ inline int64_t pw8_code(int64_t block, int half, int64_t rows, int64_t row) {
  return ((block * 2 + half) * rows + row) * (kPw8Block / 2);
}
__host__ __device__ inline int64_t pw8_scale_rows(int64_t rows) { return (rows + 15) & ~(int64_t)15; }
struct Pw8Matrix {
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t rows;
};
struct Pw8QuantiseArgs {
  const void* src;        // [lines][near], or channels first [images][lines][positions]
  int64_t lines, near;    // near: values along memory, over all images
  int64_t pitch;          // from line to line
  int64_t positions;      // of an image, channels first; else 0
  uint32_t tiles_near;
  uint8_t* near_codes;    // nullable: rows are lines, the depth is near
  uint8_t* near_scales;
  uint8_t* far_codes;     // nullable: rows are near, the depth is lines
  uint8_t* far_scales;
  float* sums;            // nullable: [tiles of the rows][channels] sums over a tile's rows
};
hipError_t launch_pw8_quantise(const Pw8QuantiseArgs& a, uint32_t blocks, int dtype, bool tile, hipStream_t st);
hipError_t launch_pw8_bias(const float* sums, int64_t tiles, int c, void* db, int dtype, hipStream_t st);
hipError_t launch_pw8_zero(void* p, size_t bytes, hipStream_t st);
struct Pw8Out {
  void* p;
  const void* bias;       // nullable: per column; with positions per row
  int64_t rows, cols;
  int64_t positions;      // channels first: columns are the positions of all images; else 0
};
struct Pw8GemmArgs {
  Pw8Matrix a, b;         // out[i][j] = sum over the depth of a[i] b[j]
  Pw8Out out;
  float* part;            // nullable: [splits][rows][part_cols], joined by a second launch
  int part_cols;
  int blocks;             // of the depth
  int splits, per_split;  // blocks of a split
  int tiles_m, tiles_n;
};
hipError_t launch_pw8_gemm(const Pw8GemmArgs& g, int bm, int bn, int dtype, hipStream_t st);
// Up to kPw8Few rows: x is quantised where it is used.
constexpr int kPw8Few = 16;
struct Pw8FewArgs {
  const void* x;
  Pw8Matrix w;
  const void* bias;       // nullable
  void* y;
  int rows, c_in;
  int positions;          // channels first: of an image; else 0
};
hipError_t launch_pw8_few(const Pw8FewArgs& a, int dtype, int cus, hipStream_t st);

// Muon over a list of matrices (deft_muon.hip).  A matrix's share of the
// workspace: X twice, kMuonSquares matrices of the smaller side, partial sums of
// squares and of products.  X has the smaller side first (m <= n), so it is a tall
// matrix's transpose.  Sides are rounded up to 32 with zeros (mp, np), values are
// pairs of fp16.
constexpr int kMuonList = 48;      // matrices of a launch
constexpr int kMuonPad = 32, kMuonSquares = 6, kMuonSums = 256;
struct MuonItem {
  char* base;                      // its share of the workspace
  void* p;
  const void* g;
  float* mom;
  float* master;
  double decay;                    // weight decay
  double scale;                    // of the update, lr apart
  int m, n;
  int tall;                        // p is [n][m]
  int splits;                      // of the sum over n
};
struct MuonArgs {
  MuonItem it[kMuonList];
  uint32_t first[kMuonList];       // first workgroup of each matrix
  int count;
  float mu, nu;                    // momentum and 1 - momentum
  int nesterov;
  double eps, lr;
  const float* control;            // nullable
  const double* schedule;          // nullable
  // products: out = f A B + fd I + fb add, by numbers of buffers: 0 and 1 are X, the others squares
  struct Phase {
    int a, b, out, add;
    float f, fd, fb;
  } ph;
};
static_assert(sizeof(MuonArgs) <= 4096, "kernel arguments");
__host__ __device__ inline int64_t muon_pad(int64_t v) { return (v + kMuonPad - 1) / kMuonPad * kMuonPad; }
__host__ __device__ inline int64_t muon_x_bytes(int m, int n) { return 4 * muon_pad(m) * muon_pad(n); }
__host__ __device__ inline int64_t muon_square_bytes(int m) { return 4 * muon_pad(m) * muon_pad(m); }
__host__ __device__ inline int64_t muon_buffer(int id, int m, int n) {
  return id < 2 ? id * muon_x_bytes(m, n) : 2 * muon_x_bytes(m, n) + (id - 2) * muon_square_bytes(m);
}
__host__ __device__ inline int64_t muon_sums(int m, int n) { return muon_buffer(2 + kMuonSquares, m, n); }
__host__ __device__ inline int64_t muon_parts(int m, int n) { return muon_sums(m, n) + kMuonSums * 8; }
inline int64_t muon_item_bytes(int m, int n, int splits) {
  return (muon_parts(m, n) + (splits > 1 ? splits * muon_square_bytes(m) : 0) + 255) / 256 * 256;
}
// Elements whose squares a workgroup sums, at most kMuonSums workgroups a matrix.
__host__ __device__ inline int64_t muon_chunk(int64_t n) {
  const int64_t least = 4096, c = (n + kMuonSums - 1) / kMuonSums;
  return c <= least ? least : (c + 1023) / 1024 * 1024;
}
// A matrix whose step one workgroup does in LDS: 64 rows at most, and the bytes of X, two
// squares and, for 32 rows, four waves' sums.
constexpr int kMuonSmallSide = 64, kMuonSmallLds = 150 * 1024;
inline int64_t muon_small_lds(int m, int n) {
  return muon_x_bytes(m, n) + 2 * muon_square_bytes(m) + (m <= 32 ? 4 * 32 * 33 * 4 : 0);
}
struct MuonSmall {
  int steps, lds;
  float g, a, b, c, x, o;  // factors of sums: G; Q = a I + b G + c G^2; X; the update
};
hipError_t launch_muon_small(const MuonArgs& a, const MuonSmall& c, int p_dtype, int g_dtype, bool master, hipStream_t st);
hipError_t launch_muon_momentum(const MuonArgs& a, uint32_t blocks, int g_dtype, hipStream_t st);
hipError_t launch_muon_scale(const MuonArgs& a, uint32_t blocks, int g_dtype, hipStream_t st);
// tile: 64, 128 or 256
hipError_t launch_muon_square(const MuonArgs& a, uint32_t blocks, int tile, bool split, hipStream_t st);
hipError_t launch_muon_join(const MuonArgs& a, uint32_t blocks, hipStream_t st);
hipError_t launch_muon_apply(const MuonArgs& a, uint32_t blocks, int tile, bool last, int p_dtype, bool master,
                             hipStream_t st);

}  // namespace deft
