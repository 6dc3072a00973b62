// C ABI of the training operators around the convolutions: argument checks,
// workspace sizes and launch sequencing.  Kernels live in deft_optim.hip,
// deft_norm_fwd.hip and deft_norm_bwd.hip.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "deft.h"
#include "deft_internal.h"

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
bool dtype_ok(int t) { return t == DEFT_F32 || t == DEFT_BF16; }
int status_of(hipError_t e) { return e == hipSuccess ? DEFT_OK : deft::report_hip_error(e); }

// Workgroups of one launch stay below 2^31.
constexpr uint64_t kMaxBlocks = 0x7fffffffu;

uint64_t blocks_of(int64_t n, int64_t per) { return ((uint64_t)n + per - 1) / per; }

int norm_launches(int count) { return std::max(1, (count + deft::kNormList - 1) / deft::kNormList); }

// ---- group norm: how a call is cut ----

constexpr int kMaxU = 16;          // accesses per thread of the widest kernels
constexpr int kMaxPer = 2048;      // channels per group: a row of one group fits a workgroup
constexpr uint64_t kFill = 512;    // workgroups that fill the chip, two on each compute unit
constexpr size_t kAlign = 256;

size_t round_up(size_t v, size_t m) { return (v + m - 1) / m * m; }
int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
int elem_size(int dtype) { return dtype == DEFT_BF16 ? 2 : 4; }

int norm_desc_status(const deft_norm_desc* d) {
  if (!d) return DEFT_ERR_NULLPTR;
  if (!dtype_ok(d->dtype)) return DEFT_ERR_DTYPE;
  if (d->n < 0 || d->s < 0 || d->c < 1 || !(d->eps >= 0.0) || !std::isfinite(d->eps) ||
      (d->layout != DEFT_CHANNELS_FIRST && d->layout != DEFT_CHANNELS_LAST) || d->act < DEFT_ACT_NONE ||
      d->act > DEFT_ACT_GELU)
    return DEFT_ERR_BAD_DESC;
  if (d->groups < 1 || d->c % d->groups) return DEFT_ERR_GROUPS;
  if (d->c / d->groups > kMaxPer) return DEFT_ERR_UNSUPPORTED;
  return DEFT_OK;
}

struct NormCut {
  deft::NormArgs a;
  deft::NormPlan p;
  bool whole;
};

// Channels last.  One slice where a band of whole groups, 128 bytes of each
// row or more, fits the registers; else slices of whole rows (of 1024 channels
// at most), as many as fill the chip.
void cut_last(const deft_norm_desc& d, bool back, NormCut& r) {
  const int nt = deft::kNormThreads, per = r.a.per, g = d.groups, esz = elem_size(d.dtype);
  const int V = d.c >= 16 / esz ? 16 / esz : 1;
  r.p.vec = V;
  r.p.threads = nt;
  // chunks across the widest of `bands` bands
  auto widest = [&](int bands) { return ceil_div((int64_t)ceil_div(g, bands) * per, V); };
  int bands = std::max(1, g / std::min(g, ceil_div(128, per * esz)));
  int rounds = ceil_div(d.s, nt / widest(bands));
  r.whole = rounds <= kMaxU && (rounds <= 4 || (uint64_t)d.n * bands >= kFill / 4);
  r.a.slices = 1;
  r.a.rp = d.s;
  if (!r.whole) {
    bands = ceil_div(g, std::max(1, 1024 / per));
    const int ty = nt / widest(bands);
    rounds = 8;
    while (rounds > 1 && (uint64_t)d.n * bands * ceil_div(d.s, (int64_t)ty * rounds) < kFill) rounds /= 2;
    r.a.rp = ty * rounds;
    r.a.slices = ceil_div(d.s, r.a.rp);
  }
  r.a.bands = bands;
  r.p.u = rounds;
  const int cols = ceil_div(g, bands) * per, ng = ceil_div(g, bands);
  // thread rows and odd pitch: at most nt * V elements and one more per row
  const size_t red = (size_t)nt * V + nt;
  r.p.lds = sizeof(float) * (back ? 2 * red + 2 * (size_t)cols + 2 * (size_t)ng : red + 2 * (size_t)ng);
}

// Accesses per thread of `rows` channels with `chunks` chunks each, and the
// team size that takes the fewest.
int best_team(int nt, int rows, int chunks, int* lt) {
  int best = 0;
  for (int l = 0; (1 << l) <= nt; ++l) {
    const int64_t rounds = (int64_t)ceil_div(rows, nt >> l) * ceil_div(chunks, 1 << l);
    // at equal counts the wider team: its accesses are nearer to each other
    if (l == 0 || rounds <= best) {
      best = (int)std::min<int64_t>(rounds, 1 << 30);
      *lt = l;
    }
  }
  return best;
}

// Channels first.  One slice where a group fits the registers; else slices of
// whole channels, or of a channel's positions where one is long.
void cut_first(const deft_norm_desc& d, bool back, NormCut& r) {
  const int per = r.a.per, esz = elem_size(d.dtype), V = d.s >= 16 / esz ? 16 / esz : 1;
  const int chunks = ceil_div(d.s, V);
  r.p.vec = V;
  int nt = 64;
  int rounds = best_team(nt, per, chunks, &r.a.lt);
  while (rounds > 4 && nt < deft::kNormThreads) rounds = best_team(nt *= 2, per, chunks, &r.a.lt);
  r.whole = rounds <= kMaxU && (rounds <= 4 || (uint64_t)d.n * d.groups >= kFill / 4);
  r.a.rp = per;
  r.a.ws = 1;
  r.a.cp = d.s;
  if (!r.whole) {
    nt = deft::kNormThreads;
    int cpc = ceil_div(chunks, ceil_div(chunks, 4 * nt));  // chunks of a channel in a slice
    int rp = std::min(per, std::max(1, 8 * nt / cpc));
    auto slices = [&] { return (uint64_t)ceil_div(per, rp) * ceil_div(chunks, cpc); };
    while ((uint64_t)d.n * d.groups * slices() < kFill && rp * (int64_t)cpc > nt) {
      if (rp > 1) rp = (rp + 1) / 2;
      else cpc = (cpc + 1) / 2;
    }
    while ((rounds = best_team(nt, rp, cpc, &r.a.lt)) > kMaxU) --rp;  // rp = 1: four at most
    r.a.rp = rp;
    r.a.cp = cpc * V;
    r.a.ws = ceil_div(chunks, cpc);
  }
  r.a.slices = ceil_div(per, r.a.rp) * r.a.ws;
  r.p.threads = nt;
  r.p.u = rounds;
  const int subs = std::max(1, (1 << r.a.lt) >> 6);
  r.p.lds = sizeof(float) * (back ? 16 + (2 + 2 * (size_t)subs) * r.a.rp : 8 + 2 * (size_t)r.a.rp);
}

int norm_cut(const deft_norm_desc& d, bool back, NormCut& r) {
  std::memset(&r, 0, sizeof(r));
  r.a.n = d.n; r.a.c = d.c; r.a.s = d.s; r.a.g = d.groups;
  r.a.per = d.c / d.groups;
  r.a.act = d.act;
  r.a.eps = (float)d.eps;
  if (d.layout == DEFT_CHANNELS_LAST) cut_last(d, back, r);
  else cut_first(d, back, r);
  const uint64_t units = (uint64_t)d.n * (d.layout == DEFT_CHANNELS_LAST ? r.a.bands : d.groups);
  if (units > kMaxBlocks || (uint64_t)d.n * d.groups > kMaxBlocks || units * r.a.slices > kMaxBlocks)
    return DEFT_ERR_UNSUPPORTED;
  r.p.blocks = (uint32_t)(units * r.a.slices);
  return DEFT_OK;
}

// Slices whose channel sums stand apart.
int norm_parts(const deft_norm_desc& d, const NormCut& r) {
  return d.layout == DEFT_CHANNELS_LAST ? r.a.slices : r.a.ws;
}
size_t norm_part_bytes(const deft_norm_desc& d, const NormCut& r, bool back) {
  if (back) return round_up((size_t)d.n * norm_parts(d, r) * 2 * d.c * sizeof(float), kAlign);
  return r.whole ? 0 : (size_t)d.n * d.groups * r.a.slices * 2 * sizeof(float);
}
size_t norm_ws_bytes(const deft_norm_desc& d, const NormCut& r, bool back) {
  const size_t sums = back && !r.whole ? (size_t)d.n * d.groups * 2 * sizeof(float) : 0;
  return round_up(norm_part_bytes(d, r, back) + sums, kAlign);
}

bool overlap(const void* a, const void* b, size_t bytes) {
  const uintptr_t p = (uintptr_t)a, q = (uintptr_t)b;
  return p && q && p < q + bytes && q < p + bytes;
}

}  // namespace

extern "C" {

int deft_adamw_step(const deft_adamw_desc* d, const deft_adamw_tensor* t, int count, const float* control,
                    const double* schedule, void* stream) {
  if (!d || (count > 0 && !t)) return DEFT_ERR_NULLPTR;
  if (!dtype_ok(d->p_dtype) || !dtype_ok(d->g_dtype)) return DEFT_ERR_DTYPE;
  // negated comparisons refuse NaN
  if (count < 0 || (d->state_bits != 8 && d->state_bits != 32) || d->step < 1 || !(d->lr >= 0.0) ||
      !(d->beta1 >= 0.0 && d->beta1 < 1.0) || !(d->beta2 >= 0.0 && d->beta2 < 1.0) || !(d->eps >= 0.0) ||
      !std::isfinite(d->lr) || !std::isfinite(d->eps) || (d->master != 0 && d->p_dtype == DEFT_F32))
    return DEFT_ERR_BAD_DESC;
  if (!aligned4(control) || ((uintptr_t)schedule & 7u)) return DEFT_ERR_ALIGN;
  for (int i = 0; i < count; ++i) {
    const deft_adamw_tensor& x = t[i];
    if (x.n < 0 || !(x.weight_decay >= 0.0) || !std::isfinite(x.weight_decay)) return DEFT_ERR_BAD_DESC;
    if (x.n == 0) continue;
    if (blocks_of(x.n, deft::kAdamwElems) > kMaxBlocks) return DEFT_ERR_UNSUPPORTED;
    if (!x.p || !x.g || !x.m || !x.v || (d->master && !x.master)) return DEFT_ERR_NULLPTR;
    if (d->state_bits == 8 && (!x.m_scale || !x.v_scale)) return DEFT_ERR_NULLPTR;
    if (!aligned16(x.p) || !aligned16(x.g) || !aligned16(x.m) || !aligned16(x.v) ||
        (d->master && !aligned16(x.master)) ||
        (d->state_bits == 8 && (!aligned4(x.m_scale) || !aligned4(x.v_scale))))
      return DEFT_ERR_ALIGN;
  }
  deft::AdamwArgs a;
  std::memset(&a, 0, sizeof(a));
  const double bc1 = 1.0 - std::pow(d->beta1, (double)d->step), bc2 = 1.0 - std::pow(d->beta2, (double)d->step);
  a.b1 = (float)d->beta1; a.c1 = (float)(1.0 - d->beta1);
  a.b2 = (float)d->beta2; a.c2 = (float)(1.0 - d->beta2);
  a.eps = (float)d->eps;
  a.rate = (float)(d->lr / bc1);
  a.low = (float)(1.0 / std::sqrt(bc2));
  a.seed = d->seed;
  a.control = control;
  a.schedule = schedule;
  uint64_t blocks = 0;
  for (int i = 0; i <= count; ++i) {
    const uint64_t more = i < count ? blocks_of(t[i].n, deft::kAdamwElems) : 0;
    // the list is full, or at its end: launch what it holds
    if (a.count && (i == count || (more && (a.count == deft::kAdamwList || blocks + more > kMaxBlocks)))) {
      const hipError_t e = deft::launch_adamw(a, (uint32_t)blocks, d->p_dtype, d->g_dtype, d->state_bits,
                                              d->master != 0, (hipStream_t)stream);
      if (e != hipSuccess) return status_of(e);
      a.count = 0;
      blocks = 0;
    }
    if (!more) continue;
    const deft_adamw_tensor& x = t[i];
    deft::AdamwTensor& y = a.t[a.count];
    y.p = x.p; y.g = x.g; y.m = x.m; y.v = x.v;
    y.m_scale = x.m_scale; y.v_scale = x.v_scale;
    y.master = x.master;
    y.n = x.n;
    y.wd = x.weight_decay;
    y.decay = (float)(1.0 - d->lr * x.weight_decay);
    y.id = (uint32_t)i;
    a.first[a.count++] = (uint32_t)blocks;
    blocks += more;
  }
  return DEFT_OK;
}

size_t deft_grad_norm_workspace_bytes(int count) {
  return (size_t)norm_launches(std::max(count, 0)) * deft::kNormGrid * sizeof(double);
}

int deft_grad_norm(const void* const* g, const int64_t* n, int count, int g_dtype, double max_norm,
                   double inv_scale, float* control, void* workspace, size_t ws_bytes, void* stream) {
  if (!control || (count > 0 && (!g || !n))) return DEFT_ERR_NULLPTR;
  if (!dtype_ok(g_dtype)) return DEFT_ERR_DTYPE;
  if (count < 0 || !(max_norm > 0.0) || !(inv_scale > 0.0) || !std::isfinite(inv_scale)) return DEFT_ERR_BAD_DESC;
  uint64_t all = 0;
  for (int i = 0; i < count; ++i) {
    if (n[i] < 0) return DEFT_ERR_BAD_DESC;
    if (n[i] == 0) continue;
    all += blocks_of(n[i], deft::kNormPiece);
    if (all > kMaxBlocks) return DEFT_ERR_UNSUPPORTED;
    if (!g[i]) return DEFT_ERR_NULLPTR;
    if (!aligned16(g[i])) return DEFT_ERR_ALIGN;
  }
  if (!aligned16(control)) return DEFT_ERR_ALIGN;
  if (!workspace || ws_bytes < deft_grad_norm_workspace_bytes(count)) return DEFT_ERR_WORKSPACE;
  if (!aligned16(workspace)) return DEFT_ERR_ALIGN;
  deft::GradNormArgs a;
  std::memset(&a, 0, sizeof(a));
  double* partials = (double*)workspace;
  int sums = 0;
  uint64_t pieces = 0;
  for (int i = 0; i <= count; ++i) {
    const uint64_t more = i < count ? blocks_of(n[i], deft::kNormPiece) : 0;
    if (a.count && (i == count || (more && a.count == deft::kNormList))) {
      a.pieces = (uint32_t)pieces;
      a.partials = partials + sums;
      const uint32_t grid = (uint32_t)std::min<uint64_t>(pieces, deft::kNormGrid);
      const hipError_t e = deft::launch_grad_squares(a, g_dtype, grid, (hipStream_t)stream);
      if (e != hipSuccess) return status_of(e);
      sums += (int)grid;
      a.count = 0;
      pieces = 0;
    }
    if (!more) continue;
    a.g[a.count] = g[i];
    a.n[a.count] = n[i];
    a.first[a.count++] = (uint32_t)pieces;
    pieces += more;
  }
  return status_of(
      deft::launch_grad_norm(partials, sums, max_norm, inv_scale, control, (hipStream_t)stream));
}

int deft_norm_desc_validate(const deft_norm_desc* d) {
  const int st = norm_desc_status(d);
  NormCut r;
  if (st != DEFT_OK || d->n == 0 || d->s == 0) return st;
  const int fwd = norm_cut(*d, false, r);
  return fwd != DEFT_OK ? fwd : norm_cut(*d, true, r);
}

size_t deft_norm_workspace_bytes(const deft_norm_desc* d, int training) {
  NormCut r;
  if (norm_desc_status(d) != DEFT_OK || d->n == 0 || d->s == 0 || norm_cut(*d, training != 0, r) != DEFT_OK) return 0;
  return norm_ws_bytes(*d, r, training != 0);
}

int deft_norm_forward(const deft_norm_desc* d, const void* x, const void* gamma, const void* beta, void* y,
                      float* mean, float* rstd, void* workspace, size_t ws_bytes, void* stream) {
  int st = norm_desc_status(d);
  if (st != DEFT_OK) return st;
  if (d->n == 0 || d->s == 0) return DEFT_OK;
  NormCut r;
  if ((st = norm_cut(*d, false, r)) != DEFT_OK) return st;
  if (!x || !gamma || !beta || !y || !mean || !rstd) return DEFT_ERR_NULLPTR;
  if (!aligned16(x) || !aligned16(gamma) || !aligned16(beta) || !aligned16(y) || !aligned16(mean) ||
      !aligned16(rstd))
    return DEFT_ERR_ALIGN;
  if (overlap(x, y, (size_t)d->n * d->s * d->c * elem_size(d->dtype))) return DEFT_ERR_BAD_DESC;
  const size_t need = norm_ws_bytes(*d, r, false);
  if (need && (!workspace || ws_bytes < need)) return DEFT_ERR_WORKSPACE;
  if (need && !aligned16(workspace)) return DEFT_ERR_ALIGN;
  r.a.x = x; r.a.gamma = gamma; r.a.beta = beta; r.a.out = y;
  r.a.mean = mean; r.a.rstd = rstd;
  r.a.part = (float*)workspace;
  const hipStream_t s = (hipStream_t)stream;
  if (r.whole) return status_of(deft::launch_norm_fwd(r.a, r.p, d->layout, d->dtype, deft::kNormWhole, s));
  hipError_t e = deft::launch_norm_fwd(r.a, r.p, d->layout, d->dtype, deft::kNormStats, s);
  if (e == hipSuccess) e = deft::launch_norm_combine(r.a, d->layout, s);
  if (e == hipSuccess) e = deft::launch_norm_fwd(r.a, r.p, d->layout, d->dtype, deft::kNormApply, s);
  return status_of(e);
}

int deft_norm_backward(const deft_norm_desc* d, const void* x, const void* gamma, const void* beta,
                       const float* mean, const float* rstd, const void* dy, void* dx, void* dgamma, void* dbeta,
                       void* workspace, size_t ws_bytes, void* stream) {
  int st = norm_desc_status(d);
  if (st != DEFT_OK) return st;
  if (!aligned16(dx) || !aligned16(dgamma) || !aligned16(dbeta)) return DEFT_ERR_ALIGN;
  const hipStream_t s = (hipStream_t)stream;
  const bool params = dgamma || dbeta;
  if (d->n == 0 || d->s == 0)
    return params ? status_of(deft::launch_norm_params(nullptr, 0, d->c, dgamma, dbeta, d->dtype, s)) : DEFT_OK;
  NormCut r;
  if ((st = norm_cut(*d, true, r)) != DEFT_OK) return st;
  if (!x || !gamma || !beta || !mean || !rstd || !dy) return DEFT_ERR_NULLPTR;
  if (!aligned16(x) || !aligned16(gamma) || !aligned16(beta) || !aligned16(mean) || !aligned16(rstd) ||
      !aligned16(dy))
    return DEFT_ERR_ALIGN;
  const size_t bytes = (size_t)d->n * d->s * d->c * elem_size(d->dtype);
  if (overlap(dx, x, bytes) || overlap(dx, dy, bytes)) return DEFT_ERR_BAD_DESC;
  if (!workspace || ws_bytes < norm_ws_bytes(*d, r, true)) return DEFT_ERR_WORKSPACE;
  if (!aligned16(workspace)) return DEFT_ERR_ALIGN;
  if (!dx && !params) return DEFT_OK;
  r.a.x = x; r.a.gamma = gamma; r.a.beta = beta; r.a.dy = dy; r.a.out = dx;
  r.a.mean = const_cast<float*>(mean); r.a.rstd = const_cast<float*>(rstd);  // only read
  r.a.part = (float*)workspace;
  r.a.sums = (float*)((char*)workspace + norm_part_bytes(*d, r, true));
  hipError_t e;
  if (r.whole) {
    e = deft::launch_norm_bwd(r.a, r.p, d->layout, d->dtype, deft::kNormWhole, s);
  } else {
    e = deft::launch_norm_bwd(r.a, r.p, d->layout, d->dtype, deft::kNormStats, s);
    if (e == hipSuccess && dx) e = deft::launch_norm_bwd_sums(r.a, d->layout, d->dtype, s);
    if (e == hipSuccess && dx) e = deft::launch_norm_bwd(r.a, r.p, d->layout, d->dtype, deft::kNormApply, s);
  }
  if (e == hipSuccess && params)
    e = deft::launch_norm_params(r.a.part, d->n * norm_parts(*d, r), d->c, dgamma, dbeta, d->dtype, s);
  return status_of(e);
}

}  // extern "C"
