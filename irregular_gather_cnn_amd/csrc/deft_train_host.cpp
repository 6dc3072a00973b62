// C ABI of the training operators around the convolutions: argument checks,
// workspace sizes and launch sequencing.  Kernels live in deft_optim.hip,
// deft_norm_fwd.hip and deft_norm_bwd.hip.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "deft.h"
#include "deft_internal.h"

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned8(const void* p) { return ((uintptr_t)p & 7u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
bool dtype_ok(int t) { return t == DEFT_F32 || t == DEFT_BF16; }
int status_of(hipError_t e) { return e == hipSuccess ? DEFT_OK : deft::report_hip_error(e); }

// A launch has fewer than 2^32 threads.
constexpr uint64_t max_blocks(int threads) { return 0xffffffffu / (uint32_t)threads; }

constexpr uint64_t kAdamwBlocks = max_blocks(deft::kAdamwThreads);

// Gradients of one norm; their pieces stay below 2^31.
constexpr uint64_t kMaxElems = 1ull << 44;
constexpr double kCacheBytes = 256e6;

int elem_size(int dtype) { return dtype == DEFT_BF16 ? 2 : 4; }
uint64_t blocks_of(int64_t n, int64_t per) { return ((uint64_t)n + per - 1) / per; }

int norm_launches(int count) { return std::max(1, (count + deft::kNormList - 1) / deft::kNormList); }

// ---- group norm: how a call is cut ----

constexpr int kMaxPer = 2048;      // channels per group: a row of one group fits a workgroup
constexpr size_t kAlign = 256;

size_t round_up(size_t v, size_t m) { return (v + m - 1) / m * m; }
int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

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
  int mode;  // kNormWhole, kNormJoint, or kNormStats: statistics, then a second launch
  int cus;   // compute units of the device that it is cut for
};

// Workgroups of `threads` that the chip holds at once: the forward's joint
// kernels take up to 128 registers, the backward's up to 256.
int resident(const NormCut& r, bool back, int threads) { return r.cus * (back ? 512 : 1024) / threads; }

// One slice for a group (or a band of groups), where it fits the registers: 32
// accesses a thread forward, 16 of x and of dy backward.  It needs no
// exchange, which costs 3 to 5 us, but only as many compute units work as there
// are groups; so where these leave units idle, it pays up to about 5 us of one
// unit's work, counted in vector operations an element, of which reading and
// writing it forward cost as much as 26 in bf16 and 52 in fp32.  Measured forward
// (us in one slice and joined): 12 bands of 9000 elements, gelu fp32, 8.6 and 10.7;
// 5 groups of 20252, relu bf16, 6.1 and 7.1; 10 of 43590, none bf16, 10.2 and 8.6; 50
// of 42476, none fp32, 18.7 and 10.9.
//
// 17 to 32 accesses forward fill a unit with one workgroup (and 7 to 24 registers
// of a thread spill, but for fp32 channels last, which takes 177).  That pays
// where all run at once: against slices, 240 groups channels first fp32 23.5 us
// and 24.4, 240 bands channels last bf16 30.9 and 33.1, 231 groups channels first
// bf16 23.9 and 33.1.  A second round that is not full loses it: 309 groups
// channels first fp32 37 and 28, 574 66 and 43, 1024 100 and 84; channels last bf16
// 8 images of 7000 x 640 69 and 47.  Channels first in bf16 gains over full rounds: 512 groups
// 48 and 52, 670 60 and 77, but 578 67 and 57, 308 48 and 39.
bool whole_pays(const deft_norm_desc& d, const NormCut& r, bool back, int V, int rounds, int64_t units, int64_t elems) {
  if (rounds > (V == 1 || back ? 16 : 32)) return false;
  if (rounds > 16 && units > r.cus) {
    const int64_t room = (units + r.cus - 1) / r.cus * r.cus;
    if (d.layout != DEFT_CHANNELS_FIRST || d.dtype != DEFT_BF16 || units * 5 < room * 4) return false;
  }
  if (units >= r.cus * 3 / 4) return true;
  const int act = d.act == DEFT_ACT_GELU ? 40 : d.act == DEFT_ACT_SILU ? 24 : 12;
  const int bytes = d.dtype == DEFT_F32 ? 52 : 26;
  if (back) return elems * std::max(2 * act, bytes * 3 / 2) <= 1000000;
  return elems * std::max(act, bytes) <= 800000;
}

// 9 to 16 accesses of 512 threads as up to 8 of 1024.
bool goes_wide(const deft_norm_desc& d, bool back, int V, int rounds) {
  const bool keep = d.dtype == DEFT_BF16 && d.act >= DEFT_ACT_SILU;
  return back && V > 1 && rounds > 8 && rounds <= 16 &&
         deft::norm_bwd_wide(d.dtype == DEFT_F32, d.layout == DEFT_CHANNELS_LAST, keep);
}

// Channels last.  Whole: bands of groups, 32 bytes of each row or more (64
// backward from 2^20 elements on, where the lines that bands share no longer
// come from the cache: 16x784x512 bf16 takes 20 us against 24).  Else slices of
// whole rows, of 1024 channels at most, of 4 to 8 accesses a thread (fewer when
// they would leave compute units idle: 443 slices of 4 rows took 18 us where 111
// of 16 take 14).  Every slice has all groups here, so the exchange grows with
// both, and from 2^21 elements on a second read costs less: forward 33.5 M elements
// in bf16 with gelu 94 us joined and 56 read twice, 8.9 M 24 and 19, 1.4 M 11.3 and
// 12.2; backward 24.4 M 93 and 78, 7.1 M in fp32 48 and 38, 1.3 M 18 and 19.
void cut_last(const deft_norm_desc& d, bool back, NormCut& r) {
  const int per = r.a.per, g = d.groups, esz = elem_size(d.dtype);
  const int V = d.c >= 16 / esz ? 16 / esz : 1;
  r.p.vec = V;
  // chunks across the widest of `bands` bands
  auto widest = [&](int bands) { return ceil_div((int64_t)ceil_div(g, bands) * per, V); };
  int nt;
  const int wide = back && (int64_t)d.n * d.s * d.c >= 1 << 20 ? 64 : 32;
  int bands = std::max(1, g / std::min(g, ceil_div(wide, per * esz)));
  while (bands > 1 && g / bands * per < V) --bands;
  // no more threads than four accesses each need: with 512 the backward of 21x29x504 in
  // bf16 takes 19 us where it takes 10
  nt = 64;
  while (nt < deft::kNormThreads && (widest(bands) > nt || ceil_div(d.s, nt / widest(bands)) > 4)) nt *= 2;
  int rounds = ceil_div(d.s, nt / widest(bands));
  if (goes_wide(d, back, V, rounds)) {
    nt = deft::kNormWide;
    rounds = 8;  // the kernel for it; half as many as before are needed
  }
  r.mode = deft::kNormWhole;
  r.a.slices = 1;
  r.a.rp = d.s;
  if (!whole_pays(d, r, back, V, rounds, (int64_t)d.n * bands, (int64_t)ceil_div(g, bands) * per * d.s)) {
    bands = ceil_div(g, std::max(1, 1024 / per));
    nt = back && widest(bands) <= 256 ? 256 : deft::kNormThreads;
    int ty = nt / widest(bands);
    rounds = 8;
    auto slices = [&] { return ceil_div(d.s, (int64_t)ty * rounds); };
    while (rounds > 4 && (int64_t)d.n * bands * slices() < r.cus) rounds /= 2;
    const bool joint = (int64_t)d.n * d.s * d.c < 1 << 21 && slices() <= resident(r, back, nt);
    r.mode = joint ? deft::kNormJoint : deft::kNormStats;
    r.a.rp = ty * rounds;
    if (back && r.mode == deft::kNormStats) {
      // read twice: small accumulating workgroups, two on each unit (20.4 M elements in
      // bf16 take 48 us; four or one a unit 52 and 64), whose slices' sums are few; no
      // slice over 64 accesses, to keep the chains of sums short
      nt = widest(bands) <= 256 ? 256 : deft::kNormThreads;
      ty = nt / widest(bands);
      rounds = 4;
      const int blocks = ceil_div(d.s, ty * rounds), want = (int)std::max<int64_t>(1, 2 * r.cus / ((int64_t)d.n * bands));
      r.a.rp = std::min(ceil_div(blocks, std::min(blocks, want)), 16) * ty * rounds;
    }
    r.a.slices = ceil_div(d.s, r.a.rp);
    // with more words than this it takes a workgroup longer to read them all than to
    // wait until others have added them up
    r.a.direct = r.a.slices * ceil_div(g, bands) <= 2048;
  }
  r.a.bands = bands;
  r.p.u = rounds;
  r.p.threads = nt;
  const size_t cols = (size_t)ceil_div(g, bands) * per, ng = ceil_div(g, bands);
  // two matrices of thread rows and odd pitch: at most nt * V elements and one more per row
  r.p.lds = sizeof(float) * (2 * ((size_t)nt * V + nt) + (back ? 4 : 2) * (ng + cols));
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

// Channels first.  Whole: one workgroup a group, no larger than four accesses a
// thread need.  Else slices of whole channels, or of a channel's positions where
// one is long, of 4 to 8 accesses a thread.
void cut_first(const deft_norm_desc& d, bool back, NormCut& r) {
  const int per = r.a.per, esz = elem_size(d.dtype), V = d.s >= 16 / esz ? 16 / esz : 1;
  const int chunks = ceil_div(d.s, V);
  r.p.vec = V;
  int nt = 64;
  int rounds = best_team(nt, per, chunks, &r.a.lt);
  while (rounds > 4 && nt < deft::kNormThreads) rounds = best_team(nt *= 2, per, chunks, &r.a.lt);
  int lt = 0;
  if (goes_wide(d, back, V, rounds) && best_team(deft::kNormWide, per, chunks, &lt) <= 8) {
    nt = deft::kNormWide;
    rounds = 8;  // the kernel for it
    r.a.lt = lt;
  }
  r.mode = deft::kNormWhole;
  r.a.rp = per;
  r.a.ws = 1;
  r.a.cp = d.s;
  if (!whole_pays(d, r, back, V, rounds, (int64_t)d.n * d.groups, (int64_t)per * d.s)) {
    nt = back ? 256 : deft::kNormThreads;
    int cpc = ceil_div(chunks, ceil_div(chunks, nt * 4));  // chunks of a channel in a slice
    int rp = std::min(per, std::max(1, nt * 8 / cpc));
    auto slices = [&] { return (int64_t)ceil_div(per, rp) * ceil_div(chunks, cpc); };
    while ((int64_t)d.n * d.groups * slices() < r.cus && rp * (int64_t)cpc > nt * 4) {
      if (rp > 1) rp = (rp + 1) / 2;
      else cpc = (cpc + 1) / 2;
    }
    while ((rounds = best_team(nt, rp, cpc, &r.a.lt)) > 8) --rp;  // rp = 1: four at most
    r.a.rp = rp;
    r.a.cp = cpc * V;
    r.a.ws = ceil_div(chunks, cpc);
    r.mode = slices() <= resident(r, back, nt) ? deft::kNormJoint : deft::kNormStats;
    r.a.direct = 1;
  }
  r.a.slices = ceil_div(per, r.a.rp) * r.a.ws;
  r.p.threads = nt;
  r.p.u = rounds;
  const int subs = std::max(1, (1 << r.a.lt) >> 6);
  r.p.lds = sizeof(float) * (back ? std::max(2 * nt, 32 + (2 + 2 * subs) * r.a.rp) : 32 + 2 * r.a.rp);
}

int norm_cut(const deft_norm_desc& d, bool back, NormCut& r, int cus = deft::compute_units()) {
  std::memset(&r, 0, sizeof(r));
  r.cus = cus;
  r.a.n = d.n; r.a.c = d.c; r.a.s = d.s; r.a.g = d.groups;
  r.a.per = d.c / d.groups;
  r.a.act = d.act;
  r.a.eps = (float)d.eps;
  if (d.layout == DEFT_CHANNELS_LAST) cut_last(d, back, r);
  else cut_first(d, back, r);
  const uint64_t units = (uint64_t)d.n * (d.layout == DEFT_CHANNELS_LAST ? r.a.bands : d.groups);
  // units first: with the slices of one unit, under 2^31, their product stays in 64 bits;
  // a call that is read twice also has launches of one workgroup a group
  const uint64_t groups = (uint64_t)d.n * d.groups;  // numbered in 31 bits
  if (units > max_blocks(r.p.threads) || units * r.a.slices > max_blocks(r.p.threads) || groups > 0x7fffffffu ||
      (r.mode == deft::kNormStats && groups > max_blocks(back ? 1024 : 256)))
    return DEFT_ERR_UNSUPPORTED;
  r.p.blocks = (uint32_t)(units * r.a.slices);
  return DEFT_OK;
}

// Slices whose channel sums stand apart.
int norm_parts(const deft_norm_desc& d, const NormCut& r) {
  return d.layout == DEFT_CHANNELS_LAST ? r.a.slices : r.a.ws;
}

// One direction's share of a workspace, at `base`: what joint workgroups share
// (kept from call to call), then the partial sums.  Fills in the pointers and
// returns the bytes.
size_t norm_layout(const deft_norm_desc& d, bool back, NormCut& r, char* base) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = base + at;
    at = round_up(at + bytes, kAlign);
    return p;
  };
  const size_t groups = (size_t)d.n * d.groups;
  if (r.mode == deft::kNormJoint) {
    const size_t clusters = d.layout == DEFT_CHANNELS_LAST ? (size_t)d.n * r.a.bands : groups;
    r.a.counter = (uint64_t*)take(clusters * 8);
    r.a.words = (uint64_t*)take(groups * r.a.slices * 16);
    r.a.totals = (uint64_t*)take(r.a.direct ? 0 : groups * 16);
  }
  // Small calls: the last workgroup sums up dgamma and dbeta.  That saves a launch
  // (3 us on the host), and costs 1 to 3 us on the device, which has time here.
  if (back && r.mode == deft::kNormWhole && (int64_t)d.n * d.s * d.c <= 200000)
    r.a.arrivals = (uint64_t*)take((d.layout == DEFT_CHANNELS_LAST ? r.a.bands : d.groups) * 8);
  if (back) {
    r.a.part = (float*)take((size_t)d.n * norm_parts(d, r) * 2 * d.c * 4);
    r.a.sums = (float*)take(r.mode == deft::kNormStats ? groups * 8 : 0);
  } else {
    r.a.part = (float*)take(r.mode == deft::kNormStats ? groups * r.a.slices * 8 : 0);
  }
  return at;
}

std::atomic<uint32_t> g_patience{200000};  // 2 ms

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
  if (!aligned4(control) || !aligned8(d->skipped) || !aligned8(schedule)) return DEFT_ERR_ALIGN;
  for (int i = 0; i < count; ++i) {
    const deft_adamw_tensor& x = t[i];
    if (x.n < 0 || !(x.weight_decay >= 0.0) || !std::isfinite(x.weight_decay)) return DEFT_ERR_BAD_DESC;
    if (x.n == 0) continue;
    if (blocks_of(x.n, deft::kAdamwElems) > kAdamwBlocks) return DEFT_ERR_UNSUPPORTED;
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
  a.skips = (deft::AdamwSkips*)d->skipped;
  a.lr = d->lr;
  a.log1 = std::log2(d->beta1);
  a.log2 = std::log2(d->beta2);
  a.step = d->step;
  a.lead = 1;
  // A step over more than the last-level cache holds leaves nothing of itself there
  // for the next one.
  double elems = 0.0;
  for (int i = 0; i < count; ++i) elems += (double)t[i].n;
  const int weights = d->master ? 8 + elem_size(d->p_dtype) : 2 * elem_size(d->p_dtype);
  const bool once = elems * (elem_size(d->g_dtype) + weights + (d->state_bits == 8 ? 4 : 16)) > kCacheBytes;
  uint64_t blocks = 0;
  for (int i = 0; i <= count; ++i) {
    const uint64_t more = i < count ? blocks_of(t[i].n, deft::kAdamwElems) : 0;
    // the list is full, or at its end: launch what it holds
    if (a.count && (i == count || (more && (a.count == deft::kAdamwList || blocks + more > kAdamwBlocks)))) {
      const hipError_t e = deft::launch_adamw(a, (uint32_t)blocks, d->p_dtype, d->g_dtype, d->state_bits,
                                              d->master != 0, once, (hipStream_t)stream);
      if (e != hipSuccess) return status_of(e);
      a.count = a.lead = 0;
      blocks = 0;
    }
    if (!more) continue;
    const deft_adamw_tensor& x = t[i];
    deft::AdamwTensor& y = a.t[a.count];
    y.p = x.p; y.g = x.g; y.m = x.m; y.v = x.v;
    y.m_scale = x.m_scale; y.v_scale = x.v_scale;
    y.master = x.master;
    y.n = x.n;
    y.decay = schedule ? x.weight_decay : 1.0 - d->lr * x.weight_decay;
    a.id[a.count] = (uint32_t)i;
    a.first[a.count++] = (uint32_t)blocks;
    blocks += more;
  }
  return DEFT_OK;
}

// The workgroups' counter, then their sums: 8 KB for each launch hold both.
static_assert(kAlign + deft::kNormGrid * sizeof(double) <= 8192, "grad norm workspace");
size_t deft_grad_norm_workspace_bytes(int count) { return (size_t)norm_launches(std::max(count, 0)) * 8192; }

int deft_grad_norm(const void* const* g, const int64_t* n, int count, int g_dtype, double max_norm,
                   double inv_scale, float* control, void* workspace, size_t ws_bytes, void* stream) {
  if (!control || (count > 0 && (!g || !n))) return DEFT_ERR_NULLPTR;
  if (!dtype_ok(g_dtype)) return DEFT_ERR_DTYPE;
  if (count < 0 || !(max_norm > 0.0) || !(inv_scale > 0.0) || !std::isfinite(inv_scale)) return DEFT_ERR_BAD_DESC;
  uint64_t all = 0;
  for (int i = 0; i < count; ++i) {
    if (n[i] < 0) return DEFT_ERR_BAD_DESC;
    if (n[i] == 0) continue;
    all += (uint64_t)n[i];
    if ((uint64_t)n[i] > kMaxElems || all > kMaxElems) return DEFT_ERR_UNSUPPORTED;
    if (!g[i]) return DEFT_ERR_NULLPTR;
    if (!aligned16(g[i])) return DEFT_ERR_ALIGN;
  }
  if (!aligned16(control)) return DEFT_ERR_ALIGN;
  if (!workspace || ws_bytes < deft_grad_norm_workspace_bytes(count)) return DEFT_ERR_WORKSPACE;
  if (!aligned16(workspace)) return DEFT_ERR_ALIGN;
  deft::GradNormArgs a;
  std::memset(&a, 0, sizeof(a));
  a.arrived = (uint64_t*)workspace;
  a.partials = (double*)((char*)workspace + kAlign);
  a.max_norm = max_norm;
  a.inv_scale = inv_scale;
  a.control = control;
  // first how many workgroups the launches have in all, then the launches; a list
  // of no elements has one workgroup
  for (int pass = 0; pass < 2; ++pass) {
    uint32_t sums = 0;
    uint64_t pieces = 0;
    a.count = 0;
    for (int i = 0; i <= count; ++i) {
      const uint64_t more = i < count ? blocks_of(n[i], deft::kNormPiece) : 0;
      if ((a.count && (i == count || (more && a.count == deft::kNormList))) || (i == count && !sums)) {
        const uint32_t grid = (uint32_t)std::min<uint64_t>(std::max<uint64_t>(pieces, 1), deft::kNormGrid);
        a.pieces = (uint32_t)pieces;
        a.at = sums;
        if (pass == 1) {
          const hipError_t e = deft::launch_grad_norm(a, g_dtype, grid, (hipStream_t)stream);
          if (e != hipSuccess) return status_of(e);
        }
        sums += grid;
        a.count = 0;
        pieces = 0;
      }
      if (!more) continue;
      a.g[a.count] = g[i];
      a.n[a.count] = n[i];
      a.first[a.count++] = (uint32_t)pieces;
      pieces += more;
    }
    a.sums = sums;
  }
  return DEFT_OK;
}

int deft_norm_desc_validate(const deft_norm_desc* d) {
  const int st = norm_desc_status(d);
  NormCut r;
  if (st != DEFT_OK || d->n == 0 || d->s == 0) return st;
  const int fwd = norm_cut(*d, false, r);
  return fwd != DEFT_OK ? fwd : norm_cut(*d, true, r);
}

size_t deft_norm_workspace_bytes(const deft_norm_desc* d, int training) {
  NormCut f, b;
  if (norm_desc_status(d) != DEFT_OK || d->n == 0 || d->s == 0 || norm_cut(*d, false, f) != DEFT_OK) return 0;
  const size_t fwd = norm_layout(*d, false, f, nullptr);
  if (!training) return fwd;
  return norm_cut(*d, true, b) == DEFT_OK ? fwd + norm_layout(*d, true, b, nullptr) : 0;
}

int deft_debug_norm_cut(const deft_norm_desc* d, int back, int cus, int* cut) {
  const int st = norm_desc_status(d);
  if (st != DEFT_OK) return st;
  if (!cut) return DEFT_ERR_NULLPTR;
  if (cus < 0 || d->n == 0 || d->s == 0) return DEFT_ERR_BAD_DESC;
  NormCut r;
  const int e = norm_cut(*d, back != 0, r, cus ? cus : deft::compute_units());
  if (e != DEFT_OK) return e;
  const int out[8] = {r.mode, r.p.vec, r.p.u, r.p.threads, r.a.slices, (int)r.p.blocks, r.a.direct, r.cus};
  std::memcpy(cut, out, sizeof(out));
  return DEFT_OK;
}

void deft_debug_norm_patience(uint32_t ticks) { g_patience = ticks; }

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
  const size_t need = norm_layout(*d, false, r, (char*)workspace);
  if (need && (!workspace || ws_bytes < need)) return DEFT_ERR_WORKSPACE;
  if (need && !aligned16(workspace)) return DEFT_ERR_ALIGN;
  r.a.x = x; r.a.gamma = gamma; r.a.beta = beta; r.a.out = y;
  r.a.mean = mean; r.a.rstd = rstd;
  r.a.patience = g_patience;
  const hipStream_t s = (hipStream_t)stream;
  hipError_t e = deft::launch_norm_fwd(r.a, r.p, d->layout, d->dtype, r.mode, s);
  if (r.mode == deft::kNormStats) {
    if (e == hipSuccess) e = deft::launch_norm_combine(r.a, d->layout, s);
    if (e == hipSuccess) e = deft::launch_norm_fwd(r.a, r.p, d->layout, d->dtype, deft::kNormApply, s);
  }
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
  NormCut f, r;
  const int cus = deft::compute_units();
  if ((st = norm_cut(*d, false, f, cus)) != DEFT_OK || (st = norm_cut(*d, true, r, cus)) != DEFT_OK) return st;
  if (!x || !gamma || !beta || !mean || !rstd || !dy) return DEFT_ERR_NULLPTR;
  if (!aligned16(x) || !aligned16(gamma) || !aligned16(beta) || !aligned16(mean) || !aligned16(rstd) ||
      !aligned16(dy))
    return DEFT_ERR_ALIGN;
  const size_t bytes = (size_t)d->n * d->s * d->c * elem_size(d->dtype);
  if (overlap(dx, x, bytes) || overlap(dx, dy, bytes)) return DEFT_ERR_BAD_DESC;
  // the forward's share comes first
  const size_t fwd = norm_layout(*d, false, f, (char*)workspace);
  if (!workspace || ws_bytes < fwd + norm_layout(*d, true, r, (char*)workspace + fwd)) return DEFT_ERR_WORKSPACE;
  if (!aligned16(workspace)) return DEFT_ERR_ALIGN;
  if (!dx && !params) return DEFT_OK;
  r.a.x = x; r.a.gamma = gamma; r.a.beta = beta; r.a.dy = dy; r.a.out = dx;
  r.a.mean = const_cast<float*>(mean); r.a.rstd = const_cast<float*>(rstd);  // only read
  r.a.patience = g_patience;
  const bool after = params && !r.a.arrivals;
  if (!params) r.a.arrivals = nullptr;
  r.a.dgamma = dgamma; r.a.dbeta = dbeta;
  hipError_t e = deft::launch_norm_bwd(r.a, r.p, d->layout, d->dtype, r.mode, s);
  if (r.mode == deft::kNormStats && dx) {
    if (e == hipSuccess) e = deft::launch_norm_bwd_sums(r.a, d->layout, d->dtype, s);
    if (e == hipSuccess) e = deft::launch_norm_bwd(r.a, r.p, d->layout, d->dtype, deft::kNormApply, s);
  }
  if (e == hipSuccess && after)
    e = deft::launch_norm_params(r.a.part, d->n * norm_parts(*d, r), d->c, dgamma, dbeta, d->dtype, s);
  return status_of(e);
}

}  // extern "C"
