// C ABI of the training operators around the convolutions: argument checks,
// workspace sizes and launch sequencing.  Kernels live in deft_optim.hip.
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

}  // extern "C"
