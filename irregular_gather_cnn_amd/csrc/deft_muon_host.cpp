// C ABI of the Muon step: argument checks, the matrices' shares of the workspace
// and the sequence of launches.  Kernels live in deft_muon.hip.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "deft.h"
#include "deft_internal.h"

namespace {

// Smaller and larger side, and elements: tiles are counted and offsets inside them
// made in 32 bits.
constexpr int64_t kMaxSide = 1 << 15, kMaxLong = 1 << 22, kMaxElems = (int64_t)1 << 32;
constexpr int64_t kChunkBytes = (int64_t)2 << 30;          // workspace, but for single matrices that need more
constexpr int kMaxSteps = 32;
// Newton-Schulz coefficients: sigma -> a sigma + b sigma^3 + c sigma^5 takes
// singular values of (0, 1] to 0.68 .. 1.21 in five steps where they were over 0.002.
constexpr double kA = 3.4445, kB = -4.7750, kC = 2.0315;
// Powers of two by which X and G, Q and P are held (deft_muon.hip).
constexpr double kSx = 16384.0, kSg = 16384.0, kSq = 8192.0, kSp = 1024.0;

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool dtype_ok(int t) { return t == DEFT_F32 || t == DEFT_BF16; }
int status_of(hipError_t e) { return e == hipSuccess ? DEFT_OK : deft::report_hip_error(e); }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int shape_status(const deft_muon_tensor& t) {
  if (t.rows < 0 || t.cols < 0) return DEFT_ERR_BAD_DESC;
  if (t.rows == 0 || t.cols == 0) return DEFT_OK;
  if (std::min(t.rows, t.cols) > kMaxSide || std::max(t.rows, t.cols) > kMaxLong || t.rows * t.cols > kMaxElems)
    return DEFT_ERR_UNSUPPORTED;
  return DEFT_OK;
}

int64_t triangle(int64_t tiles) { return tiles * (tiles + 1) / 2; }
int64_t square_tiles(int m, int tile) { return triangle(ceil_div(deft::muon_pad(m), tile)); }

// Matrices whose launches go together: first and number in the list, their shape
// and shares of the workspace.
struct Chunk {
  deft::MuonItem it[deft::kMuonList];
  int id[deft::kMuonList];
  int count = 0, next = 0;  // next: where in the list the following chunk starts
  int gram = 64, square = 64, apply = 64;  // tiles of the three kinds of product
  bool split = false;       // Gram products in parts
  bool small = false;       // every matrix fits one workgroup
  int fused = 1;            // steps between two products with X
  int64_t bytes = 0;
};

int64_t apply_tiles(int m, int n, int tile) {
  return ceil_div(deft::muon_pad(m), tile) * ceil_div(deft::muon_pad(n), tile);
}
template <typename F>
int64_t sum(const Chunk& c, F of) {
  int64_t n = 0;
  for (int i = 0; i < c.count; ++i) n += of(c.it[i]);
  return n;
}
void choose_tiles(Chunk& c, int cus) {
  auto squares = [&](int t) { return sum(c, [&](const deft::MuonItem& i) { return square_tiles(i.m, t); }); };
  auto applies = [&](int t) { return sum(c, [&](const deft::MuonItem& i) { return apply_tiles(i.m, i.n, t); }); };
  // Large tiles read less from LDS for a product, small ones fill the units: 8 matrices
  // of 256 x 2304 take 240 us with these, 281 with 64 in P X, 300 with 128 in squares, 4
  // of 1024 x 9216 1715, 2325 and 1860 (64 in squares); 256 there 2176.
  c.square = squares(128) >= cus / 2 ? 128 : 64;
  c.apply = applies(256) >= cus ? 256 : applies(128) >= cus / 2 ? 128 : 64;
  // these are split over n as well: 4 of 1024 x 9216 1715 us with 256, 1823 with 128
  c.gram = squares(256) >= cus / 8 ? 256 : squares(128) >= cus / 8 ? 128 : 64;
  // Two steps between products with X take 4 products of squares more and, of 3 m^2 n
  // operations, one Gram product and one with X fewer than two single ones. Three at a
  // time would take a quarter off where n = 9 m, but for some spectra the directions are
  // off by 6 times as much as those of single steps in fp32, not by up to twice.
  double wide = 0.0, square = 0.0;
  for (int i = 0; i < c.count; ++i) {
    wide += (double)c.it[i].m * c.it[i].m * c.it[i].n;
    square += (double)c.it[i].m * c.it[i].m * c.it[i].m;
  }
  c.fused = wide > 2.0 * square ? 2 : 1;
}

// The next chunk of the list from `at` on; its items' shares start at `base`.
void next_chunk(const deft_muon_tensor* t, int count, int at, int cus, char* base, Chunk& c) {
  c.count = 0;
  c.bytes = 0;
  int64_t most = 0;
  for (c.next = at; c.next < count && c.count < deft::kMuonList; ++c.next) {
    const deft_muon_tensor& x = t[c.next];
    if (x.rows == 0 || x.cols == 0) continue;
    deft::MuonItem& y = c.it[c.count];
    y.m = (int)std::min(x.rows, x.cols);
    y.n = (int)std::max(x.rows, x.cols);
    y.tall = x.rows > x.cols;
    y.splits = 1;
    const int64_t need = deft::muon_item_bytes(y.m, y.n, 1);
    if (c.count && most + need > kChunkBytes) break;
    most += need;
    c.id[c.count++] = c.next;
  }
  c.small = true;
  for (int i = 0; i < c.count; ++i)
    c.small &= c.it[i].m <= deft::kMuonSmallSide && deft::muon_small_lds(c.it[i].m, c.it[i].n) <= deft::kMuonSmallLds;
  if (c.small) {  // no workspace
    c.bytes = 0;
    return;
  }
  // the sums over n are split where their tiles leave compute units idle, into no
  // fewer than 16 stages
  choose_tiles(c, cus);
  const int64_t tiles = sum(c, [&](const deft::MuonItem& i) { return square_tiles(i.m, c.gram); });
  const int64_t splits = tiles ? std::max<int64_t>(1, (c.gram == 256 ? 1 : 2) * cus / tiles) : 1;
  c.split = false;
  for (int i = 0; i < c.count; ++i) {
    c.it[i].splits = (int)std::max<int64_t>(1, std::min<int64_t>(splits, deft::muon_pad(c.it[i].n) / 256));
    c.split |= c.it[i].splits > 1;
  }
  for (int i = 0; i < c.count; ++i) {
    c.it[i].base = base + c.bytes;
    c.bytes += deft::muon_item_bytes(c.it[i].m, c.it[i].n, c.split ? std::max(2, c.it[i].splits) : 1);
  }
}

// Sets the first workgroups of the items, `of` each; the sum.
template <typename F>
uint32_t lay(deft::MuonArgs& a, F of) {
  int64_t at = 0;
  for (int i = 0; i < a.count; ++i) {
    a.first[i] = (uint32_t)at;
    at += of(a.it[i]);
  }
  return (uint32_t)at;
}

struct Launcher {
  deft::MuonArgs& a;
  const Chunk& c;
  int p_dtype;
  bool master;
  hipStream_t st;
  hipError_t e = hipSuccess;

  void gram(int x, int out) {
    if (e != hipSuccess) return;
    a.ph = {x, x, out, -1, (float)(kSg / (kSx * kSx)), 0.f, 0.f};
    const uint32_t n = lay(a, [&](const deft::MuonItem& i) { return square_tiles(i.m, c.gram) * (c.split ? i.splits : 1); });
    e = deft::launch_muon_square(a, n, c.gram, c.split, st);
    if (e != hipSuccess || !c.split) return;
    e = deft::launch_muon_join(a, lay(a, [](const deft::MuonItem& i) { return square_tiles(i.m, 32); }), st);
  }
  void squares() {
    if (e != hipSuccess) return;
    e = deft::launch_muon_square(a, lay(a, [&](const deft::MuonItem& i) { return square_tiles(i.m, c.square); }), c.square,
                                 false, st);
  }
  void apply(int p, double scale, int x, int out, bool last) {
    if (e != hipSuccess) return;
    a.ph = {p, x, out, -1, (float)(last ? 1.0 / (scale * kSx) : 1.0 / scale), 0.f, 0.f};
    e = deft::launch_muon_apply(a, lay(a, [&](const deft::MuonItem& i) { return apply_tiles(i.m, i.n, c.apply); }), c.apply,
                                last, p_dtype, master, st);
  }

  // One or two steps on the X in buffer x; the result goes to the other one, or to the
  // weights.
  void fused(int steps, int x, bool last) {
    // buffers of the squares: G, Q1 and Q2, the second G, Q1 G, Q2 Q1
    const int g = 2, q1 = 3, q2 = 4, g2 = 5, r = 6, both = 7;
    auto poly = [&](int of, int to) {
      a.ph = {of, of, to, of, (float)(kC * kSq / (kSg * kSg)), (float)(kA * kSq), (float)(kB * kSq / kSg)};
      squares();
    };
    auto times = [&](int left, int right, int to, double factor) {
      a.ph = {left, right, to, -1, (float)factor, 0.f, 0.f};
      squares();
    };
    gram(x, g);
    poly(g, q1);
    int p = q1;
    double scale = kSq;
    if (steps == 2) {
      times(q1, g, r, 1.0 / kSq);
      times(q1, r, g2, 1.0 / kSq);
      poly(g2, q2);
      times(q2, q1, both, kSp / (kSq * kSq));
      p = both;
      scale = kSp;
    }
    apply(p, scale, x, 1 - x, last);
  }
};

}  // namespace

extern "C" {

size_t deft_muon_workspace_bytes(const deft_muon_tensor* t, int count) {
  if (count <= 0 || !t) return 0;
  for (int i = 0; i < count; ++i)
    if (shape_status(t[i]) != DEFT_OK) return 0;
  int64_t most = 0;
  Chunk c;
  const int cus = deft::compute_units();
  for (int at = 0; at < count; at = c.next) {
    next_chunk(t, count, at, cus, nullptr, c);
    most = std::max(most, c.bytes);
  }
  return (size_t)most;
}

int deft_muon_step(const deft_muon_desc* d, const deft_muon_tensor* t, int count, const float* control,
                   const double* schedule, void* workspace, size_t ws_bytes, void* stream) {
  if (!d || (count > 0 && !t)) return DEFT_ERR_NULLPTR;
  if (!dtype_ok(d->p_dtype) || !dtype_ok(d->g_dtype)) return DEFT_ERR_DTYPE;
  // negated comparisons refuse NaN
  if (count < 0 || d->steps < 1 || d->steps > kMaxSteps || (d->nesterov != 0 && d->nesterov != 1) || !(d->lr >= 0.0) ||
      !std::isfinite(d->lr) || !(d->momentum >= 0.0 && d->momentum < 1.0) || !(d->eps >= 1e-30) || !std::isfinite(d->eps) ||
      (d->master != 0 && d->master != 1) || (d->master && d->p_dtype == DEFT_F32))
    return DEFT_ERR_BAD_DESC;
  if (!aligned(control, 4) || !aligned(schedule, 8)) return DEFT_ERR_ALIGN;
  for (int i = 0; i < count; ++i) {
    const deft_muon_tensor& x = t[i];
    const int st = shape_status(x);
    if (st != DEFT_OK) return st;
    if (!(x.weight_decay >= 0.0) || !std::isfinite(x.weight_decay) || !std::isfinite(x.scale)) return DEFT_ERR_BAD_DESC;
    if (x.rows == 0 || x.cols == 0) continue;
    if (!x.p || !x.g || !x.m || (d->master && !x.master)) return DEFT_ERR_NULLPTR;
    if (!aligned(x.p, 16) || !aligned(x.g, 16) || !aligned(x.m, 16) || (d->master && !aligned(x.master, 16)))
      return DEFT_ERR_ALIGN;
  }
  const size_t need = deft_muon_workspace_bytes(t, count);
  if (need && (!workspace || ws_bytes < need)) return DEFT_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return DEFT_ERR_ALIGN;
  const int cus = deft::compute_units();
  const hipStream_t st = (hipStream_t)stream;
  Chunk c;
  for (int at = 0; at < count; at = c.next) {
    next_chunk(t, count, at, cus, (char*)workspace, c);
    if (!c.count) continue;
    deft::MuonArgs a;
    std::memset(&a, 0, sizeof(a));
    a.count = c.count;
    a.mu = (float)d->momentum;
    a.nu = (float)(1.0 - d->momentum);
    a.nesterov = d->nesterov;
    a.eps = d->eps;
    a.lr = d->lr;
    a.control = control;
    a.schedule = schedule;
    for (int i = 0; i < c.count; ++i) {
      const deft_muon_tensor& x = t[c.id[i]];
      deft::MuonItem& y = a.it[i] = c.it[i];
      y.p = x.p;
      y.g = x.g;
      y.mom = x.m;
      y.master = x.master;
      y.decay = x.weight_decay;
      y.scale = x.scale;
    }
    if (c.small) {
      deft::MuonSmall f;
      f.steps = d->steps;
      f.lds = 0;
      for (int i = 0; i < c.count; ++i) f.lds = std::max<int>(f.lds, (int)deft::muon_small_lds(c.it[i].m, c.it[i].n));
      f.g = (float)(kSg / (kSx * kSx));
      f.a = (float)(kA * kSq);
      f.b = (float)(kB * kSq / kSg);
      f.c = (float)(kC * kSq / (kSg * kSg));
      f.x = (float)(1.0 / kSq);
      f.o = (float)(1.0 / (kSq * kSx));
      const hipError_t e = deft::launch_muon_small(a, f, d->p_dtype, d->g_dtype, d->master != 0, st);
      if (e != hipSuccess) return status_of(e);
      continue;
    }
    hipError_t e = deft::launch_muon_momentum(
        a, lay(a, [](const deft::MuonItem& i) {
          const int64_t n = (int64_t)i.m * i.n;
          return ceil_div(n, deft::muon_chunk(n));
        }), d->g_dtype, st);
    if (e == hipSuccess)
      e = deft::launch_muon_scale(
          a, lay(a, [](const deft::MuonItem& i) { return ceil_div(deft::muon_pad(i.m), 64) * ceil_div(deft::muon_pad(i.n), 64); }),
          d->g_dtype, st);
    if (e != hipSuccess) return status_of(e);
    Launcher l{a, c, d->p_dtype, d->master != 0, st};
    // as few parts as there may be, the larger ones first
    int parts = (d->steps + c.fused - 1) / c.fused, left = d->steps, x = 0;
    for (; parts > 0; --parts) {
      const int k = (left + parts - 1) / parts;
      l.fused(k, x, parts == 1);
      x = 1 - x;
      left -= k;
    }
    if (l.e != hipSuccess) return status_of(l.e);
  }
  return DEFT_OK;
}

}  // extern "C"
