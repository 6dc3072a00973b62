// C ABI of the 8-bit pointwise convolution: argument checks, the layout of codes
// in the caller's buffers, the choice of tiles and splits, and launch
// sequencing.  Kernels live in deft_pw8_quantise.hip, deft_pw8_gemm.hip and
// deft_pw8_few.hip.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "deft.h"
#include "deft_internal.h"

namespace {

constexpr size_t kAlign = 256;
constexpr int64_t kMaxRows = 0x7fffffffLL - 128, kMaxChannels = 1 << 20;
constexpr int64_t kMaxBlocks = 0xffffffffu / 256;  // a launch has fewer than 2^32 threads

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
int status_of(hipError_t e) { return e == hipSuccess ? DEFT_OK : deft::report_hip_error(e); }
size_t round_up(size_t v, size_t m) { return (v + m - 1) / m * m; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t blocks_of(int64_t depth) { return ceil_div(depth, deft::kPw8Block); }
int elem_size(int dtype) { return dtype == DEFT_BF16 ? 2 : 4; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t p = (uintptr_t)a, q = (uintptr_t)b;
  return p && q && p < q + nb && q < p + na;
}

struct Span {
  const void* p;  // nullptr: none
  size_t bytes;
};
// Whether something that is written lies over anything else.
bool overlap(std::initializer_list<Span> written, std::initializer_list<Span> read) {
  for (const Span* a = written.begin(); a != written.end(); ++a) {
    for (const Span* b = a + 1; b != written.end(); ++b)
      if (overlap(a->p, a->bytes, b->p, b->bytes)) return true;
    for (const Span& b : read)
      if (overlap(a->p, a->bytes, b.p, b.bytes)) return true;
  }
  return false;
}

// A matrix of codes inside a buffer.
struct Part {
  size_t codes, scales, end;
  int64_t rows;
};
Part part_at(size_t at, int64_t rows, int64_t depth) {
  Part p;
  p.rows = rows;
  p.codes = at;
  p.scales = round_up(at + (size_t)blocks_of(depth) * rows * deft::kPw8Block, kAlign);
  p.end = round_up(p.scales + (size_t)blocks_of(depth) * deft::pw8_scale_rows(rows), kAlign);
  return p;
}
deft::Pw8Matrix matrix(const void* base, const Part& p) {
  return {(const uint8_t*)base + p.codes, (const uint8_t*)base + p.scales, p.rows};
}

int desc_status(const deft_pw8_desc* d) {
  if (!d) return DEFT_ERR_NULLPTR;
  if (d->dtype != DEFT_F32 && d->dtype != DEFT_BF16) return DEFT_ERR_DTYPE;
  if (d->n < 0 || d->s < 0 || d->c_in < 1 || d->c_out < 1 ||
      (d->layout != DEFT_CHANNELS_FIRST && d->layout != DEFT_CHANNELS_LAST) || (d->training != 0 && d->training != 1))
    return DEFT_ERR_BAD_DESC;
  const int64_t rows = (int64_t)d->n * d->s, most = std::max(d->c_in, d->c_out);
  if (rows > kMaxRows || most > kMaxChannels) return DEFT_ERR_UNSUPPORTED;
  // quantising launches one workgroup for 128 x 128 values, the products one for 64
  // rows by 128 outputs or more
  if (blocks_of(rows) * blocks_of(most) > kMaxBlocks || ceil_div(rows, 64) * blocks_of(most) > kMaxBlocks ||
      ceil_div(d->c_in, 64) * blocks_of(d->c_out) > kMaxBlocks)
    return DEFT_ERR_UNSUPPORTED;
  return DEFT_OK;
}

// ---- products ----

struct Product {
  int bm, bn, tiles_m, tiles_n, splits, per_split, part_cols;
  size_t part_bytes;
};

// Tile and split of a product of m x n outputs over `blocks` of the depth.
Product plan_product(int64_t m, int64_t n, int64_t blocks, int cus) {
  Product p;
  auto tiles = [&](int bm, int bn) { return ceil_div(m, bm) * ceil_div(n, bn); };
  // A unit has one workgroup of 256 x 256, whose outputs wait for its products and its
  // products for its first loads: it pays from a depth of 1024 on (a training step of
  // 32768 rows, 512 channels to 512 takes 124 us with them and 111 with 128 x 128).
  if (tiles(256, 256) >= cus && blocks >= 8) { p.bm = 256; p.bn = 256; }
  else if (m > 64) { p.bm = 128; p.bn = 128; }
  else { p.bm = 64; p.bn = 128; }
  p.tiles_m = (int)ceil_div(m, p.bm);
  p.tiles_n = (int)ceil_div(n, p.bn);
  // the depth is split where the tiles leave compute units idle, into no fewer than
  // 4 blocks; twice as many splits, two workgroups a unit, write twice the partial
  // sums (dw of 50176 rows, 1024 to 256: a step of 177 us takes 183)
  const int64_t t = tiles(p.bm, p.bn);
  int64_t splits = std::min<int64_t>(t < cus ? cus / t : 1, blocks / 4);
  splits = std::max<int64_t>(1, splits);
  p.per_split = (int)ceil_div(blocks, splits);
  p.splits = (int)ceil_div(blocks, p.per_split);
  p.part_cols = (int)std::min<int64_t>(round_up((size_t)n, 8), 0x7ffffff8);
  p.part_bytes = p.splits > 1 ? round_up((size_t)p.splits * m * p.part_cols * 4, kAlign) : 0;
  return p;
}

struct Sides {
  int64_t m, n, depth;
};
// Rows, columns and depth of each product as it is launched: channels first
// the columns are positions.
Sides forward_sides(const deft_pw8_desc& d, int64_t rows) {
  return d.layout == DEFT_CHANNELS_LAST ? Sides{rows, d.c_out, d.c_in} : Sides{d.c_out, rows, d.c_in};
}
Sides dx_sides(const deft_pw8_desc& d, int64_t rows) {
  return d.layout == DEFT_CHANNELS_LAST ? Sides{rows, d.c_in, d.c_out} : Sides{d.c_in, rows, d.c_out};
}
Sides dw_sides(const deft_pw8_desc& d, int64_t rows) { return {d.c_out, d.c_in, rows}; }

hipError_t product(const Sides& s, const deft::Pw8Matrix& a, const deft::Pw8Matrix& b, void* out, const void* bias,
                   int64_t positions, int dtype, float* part, hipStream_t st) {
  const Product p = plan_product(s.m, s.n, blocks_of(s.depth), deft::compute_units());
  deft::Pw8GemmArgs g;
  std::memset(&g, 0, sizeof(g));
  g.a = a;
  g.b = b;
  g.out.p = out;
  g.out.bias = bias;
  g.out.rows = s.m;
  g.out.cols = s.n;
  g.out.positions = positions;
  g.part = p.splits > 1 ? part : nullptr;
  g.part_cols = p.part_cols;
  g.blocks = (int)blocks_of(s.depth);
  g.splits = p.splits;
  g.per_split = p.per_split;
  g.tiles_m = p.tiles_m;
  g.tiles_n = p.tiles_n;
  return deft::launch_pw8_gemm(g, p.bm, p.bn, dtype, st);
}
size_t part_bytes(const Sides& s, int cus) { return plan_product(s.m, s.n, blocks_of(s.depth), cus).part_bytes; }

// ---- buffers ----

struct Packed {
  Part rows, turned;  // [c_out] over c_in for y, [c_in] over c_out for dx
  size_t end;
};
Packed packed_of(const deft_pw8_desc& d) {
  Packed p;
  p.rows = part_at(0, d.c_out, d.c_in);
  p.turned = part_at(p.rows.end, d.c_in, d.c_out);
  p.end = d.training ? p.turned.end : p.rows.end;
  return p;
}
bool few_rows(const deft_pw8_desc& d) { return !d.training && (int64_t)d.n * d.s <= deft::kPw8Few; }

// Workspace: the codes of x forward; of dy, in both forms, and its tiles' sums
// backward; behind them a product's partial sums.
struct Space {
  Part a, b;
  size_t sums, part, end;
};
Space forward_space(const deft_pw8_desc& d, int64_t rows, int cus) {
  Space w;
  w.a = part_at(0, rows, d.c_in);
  w.part = w.a.end;
  w.end = w.part + part_bytes(forward_sides(d, rows), cus);
  return w;
}
Space backward_space(const deft_pw8_desc& d, int64_t rows, int cus) {
  Space w;
  w.a = part_at(0, rows, d.c_out);
  w.b = part_at(w.a.end, d.c_out, rows);
  w.sums = w.b.end;
  w.part = round_up(w.sums + (size_t)blocks_of(rows) * d.c_out * 4, kAlign);
  w.end = w.part + std::max(part_bytes(dx_sides(d, rows), cus), part_bytes(dw_sides(d, rows), cus));
  return w;
}

// Codes of an image tensor of c channels: over the channels (`rows`), over the
// rows (`columns`), or both; sums over the rows of each tile.
hipError_t quantise(const deft_pw8_desc& d, int c, const void* x, char* rows_base, const Part* rows, char* cols_base,
                    const Part* columns, float* sums, hipStream_t st) {
  deft::Pw8QuantiseArgs q;
  std::memset(&q, 0, sizeof(q));
  const int64_t n = (int64_t)d.n * d.s;
  const bool last = d.layout == DEFT_CHANNELS_LAST;
  q.src = x;
  q.lines = last ? n : c;
  q.near = last ? c : n;
  q.pitch = last ? c : d.s;
  q.positions = last ? 0 : d.s;
  q.tiles_near = (uint32_t)blocks_of(q.near);
  uint8_t* code[2] = {rows ? (uint8_t*)rows_base + rows->codes : nullptr,
                      columns ? (uint8_t*)cols_base + columns->codes : nullptr};
  uint8_t* scale[2] = {rows ? (uint8_t*)rows_base + rows->scales : nullptr,
                       columns ? (uint8_t*)cols_base + columns->scales : nullptr};
  q.near_codes = code[last ? 0 : 1];
  q.near_scales = scale[last ? 0 : 1];
  q.far_codes = code[last ? 1 : 0];
  q.far_scales = scale[last ? 1 : 0];
  q.sums = sums;
  return deft::launch_pw8_quantise(q, (uint32_t)(blocks_of(q.lines) * q.tiles_near), d.dtype, false, st);
}

size_t image_bytes(const deft_pw8_desc& d, int c) { return (size_t)d.n * d.s * c * elem_size(d.dtype); }
size_t saved_bytes(const deft_pw8_desc& d) { return d.training ? part_at(0, d.c_in, (int64_t)d.n * d.s).end : 0; }

}  // namespace

extern "C" {

int deft_pw8_desc_validate(const deft_pw8_desc* d) { return desc_status(d); }

size_t deft_pw8_packed_bytes(const deft_pw8_desc* d) { return desc_status(d) == DEFT_OK ? packed_of(*d).end : 0; }

size_t deft_pw8_saved_bytes(const deft_pw8_desc* d) {
  return desc_status(d) == DEFT_OK ? saved_bytes(*d) : 0;
}

size_t deft_pw8_workspace_bytes(const deft_pw8_desc* d) {
  if (desc_status(d) != DEFT_OK || few_rows(*d)) return 0;
  const int64_t rows = (int64_t)d->n * d->s;
  const int cus = deft::compute_units();
  if (rows == 0) return 0;
  const size_t fwd = forward_space(*d, rows, cus).end;
  return d->training ? std::max(fwd, backward_space(*d, rows, cus).end) : fwd;
}

int deft_pw8_pack(const deft_pw8_desc* d, const void* w, void* packed, void* stream) {
  const int e = desc_status(d);
  if (e != DEFT_OK) return e;
  if (!w || !packed) return DEFT_ERR_NULLPTR;
  if (!aligned16(w) || !aligned16(packed)) return DEFT_ERR_ALIGN;
  const Packed p = packed_of(*d);
  if (overlap(w, (size_t)d->c_out * d->c_in * elem_size(d->dtype), packed, p.end)) return DEFT_ERR_BAD_DESC;
  deft::Pw8QuantiseArgs q;
  std::memset(&q, 0, sizeof(q));
  uint8_t* base = (uint8_t*)packed;
  q.src = w;
  q.lines = d->c_out;
  q.near = q.pitch = d->c_in;
  q.tiles_near = (uint32_t)blocks_of(q.near);
  q.near_codes = base + p.rows.codes;
  q.near_scales = base + p.rows.scales;
  if (d->training) {
    q.far_codes = base + p.turned.codes;
    q.far_scales = base + p.turned.scales;
  }
  return status_of(deft::launch_pw8_quantise(q, (uint32_t)(blocks_of(q.lines) * q.tiles_near), d->dtype, true,
                                             (hipStream_t)stream));
}

int deft_pw8_forward(const deft_pw8_desc* d, const void* x, const void* packed, const void* bias, void* y, void* saved,
                     void* workspace, size_t ws_bytes, void* stream) {
  const int e = desc_status(d);
  if (e != DEFT_OK) return e;
  const int64_t rows = (int64_t)d->n * d->s;
  if (rows == 0) return DEFT_OK;
  if (!x || !packed || !y || (d->training && !saved)) return DEFT_ERR_NULLPTR;
  if (!aligned16(x) || !aligned16(packed) || !aligned16(bias) || !aligned16(y) || !aligned16(saved)) return DEFT_ERR_ALIGN;
  const Packed p = packed_of(*d);
  const Span out{y, image_bytes(*d, d->c_out)}, kept{d->training ? saved : nullptr, saved_bytes(*d)}, in{x, image_bytes(*d, d->c_in)};
  const Span codes{packed, p.end}, biases{bias, (size_t)d->c_out * elem_size(d->dtype)};
  if (overlap({out, kept}, {in, codes, biases})) return DEFT_ERR_BAD_DESC;
  const hipStream_t st = (hipStream_t)stream;
  const int64_t positions = d->layout == DEFT_CHANNELS_FIRST ? d->s : 0;
  const int cus = deft::compute_units();
  if (few_rows(*d)) {
    deft::Pw8FewArgs f;
    std::memset(&f, 0, sizeof(f));
    f.x = x;
    f.w = matrix(packed, p.rows);
    f.bias = bias;
    f.y = y;
    f.rows = (int)rows;
    f.c_in = d->c_in;
    f.positions = (int)positions;
    return status_of(deft::launch_pw8_few(f, d->dtype, cus, st));
  }
  const Space w = forward_space(*d, rows, cus);
  if (!workspace || ws_bytes < w.end) return DEFT_ERR_WORKSPACE;
  if (!aligned16(workspace)) return DEFT_ERR_ALIGN;
  if (overlap({{workspace, w.end}}, {out, kept, in, codes, biases})) return DEFT_ERR_BAD_DESC;
  char* ws = (char*)workspace;
  const Part keep = part_at(0, d->c_in, rows);
  hipError_t err = quantise(*d, d->c_in, x, ws, &w.a, (char*)saved, d->training ? &keep : nullptr, nullptr, st);
  if (err != hipSuccess) return status_of(err);
  const deft::Pw8Matrix mx = matrix(ws, w.a), mw = matrix(packed, p.rows);
  const bool last = d->layout == DEFT_CHANNELS_LAST;
  return status_of(product(forward_sides(*d, rows), last ? mx : mw, last ? mw : mx, y, bias, positions, d->dtype,
                           (float*)(ws + w.part), st));
}

int deft_pw8_backward(const deft_pw8_desc* d, const void* saved, const void* packed, const void* dy, void* dx, void* dw,
                      void* db, void* workspace, size_t ws_bytes, void* stream) {
  const int e = desc_status(d);
  if (e != DEFT_OK) return e;
  if (!d->training) return DEFT_ERR_BAD_DESC;
  if (!aligned16(dx) || !aligned16(dw) || !aligned16(db)) return DEFT_ERR_ALIGN;
  const int64_t rows = (int64_t)d->n * d->s;
  const hipStream_t st = (hipStream_t)stream;
  if (rows == 0) {
    hipError_t err = hipSuccess;
    if (db) err = deft::launch_pw8_bias(nullptr, 0, d->c_out, db, d->dtype, st);
    if (err == hipSuccess && dw) err = deft::launch_pw8_zero(dw, (size_t)d->c_out * d->c_in * elem_size(d->dtype), st);
    return status_of(err);
  }
  if ((dw && !saved) || (dx && !packed) || ((dx || dw || db) && !dy)) return DEFT_ERR_NULLPTR;
  if (!aligned16(saved) || !aligned16(packed) || !aligned16(dy)) return DEFT_ERR_ALIGN;
  const Span in{dy, image_bytes(*d, d->c_out)}, of_x{dx, image_bytes(*d, d->c_in)};
  if (overlap({of_x}, {in})) return DEFT_ERR_BAD_DESC;
  const int cus = deft::compute_units();
  const Space w = backward_space(*d, rows, cus);
  if (!workspace || ws_bytes < w.end) return DEFT_ERR_WORKSPACE;
  if (!aligned16(workspace)) return DEFT_ERR_ALIGN;
  const size_t es = elem_size(d->dtype);
  if (overlap({of_x, {dw, d->c_out * es * d->c_in}, {db, d->c_out * es}, {workspace, w.end}},
              {in, {saved, saved_bytes(*d)}, {packed, packed_of(*d).end}}))
    return DEFT_ERR_BAD_DESC;
  if (!dx && !dw && !db) return DEFT_OK;
  char* ws = (char*)workspace;
  float* sums = db ? (float*)(ws + w.sums) : nullptr;
  float* part = (float*)(ws + w.part);
  hipError_t err = quantise(*d, d->c_out, dy, ws, dx ? &w.a : nullptr, ws, dw ? &w.b : nullptr, sums, st);
  if (err == hipSuccess && db) err = deft::launch_pw8_bias(sums, blocks_of(rows), d->c_out, db, d->dtype, st);
  if (err == hipSuccess && dx) {
    const bool last = d->layout == DEFT_CHANNELS_LAST;
    const deft::Pw8Matrix md = matrix(ws, w.a), mw = matrix(packed, packed_of(*d).turned);
    err = product(dx_sides(*d, rows), last ? md : mw, last ? mw : md, dx, nullptr, last ? 0 : d->s, d->dtype, part, st);
  }
  if (err == hipSuccess && dw)
    err = product(dw_sides(*d, rows), matrix(ws, w.b), matrix(saved, part_at(0, d->c_in, rows)), dw, nullptr, 0, d->dtype,
                  part, st);
  return status_of(err);
}

}  // extern "C"
