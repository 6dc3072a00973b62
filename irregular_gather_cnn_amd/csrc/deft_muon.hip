// Muon: momentum, and an update with its singular values brought near 1 by
// Newton-Schulz steps (gfx950).
//
// For each matrix, with u the momentum's direction,
//   X = u / max(|u|_F, eps);  per step  G = X X^T,  Q = a I + b G + c G^2,  X <- Q X
//   p <- p (1 - lr wd) - lr s X
// with the smaller side first.  All Q are polynomials of the first G, so they
// commute, and two steps can go with one product with X:
//   P = Q2 Q1,  where Q2 is made of G2 = Q1 G Q1,  and X <- P X.
// For m x n matrices two single steps take 6 m^2 n + 2 m^3 operations (symmetric
// products by halves), the two together 3 m^2 n + 5 m^3.  G2's error in the directions
// of small singular values is G's times a^2 = 12; results stay within twice the error
// of single steps in fp32 (three together: up to 6 times).
//
// Operands are pairs of fp16, hi + lo with 22 bits together, and a product is
// three of the matrix instructions', hi hi + hi lo + lo hi, in fp32.  One fp16
// alone (or bf16) leaves 2.7e-2 rms of an update of low rank, pairs 2e-5, as fp32
// does, at four times its rate.  fp16's range is kept by powers of two: X and G are
// held times 2^14 (entries under 1.5, as singular values stay under 1.21), Q times
// 2^13 (a = 3.4445), Q2 Q1 times 2^10 (a^2 = 12).
#include <type_traits>

#include "deft_device.h"
#include "deft_internal.h"

namespace deft {

namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

constexpr float kScaleX = 16384.f;

// Number of the matrix that a workgroup works on.
__device__ __forceinline__ int item_of(const MuonArgs& a, uint32_t block) {
  const int lane = threadIdx.x & 63;
  const uint32_t first = lane < a.count ? a.first[lane] : 0;
  return uniform(__popcll(__ballot(lane < a.count && first <= block)) - 1);
}

// Two values as pairs of fp16, hi + lo, packed.  The values are settled first: the
// compiler would round a product to the high part in one instruction, without its
// rounding to fp32, and take the low part from the product that was rounded; near
// ties the two then do not belong together, and the pair is off by 2^-11.
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  asm volatile("" : "+v"(x), "+v"(y));
  const f16x2_t h = {(_Float16)x, (_Float16)y};
  const f16x2_t l = {(_Float16)(x - (float)h[0]), (_Float16)(y - (float)h[1])};
  hi = __builtin_bit_cast(uint32_t, h);
  lo = __builtin_bit_cast(uint32_t, l);
}
__device__ __forceinline__ void split8(const float* f, uint4& hi, uint4& lo) {
  split2(f[0], f[1], hi.x, lo.x);
  split2(f[2], f[3], hi.y, lo.y);
  split2(f[4], f[5], hi.z, lo.z);
  split2(f[6], f[7], hi.w, lo.w);
}
__device__ __forceinline__ void join8(const uint4 hi, const uint4 lo, float* f) {
  const f16x8_t a = __builtin_bit_cast(f16x8_t, hi), b = __builtin_bit_cast(f16x8_t, lo);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = (float)a[j] + (float)b[j];
}

// An operand, of `rows` rows and `cols` columns, multiples of 32.
struct Operand {
  char* p;
  int64_t rows, cols;
  // where the 8 high parts of a run of columns (a multiple of 8) start; the low parts are 32 bytes on
  __device__ __forceinline__ char* run(int64_t row, int64_t col) const {
    return p + ((col >> 4) * rows + row) * 64 + (col & 8) * 2;
  }
  __device__ __forceinline__ void put(int64_t row, int64_t col, const float* v) const {
    uint4 hi, lo;
    split8(v, hi, lo);
    char* q = run(row, col);
    *(uint4*)q = hi;
    *(uint4*)(q + 32) = lo;
  }
};
__device__ __forceinline__ Operand operand_of(const MuonItem& t, int id) {
  const int64_t mp = muon_pad(t.m);
  return {t.base + muon_buffer(id, t.m, t.n), mp, id < 2 ? muon_pad(t.n) : mp};
}

__device__ __forceinline__ float grad_factor(const float* control) { return control ? control[1] : 1.f; }
__device__ __forceinline__ bool skipped(const float* control) { return control && !(control[2] > 0.f); }

// One new value of the momentum and the update's direction there; every operation
// one IEEE fp32 operation in this order.
__device__ __forceinline__ float scaled_by(float g, float coef) {
#pragma clang fp contract(off)
  return g * coef;
}
__device__ __forceinline__ float momentum_of(float m, float g, float mu, float nu) {
#pragma clang fp contract(off)
  return m * mu + g * nu;
}
__device__ __forceinline__ float direction_of(float m, float g, float mu, float nu, int nesterov) {
  return nesterov ? momentum_of(m, g, mu, nu) : m;
}
__device__ __forceinline__ float moved(float p, float x, float keep, float rate) {
#pragma clang fp contract(off)
  return p * keep - x * rate;
}

// m <- mu m + (1 - mu) g, and the sum of squares of u over each workgroup's share
// in fp64.  Bound by memory.
template <typename G>
__global__ __launch_bounds__(256) void k_muon_momentum(const MuonArgs a) {
  __shared__ double part[4];
  const int k = item_of(a, blockIdx.x);
  const MuonItem& t = a.it[k];
  const int64_t all = (int64_t)t.m * t.n;
  const uint32_t share = blockIdx.x - a.first[k];
  const int64_t chunk = muon_chunk(all);
  const int64_t i0 = share * chunk, i1 = min(all, i0 + chunk);
  const bool skip = skipped(a.control);
  const float coef = grad_factor(a.control);
  double sum = 0.0;
  for (int64_t i = i0 + threadIdx.x * 4; i < i1; i += 1024) {
    float g[4], m[4];
    const bool whole = i + 4 <= i1;
    if (whole) {
      const float4 q = *(const float4*)(t.mom + i);
      m[0] = q.x; m[1] = q.y; m[2] = q.z; m[3] = q.w;
      if constexpr (sizeof(G) == 4) {
        const float4 w = *(const float4*)((const float*)t.g + i);
        g[0] = w.x; g[1] = w.y; g[2] = w.z; g[3] = w.w;
      } else {
        const uint2 w = *(const uint2*)((const bf16_t*)t.g + i);
        g[0] = bf16_lo(w.x); g[1] = bf16_hi(w.x); g[2] = bf16_lo(w.y); g[3] = bf16_hi(w.y);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        m[j] = i + j < i1 ? t.mom[i + j] : 0.f;
        g[j] = i + j < i1 ? Elem<G>::to_f32(((const G*)t.g)[i + j]) : 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float f = a.control ? scaled_by(g[j], coef) : g[j];
      m[j] = momentum_of(m[j], f, a.mu, a.nu);
      const double u = direction_of(m[j], f, a.mu, a.nu, a.nesterov);
      sum = __builtin_fma(u, u, sum);
    }
    if (!skip) {
      if (whole) {
        *(float4*)(t.mom + i) = make_float4(m[0], m[1], m[2], m[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i + j < i1) t.mom[i + j] = m[j];
      }
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) ((double*)(t.base + muon_sums(t.m, t.n)))[share] = (part[0] + part[1]) + (part[2] + part[3]);
}

// X = u 2^14 / max(|u|, eps) as pairs, with zeros around it, a 64 x 64 tile of p a
// workgroup; a tall matrix is turned through LDS.
template <typename G>
__global__ __launch_bounds__(256) void k_muon_scale(const MuonArgs a) {
  __shared__ float turned[64][65];
  __shared__ double part[4];
  const int k = item_of(a, blockIdx.x);
  const MuonItem& t = a.it[k];
  const int tid = threadIdx.x;
  const int64_t mp = muon_pad(t.m), np = muon_pad(t.n);
  const int64_t all = (int64_t)t.m * t.n;
  const int64_t chunk = muon_chunk(all);
  const int sums = (int)((all + chunk - 1) / chunk);
  double sum = tid < sums ? ((const double*)(t.base + muon_sums(t.m, t.n)))[tid] : 0.0;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
  if ((tid & 63) == 0) part[tid >> 6] = sum;
  __syncthreads();
  const double norm = sqrt((part[0] + part[1]) + (part[2] + part[3]));
  const float inv = (float)(kScaleX / (norm > a.eps || norm != norm ? norm : a.eps));
  const float coef = grad_factor(a.control);

  // rows and columns of p; its padded columns
  const int rows = t.tall ? t.n : t.m, cols = t.tall ? t.m : t.n;
  const int64_t pc = t.tall ? mp : np;
  const uint32_t tiles_c = (uint32_t)((pc + 63) / 64), tile = blockIdx.x - a.first[k];
  const int64_t r0 = (int64_t)(tile / tiles_c) * 64, c0 = (int64_t)(tile % tiles_c) * 64;
  const Operand x = operand_of(t, 0);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t r = r0 + u * 32 + tid / 8, c = c0 + (tid % 8) * 8;
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.f;
    if (r < rows && c < cols) {
      const int64_t at = r * cols + c;
      const int left = (int)min<int64_t>(8, cols - c);
      float m[8], g[8];
      if (left == 8) {
        typedef float word4 __attribute__((ext_vector_type(4), aligned(4)));
        typedef uint32_t half4 __attribute__((ext_vector_type(4), aligned(2)));
        const word4 p = *(const word4*)(t.mom + at), q = *(const word4*)(t.mom + at + 4);
#pragma unroll
        for (int j = 0; j < 4; ++j) { m[j] = p[j]; m[4 + j] = q[j]; }
        if constexpr (sizeof(G) == 4) {
          const word4 v = *(const word4*)((const float*)t.g + at), w = *(const word4*)((const float*)t.g + at + 4);
#pragma unroll
          for (int j = 0; j < 4; ++j) { g[j] = v[j]; g[4 + j] = w[j]; }
        } else {
          const half4 w = *(const half4*)((const bf16_t*)t.g + at);
          unpack8(make_uint4(w.x, w.y, w.z, w.w), g);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          m[j] = j < left ? t.mom[at + j] : 0.f;
          g[j] = j < left ? Elem<G>::to_f32(((const G*)t.g)[at + j]) : 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        f[j] = direction_of(m[j], a.control ? scaled_by(g[j], coef) : g[j], a.mu, a.nu, a.nesterov) * inv;
    }
    if (!t.tall) {
      if (r < mp && c < np) {
        x.put(r, c, f);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) turned[(tid % 8) * 8 + j][u * 32 + tid / 8] = f[j];
    }
  }
  if (!t.tall) return;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = u * 32 + tid / 8, j0 = (tid % 8) * 8;
    const int64_t r = c0 + i, c = r0 + j0;
    if (r < mp && c < np) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = turned[i][j0 + j];
      x.put(r, c, f);
    }
  }
}

// ---- products of pairs ----
//
// A matrix of pairs over rows and columns is stored by panels of 16 columns:
// [columns / 16][rows][hi 16, lo 16], so that 16 of a product's depth are one piece
// of memory, in whole lines, whether the depth runs along the columns (squares and
// Gram matrices) or the rows (X in P X).
//
// One workgroup of 2 x 2 waves makes a BT x BT tile of A B.  Stages of one or four
// panels go straight into LDS in a ring of four.  A is read by rows; B by rows (its
// transpose's columns), or, DEEP, as it lies, its fragments turned by
// ds_read_b64_tr_b16.  16-byte pieces are XOR-swizzled so that the 16 rows of a
// read's phase lie in 16 places of a 256-byte bank window.  The fragments of the
// next stage are read, and a later one's loads issued, between the matrix
// instructions, of which a stage has three for each 32 x 32 block.
//
// What bounds it is the tile: a wave of 64 x 64 reads as long from LDS as it
// multiplies, one of 128 x 128 (BT 256, 256 accumulators) half as long.  4 matrices of
// 1024 x 9216: P X in 245 us and 314 with the weights (950 TFLOP/s of fp16, where the
// instructions alone reach 1560 on random values), Gram products 135 (1070), squares
// of 1024 by tiles of 128, which fill 144 units, 32 each.
template <int BT>
struct Tile {
  // Panels of a stage, and stages: small tiles take more of the depth between two
  // meetings of the waves.
  static constexpr int kSteps = BT == 64 ? 4 : 1, kRing = BT == 128 ? 5 : 4;
  static constexpr int kAhead = kRing - 1;            // stages that loads run ahead of the products
  static constexpr int MI = BT / 64;                  // 32 x 32 blocks of a wave, each way
  static constexpr int kPanel = BT * 64;              // bytes of an operand's panel
  static constexpr int kStage = 2 * kSteps * kPanel;
  static constexpr int kLoads = 2 * MI * kSteps;      // of a wave, per stage
  static constexpr int kPitch = BT / 2 + 4;           // floats of a row of a wave's block on its way out
  static constexpr int kOut = 4 * 32 * kPitch * 4;
  static constexpr int kLds = kRing * kStage > kOut ? kRing * kStage : kOut;
  static_assert((kAhead - 1) * kLoads <= 60, "waits count so far");
};

__device__ __forceinline__ int row_swizzle(int r) { return (r >> 2) & 3; }

// The sum over 32 * stages_of_two of the depth from k0 on.
// acc[i][j]: rows (i) of A in the lanes, columns (j) of B in the registers: a lane
// has 4 consecutive columns of a row.
template <int BT, bool DEEP>
__device__ __forceinline__ void multiply(unsigned char* smem, const Operand a, const Operand b, int64_t m0, int64_t n0,
                                         int64_t k0, int stages_of_two, f32x16_t (&acc)[BT / 64][BT / 64]) {
  using C = Tile<BT>;
  constexpr int MI = C::MI, kSlots = 3 * MI * MI;
  const int stages = C::kSteps == 4 ? (stages_of_two + 1) / 2 : 2 * stages_of_two;
  // one block a wave: its three products a stage have sums of their own, as each
  // would wait for the one before
  constexpr int kSums = MI == 1 ? 3 : 1;
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6), wm = wave >> 1, wn = wave & 1;
  f32x16_t more[kSums][MI][MI];
#pragma unroll
  for (int q = 0; q < kSums; ++q)
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < MI; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) more[q][i][j][r] = 0.f;

  const uint32_t lds0 = lds_addr_of(smem);
  // 16 rows of 64 bytes a load; a piece's place in its row depends on the row, or,
  // DEEP, high and low parts change places from panel to panel
  const int lrow = lane >> 2, va = lrow * 64 + (((lane & 3) ^ row_swizzle(lrow)) << 4);
  const int vdeep[2] = {lane * 16, (lane * 16) ^ 32};
  const uint32_t panel_a = uniform((uint32_t)a.rows * 64), panel_b = uniform((uint32_t)b.rows * 64);
  uint64_t pa = uniform64((uint64_t)a.p + ((k0 >> 4) * a.rows + m0) * 64);
  uint64_t pb = uniform64((uint64_t)b.p + (DEEP ? (n0 >> 4) * b.rows + k0 : (k0 >> 4) * b.rows + n0) * 64);
  const uint32_t bytes_a = uniform((uint32_t)min<int64_t>(a.rows - m0, BT) * 64u);
  uint32_t bytes_b = uniform(DEEP ? (uint32_t)min<int64_t>((b.cols - n0) >> 4, BT / 16) * panel_b - (uint32_t)k0 * 64u
                                  : (uint32_t)min<int64_t>(b.rows - n0, BT) * 64u);

  // Panels past the last one are read as zeros.
  const int panels = 2 * stages_of_two;
  int issued = 0;
  rsrc_t ra, rb;
  auto load = [&](int s, int u) {  // u-th load of stage s; in order, one stage after the other
    const int step = u / (2 * MI), v = u % (2 * MI);
    const uint32_t at = lds0 + (s % C::kRing) * C::kStage + step * 2 * C::kPanel;
    if (v == 0) {
      const bool in = C::kSteps == 1 || issued < panels;
      ra = uniform_rsrc(pa, in ? bytes_a : 0u);
      rb = uniform_rsrc(pb, in ? bytes_b : 0u);
      ++issued;
      pa += panel_a;
      pb += DEEP ? 1024u : panel_b;
      if (DEEP) bytes_b -= 1024u;
    }
    const int q = wave * MI + v % MI;
    if (v < MI) load_lds16_so(ra, at + q * 1024, va, q * 1024);
    else if (DEEP) load_lds16_so(rb, at + C::kPanel + q * 1024, vdeep[MI > 1 ? v & 1 : wave & 1], q * (int)panel_b);
    else load_lds16_so(rb, at + C::kPanel + q * 1024, va, q * 1024);
  };

  struct Frags {
    f16x8_t a[2][MI], b[2][MI];
  };
  const int frow = lane & 31, fh = lane >> 5, fs = row_swizzle(frow);
  const int dg = lane >> 4, dj = lane & 15;
  // fragment u of step k of stage s in the order of use: high parts of A's first rows,
  // of B, of A's other rows, then the low parts
  auto read = [&](int s, int k, int u, Frags& f) {
    const unsigned char* st = smem + (s % C::kRing) * C::kStage + k * 2 * C::kPanel;
    const int plane = u / (2 * MI), v = u % (2 * MI);
    if (v == 0 || v > MI) {
      const int i = v ? v - MI : 0;
      f.a[plane][i] = __builtin_bit_cast(
          f16x8_t, *(const uint4*)(st + (wm * MI * 32 + i * 32 + frow) * 64 + (((2 * plane + fh) ^ fs) << 4)));
      return;
    }
    const int j = v - 1;
    st += C::kPanel;
    if (!DEEP) {
      f.b[plane][j] = __builtin_bit_cast(
          f16x8_t, *(const uint4*)(st + (wn * MI * 32 + j * 32 + frow) * 64 + (((2 * plane + fh) ^ fs) << 4)));
      return;
    }
    const int p = (wn * MI + j) * 2 + (dg & 1);
    uint2 h[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const unsigned char* q =
          st + p * 1024 + (8 * (dg >> 1) + 4 * t + (dj >> 2)) * 64 + ((plane ^ (dg & 1)) << 5) + (dj & 3) * 8;
      h[t] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((__attribute__((address_space(3))) bf16x4_t*)q));
    }
    f.b[plane][j] = __builtin_bit_cast(f16x8_t, make_uint4(h[0].x, h[0].y, h[1].x, h[1].y));
  };

  // Step k (of a period: a stage, or two stages of one step) of stage s: the products
  // of a panel, from registers.  Under them the next panel's fragments are read; after
  // a stage's last one, from the next stage, once it has landed in all waves' LDS.
  // Loads go over the stage before this one, which every wave has used up: where a
  // stage has several steps the meeting at its end says so, as each wave has waited
  // for its reads by then; where it has one, the meeting in this step does.
  // FULL: there are such stages; else that is looked at.
  constexpr int kSteps = C::kSteps, kPeriod = kSteps == 1 ? 2 : kSteps;
  constexpr int kAfter = kSlots > 4 ? 1 : 0, kFrags = 4 * MI;
  Frags f[2];
  auto step = [&](int s, auto k_, auto full_) {
    constexpr int k = decltype(k_)::value;
    constexpr bool FULL = decltype(full_)::value, END = (k + 1) % kSteps == 0;
    const Frags& now = f[k & 1];
    Frags& next = f[(k + 1) & 1];
    const bool go = !END || FULL || s + 1 < stages, ahead = FULL || s + C::kAhead < stages;
    // loads of this step of several: all of them before the stage's last one
    constexpr int kRest = kSteps > 1 ? kSteps - 1 : 1;
    constexpr int l0 = C::kLoads * k / kRest, l1 = END ? l0 : C::kLoads * (k + 1) / kRest;
#pragma unroll
    for (int t = 0; t < kSlots; ++t) {
      const int q = t / (MI * MI), i = t / MI % MI, j = t % MI;  // hi hi, lo hi, hi lo
      more[q % kSums][i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(now.b[q == 2][j], now.a[q == 1][i], more[q % kSums][i][j], 0, 0, 0);
      if (go) {
        if (END && t == kAfter) {
          constexpr int kLater = kSteps == 1 ? C::kAhead - 2 : C::kAhead - 1;  // stages that may still be under way
          if (FULL || stages - 2 - s >= kLater) wait_vm<kLater * C::kLoads>();
          else wait_vm_atmost((stages - 2 - s) * C::kLoads);
          if (kSteps > 1) __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this stage is in registers
          __builtin_amdgcn_s_barrier();
          asm volatile("" ::: "memory");
        }
        constexpr int kFrom = END ? kAfter : 0, kTake = kSlots - kFrom;
        if (t >= kFrom) {
          const int r = t - kFrom;
#pragma unroll
          for (int u = r * kFrags / kTake; u < (r + 1) * kFrags / kTake; ++u) {
            read(END ? s + 1 : s, (k + 1) % kSteps, u, next);
            if (kSteps == 1 && ahead && u % 2) load(s + C::kAhead, u / 2);
          }
          if (kSteps > 1 && ahead) {
#pragma unroll
            for (int u = l0 + r * (l1 - l0) / kTake; u < l0 + (r + 1) * (l1 - l0) / kTake; ++u) load(s + C::kAhead, u);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  using Yes = std::integral_constant<bool, true>;
  using No = std::integral_constant<bool, false>;
  auto period = [&](int s, auto full) {
    step(s, std::integral_constant<int, 0>(), full);
    if constexpr (kSteps == 1) {
      if (decltype(full)::value || s + 1 < stages) step(s + 1, std::integral_constant<int, 1>(), full);
    } else {
      step(s, std::integral_constant<int, 1>(), full);
      step(s, std::integral_constant<int, 2>(), full);
      step(s, std::integral_constant<int, 3>(), full);
    }
  };
#pragma unroll
  for (int s = 0; s < C::kAhead; ++s)
    if (s < stages) {
#pragma unroll
      for (int u = 0; u < C::kLoads; ++u) load(s, u);
    }
  wait_vm_atmost((min(C::kAhead, stages) - 1) * C::kLoads);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  if (stages > 0) {
#pragma unroll
    for (int u = 0; u < kFrags; ++u) read(0, 0, u, f[0]);
  }
  constexpr int kStride = kPeriod / kSteps;
  int s = 0;
  for (; s + C::kAhead + kStride - 1 < stages; s += kStride) period(s, Yes());
  for (; s < stages; s += kStride) period(s, No());
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < MI; ++j) {
      acc[i][j] = more[0][i][j];
      if constexpr (kSums == 3) acc[i][j] = more[0][i][j] + (more[1][i][j] + more[2][i][j]);
    }
}

// This wave's rows i * 32 .. + 31 of the tile into its LDS, for stores along either side.
template <int BT>
__device__ __forceinline__ float* block_out(unsigned char* smem, const f32x16_t (&acc)[BT / 64]) {
  using C = Tile<BT>;
  const int lane = threadIdx.x & 63;
  float* mine = (float*)smem + (threadIdx.x >> 6) * 32 * C::kPitch;
#pragma unroll
  for (int j = 0; j < C::MI; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *(float4*)(mine + (lane & 31) * C::kPitch + j * 32 + 8 * q + 4 * (lane >> 5)) =
          make_float4(acc[j][4 * q], acc[j][4 * q + 1], acc[j][4 * q + 2], acc[j][4 * q + 3]);
  __builtin_amdgcn_s_waitcnt(0xc07f);
  return mine;
}

// Tile t of the lower triangle by rows.
__device__ __forceinline__ void triangle(uint32_t t, uint32_t& ti, uint32_t& tj) {
  uint32_t i = (uint32_t)((__builtin_amdgcn_sqrtf(8.f * t + 1.f) - 1.f) * 0.5f);
  while ((uint64_t)i * (i + 1) / 2 > t) --i;
  while ((uint64_t)(i + 1) * (i + 2) / 2 <= t) ++i;
  ti = uniform(i);
  tj = uniform(t - i * (i + 1) / 2);
}

// 8 values of the symmetric result: f acc + fd I + fb add.
__device__ __forceinline__ void finish8(const MuonArgs::Phase& ph, const MuonItem& t, const Operand& add, int64_t i, int64_t j,
                                        float* v) {
#pragma unroll
  for (int u = 0; u < 8; ++u) v[u] *= ph.f;
  if (ph.add >= 0) {
    const char* p = add.run(i, j);
    float w[8];
    join8(*(const uint4*)p, *(const uint4*)(p + 32), w);
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = __builtin_fmaf(ph.fb, w[u], v[u]);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i == j + u && i < t.m) v[u] += ph.fd;
  }
}

// A symmetric product: tiles of the lower triangle, stored on both sides of the
// diagonal.  SPLIT: partial sums over n, joined by k_muon_join.
template <int BT, bool SPLIT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(BT == 256 ? 1 : 2))) void k_muon_square(const MuonArgs a) {
  using C = Tile<BT>;
  extern __shared__ __align__(16) unsigned char smem[];
  const int k = item_of(a, blockIdx.x);
  const MuonItem& t = a.it[k];
  const MuonArgs::Phase& ph = a.ph;
  const uint32_t tiles = (uint32_t)((muon_pad(t.m) + BT - 1) / BT);
  uint32_t at = blockIdx.x - a.first[k], split = 0, ti, tj;
  if (SPLIT) {
    split = uniform(at / (tiles * (tiles + 1) / 2));
    at -= split * (tiles * (tiles + 1) / 2);
  }
  triangle(at, ti, tj);
  const Operand oa = operand_of(t, ph.a), ob = operand_of(t, ph.b), out = operand_of(t, ph.out);
  const int64_t m0 = (int64_t)ti * BT, n0 = (int64_t)tj * BT;
  const int all = (int)(oa.cols / 32), per = SPLIT ? (all + t.splits - 1) / t.splits : all;
  const int s0 = split * per, depth = uniform(max(0, min(all - s0, per)));
  f32x16_t acc[C::MI][C::MI];
  multiply<BT, false>(smem, oa, ob, m0, n0, (int64_t)s0 * 32, depth, acc);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t mw = m0 + (wave >> 1) * C::MI * 32, nw = n0 + (wave & 1) * C::MI * 32;
  const Operand add = operand_of(t, ph.add < 0 ? ph.out : ph.add);
#pragma unroll
  for (int i = 0; i < C::MI; ++i) {
    float* mine = block_out<BT>(smem, acc[i]);
    if (SPLIT) {
      constexpr int kRuns = C::MI * 4, kAt = 64 / kRuns;  // runs of 8 columns, rows a pass
      float* part = (float*)(t.base + muon_parts(t.m, t.n)) + (int64_t)split * out.rows * out.rows;
#pragma unroll
      for (int u = 0; u < 32 / kAt; ++u) {
        const int r = u * kAt + lane / kRuns, c = lane % kRuns * 8;
        const int64_t row = mw + i * 32 + r, col = nw + c;
        if (row < out.rows && col < out.rows) {
          const float* src = mine + r * C::kPitch + c;
          *(float4*)(part + row * out.rows + col) = *(const float4*)src;
          *(float4*)(part + row * out.rows + col + 4) = *(const float4*)(src + 4);
        }
      }
    } else {
      const int64_t row = mw + i * 32 + (lane & 31);
#pragma unroll
      for (int u = 0; u < C::MI * 2; ++u) {
        const int c = u * 16 + (lane >> 5) * 8;
        const int64_t col = nw + c;
        if (row < out.rows && col < out.rows) {
          float v[8];
          float* src = mine + (lane & 31) * C::kPitch + c;
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = src[j];
          finish8(ph, t, add, row, col, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) src[j] = v[j];
          out.put(row, col, v);
        }
      }
    }
    __builtin_amdgcn_s_waitcnt(0xc07f);
    if (!SPLIT && ti != tj) {
      // the other side: runs of 8 rows
#pragma unroll
      for (int u = 0; u < C::MI * 2; ++u) {
        const int c = u / 2 * 32 + (lane & 31), r = (u % 2) * 16 + (lane >> 5) * 8;
        const int64_t row = mw + i * 32 + r, col = nw + c;
        if (row < out.rows && col < out.rows) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = mine[(r + j) * C::kPitch + c];
          out.put(col, row, v);
        }
      }
      __builtin_amdgcn_s_waitcnt(0xc07f);
    }
  }
}

// Sums of the splits in their order: a 32 x 32 tile of the lower triangle a
// workgroup, stored on both sides.
__global__ __launch_bounds__(128) void k_muon_join(const MuonArgs a) {
  __shared__ float turned[32][33];
  const int k = item_of(a, blockIdx.x), tid = threadIdx.x;
  const MuonItem& t = a.it[k];
  uint32_t ti, tj;
  triangle(blockIdx.x - a.first[k], ti, tj);
  const Operand out = operand_of(t, a.ph.out);
  const int r = tid / 4, c = tid % 4 * 8;
  const int64_t row = (int64_t)ti * 32 + r, col = (int64_t)tj * 32 + c;
  const float* p = (const float*)(t.base + muon_parts(t.m, t.n)) + row * out.rows + col;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll 4
  for (int s = 0; s < t.splits; ++s) {
    const float4 lo = *(const float4*)(p + s * out.rows * out.rows), hi = *(const float4*)(p + s * out.rows * out.rows + 4);
    v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
    v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    v[e] *= a.ph.f;
    turned[c + e][r] = v[e];
  }
  out.put(row, col, v);
  if (ti == tj) return;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = turned[r][c + e];
  out.put((int64_t)tj * 32 + r, (int64_t)ti * 32 + c, v);
}

// 8 weights in sequence from any element address.
__device__ __forceinline__ void load_run(const bf16_t* p, float* f) {
  typedef uint32_t word4 __attribute__((ext_vector_type(4), aligned(2)));
  const word4 w = *(const word4*)p;
  unpack8(make_uint4(w.x, w.y, w.z, w.w), f);
}
__device__ __forceinline__ void load_run(const float* p, float* f) {
  typedef float word4 __attribute__((ext_vector_type(4), aligned(4)));
  const word4 a = *(const word4*)p, b = *(const word4*)(p + 4);
#pragma unroll
  for (int j = 0; j < 4; ++j) { f[j] = a[j]; f[4 + j] = b[j]; }
}
// X <- P X, or, LAST, p <- p (1 - lr wd) - lr s (P X).
template <int BT, bool LAST, typename T, bool MASTER>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(BT == 256 ? 1 : 2))) void k_muon_apply(const MuonArgs a) {
  using C = Tile<BT>;
  extern __shared__ __align__(16) unsigned char smem[];
  const int k = item_of(a, blockIdx.x);
  const MuonItem& t = a.it[k];
  const MuonArgs::Phase& ph = a.ph;
  if (LAST && skipped(a.control)) return;
  // tiles of a column of X follow each other: they share it in the L2
  const uint32_t tiles_m = (uint32_t)((muon_pad(t.m) + BT - 1) / BT), at = blockIdx.x - a.first[k];
  const uint32_t tn = uniform(at / tiles_m), tm = at - tn * tiles_m;
  const Operand oa = operand_of(t, ph.a), ob = operand_of(t, ph.b);
  const int64_t m0 = (int64_t)tm * BT, n0 = (int64_t)tn * BT;
  f32x16_t acc[C::MI][C::MI];
  multiply<BT, true>(smem, oa, ob, m0, n0, 0, (int)(oa.cols / 32), acc);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t mw = m0 + (wave >> 1) * C::MI * 32, nw = n0 + (wave & 1) * C::MI * 32;
  const double lr = LAST ? (a.schedule ? a.schedule[0] : a.lr) : 0.0;
  const float keep = (float)(1.0 - lr * t.decay), rate = (float)(lr * t.scale);
  // o: X of `left` weights from `at` on
  auto update = [&](int64_t at, int64_t left, const float* o) {
    T* p = (T*)t.p + at;
    float w[8];
    if (left >= 8) {
      if constexpr (MASTER) load_run(t.master + at, w);
      else load_run(p, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = moved(w[j], o[j], keep, rate);
      if constexpr (MASTER) store_run(t.master + at, w);
      store_run(p, w);
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) {
        const float v = moved(MASTER ? t.master[at + j] : Elem<T>::to_f32(p[j]), o[j], keep, rate);
        if (MASTER) t.master[at + j] = v;
        p[j] = Elem<T>::from_f32(v);
      }
  };
#pragma unroll
  for (int i = 0; i < C::MI; ++i) {
    const float* mine = block_out<BT>(smem, acc[i]);
    float v[8];
    if (!LAST) {
      const Operand out = operand_of(t, ph.out);
      const int64_t row = mw + i * 32 + (lane & 31);
#pragma unroll
      for (int u = 0; u < C::MI * 2; ++u) {
        const int c = u * 16 + (lane >> 5) * 8;
        if (row < out.rows && nw + c < out.cols) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = mine[(lane & 31) * C::kPitch + c + j] * ph.f;
          out.put(row, nw + c, v);
        }
      }
    } else if (!t.tall) {
      constexpr int kRuns = C::MI * 4, kAt = 64 / kRuns;  // runs of 8 columns, rows a pass
#pragma unroll 4
      for (int u = 0; u < 32 / kAt; ++u) {
        const int r = u * kAt + lane / kRuns, c = lane % kRuns * 8;
        const int64_t row = mw + i * 32 + r, col = nw + c;
        if (row < t.m && col < t.n) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = mine[r * C::kPitch + c + j] * ph.f;
          update(row * t.n + col, t.n - col, v);
        }
      }
    } else {
      // p is [n][m]: runs of 8 rows of X
#pragma unroll 4
      for (int u = 0; u < C::MI * 2; ++u) {
        const int c = u * 16 + lane / 4, r = lane % 4 * 8;
        const int64_t row = mw + i * 32 + r, col = nw + c;
        if (row < t.m && col < t.n) {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = mine[(r + j) * C::kPitch + c] * ph.f;
          update(col * t.m + row, t.m - row, v);
        }
      }
    }
    __builtin_amdgcn_s_waitcnt(0xc07f);
  }
}

// ---- small matrices ----
//
// A workgroup does all of a matrix that fits its LDS: momentum, norm, the steps one
// by one, the weights.  X lies in LDS in its panels, so a step is a product over n
// for G (32 rows: the waves share n and add up; 64: a wave for each 32 x 32 block), a
// small one for Q and one that replaces X's columns, each by one wave.  22 launches
// of 4 us become one: [16][144] and [18][144] take 23 us where they took 90, 2.6 for
// each step and the rest for the launch, the loads and the stores.
constexpr int kSmallThreads = 256;

// A run's place in a matrix of panels in LDS: 16-byte pieces, high 0 and 1, low 2 and 3.
__device__ __forceinline__ unsigned char* small_piece(unsigned char* x, int rows, int row, int col, int piece) {
  return x + (col >> 4) * rows * 64 + row * 64 + ((piece ^ row_swizzle(row)) << 4);
}
// The place of a value before it is split: the same 32 bytes hold a run of 8.
__device__ __forceinline__ float* small_value(unsigned char* x, int rows, int row, int col) {
  return (float*)small_piece(x, rows, row, col, ((col >> 3) & 1) + ((col >> 1) & 2)) + (col & 3);
}
__device__ __forceinline__ f16x8_t small_rows(unsigned char* x, int rows, int row0, int panel, int plane, int lane) {
  return __builtin_bit_cast(f16x8_t, *(const uint4*)small_piece(x, rows, row0 + (lane & 31), panel * 16, 2 * plane + (lane >> 5)));
}
__device__ __forceinline__ f16x8_t small_columns(unsigned char* x, int rows, int row0, int col0, int plane, int lane) {
  const int g = lane >> 4, j = lane & 15;
  uint2 h[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int row = row0 + 8 * (g >> 1) + 4 * t + (j >> 2);
    unsigned char* q = small_piece(x, rows, row, col0 + 16 * (g & 1), 2 * plane + ((j >> 1) & 1)) + (j & 1) * 8;
    h[t] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((__attribute__((address_space(3))) bf16x4_t*)q));
  }
  return __builtin_bit_cast(f16x8_t, make_uint4(h[0].x, h[0].y, h[1].x, h[1].y));
}
// 4 values at columns col .. col + 3, a multiple of 4, as pairs.
__device__ __forceinline__ void small_put4(unsigned char* x, int rows, int row, int col, const float* v) {
  uint32_t h[2], l[2];
  split2(v[0], v[1], h[0], l[0]);
  split2(v[2], v[3], h[1], l[1]);
  const int c = (col >> 3) & 1, o = (col & 4) * 2;
  *(uint2*)(small_piece(x, rows, row, col, c) + o) = make_uint2(h[0], h[1]);
  *(uint2*)(small_piece(x, rows, row, col, c + 2) + o) = make_uint2(l[0], l[1]);
}
__device__ __forceinline__ void small_get4(unsigned char* x, int rows, int row, int col, float* v) {
  const int c = (col >> 3) & 1, o = (col & 4) * 2;
  const uint2 h = *(const uint2*)(small_piece(x, rows, row, col, c) + o);
  const uint2 l = *(const uint2*)(small_piece(x, rows, row, col, c + 2) + o);
  const f16x2_t h0 = __builtin_bit_cast(f16x2_t, h.x), h1 = __builtin_bit_cast(f16x2_t, h.y);
  const f16x2_t l0 = __builtin_bit_cast(f16x2_t, l.x), l1 = __builtin_bit_cast(f16x2_t, l.y);
  v[0] = (float)h0[0] + (float)l0[0]; v[1] = (float)h0[1] + (float)l0[1];
  v[2] = (float)h1[0] + (float)l1[0]; v[3] = (float)h1[1] + (float)l1[1];
}
struct Sums3 {
  f32x16_t s[3];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
      for (int r = 0; r < 16; ++r) s[q][r] = 0.f;
  }
  // rows of a in the lanes, b's in the registers
  __device__ __forceinline__ void add(const f16x8_t ah, const f16x8_t al, const f16x8_t bh, const f16x8_t bl) {
    s[0] = __builtin_amdgcn_mfma_f32_32x32x16_f16(bh, ah, s[0], 0, 0, 0);
    s[1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(bh, al, s[1], 0, 0, 0);
    s[2] = __builtin_amdgcn_mfma_f32_32x32x16_f16(bl, ah, s[2], 0, 0, 0);
  }
  __device__ __forceinline__ f32x16_t all() const { return s[0] + (s[1] + s[2]); }
};

// X has 32 * blocks rows.
template <typename T, typename G, bool MASTER, int blocks>
__device__ __forceinline__ void small_step(unsigned char* smem, double* part, const MuonArgs& a, const MuonSmall& c) {
  const MuonItem& t = a.it[blockIdx.x];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int mp = 32 * blocks;
  const int m = t.m, n = t.n, np = (int)muon_pad(n);
  unsigned char* x = smem;
  unsigned char* g = x + 4 * mp * np;
  unsigned char* q = g + 4 * mp * mp;
  float* sums = (float*)(q + 4 * mp * mp);  // 32 rows: the waves' shares of G
  const bool skip = skipped(a.control);
  if (skip) return;
  const float coef = grad_factor(a.control);

  // momentum and direction
  for (int i = tid * 16; i < 4 * mp * np; i += kSmallThreads * 16) *(uint4*)(x + i) = make_uint4(0, 0, 0, 0);
  __syncthreads();
  double sum = 0.0;
  const int cols = t.tall ? m : n;  // of p
  const FastDiv by_cols = make_fastdiv((uint32_t)cols);
  for (int i0 = tid; i0 < m * n; i0 += 8 * kSmallThreads) {
    float gr[8], mo[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j * kSmallThreads;
      gr[j] = i < m * n ? Elem<G>::to_f32(((const G*)t.g)[i]) : 0.f;
      mo[j] = i < m * n ? t.mom[i] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j * kSmallThreads;
      if (i < m * n) {
        const float f = a.control ? scaled_by(gr[j], coef) : gr[j];
        const float v = momentum_of(mo[j], f, a.mu, a.nu);
        t.mom[i] = v;
        const float u = direction_of(v, f, a.mu, a.nu, a.nesterov);
        sum = __builtin_fma((double)u, (double)u, sum);
        const int r = fdiv(i, by_cols), k = i - r * cols;
        *small_value(x, mp, t.tall ? k : r, t.tall ? r : k) = u;
      }
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
  if (lane == 0) part[wave] = sum;
  __syncthreads();
  const double norm = sqrt((part[0] + part[1]) + (part[2] + part[3]));
  const float inv = (float)(kScaleX / (norm > a.eps || norm != norm ? norm : a.eps));
  for (int i = tid; i < mp * np / 8; i += kSmallThreads) {
    const int row = i % mp, col = i / mp * 8, piece = (col >> 3) & 1;
    uint4* ph = (uint4*)small_piece(x, mp, row, col, piece);
    uint4* pl = (uint4*)small_piece(x, mp, row, col, piece + 2);
    const float4 lo = __builtin_bit_cast(float4, *ph), hi = __builtin_bit_cast(float4, *pl);
    const float v[8] = {lo.x * inv, lo.y * inv, lo.z * inv, lo.w * inv, hi.x * inv, hi.y * inv, hi.z * inv, hi.w * inv};
    split8(v, *ph, *pl);
  }
  __syncthreads();

  const int bi = wave / blocks % blocks * 32, bj = wave % blocks * 32;  // this wave's block of a square
  const int row = lane & 31, fh = lane >> 5;
  const double lr = a.schedule ? a.schedule[0] : a.lr;
  const float keep = (float)(1.0 - lr * t.decay), rate = (float)(lr * t.scale);
  Sums3 acc;
  for (int step = 0; step < c.steps; ++step) {
    // G = X X^T
    acc.clear();
    if (blocks == 1) {
      for (int k = wave; k < np / 16; k += 4) {
        const f16x8_t h = small_rows(x, mp, 0, k, 0, lane), l = small_rows(x, mp, 0, k, 1, lane);
        acc.add(h, l, h, l);
      }
      const f32x16_t s = acc.all();
#pragma unroll
      for (int r = 0; r < 16; ++r) sums[(wave * 32 + row) * 33 + 8 * (r >> 2) + 4 * fh + (r & 3)] = s[r];
      __syncthreads();
      const int gi = tid >> 3, gj = (tid & 7) * 4;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float* p = sums + gi * 33 + gj + e;
        v[e] = ((p[0] + p[32 * 33]) + (p[64 * 33] + p[96 * 33])) * c.g;
      }
      small_put4(g, mp, gi, gj, v);
    } else {
      for (int k = 0; k < np / 16; ++k)
        acc.add(small_rows(x, mp, bi, k, 0, lane), small_rows(x, mp, bi, k, 1, lane), small_rows(x, mp, bj, k, 0, lane),
                small_rows(x, mp, bj, k, 1, lane));
      const f32x16_t s = acc.all();
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v[4] = {s[4 * e] * c.g, s[4 * e + 1] * c.g, s[4 * e + 2] * c.g, s[4 * e + 3] * c.g};
        small_put4(g, mp, bi + row, bj + 8 * e + 4 * fh, v);
      }
    }
    __syncthreads();
    // Q = a I + b G + c G^2
    if (wave < blocks * blocks) {
      acc.clear();
#pragma unroll
      for (int k = 0; k < mp / 16; ++k)
        acc.add(small_rows(g, mp, bi, k, 0, lane), small_rows(g, mp, bi, k, 1, lane), small_rows(g, mp, bj, k, 0, lane),
                small_rows(g, mp, bj, k, 1, lane));
      const f32x16_t s = acc.all();
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int col = bj + 8 * e + 4 * fh;
        float v[4];
        small_get4(g, mp, bi + row, col, v);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          v[r] = __builtin_fmaf(c.b, v[r], c.c * s[4 * e + r]);
          if (bi + row == col + r && bi + row < m) v[r] += c.a;
        }
        small_put4(q, mp, bi + row, col, v);
      }
    }
    __syncthreads();
    // X <- Q X, or the weights
    const bool last = step + 1 == c.steps;
    for (int tile = wave; tile < np / 32; tile += 4) {
      f32x16_t s[blocks];
#pragma unroll
      for (int b = 0; b < blocks; ++b) {
          acc.clear();
#pragma unroll
          for (int k = 0; k < mp / 16; ++k)
            acc.add(small_rows(q, mp, b * 32, k, 0, lane), small_rows(q, mp, b * 32, k, 1, lane),
                    small_columns(x, mp, k * 16, tile * 32, 0, lane), small_columns(x, mp, k * 16, tile * 32, 1, lane));
          s[b] = acc.all();
        }
#pragma unroll
      for (int b = 0; b < blocks; ++b) {
          const int i = b * 32 + row, j0 = tile * 32 + 4 * fh;
          if (!last) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float v[4] = {s[b][4 * e] * c.x, s[b][4 * e + 1] * c.x, s[b][4 * e + 2] * c.x, s[b][4 * e + 3] * c.x};
              small_put4(x, mp, i, j0 + 8 * e, v);
            }
          } else if (i < m) {
            const int first = t.tall ? j0 * m + i : i * n + j0, pitch = t.tall ? m : 1;
            float w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int j = 8 * (e >> 2) + (e & 3), at = first + j * pitch;
              w[e] = j0 + j < n ? MASTER ? t.master[at] : Elem<T>::to_f32(((const T*)t.p)[at]) : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int j = 8 * (e >> 2) + (e & 3), at = first + j * pitch;
              if (j0 + j < n) {
                const float v = moved(w[e], s[b][e] * c.o, keep, rate);
                if (MASTER) t.master[at] = v;
                ((T*)t.p)[at] = Elem<T>::from_f32(v);
              }
            }
          }
        }
    }
    __syncthreads();
  }
}

template <typename T, typename G, bool MASTER>
__global__ __launch_bounds__(kSmallThreads) void k_muon_small(const MuonArgs a, const MuonSmall c) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ double part[4];
  if (a.it[blockIdx.x].m <= 32) small_step<T, G, MASTER, 1>(smem, part, a, c);
  else small_step<T, G, MASTER, 2>(smem, part, a, c);
}

template <typename K>
hipError_t big_lds(K kernel, int lds) {
  return hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
}

template <int BT>
hipError_t square(const MuonArgs& a, uint32_t blocks, bool split, hipStream_t st) {
  constexpr int lds = Tile<BT>::kLds;
  const dim3 grid(blocks);
  hipError_t e = split ? big_lds(k_muon_square<BT, true>, lds) : big_lds(k_muon_square<BT, false>, lds);
  if (e != hipSuccess) return e;
  if (split) DEFT_LAUNCH("muon_gram", (k_muon_square<BT, true>), grid, dim3(256), lds, st, a);
  else DEFT_LAUNCH("muon_square", (k_muon_square<BT, false>), grid, dim3(256), lds, st, a);
  return hipGetLastError();
}

template <int BT, bool LAST, typename T, bool MASTER>
hipError_t apply(const MuonArgs& a, uint32_t blocks, hipStream_t st) {
  constexpr int lds = Tile<BT>::kLds;
  hipError_t e = big_lds(k_muon_apply<BT, LAST, T, MASTER>, lds);
  if (e != hipSuccess) return e;
  DEFT_LAUNCH("muon_apply", (k_muon_apply<BT, LAST, T, MASTER>), dim3(blocks), dim3(256), lds, st, a);
  return hipGetLastError();
}
template <int BT>
hipError_t apply_of(const MuonArgs& a, uint32_t blocks, bool last, int p_dtype, bool master, hipStream_t st) {
  if (!last) return apply<BT, false, float, false>(a, blocks, st);
  if (p_dtype == DEFT_F32) return apply<BT, true, float, false>(a, blocks, st);
  return master ? apply<BT, true, bf16_t, true>(a, blocks, st) : apply<BT, true, bf16_t, false>(a, blocks, st);
}

template <typename T, typename G, bool MASTER>
hipError_t small(const MuonArgs& a, const MuonSmall& c, hipStream_t st) {
  hipError_t e = big_lds(k_muon_small<T, G, MASTER>, c.lds);
  if (e != hipSuccess) return e;
  DEFT_LAUNCH("muon_small", (k_muon_small<T, G, MASTER>), dim3(a.count), dim3(kSmallThreads), c.lds, st, a, c);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_muon_small(const MuonArgs& a, const MuonSmall& c, int p_dtype, int g_dtype, bool master, hipStream_t st) {
  const bool gb = g_dtype == DEFT_BF16;
  if (p_dtype == DEFT_F32) return gb ? small<float, bf16_t, false>(a, c, st) : small<float, float, false>(a, c, st);
  if (master) return gb ? small<bf16_t, bf16_t, true>(a, c, st) : small<bf16_t, float, true>(a, c, st);
  return gb ? small<bf16_t, bf16_t, false>(a, c, st) : small<bf16_t, float, false>(a, c, st);
}

hipError_t launch_muon_momentum(const MuonArgs& a, uint32_t blocks, int g_dtype, hipStream_t st) {
  if (g_dtype == DEFT_F32) DEFT_LAUNCH("muon_momentum", k_muon_momentum<float>, dim3(blocks), dim3(256), 0, st, a);
  else DEFT_LAUNCH("muon_momentum", k_muon_momentum<bf16_t>, dim3(blocks), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_muon_scale(const MuonArgs& a, uint32_t blocks, int g_dtype, hipStream_t st) {
  if (g_dtype == DEFT_F32) DEFT_LAUNCH("muon_scale", k_muon_scale<float>, dim3(blocks), dim3(256), 0, st, a);
  else DEFT_LAUNCH("muon_scale", k_muon_scale<bf16_t>, dim3(blocks), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_muon_square(const MuonArgs& a, uint32_t blocks, int tile, bool split, hipStream_t st) {
  if (tile == 64) return square<64>(a, blocks, split, st);
  if (tile == 128) return square<128>(a, blocks, split, st);
  return square<256>(a, blocks, split, st);
}

hipError_t launch_muon_join(const MuonArgs& a, uint32_t blocks, hipStream_t st) {
  DEFT_LAUNCH("muon_join", k_muon_join, dim3(blocks), dim3(128), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_muon_apply(const MuonArgs& a, uint32_t blocks, int tile, bool last, int p_dtype, bool master,
                             hipStream_t st) {
  if (tile == 64) return apply_of<64>(a, blocks, last, p_dtype, master, st);
  if (tile == 128) return apply_of<128>(a, blocks, last, p_dtype, master, st);
  return apply_of<256>(a, blocks, last, p_dtype, master, st);
}

}  // namespace deft
