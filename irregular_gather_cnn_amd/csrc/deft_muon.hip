// Muon: momentum, and an update with its singular values brought near 1 by
// Newton-Schulz steps (gfx950).
//
// For each matrix, with u the momentum's direction,
//   X = u / max(|u|_F, eps);  per step  G = X X^T,  Q = a I + b G + c G^2,  X <- Q X
//   p <- p (1 - lr wd) - lr s X
// with the smaller side first.  All Q are polynomials of the first G, so they
// commute, and up to three steps go without X:
//   P <- Q P,  G <- Q G Q,   and X <- P X at the end.
// For m x n that is one product over n for G and one for X instead of three
// steps' six: 5 steps as 3 + 2 take 6 m^2 n + 14 m^3 operations (symmetric products
// by halves) where they take 15 m^2 n + 5 m^3 one by one.  In a step G's error in
// the directions of small singular values grows by a^2 = 12, so G is made from X
// again after three; then results are as near to the formulas' values as those of
// single steps in fp32 are (5 steps at once: 5 to 20 times farther).
//
// Operands are pairs of fp16, hi + lo with 22 bits together, and a product is
// three of the matrix instructions', hi hi + hi lo + lo hi, in fp32.  One fp16
// alone (or bf16) leaves 2.7e-2 rms of an update of low rank, pairs 2e-5, as fp32
// does, at four times its rate.  fp16's range is kept by powers of two: X and G are
// held times 2^14 (entries under 1.5, as singular values stay under 1.21), Q times
// 2^13 (a = 3.4445), P times 2^10 (a^3 = 41).
#include "deft_device.h"
#include "deft_internal.h"

namespace deft {

namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

constexpr float kScaleX = 16384.f;

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  return (uint64_t)uniform((uint32_t)(v >> 32)) << 32 | uniform((uint32_t)v);
}
// The pause: a load may read a scalar register that a vector instruction wrote
// only five states later, and the compiler does not see the loads in the assembly.
__device__ __forceinline__ rsrc_t uniform_rsrc(uint64_t p, uint32_t bytes) {
  rsrc_t r;
  r.x = (int)uniform((uint32_t)p);
  r.y = (int)uniform((uint32_t)(p >> 32));
  r.z = (int)uniform(bytes);
  r.w = 0x00020000;
  asm volatile("s_nop 4" : "+s"(r));
  return r;
}

// Number of the matrix that a workgroup works on.
__device__ __forceinline__ int item_of(const MuonArgs& a, uint32_t block) {
  const int lane = threadIdx.x & 63;
  const uint32_t first = lane < a.count ? a.first[lane] : 0;
  return uniform(__popcll(__ballot(lane < a.count && first <= block)) - 1);
}

// 8 values as two runs of fp16, hi + lo.
__device__ __forceinline__ void split8(const float* f, uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const f16x2_t a = {(_Float16)f[2 * j], (_Float16)f[2 * j + 1]};
    const f16x2_t b = {(_Float16)(f[2 * j] - (float)a[0]), (_Float16)(f[2 * j + 1] - (float)a[1])};
    h[j] = __builtin_bit_cast(uint32_t, a);
    l[j] = __builtin_bit_cast(uint32_t, b);
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
}
__device__ __forceinline__ void join8(const uint4 hi, const uint4 lo, float* f) {
  const f16x8_t a = __builtin_bit_cast(f16x8_t, hi), b = __builtin_bit_cast(f16x8_t, lo);
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = (float)a[j] + (float)b[j];
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
  const int64_t least = (all + kMuonSums - 1) / kMuonSums, chunk = least <= 4096 ? 4096 : (least + 1023) / 1024 * 1024;
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
  const int64_t least = (all + kMuonSums - 1) / kMuonSums, chunk = least <= 4096 ? 4096 : (least + 1023) / 1024 * 1024;
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
  _Float16* x = (_Float16*)(t.base + muon_buffer(0, t.m, t.n));
  const int64_t plane = mp * np;
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
        uint4 hi, lo;
        split8(f, hi, lo);
        *(uint4*)(x + r * np + c) = hi;
        *(uint4*)(x + plane + r * np + c) = lo;
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
      uint4 hi, lo;
      split8(f, hi, lo);
      *(uint4*)(x + r * np + c) = hi;
      *(uint4*)(x + plane + r * np + c) = lo;
    }
  }
}

// ---- products of pairs ----
//
// One workgroup of 2 x 2 waves makes a BT x BT tile of A B.  Stages of 32 of the
// depth, both planes of both operands, go straight into LDS in a ring of four.  A
// is read by rows; B by rows (its transpose's columns: squares and Gram matrices)
// or, for X, as it lies, its fragments turned by ds_read_b64_tr_b16.  16-byte
// pieces are XOR-swizzled as in the convolution's products.
constexpr int kDepth = 32, kRing = 4;

template <int BT>
struct Tile {
  static constexpr int MI = BT / 64;                  // 32 x 32 blocks of a wave, each way
  static constexpr int kPlane = BT * kDepth * 2;      // bytes of one plane of an operand's stage
  static constexpr int kStage = 4 * kPlane;
  static constexpr int kLoads = kStage / 1024 / 4;    // of a wave, per stage
  static constexpr int kPitch = BT / 2 + 4;           // floats of a row of a wave's block on its way out
  static constexpr int kLds = kRing * kStage;
  static_assert(4 * 32 * kPitch * 4 <= kLds, "results leave through the stages' memory");
};

__device__ __forceinline__ int row_swizzle(int r) { return (r >> 2) & 3; }
template <int BT> __device__ __forceinline__ int depth_swizzle(int k) { return BT == 128 ? 4 * (k & 3) : 4 * ((k >> 1) & 1); }

__device__ __forceinline__ f16x8_t row_fragment(const unsigned char* plane, int rc0, int ks, int lane) {
  const int row = rc0 + (lane & 31), c = 2 * ks + (lane >> 5);
  return __builtin_bit_cast(f16x8_t, *(const uint4*)(plane + row * 64 + ((c ^ row_swizzle(row)) << 4)));
}
template <int BT>
__device__ __forceinline__ f16x8_t depth_fragment(const unsigned char* plane, int rc0, int ks, int lane) {
  const int g = lane >> 4, j = lane & 15;
  const int n = rc0 + 16 * (g & 1) + 4 * (j & 3), c = n >> 3;
  uint2 h[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int k = 16 * ks + 8 * (g >> 1) + 4 * t + (j >> 2);
    const unsigned char* p = plane + k * (2 * BT) + ((c ^ depth_swizzle<BT>(k)) << 4) + (n & 7) * 2;
    h[t] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4bf16((__attribute__((address_space(3))) bf16x4_t*)p));
  }
  return __builtin_bit_cast(f16x8_t, make_uint4(h[0].x, h[0].y, h[1].x, h[1].y));
}

// A product's operand: planes of [rows][ld], `rows` and ld multiples of 32.
struct Operand {
  uint64_t p;
  int64_t rows, ld;
};
__device__ __forceinline__ Operand operand_of(const MuonItem& t, int id) {
  const int64_t mp = muon_pad(t.m);
  return {(uint64_t)t.base + muon_buffer(id, t.m, t.n), mp, id < 2 ? muon_pad(t.n) : mp};
}

// acc[i][j]: rows (i) of A in the lanes, columns (j) of B in the registers: a lane
// has 4 consecutive columns of a row.
template <int BT, bool DEEP>
__device__ __forceinline__ void multiply(unsigned char* smem, const Operand a, const Operand b, int64_t m0, int64_t n0,
                                         int64_t k0, int stages, f32x16_t (&acc)[BT / 64][BT / 64]) {
  using C = Tile<BT>;
  constexpr int MI = C::MI;
  const int lane = threadIdx.x & 63;
  const int wave = uniform(threadIdx.x >> 6), wm = wave >> 1, wn = wave & 1;
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < MI; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  const uint32_t lds0 = lds_addr_of(smem);
  const uint32_t pitch_a = uniform((uint32_t)a.ld * 2), pitch_b = uniform((uint32_t)b.ld * 2);
  // by rows: 16 rows of 64 bytes a load
  const int lrow = lane >> 2, lpiece = ((lane & 3) ^ row_swizzle(lrow)) << 4;
  const int va = lrow * (int)pitch_a + lpiece;
  // as it lies: some rows of the depth a load, columns past the last read as zero
  constexpr int kPieces = BT / 8, kRows = 64 / kPieces;
  const int drow = lane / kPieces;
  const uint32_t left_a = uniform((uint32_t)min<int64_t>(a.rows - m0, BT));
  const uint32_t left_b = uniform((uint32_t)min<int64_t>(DEEP ? b.ld - n0 : b.rows - n0, BT));
  const uint64_t plane_a = uniform64(a.rows * a.ld * 2), plane_b = uniform64(b.rows * b.ld * 2);
  uint64_t pa = uniform64(a.p + (m0 * a.ld + k0) * 2);
  uint64_t pb = uniform64(b.p + (DEEP ? k0 * b.ld + n0 : n0 * b.ld + k0) * 2);
  // bytes from there to the end of the tile's rows
  uint32_t bytes_a = uniform(left_a * pitch_a - (uint32_t)k0 * 2);
  uint32_t bytes_b = uniform(DEEP ? kDepth * pitch_b : left_b * pitch_b - (uint32_t)k0 * 2);

  auto issue = [&](int s) {  // called for one stage after the other
    const uint32_t at = lds0 + (s % kRing) * C::kStage;
#pragma unroll
    for (int plane = 0; plane < 2; ++plane) {
      const rsrc_t ra = uniform_rsrc(pa + plane * plane_a, bytes_a);
#pragma unroll
      for (int i = 0; i < BT / 64; ++i) {
        const int q = wave * (BT / 64) + i;
        load_lds16_so(ra, at + plane * C::kPlane + q * 1024, va, q * 16 * (int)pitch_a);
      }
      // the last rows of X end with its planes: a row's pieces beyond the columns are set out of range
      const rsrc_t rb = uniform_rsrc(pb + plane * plane_b, bytes_b);
#pragma unroll
      for (int i = 0; i < BT / 64; ++i) {
        const int q = wave * (BT / 64) + i;
        if (DEEP) {
          const int k = q * kRows + drow, c = (lane % kPieces) ^ depth_swizzle<BT>(k);
          load_lds16(rb, smem + (s % kRing) * C::kStage + (2 + plane) * C::kPlane + q * 1024,
                     8 * c < (int)left_b ? k * (int)pitch_b + 16 * c : kOOB);
        } else {
          load_lds16_so(rb, at + (2 + plane) * C::kPlane + q * 1024, lrow * (int)pitch_b + lpiece, q * 16 * (int)pitch_b);
        }
      }
    }
    pa += kDepth * 2;
    bytes_a -= kDepth * 2;
    pb += DEEP ? (uint64_t)kDepth * pitch_b : kDepth * 2;
    if (!DEEP) bytes_b -= kDepth * 2;
  };

  struct Frags {
    f16x8_t a[2][MI], b[2][MI];
  };
  auto read = [&](int s, int ks, Frags& f) {
    const unsigned char* st = smem + (s % kRing) * C::kStage;
#pragma unroll
    for (int plane = 0; plane < 2; ++plane)
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        f.a[plane][i] = row_fragment(st + plane * C::kPlane, wm * MI * 32 + i * 32, ks, lane);
        const unsigned char* pb = st + (2 + plane) * C::kPlane;
        f.b[plane][i] = DEEP ? depth_fragment<BT>(pb, wn * MI * 32 + i * 32, ks, lane)
                             : row_fragment(pb, wn * MI * 32 + i * 32, ks, lane);
      }
  };
  auto product = [&](const Frags& f) {
#pragma unroll
    for (int q = 0; q < 3; ++q)  // lo hi, hi lo, hi hi
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < MI; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(f.b[q == 1][j], f.a[q == 0][i], acc[i][j], 0, 0, 0);
  };
  constexpr int kReads = 2 * MI * (DEEP ? 3 : 2);
  auto interleave = [&]() {
#pragma unroll
    for (int u = 0; u < kReads; ++u) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                                              // LDS read
      __builtin_amdgcn_sched_group_barrier(0x008, 3 * MI * MI / kReads > 0 ? 3 * MI * MI / kReads : 1, 0);  // products
    }
  };
  auto wait_stage = [&](int later) {  // how many stages may still be under way
    if (later >= 3) wait_vm<3 * C::kLoads>();
    else if (later == 2) wait_vm<2 * C::kLoads>();
    else if (later == 1) wait_vm<C::kLoads>();
    else wait_vm<0>();
  };

  Frags f0, f1;
#pragma unroll
  for (int s = 0; s < kRing; ++s)
    if (s < stages) issue(s);
  wait_stage(min(kRing, stages) - 1);
  __syncthreads();
  read(0, 0, f0);
  for (int s = 0; s < stages; ++s) {
    read(s, 1, f1);
    product(f0);
    interleave();
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave has read the stage
    if (s + 1 < stages) {
      wait_stage(min(s + kRing, stages) - 2 - s);
      __syncthreads();
      if (s + kRing < stages) issue(s + kRing);
      read(s + 1, 0, f0);
    }
    product(f1);
    interleave();
  }
  __syncthreads();
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
    const _Float16* p = (const _Float16*)add.p + i * add.ld + j;
    float w[8];
    join8(*(const uint4*)p, *(const uint4*)(p + add.rows * add.ld), w);
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
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(BT == 64 ? 2 : 1))) void k_muon_square(const MuonArgs a) {
  using C = Tile<BT>;
  extern __shared__ __align__(16) unsigned char smem[];
  const int k = item_of(a, blockIdx.x);
  const MuonItem& t = a.it[k];
  const MuonArgs::Phase& ph = a.ph[blockIdx.y];
  const uint32_t tiles = (uint32_t)((muon_pad(t.m) + BT - 1) / BT);
  uint32_t at = blockIdx.x - a.first[k], split = 0, ti, tj;
  if (SPLIT) {
    split = uniform(at / (tiles * (tiles + 1) / 2));
    at -= split * (tiles * (tiles + 1) / 2);
  }
  triangle(at, ti, tj);
  const Operand oa = operand_of(t, ph.a), ob = operand_of(t, ph.b), out = operand_of(t, ph.out);
  const int64_t m0 = (int64_t)ti * BT, n0 = (int64_t)tj * BT;
  const int all = (int)(oa.ld / kDepth), per = SPLIT ? (all + t.splits - 1) / t.splits : all;
  const int s0 = split * per, stages = max(0, min(all - s0, per));
  f32x16_t acc[C::MI][C::MI];
  multiply<BT, false>(smem, oa, ob, m0, n0, (int64_t)s0 * kDepth, stages, acc);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t mw = m0 + (wave >> 1) * C::MI * 32, nw = n0 + (wave & 1) * C::MI * 32;
  constexpr int kRuns = C::MI * 4, kAt = 64 / kRuns;  // runs of 8 columns, rows a pass
  const Operand add = operand_of(t, ph.add < 0 ? ph.out : ph.add);
#pragma unroll
  for (int i = 0; i < C::MI; ++i) {
    float* mine = block_out<BT>(smem, acc[i]);
#pragma unroll
    for (int u = 0; u < 32 / kAt; ++u) {
      const int r = u * kAt + lane / kRuns, c = lane % kRuns * 8;
      const int64_t row = mw + i * 32 + r, col = nw + c;
      if (row < out.rows && col < out.rows) {
        float v[8];
        float* src = mine + r * C::kPitch + c;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = src[j];
        if (SPLIT) {
          float* part = (float*)(t.base + muon_parts(t.m, t.n)) + (int64_t)split * out.rows * out.rows + row * out.rows + col;
          *(float4*)part = make_float4(v[0], v[1], v[2], v[3]);
          *(float4*)(part + 4) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
          finish8(ph, t, add, row, col, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) src[j] = v[j];
          uint4 hi, lo;
          split8(v, hi, lo);
          _Float16* dst = (_Float16*)out.p + row * out.ld + col;
          *(uint4*)dst = hi;
          *(uint4*)(dst + out.rows * out.ld) = lo;
        }
      }
    }
    __builtin_amdgcn_s_waitcnt(0xc07f);
    if (!SPLIT && ti != tj) {
      // the other side: runs of 8 rows
#pragma unroll
      for (int u = 0; u < C::MI * 2; ++u) {
        const int c = u * 16 + lane / 4, r = lane % 4 * 8;
        const int64_t row = mw + i * 32 + r, col = nw + c;
        if (row < out.rows && col < out.rows) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = mine[(r + j) * C::kPitch + c];
          uint4 hi, lo;
          split8(v, hi, lo);
          _Float16* dst = (_Float16*)out.p + col * out.ld + row;
          *(uint4*)dst = hi;
          *(uint4*)(dst + out.rows * out.ld) = lo;
        }
      }
      __builtin_amdgcn_s_waitcnt(0xc07f);
    }
  }
}

// Sums of the splits in their order: a 32 x 32 tile of the lower triangle a
// workgroup, stored on both sides.
__global__ __launch_bounds__(256) void k_muon_join(const MuonArgs a) {
  __shared__ float turned[32][33];
  const int k = item_of(a, blockIdx.x), tid = threadIdx.x;
  const MuonItem& t = a.it[k];
  uint32_t ti, tj;
  triangle(blockIdx.x - a.first[k], ti, tj);
  const Operand out = operand_of(t, a.ph[0].out);
  const int r = tid / 8, c = tid % 8 * 4;
  const int64_t row = (int64_t)ti * 32 + r, col = (int64_t)tj * 32 + c;
  const float* p = (const float*)(t.base + muon_parts(t.m, t.n)) + row * out.rows + col;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < t.splits; ++s) {
    const float4 q = *(const float4*)(p + s * out.rows * out.rows);
    v[0] += q.x; v[1] += q.y; v[2] += q.z; v[3] += q.w;
  }
  auto put = [&](int64_t i, int64_t j) {
    _Float16* dst = (_Float16*)out.p + i * out.ld + j;
    const int64_t plane = out.rows * out.ld;
    f16x2_t h[2], l[2];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      h[e / 2][e & 1] = (_Float16)v[e];
      l[e / 2][e & 1] = (_Float16)(v[e] - (float)h[e / 2][e & 1]);
    }
    *(uint2*)dst = make_uint2(__builtin_bit_cast(uint32_t, h[0]), __builtin_bit_cast(uint32_t, h[1]));
    *(uint2*)(dst + plane) = make_uint2(__builtin_bit_cast(uint32_t, l[0]), __builtin_bit_cast(uint32_t, l[1]));
  };
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] *= a.ph[0].f;
    turned[c + e][r] = v[e];
  }
  put(row, col);
  if (ti == tj) return;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = turned[r][c + e];
  put((int64_t)tj * 32 + r, (int64_t)ti * 32 + c);
}

// X <- P X, or, LAST, p <- p (1 - lr wd) - lr s (P X).
template <int BT, bool LAST, typename T, bool MASTER>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(BT == 64 ? 2 : 1))) void k_muon_apply(const MuonArgs a) {
  using C = Tile<BT>;
  extern __shared__ __align__(16) unsigned char smem[];
  const int k = item_of(a, blockIdx.x);
  const MuonItem& t = a.it[k];
  const MuonArgs::Phase& ph = a.ph[0];
  if (LAST && skipped(a.control)) return;
  // tiles of a column of X follow each other: they share it in the L2
  const uint32_t tiles_m = (uint32_t)((muon_pad(t.m) + BT - 1) / BT), at = blockIdx.x - a.first[k];
  const uint32_t tn = uniform(at / tiles_m), tm = at - tn * tiles_m;
  const Operand oa = operand_of(t, ph.a), ob = operand_of(t, ph.b);
  const int64_t m0 = (int64_t)tm * BT, n0 = (int64_t)tn * BT;
  f32x16_t acc[C::MI][C::MI];
  multiply<BT, true>(smem, oa, ob, m0, n0, 0, (int)(oa.ld / kDepth), acc);

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t mw = m0 + (wave >> 1) * C::MI * 32, nw = n0 + (wave & 1) * C::MI * 32;
  constexpr int kRuns = C::MI * 4, kAt = 64 / kRuns;
  const double lr = LAST ? (a.schedule ? a.schedule[0] : a.lr) : 0.0;
  const float keep = (float)(1.0 - lr * t.decay), rate = (float)(lr * t.scale);
  auto update = [&](int64_t at, float o) {
    T* p = (T*)t.p + at;
    const float w = MASTER ? t.master[at] : Elem<T>::to_f32(*p);
    const float v = moved(w, o, keep, rate);
    if (MASTER) t.master[at] = v;
    *p = Elem<T>::from_f32(v);
  };
#pragma unroll
  for (int i = 0; i < C::MI; ++i) {
    const float* mine = block_out<BT>(smem, acc[i]);
    if (!LAST || !t.tall) {
#pragma unroll
      for (int u = 0; u < 32 / kAt; ++u) {
        const int r = u * kAt + lane / kRuns, c = lane % kRuns * 8;
        const int64_t row = mw + i * 32 + r, col = nw + c;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = mine[r * C::kPitch + c + j] * ph.f;
        if (!LAST) {
          if (row < ob.rows && col < ob.ld) {
            uint4 hi, lo;
            split8(v, hi, lo);
            _Float16* dst = (_Float16*)(t.base + muon_buffer(ph.out, t.m, t.n)) + row * ob.ld + col;
            *(uint4*)dst = hi;
            *(uint4*)(dst + ob.rows * ob.ld) = lo;
          }
        } else if (row < t.m) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (col + j < t.n) update(row * t.n + col + j, v[j]);
        }
      }
    } else {
      // p is [n][m]: runs of 8 rows of X
#pragma unroll
      for (int u = 0; u < C::MI * 2; ++u) {
        const int c = u * 16 + lane / 4, r = lane % 4 * 8;
        const int64_t row = mw + i * 32 + r, col = nw + c;
        if (col < t.n) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (row + j < t.m) update(col * t.m + row + j, mine[(r + j) * C::kPitch + c] * ph.f);
        }
      }
    }
    __builtin_amdgcn_s_waitcnt(0xc07f);
  }
}

template <typename K>
hipError_t big_lds(K kernel, int lds) {
  return hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
}

template <int BT>
hipError_t square(const MuonArgs& a, uint32_t blocks, int phases, bool split, hipStream_t st) {
  constexpr int lds = Tile<BT>::kLds;
  const dim3 grid(blocks, phases);
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

}  // namespace

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

hipError_t launch_muon_square(const MuonArgs& a, uint32_t blocks, int tile, int phases, bool split, hipStream_t st) {
  return tile == 64 ? square<64>(a, blocks, phases, split, st) : square<128>(a, blocks, phases, split, st);
}

hipError_t launch_muon_join(const MuonArgs& a, uint32_t blocks, hipStream_t st) {
  DEFT_LAUNCH("muon_join", k_muon_join, dim3(blocks), dim3(256), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_muon_apply(const MuonArgs& a, uint32_t blocks, int tile, bool last, int p_dtype, bool master,
                             hipStream_t st) {
  return tile == 64 ? apply_of<64>(a, blocks, last, p_dtype, master, st)
                    : apply_of<128>(a, blocks, last, p_dtype, master, st);
}

}  // namespace deft
