// Products of 8-bit block-scaled matrices (gfx950): the pointwise convolution
// and its gradients.
//
// C[i][j] = sum_k A[i][k] B[j][k] over two matrices of e4m3 codes stored by
// half blocks of 64 of k (deft_pw8.h), each row of a block of 128 with a power of
// two.  v_mfma_scale_f32_32x32x64 multiplies 64 codes of 32 rows by 64 of 32
// others, with their powers of two, into fp32: twice the rate of bf16, and no
// vector operations for the scales.  Products for fp32 results are 16-bit ones
// (deft_pw8.h says why).
#include <algorithm>
#include <type_traits>

#include "deft_device.h"
#include "deft_internal.h"
#include "deft_pw8.h"

namespace deft {

namespace {

constexpr int kHalf = 64;  // bytes of a row in a stage: half of a block

// Bytes straight into LDS, 4 per lane.
__device__ __forceinline__ void load_lds4(const rsrc_t r, uint32_t lds_addr, int voff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds_addr), "v"(voff), "s"(r)
               : "memory");
}

// Where a lane's runs of 8 columns go: column j of row 0, and on from row to row.
// positions: columns run over the positions of all images, rows over channels
// (channels first); else row-major.  A run that passes the last column or an
// image's end goes value by value.
template <typename T>
struct Runs {
  T* p;
  int64_t j, pitch, left, room, rows, positions;
  __device__ __forceinline__ Runs(const Pw8Out& o, int64_t j_) : j(j_), rows(o.rows), positions(o.positions) {
    left = room = o.cols - j;
    pitch = o.cols;
    int64_t at = j;
    if (positions) {
      const int64_t image = (uint32_t)j / (uint32_t)positions, pos = j - image * positions;
      at = image * rows * positions + pos;
      pitch = positions;
      if (positions - pos < room) room = positions - pos;
    }
    p = (T*)o.p + at;
  }
  __device__ __forceinline__ void put(int64_t i, const float* f) const {
    if (room >= 8) {
      store_run(p + i * pitch, f);
      return;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (u < left) {
        int64_t at = i * pitch + u;
        if (positions && u >= room) {  // the next image, or, of fewer than 8 positions, a later one
          const int64_t next = positions >= 8 ? 1 : (uint32_t)(u - (int)room) / (uint32_t)positions + 1;
          at += next * (rows - 1) * positions;
        }
        p[at] = Elem<T>::from_f32(f[u]);
      }
  }
};

// One workgroup of 2 x 2 waves computes BM x BN outputs over a range of blocks.
//
// Stages are half blocks (64 bytes of each row; the first half with the block's
// scale bytes), in a ring of four filled by loads straight into LDS.  The
// fragments of the next stage are read, and a later one's loads issued, one or two
// between two matrix instructions, so one wave a SIMD keeps its matrix unit fed: 8192^3
// in 411 to 470 us from card to card, 2.3 to 2.7 PFLOP/s, where the instructions alone
// reach 3.5 on random values (461 us on a card where it takes 501 with reads and loads
// after the barrier and their order left to the compiler, as products for fp32 have
// them: those take 890, 1.2 PFLOP/s of the 16-bit instructions' 1.56).  What bounds it
// is power: the clock falls to 1.8 GHz, and matrix units are busy 63 % of its cycles.
// 16-byte pieces are XOR-swizzled: the 16 rows of a read's phase lie in 16 places of a
// 256-byte bank window.
template <int BM, int BN>
struct Pw8Tile {
  static constexpr int MI = BM / 64, NI = BN / 64;      // 32 x 32 blocks of a wave
  static constexpr int kLoads = BM / 64 + BN / 64;      // of a wave, per stage, and one for a block's scale bytes
  static constexpr int kScaleBytes = 1024;              // of A, of B, and 512 that nobody reads
  static constexpr int kStage = (BM + BN) * kHalf + kScaleBytes;
  static constexpr int kRing = 4;
  static constexpr int kEpiPitch = NI * 32 * 4 + 16;    // 32 rows of a wave's columns in fp32
  static constexpr int kLds = kRing * kStage > 4 * 32 * kEpiPitch ? kRing * kStage : 4 * 32 * kEpiPitch;
};

template <typename T, int BM, int BN, bool PARTIAL>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(BM * BN > 128 * 256 ? 1 : 2))) void k_pw8_gemm(
    const Pw8GemmArgs g) {
  using C = Pw8Tile<BM, BN>;
  constexpr int MI = C::MI, NI = C::NI;
  extern __shared__ __align__(16) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wm = wave >> 1, wn = wave & 1;

  // tiles in bands of kBand rows of tiles, so that the tiles of an XCD share
  // rows of both matrices in its L2
  constexpr int kBand = 8;
  const int id = xcd_swizzle(blockIdx.x, gridDim.x);
  const int tiles = g.tiles_m * g.tiles_n;
  const int split = uniform(id / tiles), in = id - split * tiles;
  const int band = uniform(in / (kBand * g.tiles_n)), rows = min(kBand, g.tiles_m - band * kBand);
  const int at = in - band * kBand * g.tiles_n;
  const int tn = uniform(at / rows), tm = band * kBand + at - tn * rows;
  const int64_t m0 = (int64_t)tm * BM, n0 = (int64_t)tn * BN;
  const int kb0 = split * g.per_split, kb1 = min(g.blocks, kb0 + g.per_split);
  const int stages = 2 * (kb1 - kb0);

  f32x16_t acc[MI][NI];

  // 16 rows of 64 bytes a load; a piece's place in its row depends on the row
  const int lrow = lane >> 2;
  const int voff = lrow * kHalf + (((lane & 3) ^ ((lrow >> 2) & 3)) << 4);
  const int64_t ra = g.a.rows - m0, rb = g.b.rows - n0;
  const uint32_t bytes_a = uniform((uint32_t)min<int64_t>(ra, BM) * (uint32_t)kHalf);
  const uint32_t bytes_b = uniform((uint32_t)min<int64_t>(rb, BN) * (uint32_t)kHalf);
  const int64_t srows_a = pw8_scale_rows(g.a.rows), srows_b = pw8_scale_rows(g.b.rows);
  const uint32_t scales_a = uniform((uint32_t)min<int64_t>(srows_a - m0, 256));
  const uint32_t scales_b = uniform((uint32_t)min<int64_t>(srows_b - n0, 256));
  const uint32_t lds0 = lds_addr_of(smem);

  const uint64_t step_a = uniform64(g.a.rows * kHalf), step_b = uniform64(g.b.rows * kHalf);
  const uint64_t code_a0 = uniform64((uint64_t)(g.a.codes + (2 * kb0 * g.a.rows + m0) * kHalf));
  const uint64_t code_b0 = uniform64((uint64_t)(g.b.codes + (2 * kb0 * g.b.rows + n0) * kHalf));
  // the scales that this wave loads: even waves A's, odd ones B's
  const uint64_t scale0 = uniform64((uint64_t)(wave & 1 ? g.b.scales + kb0 * srows_b + n0 : g.a.scales + kb0 * srows_a + m0));
  uint64_t code_a, code_b, scale;
  const uint64_t step_s = uniform64(wave & 1 ? srows_b : srows_a);
  const uint32_t bytes_s = wave & 1 ? scales_b : scales_a;

  // The loads of a stage, one at a time and one stage after the other: first, with
  // a block's first stage, the scale bytes; then this wave's share of A's and B's rows.
  rsrc_t pa, pb;
  auto load = [&](int s, int u) {
    const uint32_t base = lds0 + (s & 3) * C::kStage;
    if (u == 0) {
      pa = uniform_rsrc(code_a, bytes_a);
      pb = uniform_rsrc(code_b, bytes_b);
    }
    if (u < MI) {
      const int b = wave * MI + u;
      load_lds16_so(pa, base + b * 1024, voff, b * 1024);
    } else if (u < MI + NI) {
      const int b = wave * NI + u - MI;
      load_lds16_so(pb, base + BM * kHalf + b * 1024, voff, b * 1024);
    }
    if (u == MI + NI - 1) {
      code_a += step_a;
      code_b += step_b;
    }
  };
  auto load_scales = [&](int s) {
    load_lds4(uniform_rsrc(scale, bytes_s), lds0 + (s & 3) * C::kStage + (BM + BN) * kHalf + wave * 256, lane * 4);
    scale += step_s;
  };

  struct Frags {
    pw8_codes_t a[MI], b[NI];
  };
  int sa[2][MI], sb[2][NI];  // scales of a block, and of the next one
  const int frow = lane & 31, fh = lane >> 5;
  const int sw = (frow >> 2) & 3;
  const int c0 = ((2 * fh) ^ sw) << 4, c1 = ((2 * fh + 1) ^ sw) << 4;
  auto fragment = [&](const unsigned char* p) {
    const uint4 lo = *(const uint4*)(p + c0), hi = *(const uint4*)(p + c1);
    pw8_codes_t v;
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
    v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
    return v;
  };
  // One fragment of stage s, in the order of use: A's first, all of B's, the rest of A's.
  constexpr int kFrags = MI + NI;
  auto read = [&](int s, int u, Frags& f) {
    const unsigned char* st = smem + (s & 3) * C::kStage;
    if (u == 0 || u > NI) {
      const int i = u ? u - NI : 0;
      f.a[i] = fragment(st + (wm * MI * 32 + i * 32 + frow) * kHalf);
    } else {
      const int j = u - 1;
      f.b[j] = fragment(st + (BM + wn * NI * 32 + j * 32 + frow) * kHalf);
    }
  };
  auto read_scales = [&](int s, int* na, int* nb) {
    const unsigned char* sc = smem + (s & 3) * C::kStage + (BM + BN) * kHalf;
#pragma unroll
    for (int i = 0; i < MI; ++i) na[i] = sc[wm * MI * 32 + i * 32 + frow];
#pragma unroll
    for (int j = 0; j < NI; ++j) nb[j] = sc[256 + wn * NI * 32 + j * 32 + frow];
  };
  // every wave's loads for the next stage have landed, as each has waited for its own
  auto meet = [&]() {
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // the columns' operand first: a lane then holds 4 consecutive columns of a row
  auto multiply = [&](const Frags& f, int i, int j, const int* xa, const int* xb) {
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f.b[j], f.a[i], acc[i][j], 0, 0, 0, xb[j], 0, xa[i]);
  };
  // fp32, powers that do not fit bf16: one code of every eight at a time (deft_pw8.h)
  auto multiply_apart = [&](const Frags& f, const int* xa, const int* xb) {
#pragma unroll 1
    for (int which = 0; which < 8; ++which)
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        const pw8_codes_t b = pw8_one_of_8(f.b[j], which);
#pragma unroll
        for (int i = 0; i < MI; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, f.a[i], acc[i][j], 0, 0, 0, xb[j], 0, xa[i]);
      }
  };
  // fp32: whether there is a power that does not fit bf16; rows past the last one have none
  bool apart = false, row_a[MI], row_b[NI];
#pragma unroll
  for (int i = 0; i < MI; ++i) row_a[i] = wm * MI * 32 + i * 32 + frow < ra;
#pragma unroll
  for (int j = 0; j < NI; ++j) row_b[j] = wn * NI * 32 + j * 32 + frow < rb;
  auto look = [&](const int* xa, const int* xb) {
#pragma unroll
    for (int i = 0; i < MI; ++i) apart |= row_a[i] && !pw8_fits_bf16(xa[i]);
#pragma unroll
    for (int j = 0; j < NI; ++j) apart |= row_b[j] && !pw8_fits_bf16(xb[j]);
  };
  auto multiply_wide = [&](const Frags& f, const int* xa, const int* xb) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      bf16x8_t wa[MI], wb[NI];
#pragma unroll
      for (int i = 0; i < MI; ++i) wa[i] = pw8_wide(f.a[i], u, xa[i]);
#pragma unroll
      for (int j = 0; j < NI; ++j) wb[j] = pw8_wide(f.b[j], u, xb[j]);
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb[j], wa[i], acc[i][j], 0, 0, 0);
    }
  };

  // Step s of a block's two (ODD): the products of stage s, from registers. Under
  // them: wait until stage s + 1 has landed in all waves' LDS, read its fragments,
  // and load stage s + 3 over stage s - 1, which every wave has used up. FULL:
  // there are such stages; else that is looked at.
  constexpr int kSlots = MI * NI, kAfter = kSlots > 4 ? 1 : 0;  // the products before the barrier
  constexpr int kRoom = kSlots - kAfter;
  // the biases of this lane's outputs, asked for before the products
  constexpr int kRuns = NI * 32 / 8, kRowsAt = 64 / kRuns, kPasses = 32 / kRowsAt;
  const int64_t mw = m0 + wm * MI * 32, nw = n0 + wn * NI * 32;
  const int erow = lane / kRuns, ecol = (lane % kRuns) * 8;
  float bias[MI * kPasses > 8 ? MI * kPasses : 8];
  if (!PARTIAL) {
#pragma unroll
    for (int u = 0; u < (MI * kPasses > 8 ? MI * kPasses : 8); ++u) {
      // positions: the rows' (every kRowsAt-th); else the columns'
      const int64_t at = g.out.positions ? mw + u * kRowsAt + erow : nw + ecol + u;
      const bool in = g.out.bias && (g.out.positions ? u < MI * kPasses && at < g.out.rows : u < 8 && at < g.out.cols);
      bias[u] = in ? Elem<T>::to_f32(((const T*)g.out.bias)[at]) : 0.f;
    }
  }

  Frags f[2];
  auto step = [&](int s, auto odd_, auto full_, auto apart_) {
    constexpr bool ODD = decltype(odd_)::value, FULL = decltype(full_)::value, APART = decltype(apart_)::value;
    const Frags& now = f[ODD];
    Frags& next = f[!ODD];
    const bool more = FULL || s + 1 < stages, ahead = FULL || (s + 3 < stages && stages > 4);
    if constexpr (sizeof(T) == 4) {
      if (more) {
        if (FULL || s + 2 < stages) wait_vm<C::kLoads + !ODD>();
        else wait_vm<0>();
        // this wave's reads of stage s - 1, which loads go over, have ended, too: where the products
        // that wait for them stand is left to the compiler
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        meet();
        if (ODD) read_scales(s + 1, sa[1], sb[1]);
        if (ahead) {
          if (ODD) load_scales(s + 3);
#pragma unroll
          for (int u = 0; u < kFrags; ++u) load(s + 3, u);
        }
#pragma unroll
        for (int u = 0; u < kFrags; ++u) read(s + 1, u, next);
      }
      if (APART) {
        multiply_apart(now, sa[0], sb[0]);
      } else {
        if (!ODD) look(sa[0], sb[0]);
        multiply_wide(now, sa[0], sb[0]);
      }
    } else {
#pragma unroll
      for (int t = 0; t < kSlots; ++t) {
        multiply(now, t / NI, t % NI, sa[0], sb[0]);
        if (more) {
          if (t == kAfter) {
            // of stage s + 2, the only later one (but in a depth of four), its loads may still be under way
            if (FULL || s + 2 < stages) wait_vm<C::kLoads + !ODD>();
            else wait_vm<0>();
            meet();
            if (ODD) read_scales(s + 1, sa[1], sb[1]);
            if (ODD && ahead) load_scales(s + 3);
          }
          if (t >= kAfter) {
            const int r = t - kAfter;
#pragma unroll
            for (int u = r * kFrags / kRoom; u < (r + 1) * kFrags / kRoom; ++u) {
              read(s + 1, u, next);
              if (ahead) load(s + 3, u);
            }
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (ODD) {  // the next step is the next block's
#pragma unroll
      for (int i = 0; i < MI; ++i) sa[0][i] = sa[1][i];
#pragma unroll
      for (int j = 0; j < NI; ++j) sb[0][j] = sb[1][j];
    }
  };
  using Yes = std::integral_constant<bool, true>;
  using No = std::integral_constant<bool, false>;

  auto run = [&](auto apart_) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    code_a = code_a0;
    code_b = code_b0;
    scale = scale0;
    // three stages ahead, or all four that a short depth has; a block is two
    load_scales(0);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s < 3 ? s < stages : stages == 4) {
        if (s == 2) load_scales(s);
#pragma unroll
        for (int u = 0; u < kFrags; ++u) load(s, u);
      }
    }
    if (stages > 2) wait_vm<2 * C::kLoads + 1>();
    else wait_vm<C::kLoads>();
    meet();
    read_scales(0, sa[0], sb[0]);
#pragma unroll
    for (int u = 0; u < kFrags; ++u) read(0, u, f[0]);
    int s = 0;
    for (; s + 4 < stages; s += 2) {
      step(s, No(), Yes(), apart_);
      step(s + 1, Yes(), Yes(), apart_);
    }
    for (; s < stages; s += 2) {
      step(s, No(), No(), apart_);
      step(s + 1, Yes(), No(), apart_);
    }
  };
  run(No());
  if constexpr (sizeof(T) == 4) {
    __shared__ __align__(16) int met[4];
    if (lane == 0) met[wave] = 0;
    if (apart) met[wave] = 1;
    __syncthreads();
    // Once more from the start, if a wave has met powers that do not fit: 8192^3 takes
    // 930 us, where one such value in x is met 2130. A branch in each step instead would
    // leave the accumulators no registers (2200 spilled in the tile of 256 x 256).
    if (met[0] | met[1] | met[2] | met[3]) run(Yes());
  }
  __syncthreads();

  // out through LDS, 32 rows of the wave at a time, so that lanes next to each
  // other store next to each other
  unsigned char* mine = smem + wave * 32 * C::kEpiPitch;
  const int64_t col = nw + ecol;
  const Runs<T> runs(g.out, col);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
#pragma unroll
    for (int j = 0; j < NI; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 v = make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
        *(float4*)(mine + frow * C::kEpiPitch + (j * 32 + 8 * q + 4 * fh) * 4) = v;
      }
    __builtin_amdgcn_s_waitcnt(0xc07f);
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      const int r = u * kRowsAt + erow;
      const int64_t row = mw + i * 32 + r;
      if (row < g.out.rows && col < g.out.cols) {
        const float4 lo = *(const float4*)(mine + r * C::kEpiPitch + ecol * 4);
        const float4 hi = *(const float4*)(mine + r * C::kEpiPitch + ecol * 4 + 16);
        if (PARTIAL) {
          // rows of whole runs: cols is rounded up to 8
          float* p = g.part + ((int64_t)split * g.out.rows + row) * g.part_cols + col;
          *(float4*)p = lo;
          *(float4*)(p + 4) = hi;
        } else {
          float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            // values, not the places of one array, to choose from: those would be compared number by number
            const float of_row = bias[i * kPasses + u], of_column = bias[e];
            v[e] += g.out.positions ? of_row : of_column;
          }
          runs.put(row, v);
        }
      }
    }
    __builtin_amdgcn_s_waitcnt(0xc07f);
  }
}

// Sums of the splits in their order, with the bias.
template <typename T>
__global__ __launch_bounds__(256) void k_pw8_join(const Pw8Out o, const float* part, int splits, int part_cols) {
  const int64_t runs = part_cols / 8;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= o.rows * runs) return;
  const int64_t i = id / runs, j = (id - i * runs) * 8;
  const float* p = part + i * part_cols + j;
  const int64_t pitch = o.rows * part_cols;
  float v[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) v[u] = 0.f;
  int s = 0;
  for (; s + 4 <= splits; s += 4) {
    float4 f[4][2];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      f[u][0] = *(const float4*)(p + (s + u) * pitch);
      f[u][1] = *(const float4*)(p + (s + u) * pitch + 4);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      v[0] += f[u][0].x; v[1] += f[u][0].y; v[2] += f[u][0].z; v[3] += f[u][0].w;
      v[4] += f[u][1].x; v[5] += f[u][1].y; v[6] += f[u][1].z; v[7] += f[u][1].w;
    }
  }
  for (; s < splits; ++s) {
    const float4 lo = *(const float4*)(p + s * pitch), hi = *(const float4*)(p + s * pitch + 4);
    v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
    v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
  }
  if (o.bias) {
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (o.positions || j + u < o.cols) v[u] += Elem<T>::to_f32(((const T*)o.bias)[o.positions ? i : j + u]);
  }
  Runs<T>(o, j).put(i, v);
}

template <typename T, int BM, int BN>
hipError_t gemm(const Pw8GemmArgs& g, hipStream_t st) {
  const uint32_t blocks = (uint32_t)g.tiles_m * g.tiles_n * g.splits;
  constexpr int lds = Pw8Tile<BM, BN>::kLds;
  // large tiles are taken where they fill the units, and not split
  constexpr bool kSplits = BM * BN < 256 * 256;
  const void* kernel = (const void*)k_pw8_gemm<T, BM, BN, false>;
  if constexpr (kSplits) kernel = g.part ? (const void*)k_pw8_gemm<T, BM, BN, true> : kernel;
  hipError_t e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  if (!g.part) {
    DEFT_LAUNCH("pw8_gemm", (k_pw8_gemm<T, BM, BN, false>), dim3(blocks), dim3(256), lds, st, g);
    return hipGetLastError();
  }
  if constexpr (kSplits) {
    DEFT_LAUNCH("pw8_gemm", (k_pw8_gemm<T, BM, BN, true>), dim3(blocks), dim3(256), lds, st, g);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    const int64_t runs = g.out.rows * (g.part_cols / 8);
    DEFT_LAUNCH("pw8_join", k_pw8_join<T>, dim3((uint32_t)((runs + 255) / 256)), dim3(256), 0, st, g.out, g.part, g.splits,
                g.part_cols);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t gemm_of(const Pw8GemmArgs& g, int bm, int bn, hipStream_t st) {
  if (bm == 256 && bn == 256) return gemm<T, 256, 256>(g, st);
  if (bm == 128 && bn == 128) return gemm<T, 128, 128>(g, st);
  return gemm<T, 64, 128>(g, st);
}

}  // namespace

hipError_t launch_pw8_gemm(const Pw8GemmArgs& g, int bm, int bn, int dtype, hipStream_t st) {
  return dtype == DEFT_F32 ? gemm_of<float>(g, bm, bn, st) : gemm_of<bf16_t>(g, bm, bn, st);
}

}  // namespace deft
