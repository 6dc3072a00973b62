// 8-bit codes of the pointwise convolution's matrices: e4m3 values times a power
// of two for each block of 128.
//
// Codes and scales are defined in deft_pw8.h.  Scales are powers of two, because
// the matrix instruction multiplies by such scales itself and the multiplication
// by 2^-e is exact; e4m3's values keep 4 significant bits over 15 binades
// whatever the scale.
//
// One workgroup takes 128 x 128 values once and writes them in up to two forms:
// the near form, whose depth runs along memory, and the far form, whose depth
// runs across it (x for y, and x for dw).  What bounds it is memory: for bf16 in
// and one form out it has 3 bytes a value to move.
#include "deft_device.h"
#include "deft_internal.h"
#include "deft_pw8.h"

namespace deft {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = kPw8Block;
constexpr int kRun = 8;                            // values of a line that a thread holds
constexpr int kAcross = kTile / kRun;              // threads along a line
constexpr int kLines = kTile * kAcross / kThreads; // lines of a thread, in sequence
static_assert(kLines == 8, "a thread holds 8 x 8 values");

// 8 values from any element address.
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

// FAR: the far form is written, too (or alone).  TILE: one scale for the whole
// tile.
template <typename T, bool FAR, bool TILE>
__global__ __launch_bounds__(kThreads) void k_pw8_quantise(const Pw8QuantiseArgs a) {
  // the waves' maxima of the 128 columns, then their sums; the far form's codes
  __shared__ uint32_t most_of[4][kTile];
  __shared__ float sum_of[4][kTile];
  __shared__ __align__(16) unsigned char turned[FAR ? kTile * kTile : 16];
  const int tid = threadIdx.x, q = tid % kAcross, t = tid / kAcross, wave = tid >> 6;
  const uint32_t bid = blockIdx.x;
  const uint32_t lines_at = bid / a.tiles_near, near_at = bid - lines_at * a.tiles_near;
  const int64_t line0 = (int64_t)lines_at * kTile, near0 = (int64_t)near_at * kTile;
  // this thread: lines line0 + 8 t + i, values b0 .. b0 + 7 along each
  const int64_t l0 = line0 + t * kLines, b0 = near0 + q * kRun;

  float v[kLines][kRun];
  {
    // where a run starts: lines are rows or, channels first, channels whose
    // positions go from image to image
    int64_t at = b0, room = a.near - b0;  // values that lie in sequence
    if (a.positions) {
      const int64_t image = b0 / a.positions, pos = b0 - image * a.positions;
      at = image * a.positions * a.lines + pos;
      if (a.positions - pos < room) room = a.positions - pos;
    }
    const T* src = (const T*)a.src + at + l0 * a.pitch;
    const bool whole = room >= kRun;
#pragma unroll
    for (int i = 0; i < kLines; ++i) {
#pragma unroll
      for (int j = 0; j < kRun; ++j) v[i][j] = 0.f;
      if (l0 + i < a.lines && whole) load_run(src + i * a.pitch, v[i]);
    }
    if (!whole && b0 < a.near) {
      // a line's end, or the border of two images (positions of an image may be
      // fewer than a run, then there are several)
#pragma unroll 1
      for (int j = 0; j < kRun; ++j) {
        const int64_t b = b0 + j;
        if (b >= a.near) break;
        int64_t p = b;
        if (a.positions) {
          const int64_t image = b / a.positions;
          p = image * a.positions * a.lines + (b - image * a.positions);
        }
#pragma unroll
        for (int i = 0; i < kLines; ++i)
          if (l0 + i < a.lines) {
            const float w = Elem<T>::to_f32(((const T*)a.src)[p + (l0 + i) * a.pitch]);
#pragma unroll
            for (int k = 0; k < kRun; ++k)
              if (k == j) v[i][k] = w;
          }
      }
    }
  }

  // sums over the rows, for the bias's gradient
  if (a.sums) {
    if (a.positions) {  // rows run along the lines
#pragma unroll
      for (int i = 0; i < kLines; ++i) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < kRun; ++j) s += v[i][j];
#pragma unroll
        for (int d = 1; d < kAcross; d <<= 1) s += __shfl_xor(s, d);
        if (q == 0 && l0 + i < a.lines) a.sums[(int64_t)near_at * a.lines + l0 + i] = s;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kRun; ++j) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kLines; ++i) s += v[i][j];
        s += __shfl_xor(s, 16);
        s += __shfl_xor(s, 32);
        if ((tid & 63) < kAcross) sum_of[wave][q * kRun + j] = s;
      }
    }
  }

  uint32_t line_most[kLines], column_most[kRun];
#pragma unroll
  for (int j = 0; j < kRun; ++j) column_most[j] = 0;
#pragma unroll
  for (int i = 0; i < kLines; ++i) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const uint32_t b = pw8_finite_bits(v[i][j]);
      m = pw8_max(m, b);
      column_most[j] = pw8_max(column_most[j], b);
    }
    line_most[i] = m;
  }
  if (FAR || TILE) {
    // over the wave's lines, then over the waves
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      column_most[j] = pw8_max(column_most[j], __shfl_xor(column_most[j], 16));
      column_most[j] = pw8_max(column_most[j], __shfl_xor(column_most[j], 32));
      if ((tid & 63) < kAcross) most_of[wave][q * kRun + j] = column_most[j];
    }
  }
  if (FAR || TILE || (a.sums && !a.positions)) __syncthreads();
  if (a.sums && !a.positions && tid < kTile && near0 + tid < a.near)
    a.sums[(int64_t)lines_at * a.near + near0 + tid] = sum_of[0][tid] + sum_of[1][tid] + (sum_of[2][tid] + sum_of[3][tid]);
  int tile_byte = 0;
  if (TILE) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kRun; ++j)
      for (int w = 0; w < 4; ++w) m = pw8_max(m, most_of[w][q * kRun + j]);
#pragma unroll
    for (int d = 1; d < kAcross; d <<= 1) m = pw8_max(m, __shfl_xor(m, d));
    tile_byte = pw8_scale_byte(m);
  }

  if (a.near_codes) {
#pragma unroll
    for (int i = 0; i < kLines; ++i) {
      int byte = tile_byte;
      if (!TILE) {
        uint32_t m = line_most[i];
#pragma unroll
        for (int d = 1; d < kAcross; d <<= 1) m = pw8_max(m, __shfl_xor(m, d));
        byte = pw8_scale_byte(m);
      }
      const float inv = pw8_inverse_scale(byte);
      uint2 c;
      c.x = pw8_codes4(pw8_scaled(v[i][0], inv), pw8_scaled(v[i][1], inv), pw8_scaled(v[i][2], inv), pw8_scaled(v[i][3], inv));
      c.y = pw8_codes4(pw8_scaled(v[i][4], inv), pw8_scaled(v[i][5], inv), pw8_scaled(v[i][6], inv), pw8_scaled(v[i][7], inv));
      if (l0 + i < a.lines) {
        *(uint2*)(a.near_codes + pw8_code(near_at, q / 8, a.lines, l0 + i) + q % 8 * kRun) = c;
        if (q == 0) a.near_scales[(int64_t)near_at * pw8_scale_rows(a.lines) + l0 + i] = (uint8_t)byte;
      }
    }
  }
  if (FAR && a.far_codes) {
    int bytes[kRun];
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const int b = q * kRun + j;
      bytes[j] = TILE ? tile_byte
                      : pw8_scale_byte(pw8_max(pw8_max(most_of[0][b], most_of[1][b]), pw8_max(most_of[2][b], most_of[3][b])));
      const float inv = pw8_inverse_scale(bytes[j]);
      uint2 c;
      c.x = pw8_codes4(pw8_scaled(v[0][j], inv), pw8_scaled(v[1][j], inv), pw8_scaled(v[2][j], inv), pw8_scaled(v[3][j], inv));
      c.y = pw8_codes4(pw8_scaled(v[4][j], inv), pw8_scaled(v[5][j], inv), pw8_scaled(v[6][j], inv), pw8_scaled(v[7][j], inv));
      // 8 lines of column b; columns of one j take the 8-byte places of a row of
      // the turned tile in different orders, so 16 threads write to 16 banks' pairs
      *(uint2*)(turned + b * kTile + ((t ^ q) << 3)) = c;
      if (t == 0 && near0 + b < a.near)
        a.far_scales[(int64_t)lines_at * pw8_scale_rows(a.near) + near0 + b] = (uint8_t)bytes[j];
    }
    __syncthreads();
    // 16-byte pieces in the order of memory: half, column, piece
#pragma unroll
    for (int i = 0; i < kTile * kTile / 16 / kThreads; ++i) {
      const int piece = i * kThreads + tid, half = piece / (4 * kTile), b = piece / 4 % kTile, o = b >> 3;
      const int c = half * 8 + (piece & 3) * 2;
      if (near0 + b < a.near) {
        const uint2 lo = *(const uint2*)(turned + b * kTile + ((c ^ o) << 3));
        const uint2 hi = *(const uint2*)(turned + b * kTile + (((c + 1) ^ o) << 3));
        *(uint4*)(a.far_codes + pw8_code(lines_at, half, a.near, near0 + b) + (piece & 3) * 16) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    }
  }
}

// db = the tiles' sums in their order.  64 channels a workgroup, 4 shares of the
// tiles, fp64 beyond a tile.
template <typename T>
__global__ __launch_bounds__(256) void k_pw8_bias(const float* sums, int64_t tiles, int c, T* db) {
  __shared__ double part[4][64];
  const int i = threadIdx.x & 63, share = threadIdx.x >> 6, ch = blockIdx.x * 64 + i;
  double s = 0.0;
  if (ch < c) {
    int64_t k = share;
    for (; k + 28 < tiles; k += 32) {
      float f[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) f[u] = sums[(k + 4 * u) * c + ch];
#pragma unroll
      for (int u = 0; u < 8; ++u) s += (double)f[u];
    }
    for (; k < tiles; k += 4) s += (double)sums[k * c + ch];
  }
  part[share][i] = s;
  __syncthreads();
  if (share == 0 && ch < c) db[ch] = Elem<T>::from_f32((float)((part[0][i] + part[1][i]) + (part[2][i] + part[3][i])));
}

// Clears bytes (a multiple of 2) by a kernel: a memset does not belong in captured graphs.
__global__ __launch_bounds__(256) void k_pw8_zero(uint16_t* p, size_t halves) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < halves; i += (size_t)gridDim.x * 256) p[i] = 0;
}

template <typename T>
hipError_t quantise(const Pw8QuantiseArgs& a, uint32_t blocks, bool tile, hipStream_t st) {
  if (tile && a.far_codes)
    DEFT_LAUNCH("pw8_pack", (k_pw8_quantise<T, true, true>), dim3(blocks), dim3(kThreads), 0, st, a);
  else if (tile)
    DEFT_LAUNCH("pw8_pack", (k_pw8_quantise<T, false, true>), dim3(blocks), dim3(kThreads), 0, st, a);
  else if (a.far_codes)
    DEFT_LAUNCH("pw8_quantise", (k_pw8_quantise<T, true, false>), dim3(blocks), dim3(kThreads), 0, st, a);
  else
    DEFT_LAUNCH("pw8_quantise", (k_pw8_quantise<T, false, false>), dim3(blocks), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_pw8_quantise(const Pw8QuantiseArgs& a, uint32_t blocks, int dtype, bool tile, hipStream_t st) {
  return dtype == DEFT_F32 ? quantise<float>(a, blocks, tile, st) : quantise<bf16_t>(a, blocks, tile, st);
}

hipError_t launch_pw8_zero(void* p, size_t bytes, hipStream_t st) {
  const size_t halves = bytes / 2, blocks = (halves + 2047) / 2048;
  DEFT_LAUNCH("pw8_zero", k_pw8_zero, dim3((uint32_t)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, st, (uint16_t*)p, halves);
  return hipGetLastError();
}

hipError_t launch_pw8_bias(const float* sums, int64_t tiles, int c, void* db, int dtype, hipStream_t st) {
  const dim3 grid((uint32_t)((c + 63) / 64));
  if (dtype == DEFT_F32) DEFT_LAUNCH("pw8_bias", k_pw8_bias<float>, grid, dim3(256), 0, st, sums, tiles, c, (float*)db);
  else DEFT_LAUNCH("pw8_bias", k_pw8_bias<bf16_t>, grid, dim3(256), 0, st, sums, tiles, c, (bf16_t*)db);
  return hipGetLastError();
}

}  // namespace deft
