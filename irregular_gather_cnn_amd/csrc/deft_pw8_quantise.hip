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
// runs across it (x for y, and x for dw).  What bounds it is memory: 16 x 1024 x
// 3136 in bf16 to both forms takes 44 us for 205 MB, 8192^2 to one 43 us for 201 MB.
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

// 8 consecutive values of a line as they lie in memory, from any element address: half
// the registers of their fp32 values in bf16, which lets four workgroups of 256 threads
// share a unit instead of three.
template <typename T> struct Run8;
template <> struct Run8<bf16_t> {
  typedef uint32_t word4 __attribute__((ext_vector_type(4), aligned(2)));
  word4 w;
  __device__ __forceinline__ void clear() { w = word4{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ void load(const bf16_t* p) { w = *(const word4*)p; }
  __device__ __forceinline__ void set(const bf16_t* v) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = v[2 * j] | (uint32_t)v[2 * j + 1] << 16;
  }
  // Between two passes over the values: the compiler would carry them from one to the
  // other unpacked.
  __device__ __forceinline__ void keep() {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t q = w[j];
      asm volatile("" : "+v"(q));
      w[j] = q;
    }
  }
  __device__ __forceinline__ float get(int j) const { return j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]); }
};
template <> struct Run8<float> {
  typedef float word4 __attribute__((ext_vector_type(4), aligned(4)));
  word4 w[2];
  __device__ __forceinline__ void clear() { w[0] = w[1] = word4{0.f, 0.f, 0.f, 0.f}; }
  __device__ __forceinline__ void load(const float* p) { w[0] = *(const word4*)p; w[1] = *(const word4*)(p + 4); }
  __device__ __forceinline__ void set(const float* v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j >> 2][j & 3] = v[j];
  }
  __device__ __forceinline__ void keep() {}
  __device__ __forceinline__ float get(int j) const { return w[j >> 2][j & 3]; }
};

// FAR: the far form is written, too (or alone).  TILE: one scale for the whole
// tile.
template <typename T, bool FAR, bool TILE>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(sizeof(T) == 4 && FAR ? 3 : 4))) void k_pw8_quantise(const Pw8QuantiseArgs a,
                                                                                                    const FastDiv by_positions) {
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

  Run8<T> v[kLines];
  {
    // where a run starts: lines are rows or, channels first, channels whose
    // positions go from image to image
    int64_t at = b0, room = a.near - b0;  // values that lie in sequence
    const int64_t image_pitch = a.positions * a.lines;
    if (a.positions) {
      const int64_t image = fdiv((int)b0, by_positions), pos = b0 - image * a.positions;
      at = image * image_pitch + pos;
      if (a.positions - pos < room) room = a.positions - pos;
    }
    const T* src = (const T*)a.src + l0 * a.pitch;
    const bool whole = room >= kRun;
#pragma unroll
    for (int i = 0; i < kLines; ++i) {
      v[i].clear();
      if (l0 + i < a.lines && whole) v[i].load(src + at + i * a.pitch);
    }
    if (!whole && b0 < a.near && l0 < a.lines) {
      // a line's end, or the border of two images: value by value, all at once; what lies
      // outside is read from the run's first place
      int64_t p[kRun];
#pragma unroll
      for (int j = 0; j < kRun; ++j) {
        p[j] = at;
        if (b0 + j < a.near) {
          p[j] = b0 + j;
          if (a.positions) {
            const int64_t image = fdiv((int)(b0 + j), by_positions);
            p[j] = image * image_pitch + (b0 + j - image * a.positions);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kLines; ++i) {
        const T* line = src + (l0 + i < a.lines ? i : 0) * a.pitch;
        T w[kRun];
#pragma unroll
        for (int j = 0; j < kRun; ++j) w[j] = line[p[j]];
#pragma unroll
        for (int j = 0; j < kRun; ++j) w[j] = b0 + j < a.near && l0 + i < a.lines ? w[j] : T(0);
        v[i].set(w);
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
        for (int j = 0; j < kRun; ++j) s += v[i].get(j);
        s = sum_of_16(s);
        if (q == 0 && l0 + i < a.lines) a.sums[(int64_t)near_at * a.lines + l0 + i] = s;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kRun; ++j) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kLines; ++i) s += v[i].get(j);
        s = sum_across_16(s);
        if ((tid & 63) < kAcross) sum_of[wave][q * kRun + j] = s;
      }
    }
  }

  auto keep = [&]() {
#pragma unroll
    for (int i = 0; i < kLines; ++i) v[i].keep();
  };
  keep();
  uint32_t line_most[kLines], column_most[kRun];
#pragma unroll
  for (int j = 0; j < kRun; ++j) column_most[j] = 0;
#pragma unroll
  for (int i = 0; i < kLines; ++i) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const uint32_t b = pw8_finite_bits(v[i].get(j));
      m = pw8_max(m, b);
      column_most[j] = pw8_max(column_most[j], b);
    }
    line_most[i] = m;
  }
  if (FAR || TILE) {
    // over the wave's lines, then over the waves
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      column_most[j] = max_across_16(column_most[j]);
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
    tile_byte = pw8_scale_byte(max_of_16(m));
  }

  keep();
  if (a.near_codes) {
#pragma unroll
    for (int i = 0; i < kLines; ++i) {
      int byte = tile_byte;
      if (!TILE) {
        byte = pw8_scale_byte(max_of_16(line_most[i]));
      }
      const float inv = pw8_inverse_scale(byte);
      uint2 c;
      c.x = pw8_codes4(pw8_scaled(v[i].get(0), inv), pw8_scaled(v[i].get(1), inv), pw8_scaled(v[i].get(2), inv), pw8_scaled(v[i].get(3), inv));
      c.y = pw8_codes4(pw8_scaled(v[i].get(4), inv), pw8_scaled(v[i].get(5), inv), pw8_scaled(v[i].get(6), inv), pw8_scaled(v[i].get(7), inv));
      if (l0 + i < a.lines) *(uint2*)(a.near_codes + pw8_code(near_at, q / 8, a.lines, l0 + i) + q % 8 * kRun) = c;
      // the scales' rows past the last one are read, too
      if (q == 0 && l0 + i < pw8_scale_rows(a.lines))
        a.near_scales[(int64_t)near_at * pw8_scale_rows(a.lines) + l0 + i] = (uint8_t)byte;
    }
  }
  keep();
  if (FAR && a.far_codes) {
    int bytes[kRun];
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const int b = q * kRun + j;
      bytes[j] = TILE ? tile_byte
                      : pw8_scale_byte(pw8_max(pw8_max(most_of[0][b], most_of[1][b]), pw8_max(most_of[2][b], most_of[3][b])));
      const float inv = pw8_inverse_scale(bytes[j]);
      uint2 c;
      c.x = pw8_codes4(pw8_scaled(v[0].get(j), inv), pw8_scaled(v[1].get(j), inv), pw8_scaled(v[2].get(j), inv), pw8_scaled(v[3].get(j), inv));
      c.y = pw8_codes4(pw8_scaled(v[4].get(j), inv), pw8_scaled(v[5].get(j), inv), pw8_scaled(v[6].get(j), inv), pw8_scaled(v[7].get(j), inv));
      // 8 lines of column b; columns of one j take the 8-byte places of a row of
      // the turned tile in different orders, so 16 threads write to 16 banks' pairs
      *(uint2*)(turned + b * kTile + ((t ^ q) << 3)) = c;
      if (t == 0 && near0 + b < pw8_scale_rows(a.near))
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

// db = the tiles' sums: 16 channels a workgroup, 16 shares of the tiles, fp64 beyond
// a tile, in an order that does not change.
template <typename T>
__global__ __launch_bounds__(256) void k_pw8_bias(const float* sums, int64_t tiles, int c, T* db) {
  __shared__ double part[16][16];
  const int i = threadIdx.x & 15, share = threadIdx.x >> 4, ch = blockIdx.x * 16 + i;
  double s = 0.0;
  if (ch < c) {
    int64_t k = share;
    for (; k + 112 < tiles; k += 128) {
      float f[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) f[u] = sums[(k + 16 * u) * c + ch];
#pragma unroll
      for (int u = 0; u < 8; ++u) s += (double)f[u];
    }
#pragma unroll 8
    for (; k < tiles; k += 16) s += (double)sums[k * c + ch];
  }
  part[share][i] = s;
  __syncthreads();
  if (share == 0 && ch < c) {
    s = 0.0;
#pragma unroll
    for (int u = 0; u < 16; ++u) s += part[u][i];
    db[ch] = Elem<T>::from_f32((float)s);
  }
}

// Clears bytes (a multiple of 2) by a kernel: a memset does not belong in captured graphs.
__global__ __launch_bounds__(256) void k_pw8_zero(uint16_t* p, size_t halves) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < halves; i += (size_t)gridDim.x * 256) p[i] = 0;
}

template <typename T>
hipError_t quantise(const Pw8QuantiseArgs& a, uint32_t blocks, bool tile, hipStream_t st) {
  const FastDiv by = make_fastdiv(a.positions ? (uint32_t)a.positions : 1u);
  if (tile && a.far_codes)
    DEFT_LAUNCH("pw8_pack", (k_pw8_quantise<T, true, true>), dim3(blocks), dim3(kThreads), 0, st, a, by);
  else if (tile)
    DEFT_LAUNCH("pw8_pack", (k_pw8_quantise<T, false, true>), dim3(blocks), dim3(kThreads), 0, st, a, by);
  else if (a.far_codes)
    DEFT_LAUNCH("pw8_quantise", (k_pw8_quantise<T, true, false>), dim3(blocks), dim3(kThreads), 0, st, a, by);
  else
    DEFT_LAUNCH("pw8_quantise", (k_pw8_quantise<T, false, false>), dim3(blocks), dim3(kThreads), 0, st, a, by);
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
  const dim3 grid((uint32_t)((c + 15) / 16));
  if (dtype == DEFT_F32) DEFT_LAUNCH("pw8_bias", k_pw8_bias<float>, grid, dim3(256), 0, st, sums, tiles, c, (float*)db);
  else DEFT_LAUNCH("pw8_bias", k_pw8_bias<bf16_t>, grid, dim3(256), 0, st, sums, tiles, c, (bf16_t*)db);
  return hipGetLastError();
}

}  // namespace deft
