// The 8-bit pointwise convolution of at most 16 rows: single steps and short
// calls, which are bound by the weights' bytes or by the launch.
//
// One launch: y[r][o] = sum_k x[r][k] w[o][k] + b[o].  A workgroup takes 16 or 32
// outputs o, its waves share the blocks of k.  A wave reads a block of its
// weights as they lie (twice 1 KB for 16 outputs) and 32 values of a row of x a lane,
// which it turns into codes by itself, in the registers that the matrix
// instruction takes them from; the blocks' codes are those that the quantising
// launch makes.  The waves' sums meet in LDS, in their order.
#include "deft_device.h"
#include "deft_internal.h"
#include "deft_pw8.h"

namespace deft {

namespace {

constexpr int kWaves = 8;

template <typename T> struct Run32;  // 32 consecutive values as they lie
template <> struct Run32<bf16_t> {
  typedef uint32_t word4 __attribute__((ext_vector_type(4), aligned(2)));
  word4 w[4];
  __device__ __forceinline__ void load(const bf16_t* p) {
#pragma unroll
    for (int u = 0; u < 4; ++u) w[u] = *(const word4*)(p + 8 * u);
  }
  __device__ __forceinline__ float get(int j) const {
    const uint32_t q = w[j >> 3][(j >> 1) & 3];
    return j & 1 ? bf16_hi(q) : bf16_lo(q);
  }
  // Bits of the greatest magnitude, as fp32; two at a time.
  __device__ __forceinline__ uint32_t most() const {
    typedef uint16_t half2_t __attribute__((ext_vector_type(2)));
    half2_t m = {0, 0};
#pragma unroll
    for (int j = 0; j < 16; ++j)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(half2_t, w[j >> 2][j & 3] & 0x7fff7fffu));
    return (uint32_t)(m[0] > m[1] ? m[0] : m[1]) << 16;
  }
  // Codes of finite values over 2^(byte - 127), byte > 0: one instruction for two.
  __device__ __forceinline__ pw8_codes_t codes(int byte) const {
    typedef __bf16 pair_t __attribute__((ext_vector_type(2)));
    typedef short words_t __attribute__((ext_vector_type(2)));
    const float scale = __uint_as_float((uint32_t)byte << 23);
    pw8_codes_t c;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t a = w[j >> 1][2 * (j & 1)], b = w[j >> 1][2 * (j & 1) + 1];
      words_t q = {0, 0};
      q = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(q, __builtin_bit_cast(pair_t, a), scale, false);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(q, __builtin_bit_cast(pair_t, b), scale, true);
      c[j] = __builtin_bit_cast(int, q);
    }
    return c;
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int u = 0; u < 4; ++u) w[u] = word4{0u, 0u, 0u, 0u};
  }
};
template <> struct Run32<float> {
  typedef float word4 __attribute__((ext_vector_type(4), aligned(4)));
  word4 w[8];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int u = 0; u < 8; ++u) w[u] = *(const word4*)(p + 4 * u);
  }
  __device__ __forceinline__ float get(int j) const { return w[j >> 2][j & 3]; }
};

// NF: fragments of 16 outputs; AHEAD: blocks whose loads a wave has under way
template <typename T, int NF, int AHEAD>
__global__ __launch_bounds__(64 * kWaves) void k_pw8_few(const Pw8FewArgs a) {
  __shared__ float part[kWaves][NF * 16][kPw8Few + 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int row = lane & 15, h = lane >> 4;  // of x or of the weights; quarter of a block
  const int64_t o0 = (int64_t)blockIdx.x * NF * 16;
  const int blocks = (a.c_in + kPw8Block - 1) / kPw8Block;
  const int64_t spitch = pw8_scale_rows(a.w.rows);
  const bool live = row < a.rows;
  // where this lane's row of x starts, and from channel to channel
  int64_t x0 = 0, step = 1;
  if (live) {
    if (a.positions) {
      const int image = row / a.positions;
      x0 = (int64_t)image * a.c_in * a.positions + (row - image * a.positions);
      step = a.positions;
    } else {
      x0 = (int64_t)row * a.c_in;
    }
  }
  const T* x = (const T*)a.x + x0;

  f32x4_t acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[f][r] = 0.f;

  uint4 lo[AHEAD][NF], hi[AHEAD][NF];
  int ws[AHEAD][NF];
  Run32<T> run[AHEAD];
  for (int k0 = wave; k0 < blocks; k0 += kWaves * AHEAD) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int kb = k0 + u * kWaves;
      const int c0 = kb * kPw8Block + h * 32;
      if (kb < blocks) {
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          // rows beyond the last are the last one's: their outputs are not stored
          const int64_t o = min(o0 + f * 16 + row, a.w.rows - 1);
          const uint8_t* p = a.w.codes + pw8_code(kb, h >> 1, a.w.rows, o) + (h & 1) * 32;
          lo[u][f] = *(const uint4*)p;
          hi[u][f] = *(const uint4*)(p + 16);
          ws[u][f] = a.w.scales[kb * spitch + o];
        }
        if (live && step == 1 && c0 + 32 <= a.c_in) run[u].load(x + c0);
      }
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      const int kb = k0 + u * kWaves;
      if (kb < blocks) {
        const int c0 = kb * kPw8Block + h * 32;
        int byte = 0;
        pw8_codes_t q;
        bool done = false;
        if constexpr (sizeof(T) == 2) {
          // whole runs of finite values: a fifth of the operations of the general way
          if (step == 1 && (kb + 1) * kPw8Block <= a.c_in) {
            if (!live) run[u].clear();
            const uint32_t m = max_across_16(run[u].most());
            byte = pw8_scale_byte(m);
            done = !__any(m >= 0x7f800000u || byte == 0);
            if (done) q = run[u].codes(byte);
          }
        }
        if (!done) {
          float v[32];
          if (live && step == 1 && c0 + 32 <= a.c_in) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = run[u].get(j);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = live && c0 + j < a.c_in ? Elem<T>::to_f32(x[(c0 + j) * step]) : 0.f;
          }
          uint32_t m = 0;
#pragma unroll
          for (int j = 0; j < 32; ++j) m = pw8_max(m, pw8_finite_bits(v[j]));
          byte = pw8_scale_byte(max_across_16(m));
          const float inv = pw8_inverse_scale(byte);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            q[j] = (int)pw8_codes4(pw8_scaled(v[4 * j], inv), pw8_scaled(v[4 * j + 1], inv), pw8_scaled(v[4 * j + 2], inv),
                                   pw8_scaled(v[4 * j + 3], inv));
        }
#pragma unroll
        for (int f = 0; f < NF; ++f) {
          pw8_codes_t w;
          w[0] = lo[u][f].x; w[1] = lo[u][f].y; w[2] = lo[u][f].z; w[3] = lo[u][f].w;
          w[4] = hi[u][f].x; w[5] = hi[u][f].y; w[6] = hi[u][f].z; w[7] = hi[u][f].w;
          if constexpr (sizeof(T) == 2) {
            acc[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, q, acc[f], 0, 0, 0, ws[u][f], 0, byte);
          } else {
            if (__any(!pw8_fits_bf16(ws[u][f]) || !pw8_fits_bf16(byte))) {  // deft_pw8.h says why
#pragma unroll 1
              for (int e = 0; e < 8; ++e)
                acc[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(pw8_one_of_8(w, e), q, acc[f], 0, 0, 0, ws[u][f], 0, byte);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pw8_wide(w, e, ws[u][f]), pw8_wide(q, e, byte), acc[f], 0, 0, 0);
            }
          }
        }
      }
    }
  }
  // register r: output 4 h + r of a fragment, row `row` of x
#pragma unroll
  for (int f = 0; f < NF; ++f)
#pragma unroll
    for (int r = 0; r < 4; ++r) part[wave][f * 16 + 4 * h + r][row] = acc[f][r];
  __syncthreads();
  for (int e = tid; e < NF * 16 * kPw8Few; e += 64 * kWaves) {
    const int o = e % (NF * 16), r = e / (NF * 16);
    if (r >= a.rows || o0 + o >= a.w.rows) continue;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) s += part[w][o][r];
    if (a.bias) s += Elem<T>::to_f32(((const T*)a.bias)[o0 + o]);
    int64_t at = (int64_t)r * a.w.rows + o0 + o;
    if (a.positions) {
      const int image = r / a.positions;
      at = ((int64_t)image * a.w.rows + o0 + o) * a.positions + (r - image * a.positions);
    }
    ((T*)a.y)[at] = Elem<T>::from_f32(s);
  }
}

template <typename T>
hipError_t few(const Pw8FewArgs& a, int cus, hipStream_t st) {
  // 32 outputs a workgroup where that still leaves one for each compute unit: with 16 x is
  // turned into codes twice as often (8 rows, 8192 to 8192: 20.3 us where they take 14.5,
  // fp32 28 and 22.5)
  constexpr int kAhead = sizeof(T) == 2 ? 4 : 1;
  if (a.w.rows >= (int64_t)32 * cus)
    DEFT_LAUNCH("pw8_few", (k_pw8_few<T, 2, kAhead>), dim3((uint32_t)((a.w.rows + 31) / 32)), dim3(64 * kWaves), 0, st, a);
  else
    DEFT_LAUNCH("pw8_few", (k_pw8_few<T, 1, kAhead>), dim3((uint32_t)((a.w.rows + 15) / 16)), dim3(64 * kWaves), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_pw8_few(const Pw8FewArgs& a, int dtype, int cus, hipStream_t st) {
  return dtype == DEFT_F32 ? few<float>(a, cus, st) : few<bf16_t>(a, cus, st);
}

}  // namespace deft
