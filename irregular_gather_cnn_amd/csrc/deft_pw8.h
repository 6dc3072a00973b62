// Codes of the 8-bit pointwise convolution, shared by the kernels that make them.
//
// Block of values v: with most = max |v| over its finite ones, e is the least
// whole number >= -127 for which most <= 448 * 2^e, or 0 where most = 0; code =
// v * 2^-e rounded to the nearest e4m3, ties to even; the block's scale byte is
// e + 127.  A NaN or an infinity becomes the code NaN, and so reaches the outputs
// that it enters and no other.
//
// A matrix of codes over rows and a depth is stored by half blocks of the depth:
// codes [ceil(depth / 128)][2][rows][64], the last block filled up with zeros, and
// scale bytes [ceil(depth / 128)][round_up(rows, 16)].  What a stage of a product
// reads is then one piece of memory, in whole lines (with 128 codes of a row in
// sequence a stage read half lines: 8192^3 took 608 us and then 554), and
// offsets inside it fit 32 bits however large the matrix is.
#pragma once
#include "deft_device.h"

namespace deft {

// Bits of |v|, by which values are ordered; 0 where v is not finite.
__device__ __forceinline__ uint32_t pw8_finite_bits(float v) {
  const uint32_t b = __float_as_uint(v) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}
__device__ __forceinline__ uint32_t pw8_max(uint32_t a, uint32_t b) { return a > b ? a : b; }
// v of the lane whose number within its 16 is greater by N, cyclically.
template <int N> __device__ __forceinline__ uint32_t turn16(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xf, 0xf, false);
}
// The greatest among 16 lanes, and among the lanes of the same number in each 16.
__device__ __forceinline__ uint32_t max_of_16(uint32_t v) {
  v = pw8_max(v, turn16<8>(v));
  v = pw8_max(v, turn16<4>(v));
  v = pw8_max(v, turn16<2>(v));
  return pw8_max(v, turn16<1>(v));
}
__device__ __forceinline__ uint32_t max_across_16(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = pw8_max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return pw8_max(b[0], b[1]);
}
// Sums likewise, in an order that is the same for all lanes.
__device__ __forceinline__ float sum_of_16(float v) {
  v += __uint_as_float(turn16<8>(__float_as_uint(v)));
  v += __uint_as_float(turn16<4>(__float_as_uint(v)));
  v += __uint_as_float(turn16<2>(__float_as_uint(v)));
  return v + __uint_as_float(turn16<1>(__float_as_uint(v)));
}
__device__ __forceinline__ float sum_across_16(float v) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}
// e + 127 of a block whose largest value has these bits.
__device__ __forceinline__ int pw8_scale_byte(uint32_t most) {
  const int e = (int)(most >> 23) - 8 + ((most & 0x7fffffu) > 0x600000u);  // 448 = 1.75 * 2^8
  return most == 0 ? 127 : e < 0 ? 0 : e;
}
// 2^-e; the byte is at most 247.
__device__ __forceinline__ float pw8_inverse_scale(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }
// v * inv, NaN where v is not finite.
__device__ __forceinline__ float pw8_scaled(float v, float inv) { return __builtin_fmaf(v, inv, 0.f * v); }
__device__ __forceinline__ uint32_t pw8_codes4(float a, float b, float c, float d) {
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// How the products are summed.  The 8-bit matrix instructions add 8 products at
// a time with 13 bits below the largest of the 8, and cut the rest off; groups
// are then added in fp32.  That leaves results off by 1.5e-5 of their root mean
// square (normal values, 64 to 8192 terms; 4.6e-5 where channels differ in size and
// some values are large), where rounding to bf16 leaves 1.66e-3, for twice the rate
// of the 16-bit instructions.  fp32 results take those: codes times
// their powers of two are bf16 values, but at the ends of the range, and 16-bit
// instructions sum exact products as fp32 does (3e-8).
typedef int pw8_codes_t __attribute__((ext_vector_type(8)));

// 8 codes of words 2u and 2u + 1 times 2^(byte - 127), as bf16.
__device__ __forceinline__ bf16x8_t pw8_wide(const pw8_codes_t& c, int u, int byte) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  const float scale = __uint_as_float((uint32_t)byte << 23);
  bf16x8_t v;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const bf16x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[2 * u + k], scale, false);
    const bf16x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[2 * u + k], scale, true);
    v[4 * k] = lo[0]; v[4 * k + 1] = lo[1]; v[4 * k + 2] = hi[0]; v[4 * k + 3] = hi[1];
  }
  return v;
}

// Whether every code times 2^(byte - 127) is a normal bf16 value: codes reach from
// 2^-9 to 448.  Under the least such byte values would be lost, and over the
// greatest a code of 256 be infinite.  Products with those blocks take the 8-bit
// instructions, eight times, each with one code of every eight in place: nothing
// is cut off, then.
__device__ __forceinline__ bool pw8_fits_bf16(int byte) { return (uint32_t)(byte - 10) <= 236u; }
__device__ __forceinline__ pw8_codes_t pw8_one_of_8(const pw8_codes_t& c, int which) {
  const int mask = 0xff << 8 * (which & 3), even = which < 4 ? mask : 0, odd = mask ^ even;
  pw8_codes_t v;
#pragma unroll
  for (int w = 0; w < 8; ++w) v[w] = c[w] & (w & 1 ? odd : even);
  return v;
}

}  // namespace deft
