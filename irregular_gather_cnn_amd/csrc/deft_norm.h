// Building blocks of the group norm kernels: 16-byte chunks of a row at any
// element offset, the activations, and reductions within a workgroup.
#pragma once
#include "deft_device.h"
#include "deft_internal.h"

namespace deft {

// V consecutive elements of a row, as read.  V fills 16 bytes; rows shorter
// than that are walked element by element (V = 1).  A row may start at any
// element, so the 16-byte access has only the element's alignment.
template <typename T, int V> struct Chunk;
template <> struct Chunk<bf16_t, 8> {
  typedef uint32_t word4 __attribute__((ext_vector_type(4), aligned(2)));
  word4 q;
  __device__ __forceinline__ void zero() { q = word4(0); }
  __device__ __forceinline__ void load(const bf16_t* p) { q = *(const word4*)p; }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) { f[2 * j] = bf16_lo(q[j]); f[2 * j + 1] = bf16_hi(q[j]); }
  }
  static __device__ __forceinline__ void store(bf16_t* p, const float* f) {
    word4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(f[2 * j], f[2 * j + 1]);
    *(word4*)p = w;
  }
};
template <> struct Chunk<float, 4> {
  typedef float word4 __attribute__((ext_vector_type(4), aligned(4)));
  word4 q;
  __device__ __forceinline__ void zero() { q = word4(0.f); }
  __device__ __forceinline__ void load(const float* p) { q = *(const word4*)p; }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = q[j];
  }
  static __device__ __forceinline__ void store(float* p, const float* f) {
    word4 w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = f[j];
    *(word4*)p = w;
  }
};
template <typename T> struct Chunk<T, 1> {
  T q;
  __device__ __forceinline__ void zero() { q = T(0); }
  __device__ __forceinline__ void load(const T* p) { q = *p; }
  __device__ __forceinline__ void get(float* f) const { f[0] = Elem<T>::to_f32(q); }
  static __device__ __forceinline__ void store(T* p, const float* f) { *p = Elem<T>::from_f32(f[0]); }
};

// exp(x) as 2^(x log2 e); the product's rounding costs x 2^-24 of the result.
__device__ __forceinline__ float exp_of(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

// Upper tail Q(a) = P(N > a) of the normal distribution, a >= 0, given e =
// exp(-a^2/2): e t P(t) with t = 1 / (1 + p a), the form of Hastings' (1955)
// approximations of the normal integral; P is fitted here to the least
// relative error over 0 <= a <= 14.  bf16 results take the degree 5 (4.7e-6),
// fp32 the degree 8 (1.7e-8 before rounding).  Products with a tail keep its
// relative error, where 1 + erf loses the small values.
template <typename T> __device__ __forceinline__ float normal_tail(float a, float e) {
  if (sizeof(T) == 2) {
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.31f, a, 1.f));
    float q = -7.392986440e-02f;
    q = __builtin_fmaf(q, t, 1.804524971e-01f);
    q = __builtin_fmaf(q, t, 1.574232522e-02f);
    q = __builtin_fmaf(q, t, 1.334309906e-01f);
    q = __builtin_fmaf(q, t, 1.204410087e-01f);
    q = __builtin_fmaf(q, t, 1.238607214e-01f);
    return e * t * q;
  }
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.21f, a, 1.f));
  float q = -7.165636271e-02f;
  q = __builtin_fmaf(q, t, 2.835888902e-01f);
  q = __builtin_fmaf(q, t, -3.302541537e-01f);
  q = __builtin_fmaf(q, t, 3.494019787e-01f);
  q = __builtin_fmaf(q, t, -9.392592504e-02f);
  q = __builtin_fmaf(q, t, 1.248730502e-01f);
  q = __builtin_fmaf(q, t, 6.919208384e-02f);
  q = __builtin_fmaf(q, t, 8.506887049e-02f);
  q = __builtin_fmaf(q, t, 8.371157490e-02f);
  return e * t * q;
}

// A NaN stays a NaN in every activation.
template <typename T, int ACT> __device__ __forceinline__ float act_of(float z) {
  if (ACT == DEFT_ACT_RELU) return z < 0.f ? 0.f : z;
  if (ACT == DEFT_ACT_SILU) return z * __builtin_amdgcn_rcpf(1.f + exp_of(-z));
  if (ACT == DEFT_ACT_GELU) {
    const float q = normal_tail<T>(__builtin_fabsf(z), exp_of(-0.5f * z * z));
    return z * (z > 0.f ? 1.f - q : q);
  }
  return z;
}
// dy times the activation's slope at z.
template <typename T, int ACT> __device__ __forceinline__ float act_grad(float z, float dy) {
  if (ACT == DEFT_ACT_RELU) return z > 0.f ? dy : 0.f;
  if (ACT == DEFT_ACT_SILU) {
    const float p = __builtin_amdgcn_rcpf(1.f + exp_of(-z));
    return dy * (p * __builtin_fmaf(z, 1.f - p, 1.f));
  }
  if (ACT == DEFT_ACT_GELU) {
    const float e = exp_of(-0.5f * z * z);
    const float q = normal_tail<T>(__builtin_fabsf(z), e);
    return dy * __builtin_fmaf(z * 0.3989422804f, e, z > 0.f ? 1.f - q : q);
  }
  return dy;
}

// Calls f(constant) for the activation of the call.
template <int A> struct ActTag { static constexpr int value = A; };
template <typename F> __device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case DEFT_ACT_RELU: f(ActTag<DEFT_ACT_RELU>{}); break;
    case DEFT_ACT_SILU: f(ActTag<DEFT_ACT_SILU>{}); break;
    case DEFT_ACT_GELU: f(ActTag<DEFT_ACT_GELU>{}); break;
    default: f(ActTag<DEFT_ACT_NONE>{}); break;
  }
}

// Sum over aligned teams of `t` lanes (a power of two up to 64), in every lane.
__device__ __forceinline__ float team_sum(float v, int t) {
  for (int d = t >> 1; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// Sum over the workgroup, in every thread; `lds` holds a float per wave and is
// free again after the caller's next barrier.
__device__ __forceinline__ float block_sum(float v, float* lds) {
  v = team_sum(v, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float r = 0.f;
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) r += lds[w];
  return r;
}

// Sums of the segments of a matrix in LDS: out(seg, sum over rows r and
// columns j < len of m[r * pitch + seg * len + j]), called by one thread per
// segment.  A team of lanes walks each segment; `pitch` is odd, so that lanes
// on different rows fall on different banks.
template <typename F>
__device__ __forceinline__ void segment_sums(const float* m, int pitch, int rows, int nseg, int len, F out) {
  const int nt = blockDim.x, total = rows * len;
  int t = 64;
  while (t > 1 && t * nseg > nt) t >>= 1;
  const int l = threadIdx.x & (t - 1);
  const FastDiv by_len = make_fastdiv(len);
  for (int seg = threadIdx.x / t; seg < nseg; seg += nt / t) {
    float v = 0.f;
    for (int i = l; i < total; i += t) {
      const int r = fdiv(i, by_len);
      v += m[r * pitch + seg * len + (i - r * len)];
    }
    v = team_sum(v, t);
    if (l == 0) out(seg, v);
  }
}

// Columns c0 .. c0 + cols of one image's [s][c], as a workgroup's threads
// share them: thread (tx, ty) has the chunk tx of the rows ty, ty + TY, ...
// A ragged band's last chunk starts early enough to end at the band's end;
// its first `shift` elements are also the chunk's before it, and count there.
struct Band {
  int g0, ng, c0, cols;
  int cx, tx, ty, TY, col, shift;
  template <int V> __device__ __forceinline__ void set(int b, int bands, int g, int per) {
    g0 = (int)((int64_t)b * g / bands);
    ng = (int)((int64_t)(b + 1) * g / bands) - g0;
    c0 = g0 * per;
    cols = ng * per;
    cx = (cols + V - 1) / V;
    TY = blockDim.x / cx;
    ty = threadIdx.x / cx;
    tx = threadIdx.x - ty * cx;
    col = tx * V + V <= cols ? tx * V : cols - V;  // cols >= V
    shift = tx * V - col;
    col += c0;
  }
};

}  // namespace deft
