// Building blocks of the group norm kernels: 16-byte chunks of a row at any
// element offset, the activations, and reductions within a workgroup.
#pragma once
#include "deft_device.h"
#include "deft_internal.h"

namespace deft {

// V consecutive elements of a row, as read.  V fills 16 bytes; rows shorter
// than that are walked element by element (V = 1).  A row may start at any
// element, so the 16-byte access has only the element's alignment.  keep()
// stops the compiler from carrying the unpacked values from one pass over the
// chunks to the next, which takes twice the registers.
template <typename T, int V> struct Chunk;
template <> struct Chunk<bf16_t, 8> {
  typedef uint32_t word4 __attribute__((ext_vector_type(4), aligned(2)));
  word4 q;
  __device__ __forceinline__ void keep() { asm volatile("" : "+v"(q)); }
  __device__ __forceinline__ void load(const bf16_t* p) { q = *(const word4*)p; }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) { f[2 * j] = bf16_lo(q[j]); f[2 * j + 1] = bf16_hi(q[j]); }
  }
  __device__ __forceinline__ void zero_if(bool cond) {
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = cond ? 0u : q[j];
  }
  // The first `shift` elements become zeros.
  __device__ __forceinline__ void zero_below(int shift) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      q[j] &= (2 * j >= shift ? 0xffffu : 0u) | (2 * j + 1 >= shift ? 0xffff0000u : 0u);
  }
  // sum += elements 2j and 2j + 1, sq += their squares: two instructions, with
  // products that are exact in fp32
  __device__ __forceinline__ void moments(int j, float& sum, float& sq) const {
    typedef __bf16 pair __attribute__((ext_vector_type(2)));
    const uint32_t word = q[j];  // a bit cast of q[j] itself would read element 0
    const pair x = __builtin_bit_cast(pair, word), one = {(__bf16)1.f, (__bf16)1.f};
    sum = __builtin_amdgcn_fdot2_f32_bf16(x, one, sum, false);
    sq = __builtin_amdgcn_fdot2_f32_bf16(x, x, sq, false);
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
  __device__ __forceinline__ void keep() {}
  __device__ __forceinline__ void load(const float* p) { q = *(const word4*)p; }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = q[j];
  }
  __device__ __forceinline__ void put(const float* f) {
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = f[j];
  }
  __device__ __forceinline__ void zero_if(bool cond) {
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = cond ? 0.f : q[j];
  }
  __device__ __forceinline__ void zero_below(int shift) {
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = j >= shift ? q[j] : 0.f;
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
  __device__ __forceinline__ void keep() {}
  __device__ __forceinline__ void load(const T* p) { q = *p; }
  __device__ __forceinline__ void get(float* f) const { f[0] = Elem<T>::to_f32(q); }
  __device__ __forceinline__ void put(const float* f) { q = Elem<T>::from_f32(f[0]); }
  __device__ __forceinline__ void zero_if(bool cond) { q = cond ? T(0) : q; }
  __device__ __forceinline__ void zero_below(int) {}
  static __device__ __forceinline__ void store(T* p, const float* f) { *p = Elem<T>::from_f32(f[0]); }
};

// The same number, of which the compiler no longer knows what it was computed
// from: what each pass derives from it is derived anew and holds no registers
// between the passes.
__device__ __forceinline__ int anew(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Between the rounds of a loop over chunks: the compiler would run unrolled
// rounds into each other until registers spill.
__device__ __forceinline__ void apart() { __builtin_amdgcn_sched_barrier(0); }

// exp(x) as 2^(x log2 e), and 1 / x.  For bf16 results the hardware's
// approximations are enough: the product's rounding costs x 2^-24 of the result.
// fp32 silu takes that rounding back, and one Newton step (the error of its sums
// falls from 2.2e-7 to 1e-7 for two operations in ten more).
// gelu takes the plain exponential in fp32, too: it scales the tail, whose error it
// makes (z^2 + 2) 2^-24 of itself; for z > 0 that is at most 2^-23 of y.
template <typename T> __device__ __forceinline__ float exp_of(float x) {
  const float t = x * 1.44269504f, e = __builtin_amdgcn_exp2f(t);
  if (sizeof(T) == 2) return e;
  // what t lacks: its rounding, and log2 e beyond fp32
  const float r = __builtin_fmaf(x, 1.92596299e-8f, __builtin_fmaf(x, 1.44269504f, -t));
  const float more = e * (r * 0.693147181f);
  return e + (__builtin_fabsf(t) < 127.f ? more : 0.f);  // zeros, infinities and NaN stay
}
template <typename T> __device__ __forceinline__ float inverse_of(float x) {
  const float r = __builtin_amdgcn_rcpf(x);
  if (sizeof(T) == 2) return r;
  const float s = __builtin_fmaf(__builtin_fmaf(-x, r, 1.f), r, r);
  return x < 1e38f ? s : r;  // where x r is no longer near 1
}

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
  if (ACT == DEFT_ACT_SILU) return z * inverse_of<T>(1.f + exp_of<T>(-z));
  if (ACT == DEFT_ACT_GELU) {
    const float q = normal_tail<T>(__builtin_fabsf(z), exp_of<bf16_t>(-0.5f * z * z));
    return z * (z > 0.f ? 1.f - q : q);
  }
  return z;
}
// dy times the activation's slope at z.
template <typename T, int ACT> __device__ __forceinline__ float act_grad(float z, float dy) {
  if (ACT == DEFT_ACT_RELU) return z > 0.f ? dy : 0.f;
  if (ACT == DEFT_ACT_SILU) {
    const float p = inverse_of<T>(1.f + exp_of<T>(-z));
    return dy * (p * __builtin_fmaf(z, 1.f - p, 1.f));
  }
  if (ACT == DEFT_ACT_GELU) {
    const float e = exp_of<bf16_t>(-0.5f * z * z);
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

// v of the lane that differs in bit STEP (within 8 and 16 lanes: that is its
// mirror image, which is as good for sums), by moves that stay in the vector
// unit; through LDS a step takes ten times as long.
template <int STEP> __device__ __forceinline__ uint32_t across(uint32_t v) {
  constexpr int ctrl = STEP == 1 ? 0xB1 : STEP == 2 ? 0x4E : STEP == 4 ? 0x141 : 0x140;
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xf, 0xf, false);
}
template <int STEP> __device__ __forceinline__ float with_across(float v) {
  const uint32_t w = __float_as_uint(v);
  if constexpr (STEP <= 8) return v + __uint_as_float(across<STEP>(w));
  // the swap leaves one row's values in both rows of each result
  const auto p = STEP == 16 ? __builtin_amdgcn_permlane16_swap(w, w, false, false)
                            : __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}
template <int STEP> __device__ __forceinline__ double with_across(double v) {
  const uint64_t w = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)w, hi = (uint32_t)(w >> 32);
  if constexpr (STEP <= 8)
    return v + __builtin_bit_cast(double, (uint64_t)across<STEP>(hi) << 32 | across<STEP>(lo));
  const auto p = STEP == 16 ? __builtin_amdgcn_permlane16_swap(lo, lo, false, false)
                            : __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
  const auto q = STEP == 16 ? __builtin_amdgcn_permlane16_swap(hi, hi, false, false)
                            : __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
  return __builtin_bit_cast(double, (uint64_t)q[0] << 32 | p[0]) +
         __builtin_bit_cast(double, (uint64_t)q[1] << 32 | p[1]);
}
// Sum over aligned teams of `t` lanes (a power of two up to 64), in every lane;
// whole teams call it together.
template <typename F> __device__ __forceinline__ F team_sum(F v, int t) {
  if (t > 1) v = with_across<1>(v);
  if (t > 2) v = with_across<2>(v);
  if (t > 4) v = with_across<4>(v);
  if (t > 8) v = with_across<8>(v);
  if (t > 16) v = with_across<16>(v);
  if (t > 32) v = with_across<32>(v);
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

// The same of two fp64 values at once; `lds` holds two per wave.
__device__ __forceinline__ void block_sums(double& a, double& b, double* lds) {
  a = team_sum(a, 64);
  b = team_sum(b, 64);
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) { lds[2 * wave] = a; lds[2 * wave + 1] = b; }
  __syncthreads();
  a = b = 0.0;
  for (int w = 0; w < (int)(blockDim.x >> 6); ++w) { a += lds[2 * w]; b += lds[2 * w + 1]; }
}

// A team's walk over the entries of one segment, rows by `len` entries: lane l
// of t has the entries l, l + t, ...: f(row, entry).
template <typename F> __device__ __forceinline__ void walk(int l, int t, int rows, int len, F f) {
  int r = l / len, e = l - r * len;
  const int dr = t / len, de = t - dr * len;
  while (r < rows) {
    f(r, e);
    r += dr;
    e += de;
    if (e >= len) { e -= len; ++r; }
  }
}
// Lanes of a team where nseg segments share the workgroup, `most` at most.
__device__ __forceinline__ int team_size(int nseg, int most) {
  const int each = max((int)blockDim.x / nseg, 1);
  return min(1 << (31 - __builtin_clz(each)), most);
}

// Sums of the segments of a matrix in LDS: out(seg, sum over rows r and
// columns j < len of m[r * pitch + seg * len + j]), called by one thread per
// segment.  `pitch` is odd, so that lanes on different rows fall on different
// banks.
template <typename F>
__device__ __forceinline__ void segment_sums(const float* m, int pitch, int rows, int nseg, int len, F out) {
  const int t = team_size(nseg, 64), l = threadIdx.x & (t - 1);
  for (int seg = threadIdx.x / t; seg < nseg; seg += blockDim.x / t) {
    float v = 0.f;
    walk(l, t, rows, len, [&](int r, int e) { v += m[r * pitch + seg * len + e]; });
    v = team_sum(v, t);
    if (l == 0) out(seg, v);
  }
}

// Values that a workgroup needs after its main loads, into LDS as fp32.  They are
// asked for (ctor) before the main loads and stored (put) after those are under
// way: a load that is issued between the statistics and the result finds the
// memory busy, and took 2 to 6 us there.
template <typename T> struct Ahead {
  const T* p;
  int n;
  T v;
  __device__ __forceinline__ Ahead(const void* from, int count) : p((const T*)from), n(count) {
    if ((int)threadIdx.x < n) v = p[threadIdx.x];
  }
  __device__ __forceinline__ void put(float* lds) const {
    if ((int)threadIdx.x < n) lds[threadIdx.x] = Elem<T>::to_f32(v);
    for (int i = threadIdx.x + blockDim.x; i < n; i += blockDim.x) lds[i] = Elem<T>::to_f32(p[i]);
  }
};

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

// ---- Joining the slices of a group that several workgroups hold ----
//
// Each of a cluster's `slices` workgroups (all slices of an image's band, or of
// a group) publishes two floats per group, and each needs all of them.  A word
// is a float beside the call's tag, stored and read whole by relaxed atomics
// of agent scope: a word with the tag is the value, so nothing else has to be
// ordered, and words of earlier calls are told apart without clearing them.
// The tag counts the cluster's calls: a workgroup's ticket, one atomic add on
// a counter that is never reset, divided by the slices.
//
// Workgroups wait for each other only up to a deadline.  One that has waited
// in vain (its peers may not have been started, where other work holds the
// chip) computes the slices that it misses itself: their values have the same
// bits whoever computes them.  So no call depends on how many workgroups are
// resident.  Then all words have been stored, and the last look at them waits
// for the memory only, as long as calls on a workspace that began with zeros
// follow each other.  Where they do not, tags of two calls can replace each
// other for good; so that look has a deadline, too, and what it misses is NaN.
constexpr uint32_t kLastLook = 1000000;  // ticks: 10 ms, where some microseconds are needed
struct Joint {
  uint64_t* part;     // [slices][ng][2]
  uint64_t* total;    // [ng][2], where slices * ng is too much for each to read
  uint32_t tag;
  uint64_t deadline;

  static __device__ __forceinline__ void put(uint64_t* p, float v, uint32_t tag) {
    __hip_atomic_store(p, (uint64_t)tag << 32 | __float_as_uint(v), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __device__ __forceinline__ void publish(int slice, int ng, int g, float a, float b) const {
    uint64_t* p = part + ((size_t)slice * ng + g) * 2;
    put(p, a, tag);
    put(p + 1, b, tag);
  }
  // Both words at p; false if one has not the tag yet.
  __device__ __forceinline__ bool read(const uint64_t* p, float& a, float& b) const {
    const uint64_t u = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint64_t v = __hip_atomic_load(p + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    a = __uint_as_float((uint32_t)u);
    b = __uint_as_float((uint32_t)v);
    return (uint32_t)(u >> 32) == tag && (uint32_t)(v >> 32) == tag;
  }
  // Reads until all are there; false if they were not after the deadline.
  template <typename READ> __device__ __forceinline__ bool wait(READ all) const {
    for (bool late = false; !all(); __builtin_amdgcn_s_sleep(1)) {
      if (late) return false;
      late = __builtin_readsteadycounter() >= deadline;
    }
    return true;
  }
  // f(k, a, b) with the words of group g of the lane's slices lane, lane + 64,
  // ..., four in flight at a time.  The same answer in every lane of the wave.
  template <typename F> __device__ __forceinline__ bool gather(int slices, int ng, int g, F f) const {
    bool ok = true;
    for (int k0 = threadIdx.x & 63; k0 - (int)(threadIdx.x & 63) < slices; k0 += 256) {
      float a[4], b[4];
      ok &= wait([&] {
        bool all = true;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (k0 + 64 * i < slices) all &= read(part + ((size_t)(k0 + 64 * i) * ng + g) * 2, a[i], b[i]);
        return all;
      });
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (k0 + 64 * i < slices) f(k0 + 64 * i, a[i], b[i]);
    }
    return __ballot(!ok) == 0;
  }
  // The next slice after k that is not published for all groups, `slices` if
  // there is none.  The same answer in every thread of the workgroup.
  __device__ __forceinline__ int next(int k, int slices, int ng) const {
    while (++k < slices) {
      int ok = 1;
      for (int i = threadIdx.x; i < 2 * ng; i += blockDim.x) {
        const uint64_t u =
            __hip_atomic_load(part + (size_t)k * ng * 2 + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        ok &= (uint32_t)(u >> 32) == tag;
      }
      if (!__syncthreads_and(ok)) break;
    }
    __syncthreads();  // what LDS holds of the last slice has been read
    return k;
  }
};

// The cluster's tag for this call; one thread's work.
__device__ __forceinline__ uint32_t joint_tag(uint64_t* counter, int slices) {
  const uint64_t t = __hip_atomic_fetch_add(counter, 1ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return (uint32_t)(t / (uint32_t)slices) + 1;
}

}  // namespace deft
