// The end of a training step over a list of tensors: the norm of all gradients
// with its clipping factor, and AdamW with 32-bit or 8-bit states.
//
// AdamW at step t, element by element:
//   g  = coef * grad
//   m' = b1 m + (1 - b1) g
//   v' = b2 v + (1 - b2) g^2
//   p' = (1 - lr wd) p - lr / (1 - b1^t) * m' / (sqrt(v') / sqrt(1 - b2^t) + eps)
// Every operation is one IEEE fp32 operation in this order (no contraction
// into fused multiply-adds), so a step gives the same bits wherever an
// element lies, and the same as the formulas written out in fp32.
//
// 8-bit states hold e4m3 codes and one fp32 scale for each 256 consecutive
// elements of a tensor: m = code * scale, and for v its root, sqrt(v) = code *
// scale, which halves the exponent range v needs.  scale = max / 448, the
// largest code, so a block spans 2^-17.8 of its maximum.  m is rounded to
// nearest: a step changes it by a tenth.  A step changes sqrt(v) by 0.05 % at
// most where it decays, far below half a code step (3-6 %), so rounding to
// nearest would never let it move: it is rounded stochastically (unbiased) by
// 16 bits of a hash of the call's seed, the tensor's number and the element.
// What is not zero keeps at least the least code, so no element divides by a
// root that rounding made zero.  A block that holds a NaN or an infinity gets
// the scale NaN and zero codes.
#include "deft_device.h"
#include "deft_internal.h"

namespace deft {

namespace {

constexpr int kThreads = kAdamwThreads;
constexpr int kPer = 4;                       // consecutive elements per lane: one wave covers a scale's 256
constexpr int kWaveElems = 64 * kPer;
constexpr float kCodeMax = 448.f;             // largest e4m3 value
constexpr float kTiny = 1.17549435e-38f;      // 2^-126: a smaller scale's inverse may overflow
static_assert(kWaveElems == kStateBlock, "one wave per scale");

// Number of the tensor whose workgroups (pieces) hold `block`: each lane has the
// first one of its tensor, in ascending order, or no tensor (count <= 64).
__device__ __forceinline__ int tensor_of(bool mine, uint32_t first, uint32_t block) {
  return __builtin_amdgcn_readfirstlane(__popcll(__ballot(mine && first <= block)) - 1);
}

// Four consecutive elements from i on; zeros past n.  ONCE: the data are not
// asked for again before they have left the caches (nontemporal accesses).
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
template <bool ONCE, typename W> __device__ __forceinline__ W get(const W* p) {
  return ONCE ? __builtin_nontemporal_load(p) : *p;
}
template <bool ONCE, typename W> __device__ __forceinline__ void put(W* p, W w) {
  if (ONCE) __builtin_nontemporal_store(w, p);
  else *p = w;
}
template <bool ONCE>
__device__ __forceinline__ void load4(const float* __restrict__ p, int64_t i, int64_t n, float* f) {
  if (i + 4 <= n) {
    const f32x4 q = get<ONCE>((const f32x4*)(p + i));
    f[0] = q.x; f[1] = q.y; f[2] = q.z; f[3] = q.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = i + k < n ? p[i + k] : 0.f;
  }
}
template <bool ONCE>
__device__ __forceinline__ void load4(const bf16_t* __restrict__ p, int64_t i, int64_t n, float* f) {
  if (i + 4 <= n) {
    const u32x2 q = get<ONCE>((const u32x2*)(p + i));
    f[0] = bf16_lo(q.x); f[1] = bf16_hi(q.x); f[2] = bf16_lo(q.y); f[3] = bf16_hi(q.y);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = i + k < n ? bf16_to_f32(p[i + k]) : 0.f;
  }
}
template <bool ONCE>
__device__ __forceinline__ void store4(float* __restrict__ p, int64_t i, int64_t n, const float* f) {
  if (i + 4 <= n) {
    put<ONCE>((f32x4*)(p + i), f32x4{f[0], f[1], f[2], f[3]});
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < n) p[i + k] = f[k];
  }
}
template <bool ONCE>
__device__ __forceinline__ void store4(bf16_t* __restrict__ p, int64_t i, int64_t n, const float* f) {
  if (i + 4 <= n) {
    put<ONCE>((u32x2*)(p + i), u32x2{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3])});
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < n) p[i + k] = f32_to_bf16(f[k]);
  }
}
// Four e4m3 codes as one word.
template <bool ONCE>
__device__ __forceinline__ uint32_t load_codes(const uint8_t* __restrict__ p, int64_t i, int64_t n) {
  if (i + 4 <= n) return get<ONCE>((const uint32_t*)(p + i));
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (i + k < n) w |= (uint32_t)p[i + k] << (8 * k);
  return w;
}
template <bool ONCE>
__device__ __forceinline__ void store_codes(uint8_t* __restrict__ p, int64_t i, int64_t n, uint32_t w) {
  if (i + 4 <= n) {
    put<ONCE>((uint32_t*)(p + i), w);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < n) p[i + k] = (uint8_t)(w >> (8 * k));
  }
}
__device__ __forceinline__ void decode4(uint32_t w, float* f) {
  f[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0); f[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1);
  f[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2); f[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3);
}
// To nearest even; |f| <= 448.
__device__ __forceinline__ uint32_t encode4(const float* f) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], w, true);
}

// Largest of the wave's values, in every lane.  Bit patterns of non-negative
// floats: an infinity beats every number and a NaN beats an infinity.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
  const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xf, false);
  return x > y ? x : y;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = dpp_max<0x111, 0xf>(x);  // row_shr 1, 2, 4, 8: lane 15 of each row has the row's
  x = dpp_max<0x112, 0xf>(x);
  x = dpp_max<0x114, 0xf>(x);
  x = dpp_max<0x118, 0xf>(x);
  x = dpp_max<0x142, 0xa>(x);  // row_bcast 15, 31: lane 63 has the wave's
  x = dpp_max<0x143, 0xc>(x);
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

struct Scale {
  float s, inv;  // inv 0: all codes zero
};
__device__ __forceinline__ Scale block_scale(uint32_t most) {
  Scale r;
  if (most >= 0x7f800000u) {  // a NaN or an infinity
    r.s = __uint_as_float(0x7fc00000u);
    r.inv = 0.f;
    return r;
  }
  const float s = __uint_as_float(most) / kCodeMax;
  r.s = s >= kTiny ? s : 0.f;
  r.inv = s >= kTiny ? 1.0f / s : 0.f;
  return r;
}

__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0xBB67AE85u;
  x ^= x >> 15;
  x *= 0x6A09E667u;
  return x ^ (x >> 16);
}

// t in [0, 448] to the e4m3 grid, up with the probability of what is cut off.
// Normal codes keep 3 of the 23 fraction bits: the random number is added
// below them; under 2^-6 the codes lie 2^-9 apart.
__device__ __forceinline__ float round_random(float t, uint32_t u16) {
#pragma clang fp contract(off)
  const float normal = __uint_as_float((__float_as_uint(t) + (u16 * 16u + 8u)) & 0xfff00000u);
  float small = floorf(t * 512.f + ((float)u16 + 0.5f) * 0x1p-16f) * 0x1p-9f;
  small = t > 0.f ? fmaxf(small, 0x1p-9f) : small;
  return t < 0x1p-6f ? small : normal;
}

struct Rates {
  float b1, c1, b2, c2, eps;  // c = 1 - b
  float rate, low;            // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
};

// One element; m, v and p are updated.
__device__ __forceinline__ void adamw(float g, float& m, float& v, float& root, float& p, float decay,
                                      const Rates& r) {
#pragma clang fp contract(off)
  m = m * r.b1 + g * r.c1;
  v = v * r.b2 + (g * g) * r.c2;
  root = __builtin_sqrtf(v);
  p = p * decay - (m / (root * r.low + r.eps)) * r.rate;
}

// Where steps were skipped: the number of a call's step among those taken, the
// corrections of such a step, and those of the next call, by one thread.
__device__ __forceinline__ uint32_t taken_by(int64_t step, uint32_t skipped) {
  return step > skipped ? (uint32_t)(step - skipped) : 1;
}
__device__ __forceinline__ AdamwSkips::Next correction(const AdamwArgs& a, uint32_t taken) {
  AdamwSkips::Next r;
  r.inverse = 1.0 / (1.0 - exp2((double)taken * a.log1));
  r.low = (float)(1.0 / sqrt(1.0 - exp2((double)taken * a.log2)));
  r.taken = taken;
  return r;
}
__device__ __forceinline__ void correct_next(const AdamwArgs& a, uint32_t skipped) {
  a.skips->next[(a.step + 1) & 1] = correction(a, taken_by(a.step + 1, skipped));
}

}  // namespace

// P: weights' type, G: gradients', BITS: states', MASTER: fp32 masters beside bf16 weights.
//
// Bound by memory: 16.06 bytes an element with bf16 weights, masters and 8-bit
// states.  77 M elements take 240 us, 5.1 TB/s as a copy does, and 225 to 230
// with nontemporal accesses (ONCE); 5 M elements, 141 MB, stay in the caches from
// one step to the next and take 31 us against 34.
template <typename P, typename G, int BITS, bool MASTER, bool ONCE>
__global__ __launch_bounds__(kThreads) void k_adamw(const AdamwArgs a) {
#pragma clang fp contract(off)
  AdamwSkips* const skips = a.skips;
  float coef = 1.f, finite = 1.f;
  uint32_t skipped = 0;
  if (a.control && skips) {  // one wait for both
    coef = a.control[1];
    finite = a.control[2];
    skipped = skips->count;
  } else if (a.control) {
    coef = a.control[1];
    finite = a.control[2];
  } else if (skips) {
    skipped = skips->count;
  }
  const bool lead = a.lead && blockIdx.x == 0 && threadIdx.x == 0;
  if (finite == 0.f) {  // the step is counted, and nothing else is written
    if (skips && lead) {
      skips->count = skipped + 1;
      correct_next(a, skipped + 1);
    }
    return;
  }
  const int lane = threadIdx.x & 63;
  const int ti = tensor_of(lane < a.count, lane < a.count ? a.first[lane] : 0, blockIdx.x);
  const AdamwTensor& t = a.t[ti];
  const int64_t n = t.n;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t i0 = ((int64_t)(blockIdx.x - a.first[ti]) * (kThreads / 64) + wave) * kWaveElems;
  if (i0 >= n) return;
  const int64_t i = i0 + lane * kPer;
  Rates r{a.b1, a.c1, a.b2, a.c2, a.eps, a.rate, a.low};
  float decay = (float)t.decay;
  uint32_t seed = a.seed;
  if (a.schedule) {
    const double lr = a.schedule[0];
    r.rate = (float)(lr / a.schedule[1]);
    r.low = (float)(1.0 / sqrt(a.schedule[2]));
    decay = (float)(1.0 - lr * t.decay);
    seed = (uint32_t)(int64_t)a.schedule[3];
  } else if (skipped) {
    AdamwSkips::Next now = skips->next[a.step & 1];
    // not what the last call left where it was captured, and is replayed with one number
    if (now.taken != taken_by(a.step, skipped)) now = correction(a, taken_by(a.step, skipped));
    r.rate = (float)(a.lr * now.inverse);
    r.low = now.low;
    if (lead) correct_next(a, skipped);
  }
  float g[4], p[4], m[4], v[4], root[4];
  load4<ONCE>((const G*)t.g, i, n, g);
  if (MASTER) load4<ONCE>((const float*)t.master, i, n, p);
  else load4<ONCE>((const P*)t.p, i, n, p);
  if (BITS == 32) {
    load4<ONCE>((const float*)t.m, i, n, m);
    load4<ONCE>((const float*)t.v, i, n, v);
  } else {
    const uint32_t mw = load_codes<ONCE>((const uint8_t*)t.m, i, n), vw = load_codes<ONCE>((const uint8_t*)t.v, i, n);
    const float ms = t.m_scale[i0 / kStateBlock], vs = t.v_scale[i0 / kStateBlock];
    decode4(mw, m);
    decode4(vw, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      m[k] = m[k] * ms;
      v[k] = v[k] * vs;
      v[k] = v[k] * v[k];
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (a.control) g[k] = g[k] * coef;
    adamw(g[k], m[k], v[k], root[k], p[k], decay, r);
  }
  if (MASTER) store4<ONCE>(t.master, i, n, p);
  store4<ONCE>((P*)t.p, i, n, p);
  if (BITS == 32) {
    store4<ONCE>((float*)t.m, i, n, m);
    store4<ONCE>((float*)t.v, i, n, v);
    return;
  }
  // lanes past n hold zeros throughout
  uint32_t mm = 0, vm = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t x = __float_as_uint(m[k]) & 0x7fffffffu, y = __float_as_uint(root[k]) & 0x7fffffffu;
    mm = x > mm ? x : mm;
    vm = y > vm ? y : vm;
  }
  const Scale sm = block_scale(wave_max(mm)), sv = block_scale(wave_max(vm));
  const uint32_t key = mix(seed + a.id[ti] * 0x3C6EF373u);
  const uint32_t pair = (uint32_t)(i >> 1);
  const uint32_t h[2] = {mix(pair * 0x6A09E667u + key), mix((pair + 1) * 0x6A09E667u + key)};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float tm = sm.inv > 0.f ? m[k] * sm.inv : 0.f;
    m[k] = fminf(fmaxf(tm, -kCodeMax), kCodeMax);
    const float tv = sv.inv > 0.f ? fminf(root[k] * sv.inv, kCodeMax) : 0.f;
    v[k] = round_random(tv, (k & 1) ? h[k >> 1] >> 16 : h[k >> 1] & 0xffffu);
  }
  store_codes<ONCE>((uint8_t*)t.m, i, n, encode4(m));
  store_codes<ONCE>((uint8_t*)t.v, i, n, encode4(v));
  if (lane == 0) {
    t.m_scale[i0 / kStateBlock] = sm.s;
    t.v_scale[i0 / kStateBlock] = sv.s;
  }
}

// Sum of one workgroup's values (fp64, fixed order), in every thread.
__device__ __forceinline__ double group_sum(double x, double* lds) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  double r = 0.0;
#pragma unroll
  for (int w = 0; w < kSquareThreads / 64; ++w) r += lds[w];
  return r;
}

// 16 bytes as fp64 squares, added to sum in order.
__device__ __forceinline__ double add_squares(const float4 q, double sum, float) {
  sum = __builtin_fma((double)q.x, (double)q.x, sum);
  sum = __builtin_fma((double)q.y, (double)q.y, sum);
  sum = __builtin_fma((double)q.z, (double)q.z, sum);
  return __builtin_fma((double)q.w, (double)q.w, sum);
}
__device__ __forceinline__ double add_squares(const float4 q, double sum, bf16_t) {
  float f[8];
  unpack8(__builtin_bit_cast(uint4, q), f);
#pragma unroll
  for (int k = 0; k < 8; ++k) sum = __builtin_fma((double)f[k], (double)f[k], sum);
  return sum;
}

// Norm of all gradients and the factor that clips them.  Each workgroup sums the
// squares of its pieces in fp64 (squares of fp32 values neither overflow nor
// vanish there) and the last one that stores its sum adds all up, in their order,
// and writes control = {norm, factor, finite, 0}; so the bits do not depend on
// which is the last.
//
// Bound by reading: a piece's loads are all in flight before the first is used.
// One large workgroup on each compute unit, for the counting at the end is one
// after the other (10 ns each; with 1024 workgroups of 256 threads 77 M elements
// in bf16 took 37 us).
template <typename G>
__global__ __launch_bounds__(kSquareThreads) void k_grad_norm(const GradNormArgs a) {
  __shared__ double lds[kSquareThreads / 64];
  __shared__ int last;
  constexpr int kVec = 16 / sizeof(G), kLoads = kNormPiece / (kSquareThreads * kVec);
  const int lane = threadIdx.x & 63;
  const bool mine = lane < a.count;
  const uint32_t first = mine ? a.first[lane] : 0;
  double sum = 0.0;
  for (uint32_t b = blockIdx.x; b < a.pieces; b += gridDim.x) {
    const int ti = tensor_of(mine, first, b);
    const G* g = (const G*)a.g[ti];
    const int64_t i0 = (int64_t)(b - a.first[ti]) * kNormPiece, n = a.n[ti];
    if (i0 + kNormPiece <= n) {
      const float4* p = (const float4*)(g + i0) + threadIdx.x;
      float4 q[kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) q[u] = p[u * kSquareThreads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) sum = add_squares(q[u], sum, G());
    } else {
      for (int64_t i = i0 + threadIdx.x * 4; i < n; i += kSquareThreads * 4) {
        float f[4];
        load4<false>(g, i, n, f);
#pragma unroll
        for (int k = 0; k < 4; ++k) sum = __builtin_fma((double)f[k], (double)f[k], sum);
      }
    }
  }
  const double total = group_sum(sum, lds);
  if (threadIdx.x == 0) {
    __hip_atomic_store(a.partials + a.at + blockIdx.x, total, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // it has arrived before this workgroup is counted
    const uint64_t t = __hip_atomic_fetch_add(a.arrived, 1ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    last = t + 1 == a.sums;
    if (last) __hip_atomic_store(a.arrived, 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!last) return;
  sum = 0.0;
#pragma unroll 4
  for (uint32_t i = threadIdx.x; i < a.sums; i += kSquareThreads)
    sum += __hip_atomic_load(a.partials + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const double all = group_sum(sum, lds);
  if (threadIdx.x == 0) {
    const double norm = sqrt(all) * a.inv_scale;
    const bool finite = norm < __builtin_inf();
    double f = 1.0;
    if (a.max_norm < __builtin_inf()) f = fmin(1.0, a.max_norm / (norm + 1e-6));
    a.control[0] = (float)norm;
    a.control[1] = finite ? (float)(a.inv_scale * f) : 0.f;
    a.control[2] = finite ? 1.f : 0.f;
    a.control[3] = 0.f;
  }
}

hipError_t launch_adamw(const AdamwArgs& a, uint32_t blocks, int p_dtype, int g_dtype, int bits, bool master,
                        bool once, hipStream_t st) {
  const dim3 grid(blocks), block(kThreads);
#define DEFT_ADAMW(P, G, B, M)                                                             \
  do {                                                                                     \
    if (once) DEFT_LAUNCH("adamw", (k_adamw<P, G, B, M, true>), grid, block, 0, st, a);    \
    else DEFT_LAUNCH("adamw", (k_adamw<P, G, B, M, false>), grid, block, 0, st, a);        \
  } while (0)
#define DEFT_ADAMW_BITS(P, G, M)                                       \
  do {                                                                 \
    if (bits == 8) DEFT_ADAMW(P, G, 8, M);                             \
    else DEFT_ADAMW(P, G, 32, M);                                      \
  } while (0)
  const bool gb = g_dtype == DEFT_BF16;
  if (p_dtype == DEFT_F32) {
    if (gb) DEFT_ADAMW_BITS(float, bf16_t, false);
    else DEFT_ADAMW_BITS(float, float, false);
  } else if (master) {
    if (gb) DEFT_ADAMW_BITS(bf16_t, bf16_t, true);
    else DEFT_ADAMW_BITS(bf16_t, float, true);
  } else {
    if (gb) DEFT_ADAMW_BITS(bf16_t, bf16_t, false);
    else DEFT_ADAMW_BITS(bf16_t, float, false);
  }
#undef DEFT_ADAMW_BITS
#undef DEFT_ADAMW
  return hipGetLastError();
}

hipError_t launch_grad_norm(const GradNormArgs& a, int g_dtype, uint32_t grid, hipStream_t st) {
  if (g_dtype == DEFT_BF16) DEFT_LAUNCH("grad_norm", k_grad_norm<bf16_t>, dim3(grid), dim3(kSquareThreads), 0, st, a);
  else DEFT_LAUNCH("grad_norm", k_grad_norm<float>, dim3(grid), dim3(kSquareThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace deft
