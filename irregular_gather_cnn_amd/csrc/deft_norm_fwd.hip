// Group norm with activation, forward: y = act(gamma (x - mean) rstd + beta).
//
// A workgroup holds its slice of a group (or of a band of groups) in
// registers, so x is read once: the sum gives the mean, a second pass over the
// registers the squares about it, which loses nothing where the mean is far
// from zero, a third the result.
#include "deft_norm.h"

namespace deft {

namespace {

// Channels last: slice k of band b of image n, blocks in the order ((n, k), b),
// so that the workgroups of one XCD share the lines of neighbouring bands.
// part: [n][g][slices]{mean, M2}.
template <typename T, int V, int U, int MODE>
__global__ __launch_bounds__(kNormThreads) void k_norm_fwd_last(const NormArgs a) {
  extern __shared__ float lds[];
  const int id = xcd_swizzle(blockIdx.x, gridDim.x);
  const int b = id % a.bands, nk = id / a.bands, k = nk % a.slices, n = nk / a.slices;
  Band w;
  w.set<V>(b, a.bands, a.g, a.per);
  const int r0 = k * a.rp, rows = min(a.rp, a.s - r0);
  const int rounds = (rows + w.TY - 1) / w.TY;
  const int mine = w.ty < w.TY ? (rows - w.ty + w.TY - 1) / w.TY : 0;
  const size_t at = ((size_t)n * a.s + r0 + w.ty) * a.c + w.col, step = (size_t)w.TY * a.c;
  const T* xp = (const T*)a.x + at;
  Chunk<T, V> q[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u < mine) q[u].load(xp + u * step);
    else q[u].zero();
  }
  float* gm = lds;                // means of the band's groups
  float* gr = gm + w.ng;          // 1 / std
  float* red = gr + w.ng;         // [TY][pitch]
  float mu[V];
  const int per = a.per, ng0 = n * a.g + w.g0;
  int gi[V];
  {
    int i = w.col / per, r = w.col - i * per;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      gi[j] = i - w.g0;
      if (++r == per) { r = 0; ++i; }
    }
  }
  if (MODE != kNormApply) {
    // where a chunk lies in one group its elements are added up before LDS
    const bool solid = w.ng == 1 || per % V == 0;
    const int pitch = (solid ? w.cx : w.cols) | 1, len = solid ? (w.ng == 1 ? w.cx : per / V) : per;
    const float count = (float)rows * (float)per;
    auto spill = [&](const float* acc) {
      if (w.ty < w.TY) {
        if (solid) {
          float v = 0.f;
#pragma unroll
          for (int j = 0; j < V; ++j) v += j >= w.shift ? acc[j] : 0.f;
          red[w.ty * pitch + w.tx] = v;
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (j >= w.shift) red[w.ty * pitch + (w.col - w.c0) + j] = acc[j];
        }
      }
      __syncthreads();
    };
    float acc[V] = {};
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u < rounds) {
        float f[V];
        q[u].get(f);
  #pragma unroll
        for (int j = 0; j < V; ++j) acc[j] += f[j];
      }
    }
    spill(acc);
    segment_sums(red, pitch, w.TY, w.ng, len, [&](int seg, float v) { gm[seg] = v / count; });
    __syncthreads();
#pragma unroll
    for (int j = 0; j < V; ++j) { mu[j] = gm[gi[j]]; acc[j] = 0.f; }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u < rounds) {
        if (u < mine) {
          float f[V];
          q[u].get(f);
  #pragma unroll
          for (int j = 0; j < V; ++j) acc[j] = __builtin_fmaf(f[j] - mu[j], f[j] - mu[j], acc[j]);
        }
      }
    }
    spill(acc);
    segment_sums(red, pitch, w.TY, w.ng, len, [&](int seg, float v) {
      if (MODE == kNormStats) {
        float2* p = (float2*)a.part + (size_t)(ng0 + seg) * a.slices + k;
        *p = make_float2(gm[seg], v);
      } else {
        const float rstd = 1.f / __builtin_sqrtf(v / count + a.eps);
        gr[seg] = rstd;
        a.mean[ng0 + seg] = gm[seg];
        a.rstd[ng0 + seg] = rstd;
      }
    });
    if (MODE == kNormStats) return;
  } else {
    for (int i = threadIdx.x; i < w.ng; i += blockDim.x) {
      gm[i] = a.mean[ng0 + i];
      gr[i] = a.rstd[ng0 + i];
    }
  }
  __syncthreads();
  if (w.ty >= w.TY) return;
  float ga[V], be[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    mu[j] = gm[gi[j]];
    ga[j] = Elem<T>::to_f32(((const T*)a.gamma)[w.col + j]) * gr[gi[j]];
    be[j] = Elem<T>::to_f32(((const T*)a.beta)[w.col + j]);
  }
  T* yp = (T*)a.out + at;
  with_act(a.act, [&](auto act) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u < mine) {
        float f[V];
        q[u].get(f);
#pragma unroll
        for (int j = 0; j < V; ++j)
          f[j] = act_of<T, decltype(act)::value>(__builtin_fmaf(f[j] - mu[j], ga[j], be[j]));
        Chunk<T, V>::store(yp + u * step, f);
      }
    }
  });
}

// Channels first: slice (kr, ks) of a group of an image: channels kr * rp ...,
// positions ks * cp ....  Teams of 2^lt lanes walk a channel's positions.
// part: [n][g][slices]{mean, M2}.
template <typename T, int V, int U, int MODE>
__global__ __launch_bounds__(kNormThreads) void k_norm_fwd_first(const NormArgs a) {
  extern __shared__ float lds[];
  const int id = xcd_swizzle(blockIdx.x, gridDim.x);
  const int k = id % a.slices, ng = id / a.slices, g = ng % a.g;
  const int kr = k / a.ws, ks = k - kr * a.ws;
  const int r0 = kr * a.rp, rows = min(a.rp, a.per - r0);
  const int c0 = ks * a.cp, cols = min(a.cp, a.s - c0);
  const int t = 1 << a.lt, ln = threadIdx.x & (t - 1), tm = threadIdx.x >> a.lt, teams = blockDim.x >> a.lt;
  const int chunks = (cols + V - 1) / V, ic = (chunks + t - 1) >> a.lt;
  const int rounds = (rows + teams - 1) / teams * ic;
  const size_t base = ((size_t)ng * a.per + r0) * a.s;
  const T* xp = (const T*)a.x + base;
  float* gam = lds + 8;
  float* bet = gam + rows;
  if (MODE != kNormStats) {
    for (int i = threadIdx.x; i < rows; i += blockDim.x) {
      gam[i] = Elem<T>::to_f32(((const T*)a.gamma)[g * a.per + r0 + i]);
      bet[i] = Elem<T>::to_f32(((const T*)a.beta)[g * a.per + r0 + i]);
    }
  }
  // round u: channel tm + teams * (u / ic), chunk ln + t * (u % ic); a ragged
  // row's last chunk starts early enough to end with the row
  auto slot = [&](int row, int i, int& pos, int& shift) {
    const int want = c0 + i * V;
    pos = want + V <= a.s ? want : a.s - V;  // s >= V
    shift = want - pos;
    return row < rows && i < chunks;
  };
  Chunk<T, V> q[U];
  {
    int row = tm, i = ln;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int pos, shift;
      const bool ok = slot(row, i, pos, shift);
      if (u < rounds && ok) q[u].load(xp + (size_t)row * a.s + pos);
      else q[u].zero();
      i += t;
      if (i - ln >= ic * t) { i = ln; row += teams; }
    }
  }
  const bool ragged = a.s % V != 0;
  float mean, rstd;
  if (MODE != kNormApply) {
    const float count = (float)rows * (float)cols;
    float sum = 0.f;
    int row = tm, i = ln;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u < rounds) {
        float f[V];
        q[u].get(f);
        if (ragged) {
          int pos, shift;
          slot(row, i, pos, shift);
  #pragma unroll
          for (int j = 0; j < V; ++j) f[j] = j >= shift ? f[j] : 0.f;
          i += t;
          if (i - ln >= ic * t) { i = ln; row += teams; }
        }
  #pragma unroll
        for (int j = 0; j < V; ++j) sum += f[j];
      }
    }
    mean = block_sum(sum, lds) / count;
    __syncthreads();
    float m2 = 0.f;
    row = tm, i = ln;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u < rounds) {
        int pos, shift;
        const bool ok = slot(row, i, pos, shift);
        i += t;
        if (i - ln >= ic * t) { i = ln; row += teams; }
        if (ok) {
          float f[V];
          q[u].get(f);
  #pragma unroll
          for (int j = 0; j < V; ++j) {
            const float d = !ragged || j >= shift ? f[j] - mean : 0.f;
            m2 = __builtin_fmaf(d, d, m2);
          }
        }
      }
    }
    m2 = block_sum(m2, lds);
    if (MODE == kNormStats) {
      if (threadIdx.x == 0) ((float2*)a.part)[(size_t)ng * a.slices + k] = make_float2(mean, m2);
      return;
    }
    rstd = 1.f / __builtin_sqrtf(m2 / count + a.eps);
    if (threadIdx.x == 0) {
      a.mean[ng] = mean;
      a.rstd[ng] = rstd;
    }
  } else {
    mean = a.mean[ng];
    rstd = a.rstd[ng];
    __syncthreads();
  }
  T* yp = (T*)a.out + base;
  with_act(a.act, [&](auto act) {
    int row = tm, i = ln;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int pos, shift;
      const bool ok = slot(row, i, pos, shift);
      if (u < rounds && ok) {
        const float ga = gam[row] * rstd, be = bet[row];
        float f[V];
        q[u].get(f);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = act_of<T, decltype(act)::value>(__builtin_fmaf(f[j] - mean, ga, be));
        Chunk<T, V>::store(yp + (size_t)row * a.s + pos, f);
      }
      i += t;
      if (i - ln >= ic * t) { i = ln; row += teams; }
    }
  });
}

// Elements of a group in slice k.
__device__ __forceinline__ float slice_count(const NormArgs& a, int layout, int k) {
  if (layout == DEFT_CHANNELS_LAST) return (float)min(a.rp, a.s - k * a.rp) * (float)a.per;
  const int kr = k / a.ws, ks = k - kr * a.ws;
  return (float)min(a.rp, a.per - kr * a.rp) * (float)min(a.cp, a.s - ks * a.cp);
}

// mean and rstd of each group of each image from its slices: a wave per group.
__global__ __launch_bounds__(64) void k_norm_combine(const NormArgs a, int layout) {
  const int ng = blockIdx.x, lane = threadIdx.x;
  const float2* p = (const float2*)a.part + (size_t)ng * a.slices;
  const float count = (float)a.s * (float)a.per;
  float v = 0.f;
  for (int k = lane; k < a.slices; k += 64) v += p[k].x * slice_count(a, layout, k);
  const float mean = team_sum(v, 64) / count;
  v = 0.f;
  for (int k = lane; k < a.slices; k += 64) {
    const float d = p[k].x - mean;
    v += __builtin_fmaf(d * d, slice_count(a, layout, k), p[k].y);
  }
  v = team_sum(v, 64);
  if (lane == 0) {
    a.mean[ng] = mean;
    a.rstd[ng] = 1.f / __builtin_sqrtf(v / count + a.eps);
  }
}

template <typename T, int V, int U>
hipError_t launch(const NormArgs& a, const NormPlan& p, int layout, int mode, hipStream_t st) {
  const dim3 grid(p.blocks), block(p.threads);
#define DEFT_NORM(M)                                                                                           \
  do {                                                                                                         \
    if (layout == DEFT_CHANNELS_LAST) DEFT_LAUNCH("norm_fwd", (k_norm_fwd_last<T, V, U, M>), grid, block, p.lds, st, a); \
    else DEFT_LAUNCH("norm_fwd", (k_norm_fwd_first<T, V, U, M>), grid, block, p.lds, st, a);                   \
  } while (0)
  if (mode == kNormWhole) DEFT_NORM(kNormWhole);
  else if (mode == kNormStats) DEFT_NORM(kNormStats);
  else DEFT_NORM(kNormApply);
#undef DEFT_NORM
  return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const NormArgs& a, const NormPlan& p, int layout, int mode, hipStream_t st) {
  constexpr int V = Elem<T>::VEC;
  if (p.vec == 1) return launch<T, 1, 16>(a, p, layout, mode, st);
  if (p.u <= 4) return launch<T, V, 4>(a, p, layout, mode, st);
  if (p.u <= 8) return launch<T, V, 8>(a, p, layout, mode, st);
  return launch<T, V, 16>(a, p, layout, mode, st);
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs& a, const NormPlan& p, int layout, int dtype, int mode, hipStream_t st) {
  if (p.u > 16) return hipErrorInvalidValue;
  return dtype == DEFT_BF16 ? launch_t<bf16_t>(a, p, layout, mode, st) : launch_t<float>(a, p, layout, mode, st);
}

hipError_t launch_norm_combine(const NormArgs& a, int layout, hipStream_t st) {
  DEFT_LAUNCH("norm_combine", k_norm_combine, dim3((unsigned)(a.n * a.g)), dim3(64), 0, st, a, layout);
  return hipGetLastError();
}

}  // namespace deft
