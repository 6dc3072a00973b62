// Group norm with activation, backward.
//
// With d = x - mean, dz = dy act'(gamma d rstd + beta), per channel of an image
//   A = sum dz,  B = rstd sum dz d
// (dbeta and dgamma are their sums over the images), and per group of m elements
//   S1 = sum_channels gamma A,  S2 = sum_channels gamma B
//   dx = rstd gamma dz - rstd S1 / m - d rstd^2 S2 / m.
// So one reduction, over each channel's positions, serves all three gradients.
// A workgroup holds its slice of x and dy in registers and reads them once;
// what it keeps is as read, and dz is computed for the sums and again for dx.
#include "deft_norm.h"

namespace deft {

namespace {

// Channels last.  part: [n][slices][2][c], A and B of each slice.
template <typename T, int V, int U, int MODE>
__global__ __launch_bounds__(kNormThreads) void k_norm_bwd_last(const NormArgs a) {
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
  const T* yp = (const T*)a.dy + at;
  Chunk<T, V> q[U], h[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u < mine) {
      q[u].load(xp + u * step);
      h[u].load(yp + u * step);
    } else {
      q[u].zero();
      h[u].zero();
    }
  }
  const int per = a.per, ng0 = n * a.g + w.g0;
  float mu[V], rs[V], ga[V], be[V];
  int gi[V];
  {
    int i = w.col / per, r = w.col - i * per;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      gi[j] = i - w.g0;
      mu[j] = a.mean[n * a.g + i];
      rs[j] = a.rstd[n * a.g + i];
      ga[j] = Elem<T>::to_f32(((const T*)a.gamma)[w.col + j]) * rs[j];
      be[j] = Elem<T>::to_f32(((const T*)a.beta)[w.col + j]);
      if (++r == per) { r = 0; ++i; }
    }
  }
  float* s1 = lds;              // the band's groups
  float* s2 = s1 + w.ng;
  float* ca = s2 + w.ng;        // its columns: gamma A, gamma B
  float* cb = ca + w.cols;
  const int pitch = w.cols | 1;
  float* ra = cb + w.cols;      // [TY][pitch]
  float* rb = ra + w.TY * pitch;
  if (MODE != kNormApply) {
    float sa[V] = {}, sb[V] = {};
    with_act(a.act, [&](auto act) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u < rounds) {
          // a row past the end holds dy = 0
          float f[V], g[V];
          q[u].get(f);
          h[u].get(g);
  #pragma unroll
          for (int j = 0; j < V; ++j) {
            const float d = f[j] - mu[j];
            const float dz = act_grad<T, decltype(act)::value>(__builtin_fmaf(d, ga[j], be[j]), g[j]);
            sa[j] += dz;
            sb[j] = __builtin_fmaf(dz, d, sb[j]);
          }
        }
      }
    });
    if (w.ty < w.TY) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (j >= w.shift) {
          ra[w.ty * pitch + (w.col - w.c0) + j] = mine > 0 ? sa[j] : 0.f;
          rb[w.ty * pitch + (w.col - w.c0) + j] = mine > 0 ? sb[j] : 0.f;
        }
      }
    }
    __syncthreads();
    float* out = a.part + ((size_t)n * a.slices + k) * 2 * a.c + w.c0;
    segment_sums(ra, pitch, w.TY, w.cols, 1, [&](int col, float v) {
      out[col] = v;
      ca[col] = v * Elem<T>::to_f32(((const T*)a.gamma)[w.c0 + col]);
    });
    segment_sums(rb, pitch, w.TY, w.cols, 1, [&](int col, float v) {
      v *= a.rstd[n * a.g + (w.c0 + col) / per];
      out[a.c + col] = v;
      cb[col] = v * Elem<T>::to_f32(((const T*)a.gamma)[w.c0 + col]);
    });
    if (MODE == kNormStats) return;
    __syncthreads();
    segment_sums(ca, 0, 1, w.ng, per, [&](int seg, float v) { s1[seg] = v; });
    segment_sums(cb, 0, 1, w.ng, per, [&](int seg, float v) { s2[seg] = v; });
  } else {
    for (int i = threadIdx.x; i < w.ng; i += blockDim.x) {
      s1[i] = a.sums[2 * (size_t)(ng0 + i)];
      s2[i] = a.sums[2 * (size_t)(ng0 + i) + 1];
    }
  }
  __syncthreads();
  if (w.ty >= w.TY || !a.out) return;
  const float inv = 1.f / ((float)a.s * (float)per);
  float c1[V], c2[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    c1[j] = rs[j] * s1[gi[j]] * inv;
    c2[j] = rs[j] * rs[j] * s2[gi[j]] * inv;
  }
  T* op = (T*)a.out + at;
  with_act(a.act, [&](auto act) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u < mine) {
        float f[V], g[V];
        q[u].get(f);
        h[u].get(g);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float d = f[j] - mu[j];
          const float dz = act_grad<T, decltype(act)::value>(__builtin_fmaf(d, ga[j], be[j]), g[j]);
          f[j] = __builtin_fmaf(dz, ga[j], -__builtin_fmaf(d, c2[j], c1[j]));
        }
        Chunk<T, V>::store(op + u * step, f);
      }
    }
  });
}

// Channels first.  part: [n][ws][2][c], A and B of each slice of the positions.
template <typename T, int V, int U, int MODE>
__global__ __launch_bounds__(kNormThreads) void k_norm_bwd_first(const NormArgs a) {
  extern __shared__ float lds[];
  const int id = xcd_swizzle(blockIdx.x, gridDim.x);
  const int k = id % a.slices, ng = id / a.slices, g = ng % a.g, n = ng / a.g;
  const int kr = k / a.ws, ks = k - kr * a.ws;
  const int r0 = kr * a.rp, rows = min(a.rp, a.per - r0);
  const int c0 = ks * a.cp, cols = min(a.cp, a.s - c0);
  const int t = 1 << a.lt, ln = threadIdx.x & (t - 1), tm = threadIdx.x >> a.lt, teams = blockDim.x >> a.lt;
  const int chunks = (cols + V - 1) / V, ic = (chunks + t - 1) >> a.lt;
  const int rounds = (rows + teams - 1) / teams * ic;
  const size_t base = ((size_t)ng * a.per + r0) * a.s;
  const T* xp = (const T*)a.x + base;
  const T* yp = (const T*)a.dy + base;
  const int subs = t > 64 ? t >> 6 : 1;  // waves that share a channel
  float* gam = lds + 16;
  float* bet = gam + rows;
  float* ra = bet + rows;                // [rows][subs]
  float* rb = ra + rows * subs;
  for (int i = threadIdx.x; i < rows; i += blockDim.x) {
    gam[i] = Elem<T>::to_f32(((const T*)a.gamma)[g * a.per + r0 + i]);
    bet[i] = Elem<T>::to_f32(((const T*)a.beta)[g * a.per + r0 + i]);
  }
  auto slot = [&](int row, int i, int& pos, int& shift) {
    const int want = c0 + i * V;
    pos = want + V <= a.s ? want : a.s - V;  // s >= V
    shift = want - pos;
    return row < rows && i < chunks;
  };
  Chunk<T, V> q[U], h[U];
  {
    int row = tm, i = ln;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int pos, shift;
      const bool ok = slot(row, i, pos, shift);
      if (u < rounds && ok) {
        q[u].load(xp + (size_t)row * a.s + pos);
        h[u].load(yp + (size_t)row * a.s + pos);
      } else {
        q[u].zero();
        h[u].zero();
      }
      i += t;
      if (i - ln >= ic * t) { i = ln; row += teams; }
    }
  }
  const float mean = a.mean[ng], rstd = a.rstd[ng];
  const bool ragged = a.s % V != 0;
  __syncthreads();
  float s1, s2;
  if (MODE != kNormApply) {
    with_act(a.act, [&](auto act) {
      int row = tm, i = ln;
      float sa = 0.f, sb = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u < rounds) {
          int pos, shift;
          if (slot(row, i, pos, shift)) {
            const float ga = gam[row] * rstd, be = bet[row];
            float f[V], e[V];
            q[u].get(f);
            h[u].get(e);
  #pragma unroll
            for (int j = 0; j < V; ++j) {
              const float d = f[j] - mean;
              float dz = act_grad<T, decltype(act)::value>(__builtin_fmaf(d, ga, be), e[j]);
              if (ragged) dz = j >= shift ? dz : 0.f;
              sa += dz;
              sb = __builtin_fmaf(dz, d, sb);
            }
          }
          i += t;
          if (i - ln >= ic * t) {  // the channel's last round, for every team
            sa = team_sum(sa, t < 64 ? t : 64);
            sb = team_sum(sb, t < 64 ? t : 64);
            if ((ln & 63) == 0 && row < rows) {
              ra[row * subs + (ln >> 6)] = sa;
              rb[row * subs + (ln >> 6)] = sb;
            }
            sa = sb = 0.f;
            i = ln;
            row += teams;
          }
        }
      }
    });
    __syncthreads();
    float* out = a.part + ((size_t)n * a.ws + ks) * 2 * a.c + g * a.per + r0;
    s1 = s2 = 0.f;
    for (int row = threadIdx.x; row < rows; row += blockDim.x) {
      float va = 0.f, vb = 0.f;
      for (int i = 0; i < subs; ++i) {
        va += ra[row * subs + i];
        vb += rb[row * subs + i];
      }
      vb *= rstd;
      out[row] = va;
      out[a.c + row] = vb;
      s1 = __builtin_fmaf(va, gam[row], s1);
      s2 = __builtin_fmaf(vb, gam[row], s2);
    }
    if (MODE == kNormStats) return;
    s1 = block_sum(s1, lds);
    s2 = block_sum(s2, lds + 8);
  } else {
    s1 = a.sums[2 * (size_t)ng];
    s2 = a.sums[2 * (size_t)ng + 1];
  }
  if (!a.out) return;
  const float inv = 1.f / ((float)a.s * (float)a.per);
  const float c1 = rstd * s1 * inv, c2 = rstd * rstd * s2 * inv;
  T* op = (T*)a.out + base;
  with_act(a.act, [&](auto act) {
    int row = tm, i = ln;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      int pos, shift;
      const bool ok = slot(row, i, pos, shift);
      if (u < rounds && ok) {
        const float ga = gam[row] * rstd, be = bet[row];
        float f[V], e[V];
        q[u].get(f);
        h[u].get(e);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float d = f[j] - mean;
          const float dz = act_grad<T, decltype(act)::value>(__builtin_fmaf(d, ga, be), e[j]);
          f[j] = __builtin_fmaf(dz, ga, -__builtin_fmaf(d, c2, c1));
        }
        Chunk<T, V>::store(op + (size_t)row * a.s + pos, f);
      }
      i += t;
      if (i - ln >= ic * t) { i = ln; row += teams; }
    }
  });
}

// S1 and S2 of each group of each image from the slices' A and B.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_bwd_sums(const NormArgs a, int parts) {
  __shared__ float lds[16];
  const int ng = blockIdx.x, g = ng % a.g, n = ng / a.g, c0 = g * a.per;
  const float* p = a.part + (size_t)n * parts * 2 * a.c + c0;
  float s1 = 0.f, s2 = 0.f;
  for (int i = threadIdx.x; i < parts * a.per; i += 256) {
    const int k = i / a.per, ch = i - k * a.per;
    const float gamma = Elem<T>::to_f32(((const T*)a.gamma)[c0 + ch]);
    s1 = __builtin_fmaf(gamma, p[(size_t)k * 2 * a.c + ch], s1);
    s2 = __builtin_fmaf(gamma, p[((size_t)k * 2 + 1) * a.c + ch], s2);
  }
  s1 = block_sum(s1, lds);
  s2 = block_sum(s2, lds + 8);
  if (threadIdx.x == 0) ((float2*)a.sums)[ng] = make_float2(s1, s2);
}

// dbeta and dgamma: sums of A and B over the rows of part.  64 channels per
// workgroup, 16 shares of the rows.
template <typename T>
__global__ __launch_bounds__(1024) void k_norm_params(const float* __restrict__ part, int rows, int c, T* dgamma,
                                                      T* dbeta) {
  __shared__ float lds[2][16][64];
  const int ch = blockIdx.x * 64 + threadIdx.x % 64, share = threadIdx.x / 64;
  float va = 0.f, vb = 0.f;
  if (ch < c) {
#pragma unroll 4
    for (int r = share; r < rows; r += 16) {
      va += part[(size_t)r * 2 * c + ch];
      vb += part[((size_t)r * 2 + 1) * c + ch];
    }
  }
  lds[0][share][threadIdx.x % 64] = va;
  lds[1][share][threadIdx.x % 64] = vb;
  __syncthreads();
  if (share < 2 && ch < c) {
    float v = 0.f;
    for (int i = 0; i < 16; ++i) v += lds[share][i][threadIdx.x % 64];
    T* out = share ? dgamma : dbeta;
    if (out) out[ch] = Elem<T>::from_f32(v);
  }
}

template <typename T, int V, int U>
hipError_t launch(const NormArgs& a, const NormPlan& p, int layout, int mode, hipStream_t st) {
  const dim3 grid(p.blocks), block(p.threads);
#define DEFT_NORM(M)                                                                                           \
  do {                                                                                                         \
    const void* f = layout == DEFT_CHANNELS_LAST ? (const void*)k_norm_bwd_last<T, V, U, M>                    \
                                                 : (const void*)k_norm_bwd_first<T, V, U, M>;                  \
    if (p.lds > 65536) {                                                                                       \
      const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)p.lds);     \
      if (e != hipSuccess) return e;                                                                           \
    }                                                                                                          \
    if (layout == DEFT_CHANNELS_LAST) DEFT_LAUNCH("norm_bwd", (k_norm_bwd_last<T, V, U, M>), grid, block, p.lds, st, a); \
    else DEFT_LAUNCH("norm_bwd", (k_norm_bwd_first<T, V, U, M>), grid, block, p.lds, st, a);                   \
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

hipError_t launch_norm_bwd(const NormArgs& a, const NormPlan& p, int layout, int dtype, int mode, hipStream_t st) {
  if (p.u > 16) return hipErrorInvalidValue;
  return dtype == DEFT_BF16 ? launch_t<bf16_t>(a, p, layout, mode, st) : launch_t<float>(a, p, layout, mode, st);
}

hipError_t launch_norm_bwd_sums(const NormArgs& a, int layout, int dtype, hipStream_t st) {
  const int parts = layout == DEFT_CHANNELS_LAST ? a.slices : a.ws;
  const dim3 grid((unsigned)(a.n * a.g));
  if (dtype == DEFT_BF16) DEFT_LAUNCH("norm_bwd_sums", k_norm_bwd_sums<bf16_t>, grid, dim3(256), 0, st, a, parts);
  else DEFT_LAUNCH("norm_bwd_sums", k_norm_bwd_sums<float>, grid, dim3(256), 0, st, a, parts);
  return hipGetLastError();
}

hipError_t launch_norm_params(const float* part, int rows, int c, void* dgamma, void* dbeta, int dtype,
                              hipStream_t st) {
  const dim3 grid((c + 63) / 64);
  if (dtype == DEFT_BF16)
    DEFT_LAUNCH("norm_params", k_norm_params<bf16_t>, grid, dim3(1024), 0, st, part, rows, c, (bf16_t*)dgamma,
                (bf16_t*)dbeta);
  else
    DEFT_LAUNCH("norm_params", k_norm_params<float>, grid, dim3(1024), 0, st, part, rows, c, (float*)dgamma,
                (float*)dbeta);
  return hipGetLastError();
}

}  // namespace deft
