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
#include <algorithm>

#include "deft_norm.h"

namespace deft {

namespace {

template <typename T, int U, int MODE, bool KEEP> constexpr int bound(bool last) {
  return MODE == kNormWhole && U == 8 && norm_bwd_wide(sizeof(T) == 4, last, KEEP) ? kNormWide : kNormThreads;
}

// Sums of the words of group g of a cluster, in every lane of a wave; false if
// they did not come.
__device__ __forceinline__ bool sum_joint(const NormArgs& a, const Joint& jt, int ng, int g, float& s1, float& s2) {
  float v1 = 0.f, v2 = 0.f;
  if (!jt.gather(a.slices, ng, g, [&](int, float x, float y) { v1 += x; v2 += y; })) return false;
  s1 = team_sum(v1, 64);
  s2 = team_sum(v2, 64);
  return true;
}

// dz of the chunks between the sums and dx.  fp32 has room for it in dy's place.
// bf16 can keep it in registers of its own (KEEP) or compute it again: relu and
// none take an instruction for that, silu 15 and gelu 28 an element.
template <typename T, int V, int U, bool KEEP> struct Dz {
  float v[U][V];
};
template <typename T, int V, int U> struct Dz<T, V, U, false> {};

// d and dz at chunk u's elements; `held`: after an earlier call.
template <int ACT, typename T, int V, int U, bool KEEP>
__device__ __forceinline__ void chunk_dz(const Chunk<T, V>* x, Chunk<T, V>* y, Dz<T, V, U, KEEP>& kept, int u,
                                         bool held, const float* mu, const float* ga, const float* be, float* d,
                                         float* dz) {
  x[u].get(d);
  if constexpr (KEEP) {
    if (held) {
#pragma unroll
      for (int j = 0; j < V; ++j) { d[j] -= mu[j]; dz[j] = kept.v[u][j]; }
      return;
    }
  }
  y[u].get(dz);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    d[j] -= mu[j];
    if (!held || sizeof(T) == 2) dz[j] = act_grad<T, ACT>(__builtin_fmaf(d[j], ga[j], be[j]), dz[j]);
  }
  if (held) return;
  if constexpr (KEEP) {
#pragma unroll
    for (int j = 0; j < V; ++j) kept.v[u][j] = dz[j];
  }
  if constexpr (sizeof(T) == 4) y[u].put(dz);
}

// A and B go to memory as relaxed atomics of agent scope, so that the workgroup
// that sums them up need not be on the same part of the chip.
__device__ __forceinline__ void put_part(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// dbeta and dgamma of the channels c0 ... by the last of the images' workgroups
// that have them (one slice each): small calls, which take longer to launch than
// to run, save a launch by it.
// Each wave waits for its stores of A and B (stored), then, past a barrier, one
// thread counts the workgroup in (arrive) while dx is computed, and at the end
// the last one adds up.
__device__ __forceinline__ void stored() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ uint64_t arrive(const NormArgs& a, int unit) {
  if (!a.arrivals || threadIdx.x) return 0;
  return __hip_atomic_fetch_add(a.arrivals + unit, 1ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ void params_by_last(const NormArgs& a, uint64_t ticket, int unit, int c0, int cols, float* lds) {
  if (!a.arrivals) return;
  __shared__ int last;
  if (threadIdx.x == 0) {
    last = ticket + 1 == (uint64_t)a.n;
    if (last)  // for the next call
      __hip_atomic_store(a.arrivals + unit, 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  if (!last) return;
  const int nt = blockDim.x, rows = a.n, wide = min(cols, nt);
  const int shares = min(nt / wide, 16), share = threadIdx.x / wide, lane = threadIdx.x - share * wide;
  for (int col = lane; col - lane < cols; col += wide) {
    float va = 0.f, vb = 0.f;
    if (share < shares && col < cols) {
      const float* p = a.part + c0 + col;
      for (int r0 = share; r0 < rows; r0 += 16 * shares) {  // 16 at once: each load takes a microsecond
        float xa[16], xb[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float* at = p + (size_t)min(r0 + i * shares, rows - 1) * 2 * a.c;
          xa[i] = __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          xb[i] = __hip_atomic_load(at + a.c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          va += r0 + i * shares < rows ? xa[i] : 0.f;
          vb += r0 + i * shares < rows ? xb[i] : 0.f;
        }
      }
      lds[threadIdx.x] = va;
      lds[nt + threadIdx.x] = vb;
    }
    __syncthreads();
    if (share == 0 && col < cols) {
      for (int i = 1; i < shares; ++i) {
        va += lds[i * wide + lane];
        vb += lds[nt + i * wide + lane];
      }
      if (a.dbeta) ((T*)a.dbeta)[c0 + col] = Elem<T>::from_f32(va);
      if (a.dgamma) ((T*)a.dgamma)[c0 + col] = Elem<T>::from_f32(vb);
    }
    __syncthreads();
  }
}

// Channels last; blocks as in the forward.  part: [n][slices][2][c], A and B of
// each slice.  Joint words: a slice's shares of S1 and S2.
// Bound by memory, in phases: where a group is held whole, its x and dy fill a
// compute unit's registers, so loads, sums and stores follow each other.
// 32x1024x512 fp32 takes 51 us (3.9 TB/s; gelu 58), 16x784x512 bf16 silu 19 (2.1
// TB/s); 2x65536x320 bf16, read twice, 100 (4.2 TB/s of what it reads and writes).
template <typename T, int V, int U, int MODE, bool KEEP>
__global__ __launch_bounds__((bound<T, U, MODE, KEEP>(true))) void k_norm_bwd_last(const NormArgs a) {
  extern __shared__ float lds[];
  int b, k, n;
  if (MODE == kNormJoint) {
    const int nb = blockIdx.x / a.slices;
    k = blockIdx.x - nb * a.slices;
    n = nb / a.bands;
    b = nb - n * a.bands;
  } else {
    const int id = xcd_swizzle(blockIdx.x, gridDim.x), nk = id / a.bands;
    b = id - nk * a.bands;
    n = nk / a.slices;
    k = nk - n * a.slices;
  }
  Band w;
  w.set<V>(b, a.bands, a.g, a.per);
  const int per = a.per, ng0 = n * a.g + w.g0;
  const size_t step = (size_t)w.TY * a.c;
  Chunk<T, V> q[U], h[U];
  Dz<T, V, U, KEEP> kept;
  int rows, mine, end;
  size_t at;
  // rows r0 ... of a slice that ends before `end`, as many as the registers hold
  auto load_rows = [&](int r0) {
    rows = min(w.TY * U, end - r0);
    mine = w.ty < w.TY ? (rows - w.ty + w.TY - 1) / w.TY : 0;
    at = ((size_t)n * a.s + r0 + min(w.ty, rows - 1)) * a.c + w.col;
    const T* xp = (const T*)a.x + at;
    const T* yp = (const T*)a.dy + at;
    // rows past the end are read as the last one: no branch surrounds the loads
#pragma unroll
    for (int u = 0; u < U; ++u) {
      apart();
      q[u].load(xp);
      h[u].load(yp);
      const size_t go = u + 1 < mine ? step : 0;
      xp += go;
      yp += go;
    }
  };
  auto load = [&](int slice) {
    end = (int)min((uint32_t)(slice + 1) * (uint32_t)a.rp, (uint32_t)a.s);  // the product may pass 2^31
    load_rows(slice * a.rp);
  };
  const Ahead<T> gamma((const T*)a.gamma + w.c0, w.cols), beta((const T*)a.beta + w.c0, w.cols);
  const Ahead<float> means(a.mean + ng0, w.ng), rstds(a.rstd + ng0, w.ng);
  load(k);
  float* gm = lds;              // the band's groups: mean, 1 / std, S1, S2
  float* gr = gm + w.ng;
  float* s1 = gr + w.ng;
  float* s2 = s1 + w.ng;
  float* gam = s2 + w.ng;       // its channels: gamma, beta, gamma A, gamma B
  float* bet = gam + w.cols;
  float* ca = bet + w.cols;
  float* cb = ca + w.cols;
  means.put(gm);
  rstds.put(gr);
  gamma.put(gam);
  beta.put(bet);
  __syncthreads();
  float mu[V], ga[V], be[V];
  auto coefficients = [&](auto f) {
    const int col = anew(w.col - w.c0);
    int i = col / per, next = (i + 1) * per - col;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      f(j, i, col + j);
      if (--next == 0) { next = per; ++i; }
    }
  };
  coefficients([&](int j, int i, int col) {
    mu[j] = gm[i];
    ga[j] = gam[col] * gr[i];
    be[j] = bet[col];
  });
  const int pitch = w.cols | 1;
  float* ra = cb + w.cols;      // [TY][pitch]
  float* rb = ra + w.TY * pitch;
  // A and B of the loaded slice to part, and out(group, S1, S2) of the slice by
  // one thread a group
  auto sums = [&](int slice, auto out) {
    float sa[V] = {}, sb[V] = {};
    for (int r0 = slice * a.rp;;) {
      const int rounds = (rows + w.TY - 1) / w.TY;
      // the activation is chosen within each round: chosen outside, every branch
      // would leave its dz in registers of its own
#pragma unroll
      for (int u = 0; u < U; ++u) {
        apart();
        if (u < rounds) {
          h[u].zero_if(u >= mine);
          float d[V], dz[V];
          with_act(a.act, [&](auto act) {
            chunk_dz<decltype(act)::value>(q, h, kept, u, false, mu, ga, be, d, dz);
          });
#pragma unroll
          for (int j = 0; j < V; ++j) {
            sa[j] += dz[j];
            sb[j] = __builtin_fmaf(dz[j], d[j], sb[j]);
          }
        }
      }
      if (MODE != kNormStats || end - r0 <= w.TY * U) break;  // only slices that are read twice are longer
      r0 += w.TY * U;
      load_rows(r0);
    }
    if (w.ty < w.TY) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (j >= w.shift) {
          ra[w.ty * pitch + (w.col - w.c0) + j] = sa[j];
          rb[w.ty * pitch + (w.col - w.c0) + j] = sb[j];
        }
      }
    }
    __syncthreads();
    float* ab = a.part + ((size_t)n * a.slices + slice) * 2 * a.c + w.c0;
    segment_sums(ra, pitch, w.TY, w.cols, 1, [&](int col, float v) {
      put_part(ab + col, v);
      ca[col] = v * gam[col];
    });
    segment_sums(rb, pitch, w.TY, w.cols, 1, [&](int col, float v) {
      v *= gr[col / per];
      put_part(ab + a.c + col, v);
      cb[col] = v * gam[col];
    });
    if (MODE == kNormStats) return;
    __syncthreads();
    segment_sums(ca, 0, 1, w.ng, per, [&](int g, float v) { s1[g] = v; });
    // the same thread has the group's sum of ca
    segment_sums(cb, 0, 1, w.ng, per, [&](int g, float v) { out(g, s1[g], v); });
  };
  if (MODE == kNormWhole) {
    sums(k, [&](int g, float, float v) { s2[g] = v; });
  } else if (MODE == kNormStats) {
    sums(k, [&](int, float, float) {});
    return;
  } else if (MODE == kNormApply) {
    for (int i = threadIdx.x; i < w.ng; i += blockDim.x) {
      s1[i] = a.sums[2 * (size_t)(ng0 + i)];
      s2[i] = a.sums[2 * (size_t)(ng0 + i) + 1];
    }
  } else {
    __shared__ uint32_t tag;
    const int cluster = n * a.bands + b, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    if (threadIdx.x == 0) tag = joint_tag(a.counter + cluster, a.slices);
    __syncthreads();
    Joint jt{a.words + (size_t)ng0 * a.slices * 2, a.totals + (size_t)ng0 * 2, tag,
             __builtin_readsteadycounter() + a.patience};
    // groups first, first + step, ... of the band, a wave each
    auto totals = [&](int first, int every, bool publish, bool last) {
      bool ok = true;
      for (int g = first + every * wave; g < w.ng && ok; g += every * waves) {
        float v1, v2;
        ok = sum_joint(a, jt, w.ng, g, v1, v2);
        if (last && !ok) {
          v1 = v2 = __builtin_nanf("");
          ok = true;
        }
        if (ok && (threadIdx.x & 63) == 0) {
          s1[g] = v1;
          s2[g] = v2;
          if (publish) {
            Joint::put(jt.total + 2 * g, v1, jt.tag);
            Joint::put(jt.total + 2 * g + 1, v2, jt.tag);
          }
        }
      }
      return ok;
    };
    for (int slice = k, alone = 0;;) {
      sums(slice, [&](int g, float v1, float v2) { jt.publish(slice, w.ng, g, v1, v2); });
      __syncthreads();  // s1 is read above and written below
      if (alone == 2) {
        totals(0, 1, !a.direct, true);
        break;
      }
      if (!alone) {
        bool ok = a.direct ? totals(0, 1, false, false) : totals(k, a.slices, true, false);
        if (!a.direct)
          for (int g = threadIdx.x; g < w.ng && ok; g += blockDim.x)
            ok = jt.wait([&] { return jt.read(jt.total + 2 * g, s1[g], s2[g]); });
        if (__syncthreads_and(ok)) break;
        alone = 1;
        slice = -1;
      }
      slice = jt.next(slice, a.slices, w.ng);
      if (slice == a.slices) {  // every word has been seen or stored here
        slice = k;
        alone = 2;
        jt.deadline = __builtin_readsteadycounter() + kLastLook;
      }
      load(slice);
    }
  }
  if (MODE == kNormWhole && a.arrivals) stored();
  __syncthreads();
  const uint64_t ticket = MODE == kNormWhole ? arrive(a, b) : 0;
  const float inv = 1.f / ((float)a.s * (float)per);
  float c1[V], c2[V];
  coefficients([&](int j, int i, int) {
    const float rstd = gr[i];
    c1[j] = rstd * s1[i] * inv;
    c2[j] = rstd * rstd * s2[i] * inv;
  });
  if (a.out) with_act(a.act, [&](auto act) {
    for (int r0 = k * a.rp;;) {
      T* p = (T*)a.out + at;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        apart();
        if (u < mine) {
          float d[V], dz[V];
          q[u].keep();
          if (!KEEP) h[u].keep();
          chunk_dz<decltype(act)::value>(q, h, kept, u, MODE != kNormApply, mu, ga, be, d, dz);
#pragma unroll
          for (int j = 0; j < V; ++j) dz[j] = __builtin_fmaf(dz[j], ga[j], -__builtin_fmaf(d[j], c2[j], c1[j]));
          Chunk<T, V>::store(p, dz);
          p += step;
        }
      }
      if (MODE != kNormApply || end - r0 <= w.TY * U) break;
      r0 += w.TY * U;
      load_rows(r0);
    }
  });
  if (MODE == kNormWhole) params_by_last<T>(a, ticket, b, w.c0, w.cols, lds);
}

// Channels first; blocks as in the forward.  part: [n][ws][2][c], A and B of
// each slice of the positions.  Joint words: a slice's shares of S1 and S2.
// Bound as above: 16x256x56x56 bf16 relu takes 21 us (3.7 TB/s), gelu 33;
// 2x320x65536 bf16 75.
template <typename T, int V, int U, int MODE, bool KEEP>
__global__ __launch_bounds__((bound<T, U, MODE, KEEP>(false))) void k_norm_bwd_first(const NormArgs a) {
  extern __shared__ float lds[];
  const int id = MODE == kNormJoint ? blockIdx.x : xcd_swizzle(blockIdx.x, gridDim.x);
  const int ng = id / a.slices, k = id - ng * a.slices, n = ng / a.g, g = ng - n * a.g;
  const int t = 1 << a.lt, ln = threadIdx.x & (t - 1), tm = threadIdx.x >> a.lt, teams = blockDim.x >> a.lt;
  const int subs = t > 64 ? t >> 6 : 1;  // waves that share a channel
  float* gam = lds + 32;
  float* bet = gam + a.rp;
  float* ra = bet + a.rp;                // [rows][subs]
  float* rb = ra + a.rp * subs;
  int r0, c0, rows, cols, chunks, ic, rounds, ks;
  auto slot = [&](int row, int i, int& pos, int& shift) {
    const uint32_t want = (uint32_t)c0 + (uint32_t)i * V;  // past a row of 2^31 - 1, too
    pos = want + V <= (uint32_t)a.s ? (int)want : a.s - V;  // s >= V
    shift = (int)(want - pos);
    return row < rows && i < chunks;
  };
  Chunk<T, V> q[U], h[U];
  Dz<T, V, U, KEEP> kept;
  size_t base;
  auto load = [&](int slice) {
    const int kr = slice / a.ws;
    ks = slice - kr * a.ws;
    r0 = kr * a.rp;
    rows = min(a.rp, a.per - r0);
    c0 = ks * a.cp;
    cols = min(a.cp, a.s - c0);
    chunks = (cols + V - 1) / V;
    ic = (chunks + t - 1) >> a.lt;
    rounds = (rows + teams - 1) / teams * ic;
    base = ((size_t)ng * a.per + r0) * a.s;
    const T* xp = (const T*)a.x + base;
    const T* yp = (const T*)a.dy + base;
    const Ahead<T> gamma((const T*)a.gamma + g * a.per + r0, rows), beta((const T*)a.beta + g * a.per + r0, rows);
    const int first = anew(ln);
    int row = tm, i = first;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      apart();
      int pos, shift;
      slot(row, i, pos, shift);
      const size_t off = (size_t)min(row, rows - 1) * a.s + pos;  // past the end: what is there, unused
      q[u].load(xp + off);
      h[u].load(yp + off);
      i += t;
      if (i - first >= ic * t) { i = first; row += teams; }
    }
    gamma.put(gam);
    beta.put(bet);
    __syncthreads();
  };
  const float mean = a.mean[ng], rstd = a.rstd[ng];
  load(k);
  const bool ragged = a.s % V != 0;
  // one channel's chunk: the same coefficients for its elements
  auto dz_of = [&](auto act, int u, int row, bool held, float* d, float* dz) {
    float mu[V], ga[V], be[V];
    const float gr = gam[row] * rstd, b = bet[row];
#pragma unroll
    for (int j = 0; j < V; ++j) { mu[j] = mean; ga[j] = gr; be[j] = b; }
    chunk_dz<decltype(act)::value>(q, h, kept, u, held, mu, ga, be, d, dz);
    return gr;
  };
  // A and B of the loaded slice to part; its shares of S1 and S2 in every thread
  auto sums = [&](float& s1, float& s2) {
    const int first = anew(ln);
    int row = tm, i = first;
    float sa = 0.f, sb = 0.f;
    // the activation is chosen within each round, as above
#pragma unroll
    for (int u = 0; u < U; ++u) {
      apart();
      if (u < rounds) {
        int pos, shift;
        if (slot(row, i, pos, shift)) {
          float d[V], dz[V];
          with_act(a.act, [&](auto act) { dz_of(act, u, row, false, d, dz); });
#pragma unroll
          for (int j = 0; j < V; ++j) {
            if (ragged) dz[j] = j >= shift ? dz[j] : 0.f;
            sa += dz[j];
            sb = __builtin_fmaf(dz[j], d[j], sb);
          }
        }
        i += t;
        if (i - first >= ic * t) {  // the channel's last round, for every team
          sa = team_sum(sa, t < 64 ? t : 64);
          sb = team_sum(sb, t < 64 ? t : 64);
          if ((ln & 63) == 0 && row < rows) {
            ra[row * subs + (ln >> 6)] = sa;
            rb[row * subs + (ln >> 6)] = sb;
          }
          sa = sb = 0.f;
          i = first;
          row += teams;
        }
      }
    }
    __syncthreads();
    float* ab = a.part + ((size_t)n * a.ws + ks) * 2 * a.c + g * a.per + r0;
    s1 = s2 = 0.f;
    for (int row = threadIdx.x; row < rows; row += blockDim.x) {
      float va = 0.f, vb = 0.f;
      for (int i = 0; i < subs; ++i) {
        va += ra[row * subs + i];
        vb += rb[row * subs + i];
      }
      vb *= rstd;
      put_part(ab + row, va);
      put_part(ab + a.c + row, vb);
      s1 = __builtin_fmaf(va, gam[row], s1);
      s2 = __builtin_fmaf(vb, gam[row], s2);
    }
    if (MODE == kNormStats) return;
    s1 = block_sum(s1, lds);
    if (MODE == kNormWhole && a.arrivals) stored();
    s2 = block_sum(s2, lds + 16);
  };
  float s1, s2;
  if (MODE == kNormWhole) {
    sums(s1, s2);
  } else if (MODE == kNormStats) {
    sums(s1, s2);
    return;
  } else if (MODE == kNormApply) {
    s1 = a.sums[2 * (size_t)ng];
    s2 = a.sums[2 * (size_t)ng + 1];
  } else {
    __shared__ uint32_t tag;
    if (threadIdx.x == 0) tag = joint_tag(a.counter + ng, a.slices);
    __syncthreads();
    Joint jt{a.words + (size_t)ng * a.slices * 2, nullptr, tag, __builtin_readsteadycounter() + a.patience};
    // one wave reads the words: they lie in few lines, which all workgroups ask for
    __shared__ float got[2];
    auto join = [&] {
      bool ok = true;
      if (threadIdx.x < 64) {
        ok = sum_joint(a, jt, 1, 0, s1, s2);
        if (threadIdx.x == 0) { got[0] = s1; got[1] = s2; }
      }
      ok = __syncthreads_and(ok);
      s1 = got[0];
      s2 = got[1];
      return ok;
    };
    for (int slice = k, alone = 0;;) {
      sums(s1, s2);
      if (threadIdx.x == 0) jt.publish(slice, 1, 0, s1, s2);
      if (alone == 2) {
        if (!join()) s1 = s2 = __builtin_nanf("");
        break;
      }
      if (!alone) {
        if (join()) break;
        alone = 1;
        slice = -1;
      }
      slice = jt.next(slice, a.slices, 1);
      if (slice == a.slices) {  // every word has been seen or stored here
        slice = k;
        alone = 2;
        jt.deadline = __builtin_readsteadycounter() + kLastLook;
      }
      load(slice);
    }
  }
  const uint64_t ticket = MODE == kNormWhole ? arrive(a, g) : 0;
  const float inv = 1.f / ((float)a.s * (float)a.per);
  const float c1 = rstd * s1 * inv, c2 = rstd * rstd * s2 * inv;
  T* op = (T*)a.out + base;
  if (a.out) with_act(a.act, [&](auto act) {
    const int first = anew(ln);
    int row = tm, i = first;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      apart();
      int pos, shift;
      const bool ok = slot(row, i, pos, shift);
      if (u < rounds && ok) {
        float d[V], dz[V];
        q[u].keep();
        if (!KEEP) h[u].keep();
        const float ga = dz_of(act, u, row, MODE != kNormApply, d, dz);
#pragma unroll
        for (int j = 0; j < V; ++j) dz[j] = __builtin_fmaf(dz[j], ga, -__builtin_fmaf(d[j], c2, c1));
        Chunk<T, V>::store(op + (size_t)row * a.s + pos, dz);
      }
      i += t;
      if (i - first >= ic * t) { i = first; row += teams; }
    }
  });
  if (MODE == kNormWhole) params_by_last<T>(a, ticket, g, g * a.per, a.per, lds);
}

// S1 and S2 of each group of each image from the slices' A and B.  A thread has
// a channel and a share of the slices.
template <typename T>
__global__ __launch_bounds__(1024) void k_norm_bwd_sums(const NormArgs a, int parts) {
  __shared__ float lds[32];
  const int ng = blockIdx.x, g = ng % a.g, n = ng / a.g, c0 = g * a.per;
  const int wide = min(a.per, 1024), shares = 1024 / wide, share = threadIdx.x / wide;
  float s1 = 0.f, s2 = 0.f;
  if (share < shares) {
    for (int ch = threadIdx.x - share * wide; ch < a.per; ch += wide) {
      const float* p = a.part + (size_t)n * parts * 2 * a.c + c0 + ch;
      float va = 0.f, vb = 0.f;
#pragma unroll 8
      for (int k = share; k < parts; k += shares) {
        va += p[(size_t)k * 2 * a.c];
        vb += p[((size_t)k * 2 + 1) * a.c];
      }
      const float gamma = Elem<T>::to_f32(((const T*)a.gamma)[c0 + ch]);
      s1 = __builtin_fmaf(gamma, va, s1);
      s2 = __builtin_fmaf(gamma, vb, s2);
    }
  }
  s1 = block_sum(s1, lds);
  s2 = block_sum(s2, lds + 16);
  if (threadIdx.x == 0) ((float2*)a.sums)[ng] = make_float2(s1, s2);
}

// dbeta and dgamma: sums of A and B over the rows of part.  16 channels (a line's
// half) per workgroup, 64 shares of the rows.  `pitch` channels a row, `c` of them here.
template <typename T>
__global__ __launch_bounds__(1024) void k_norm_params(const float* __restrict__ part, int rows, int pitch, int c,
                                                      T* dgamma, T* dbeta) {
  __shared__ float lds[2][64][17];
  const int lane = threadIdx.x & 15, ch = blockIdx.x * 16 + lane, share = threadIdx.x >> 4;
  float va = 0.f, vb = 0.f;
  if (ch < c) {
#pragma unroll 8
    for (int r = share; r < rows; r += 64) {
      va += part[(size_t)r * 2 * pitch + ch];
      vb += part[((size_t)r * 2 + 1) * pitch + ch];
    }
  }
  lds[0][share][lane] = va;
  lds[1][share][lane] = vb;
  __syncthreads();
  // waves 0 and 1: four lanes a channel
  const int which = threadIdx.x >> 6, l = threadIdx.x & 63, col = l >> 2;
  if (which < 2) {
    float v = 0.f;
    for (int i = l & 3; i < 64; i += 4) v += lds[which][i][col];
    v = team_sum(v, 4);
    T* out = which ? dgamma : dbeta;
    if (out && (l & 3) == 0 && blockIdx.x * 16 + col < c) out[blockIdx.x * 16 + col] = Elem<T>::from_f32(v);
  }
}

template <typename T, int V, int U, int MODE, bool KEEP>
hipError_t launch(const NormArgs& a, const NormPlan& p, int layout, hipStream_t st) {
  const bool last = layout == DEFT_CHANNELS_LAST;
  const void* f = last ? (const void*)k_norm_bwd_last<T, V, U, MODE, KEEP>
                       : (const void*)k_norm_bwd_first<T, V, U, MODE, KEEP>;
  if (p.lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)p.lds);
    if (e != hipSuccess) return e;
  }
  const dim3 grid(p.blocks), block(p.threads);
  if (last) DEFT_LAUNCH("norm_bwd", (k_norm_bwd_last<T, V, U, MODE, KEEP>), grid, block, p.lds, st, a);
  else DEFT_LAUNCH("norm_bwd", (k_norm_bwd_first<T, V, U, MODE, KEEP>), grid, block, p.lds, st, a);
  return hipGetLastError();
}

template <typename T, int V, int U>
hipError_t launch_mode(const NormArgs& a, const NormPlan& p, int layout, int mode, hipStream_t st) {
  constexpr bool can = V == 8 && U <= 8;  // 16 chunks and their dz fill the registers
  const bool keep = can && (a.act == DEFT_ACT_SILU || a.act == DEFT_ACT_GELU);
  if (mode == kNormWhole)
    return keep ? launch<T, V, U, kNormWhole, can>(a, p, layout, st)
                : launch<T, V, U, kNormWhole, false>(a, p, layout, st);
  if constexpr (U <= 8 || V == 1) {  // slices have no more
    if (mode == kNormJoint)
      return keep ? launch<T, V, U, kNormJoint, can>(a, p, layout, st)
                  : launch<T, V, U, kNormJoint, false>(a, p, layout, st);
    return mode == kNormStats ? launch<T, V, U, kNormStats, false>(a, p, layout, st)
                              : launch<T, V, U, kNormApply, false>(a, p, layout, st);
  }
  return hipErrorInvalidValue;
}

template <typename T>
hipError_t launch_t(const NormArgs& a, const NormPlan& p, int layout, int mode, hipStream_t st) {
  constexpr int V = Elem<T>::VEC;
  if (p.vec == 1) return launch_mode<T, 1, 16>(a, p, layout, mode, st);
  if (p.u <= 4) return launch_mode<T, V, 4>(a, p, layout, mode, st);
  if (p.u <= 8) return launch_mode<T, V, 8>(a, p, layout, mode, st);
  return launch_mode<T, V, 16>(a, p, layout, mode, st);
}

}  // namespace

hipError_t launch_norm_bwd(const NormArgs& a, const NormPlan& p, int layout, int dtype, int mode, hipStream_t st) {
  if (p.u > 16) return hipErrorInvalidValue;
  return dtype == DEFT_BF16 ? launch_t<bf16_t>(a, p, layout, mode, st) : launch_t<float>(a, p, layout, mode, st);
}

hipError_t launch_norm_bwd_sums(const NormArgs& a, int layout, int dtype, hipStream_t st) {
  const int parts = layout == DEFT_CHANNELS_LAST ? a.slices : a.ws;
  const dim3 grid((unsigned)(a.n * a.g));
  if (dtype == DEFT_BF16) DEFT_LAUNCH("norm_bwd_sums", k_norm_bwd_sums<bf16_t>, grid, dim3(1024), 0, st, a, parts);
  else DEFT_LAUNCH("norm_bwd_sums", k_norm_bwd_sums<float>, grid, dim3(1024), 0, st, a, parts);
  return hipGetLastError();
}

template <typename T>
static hipError_t launch_params(const float* part, int rows, int c, T* dgamma, T* dbeta, hipStream_t st) {
  constexpr int kMost = 1 << 25;  // channels, of 64 threads each: a launch has fewer than 2^32
  for (int64_t c0 = 0; c0 < c; c0 += kMost) {
    const int cols = (int)std::min<int64_t>(c - c0, kMost);
    DEFT_LAUNCH("norm_params", k_norm_params<T>, dim3((cols + 15) / 16), dim3(1024), 0, st, part ? part + c0 : part,
                rows, c, cols, dgamma ? dgamma + c0 : dgamma, dbeta ? dbeta + c0 : dbeta);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_norm_params(const float* part, int rows, int c, void* dgamma, void* dbeta, int dtype,
                              hipStream_t st) {
  return dtype == DEFT_BF16 ? launch_params(part, rows, c, (bf16_t*)dgamma, (bf16_t*)dbeta, st)
                            : launch_params(part, rows, c, (float*)dgamma, (float*)dbeta, st);
}

}  // namespace deft
