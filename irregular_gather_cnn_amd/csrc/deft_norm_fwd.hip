// Group norm with activation, forward: y = act(gamma (x - mean) rstd + beta).
//
// A workgroup holds its slice of a group (or of a band of groups) in
// registers, so x is read once.  Statistics must not lose the variance where the
// mean is far from zero: all sums beyond a thread's are fp64.  Within a thread,
// fp32 elements give the squares about the mean of its own ones.  bf16 elements
// give plain sums of themselves and of their squares, at most 256 of each.
// Products of bf16 numbers are exact in fp32, and so are those sums where the
// numbers are near to each other, which is where the difference of the two needs
// it; this takes one instruction an element (v_dot2c_f32_bf16) in place of five.
#include "deft_norm.h"

namespace deft {

namespace {

// Elements of a group in slice k.
__device__ __forceinline__ float slice_count(const NormArgs& a, int layout, int k) {
  if (layout == DEFT_CHANNELS_LAST) return (float)min(a.rp, a.s - k * a.rp) * (float)a.per;
  const int kr = k / a.ws, ks = k - kr * a.ws;
  return (float)min(a.rp, a.per - kr * a.rp) * (float)min(a.cp, a.s - ks * a.cp);
}

// A group's mean and rstd from its slices' mean and M2: sums over the lanes'
// slices in fp64, which squares of means far from zero need.
struct Combine {
  double sum = 0.0, squares = 0.0;
  __device__ __forceinline__ void add(float count, float mean, float m2) {
    sum += (double)count * mean;
    squares += (double)m2 + (double)count * mean * mean;
  }
  // of the sums over all lanes
  __device__ __forceinline__ void finish(const NormArgs& a, float& mean, float& rstd) const {
    const double inv = 1.0 / ((double)a.s * a.per), m = sum * inv;
    double var = squares * inv - m * m;
    var = var < 0.0 ? 0.0 : var;  // a NaN stays
    mean = (float)m;
    rstd = 1.f / __builtin_sqrtf((float)var + a.eps);
  }
};
// The same from the words of group g of a cluster; false if they did not come.
__device__ __forceinline__ bool combine_joint(const NormArgs& a, int layout, const Joint& jt, int ng, int g,
                                              float& mean, float& rstd) {
  Combine c;
  if (!jt.gather(a.slices, ng, g, [&](int k, float m, float m2) { c.add(slice_count(a, layout, k), m, m2); }))
    return false;
  c.sum = team_sum(c.sum, 64);
  c.squares = team_sum(c.squares, 64);
  c.finish(a, mean, rstd);
  return true;
}

// Channels last: slice k of band b of image n.  Blocks are in the order ((n, k), b),
// so that the workgroups of one XCD share the lines of neighbouring bands; joint
// ones in the order ((n, b), k) over all XCDs, so that a cluster starts together.
// Bound by memory from a few million elements on: 32x1024x512 fp32 takes 23 us (5.8
// TB/s), 2x65536x320 bf16 53 (read twice: 4.7 TB/s the first time, then 5.7); by
// vector operations with gelu in bf16 (28 an element; 16x784x512 15 us against 11);
// by latency below: load, reduction and store take 5 us, an exchange 3 to 5 more.
// part: [n][g][slices]{mean, M2}.
template <typename T, int V, int U, int MODE>
__global__ __launch_bounds__(kNormThreads, MODE == kNormJoint ? 4 : 1) void k_norm_fwd_last(const NormArgs a) {
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
  Chunk<T, V> q[U];
  int rows, mine;
  size_t at;
  // Rows past the end are read as the last one: loads that no branch surrounds
  // are waited for one by one.
  auto load = [&](int slice) {
    const int r0 = slice * a.rp;
    rows = min(a.rp, a.s - r0);
    mine = w.ty < w.TY ? (rows - w.ty + w.TY - 1) / w.TY : 0;
    at = ((size_t)n * a.s + r0 + min(w.ty, rows - 1)) * a.c + w.col;
    const T* xp = (const T*)a.x + at;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      apart();
      q[u].load(xp);
      xp += u + 1 < mine ? step : 0;
    }
  };
  const Ahead<T> gamma((const T*)a.gamma + w.c0, MODE == kNormStats ? 0 : w.cols);
  const Ahead<T> beta((const T*)a.beta + w.c0, MODE == kNormStats ? 0 : w.cols);
  load(k);
  float* gm = lds;                // means of the band's groups
  float* gr = gm + w.ng;          // 1 / std
  float* gam = gr + w.ng;         // the band's channels
  float* bet = gam + w.cols;
  float* red = bet + w.cols;      // [2][TY][pitch]: sums, and squares about a thread's own mean
  gamma.put(gam);
  beta.put(bet);
  // Entries of a thread row in LDS: one a chunk where chunks lie in one group,
  // one a pair of columns where pairs do, else one a column.
  const bool solid = w.ng == 1 || per % V == 0;
  const bool pairs = V == 8 && !solid && per % 2 == 0;
  const int width = solid ? w.cx : pairs ? w.cols / 2 : w.cols, pitch = width | 1;
  const int len = solid ? (w.ng == 1 ? w.cx : per / V) : pairs ? per / 2 : per;
  // Statistics of the loaded slice: out(group, mean, M2) by one thread a group.
  auto statistics = [&](auto out) {
    float* rq = red + w.TY * pitch;
    float* my = red + w.ty * pitch + (solid ? w.tx : pairs ? (w.col - w.c0) / 2 : w.col - w.c0);
    auto spill = [&](int j, float sum, float sq) {
      my[j] = sum;
      my[w.TY * pitch + j] = sq;
    };
    const float inv = 1.f / (float)max(mine, 1);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      apart();
      q[u].zero_if(u >= mine);
    }
    if constexpr (sizeof(T) == 2 && V == 8) {
      if (solid || pairs) {
        const bool cut = solid && w.cols % V != 0;
        float sum[4] = {}, sq[4] = {};
#pragma unroll
        for (int u = 0; u < U; ++u) {
          apart();
          Chunk<T, V> x = q[u];
          if (cut) x.zero_below(w.shift);
#pragma unroll
          for (int j = 0; j < 4; ++j) x.moments(j, sum[j], sq[j]);
        }
        if (w.ty < w.TY) {
          if (solid) {
            spill(0, (sum[0] + sum[1]) + (sum[2] + sum[3]), (sq[0] + sq[1]) + (sq[2] + sq[3]));
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (2 * j >= w.shift) spill(j, sum[j], sq[j]);
          }
        }
      }
    }
    if (!(sizeof(T) == 2 && V == 8 && (solid || pairs))) {
      float sum[V] = {}, sq[V] = {}, whole = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        apart();
        float f[V];
        q[u].get(f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          sum[j] += f[j];
          if (sizeof(T) == 2) sq[j] = __builtin_fmaf(f[j], f[j], sq[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < V; ++j) whole += j >= w.shift ? sum[j] : 0.f;
      if (sizeof(T) == 4) {
        const float mean = whole * (inv * (w.shift ? 1.f / (float)(V - w.shift) : 1.f / V));
#pragma unroll
        for (int u = 0; u < U; ++u) {
          apart();
          float f[V];
          q[u].get(f);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float d = u < mine ? f[j] - (solid ? mean : sum[j] * inv) : 0.f;
            sq[j] = __builtin_fmaf(d, d, sq[j]);
          }
        }
      }
      if (w.ty < w.TY) {
        if (solid) {
          float v = 0.f;
#pragma unroll
          for (int j = 0; j < V; ++j) v += j >= w.shift ? sq[j] : 0.f;
          spill(0, whole, v);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j)
            if (j >= w.shift) spill(j, sum[j], sq[j]);
        }
      }
    }
    __syncthreads();
    // All of a group's entries by a team of lanes, or of whole waves where the
    // groups are few; sums in fp64: squares of means far from zero need it.
    __shared__ double of_wave[kNormThreads / 64][2];
    const int t = team_size(w.ng, blockDim.x), l = threadIdx.x & (t - 1);
    const double inv_count = 1.0 / ((double)rows * per);
    // fp32: a thread row r has most or most - 1 rows
    const int most = (rows + w.TY - 1) / w.TY, with_most = rows - (most - 1) * w.TY;
    const float inv_most = 1.f / (float)most, inv_less = 1.f / (float)max(most - 1, 1);
    auto finish = [&](int g, double v1, double v2) {
      v2 -= v1 * v1 * inv_count;
      out(g, (float)(v1 * inv_count), v2 < 0.0 ? 0.f : (float)v2);  // a NaN stays
    };
    for (int g = threadIdx.x / t; g < w.ng; g += blockDim.x / t) {
      double v1 = 0.0, v2 = 0.0;
      walk(l, t, w.TY, len, [&](int r, int e) {
        const int x = g * len + e;
        const float sum = red[r * pitch + x], sq = rq[r * pitch + x];
        v1 += (double)sum;
        v2 += (double)sq;
        if (sizeof(T) == 4) {
          // squares about the entry's mean to squares about zero: + m (2 sum - num m), which
          // takes m's rounding in its square only
          int num = r < with_most ? most : most - 1;
          float inv = r < with_most ? inv_most : inv_less;
          if (solid) {
            const int cols = x == w.cx - 1 ? w.cols - x * V : V;
            num *= cols;
            inv *= cols == V ? 1.f / V : 1.f / (float)cols;
          }
          const double m = (double)(sum * inv);
          v2 += m * (2.0 * (double)sum - (double)num * m);
        }
      });
      v1 = team_sum(v1, min(t, 64));
      v2 = team_sum(v2, min(t, 64));
      if (t <= 64) {
        if (l == 0) finish(g, v1, v2);
      } else if ((l & 63) == 0) {
        of_wave[threadIdx.x >> 6][0] = v1;
        of_wave[threadIdx.x >> 6][1] = v2;
      }
    }
    if (t > 64) {
      __syncthreads();
      if (threadIdx.x < w.ng) {
        double v1 = 0.0, v2 = 0.0;
        for (int i = 0; i < t / 64; ++i) {
          v1 += of_wave[threadIdx.x * (t / 64) + i][0];
          v2 += of_wave[threadIdx.x * (t / 64) + i][1];
        }
        finish(threadIdx.x, v1, v2);
      }
    }
  };
  if (MODE == kNormWhole) {
    statistics([&](int g, float mean, float m2) {
      const float rstd = 1.f / __builtin_sqrtf(m2 / ((float)a.s * (float)per) + a.eps);
      gm[g] = mean;
      gr[g] = rstd;
      a.mean[ng0 + g] = mean;
      a.rstd[ng0 + g] = rstd;
    });
  } else if (MODE == kNormStats) {
    statistics([&](int g, float mean, float m2) {
      ((float2*)a.part)[(size_t)(ng0 + g) * a.slices + k] = make_float2(mean, m2);
    });
    return;
  } else if (MODE == kNormApply) {
    for (int i = threadIdx.x; i < w.ng; i += blockDim.x) {
      gm[i] = a.mean[ng0 + i];
      gr[i] = a.rstd[ng0 + i];
    }
  } else {
    __shared__ uint32_t tag;
    const int cluster = n * a.bands + b, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    if (threadIdx.x == 0) tag = joint_tag(a.counter + cluster, a.slices);
    __syncthreads();
    Joint jt{a.words + (size_t)ng0 * a.slices * 2, a.totals + (size_t)ng0 * 2, tag, __builtin_readsteadycounter() + a.patience};
    // groups first, first + step, ... of the band, a wave each
    auto totals = [&](int first, int every, bool publish, bool last) {
      bool ok = true;
      for (int g = first + every * wave; g < w.ng && ok; g += every * waves) {
        float mean, rstd;
        ok = combine_joint(a, DEFT_CHANNELS_LAST, jt, w.ng, g, mean, rstd);
        if (last && !ok) {
          mean = rstd = __builtin_nanf("");
          ok = true;
        }
        if (ok && (threadIdx.x & 63) == 0) {
          gm[g] = mean;
          gr[g] = rstd;
          if (publish) {
            Joint::put(jt.total + 2 * g, mean, jt.tag);
            Joint::put(jt.total + 2 * g + 1, rstd, jt.tag);
          }
        }
      }
      return ok;
    };
    for (int slice = k, alone = 0;;) {
      statistics([&](int g, float mean, float m2) { jt.publish(slice, w.ng, g, mean, m2); });
      if (alone == 2) {
        totals(0, 1, !a.direct, true);
        break;
      }
      if (!alone) {
        bool ok = a.direct ? totals(0, 1, false, false) : totals(k, a.slices, true, false);
        if (!a.direct)
          for (int g = threadIdx.x; g < w.ng && ok; g += blockDim.x)
            ok = jt.wait([&] { return jt.read(jt.total + 2 * g, gm[g], gr[g]); });
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
    __syncthreads();
    if (k == 0)
      for (int i = threadIdx.x; i < w.ng; i += blockDim.x) {
        a.mean[ng0 + i] = gm[i];
        a.rstd[ng0 + i] = gr[i];
      }
  }
  __syncthreads();
  if (w.ty >= w.TY) return;
  float mu[V], ga[V], be[V];
  int gi = w.col / per, next = (gi + 1) * per - w.col;
  gi -= w.g0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    mu[j] = gm[gi];
    ga[j] = gam[w.col - w.c0 + j] * gr[gi];
    be[j] = bet[w.col - w.c0 + j];
    if (--next == 0) { next = per; ++gi; }
  }
  // z from x - mean, as the backward computes it: with the mean in the bias, the
  // rounding of mean * gamma * rstd would stay, 0.006 in a constant group of 1000s,
  // whose z is beta
  T* yp = (T*)a.out + at;
  with_act(a.act, [&](auto act) {
    T* p = yp;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      apart();
      if (u < mine) {
        float f[V];
        q[u].keep();
        q[u].get(f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          f[j] = act_of<T, decltype(act)::value>(__builtin_fmaf(f[j] - mu[j], ga[j], be[j]));
        }
        Chunk<T, V>::store(p, f);
        p += step;
      }
    }
  });
}

// Channels first: slice (kr, ks) of a group of an image: channels kr * rp ...,
// positions ks * cp ....  Teams of 2^lt lanes walk a channel's positions.
// Bound by memory: 16x256x56x56 bf16 takes 12 to 13 us in one slice a group (4.3
// TB/s), 2x320x65536 bf16 41 joined (4.1 TB/s).
// part: [n][g][slices]{mean, M2}.
template <typename T, int V, int U, int MODE>
__global__ __launch_bounds__(kNormThreads, MODE == kNormJoint ? 4 : 1) void k_norm_fwd_first(const NormArgs a) {
  extern __shared__ float lds[];
  const int id = MODE == kNormJoint ? blockIdx.x : xcd_swizzle(blockIdx.x, gridDim.x);
  const int ng = id / a.slices, k = id - ng * a.slices, g = ng % a.g;
  const int t = 1 << a.lt, ln = threadIdx.x & (t - 1), tm = threadIdx.x >> a.lt, teams = blockDim.x >> a.lt;
  float* gam = lds + 32;
  float* bet = gam + a.rp;
  int r0, c0, rows, cols, chunks, ic, rounds;
  // round u: channel tm + teams * (u / ic), chunk ln + t * (u % ic); a ragged
  // row's last chunk starts early enough to end with the row
  auto slot = [&](int row, int i, int& pos, int& shift) {
    const uint32_t want = (uint32_t)c0 + (uint32_t)i * V;  // past a row of 2^31 - 1, too
    pos = want + V <= (uint32_t)a.s ? (int)want : a.s - V;  // s >= V
    shift = (int)(want - pos);
    return row < rows && i < chunks;
  };
  Chunk<T, V> q[U];
  size_t base;
  auto load = [&](int slice) {
    const int kr = slice / a.ws, ks = slice - kr * a.ws;
    r0 = kr * a.rp;
    rows = min(a.rp, a.per - r0);
    c0 = ks * a.cp;
    cols = min(a.cp, a.s - c0);
    chunks = (cols + V - 1) / V;
    ic = (chunks + t - 1) >> a.lt;
    rounds = (rows + teams - 1) / teams * ic;
    base = ((size_t)ng * a.per + r0) * a.s;
    const T* xp = (const T*)a.x + base;
    const int first = anew(ln);
    int row = tm, i = first;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      apart();
      int pos, shift;
      slot(row, i, pos, shift);
      q[u].load(xp + (size_t)min(row, rows - 1) * a.s + pos);  // past the end: what is there, unused
      i += t;
      if (i - first >= ic * t) { i = first; row += teams; }
    }
  };
  const int ch = g * a.per + k / a.ws * a.rp, chs = MODE == kNormStats ? 0 : min(a.rp, a.per - k / a.ws * a.rp);
  const Ahead<T> gamma((const T*)a.gamma + ch, chs), beta((const T*)a.beta + ch, chs);
  load(k);
  gamma.put(gam);
  beta.put(bet);
  const bool ragged = a.s % V != 0;
  float mean, rstd;
  // mean and M2 of the loaded slice, in every thread
  auto statistics = [&](float& m, float& m2) {
    const double inv_count = 1.0 / ((double)rows * cols);
    float sum[4] = {}, sq[4] = {};
    int first = anew(ln);
    int row = tm, i = first;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      apart();
      int pos, shift;
      q[u].zero_if(!slot(row, i, pos, shift));
      Chunk<T, V> x = q[u];
      if (ragged) x.zero_below(shift);
      i += t;
      if (i - first >= ic * t) { i = first; row += teams; }
      if constexpr (sizeof(T) == 2 && V == 8) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x.moments(j, sum[j], sq[j]);
      } else {
        float f[V];
        x.get(f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          sum[j] += f[j];
          if (sizeof(T) == 2) sq[j] = __builtin_fmaf(f[j], f[j], sq[j]);
        }
      }
    }
    const float all = (sum[0] + sum[1]) + (sum[2] + sum[3]);
    double v1 = all, v2 = 0.0;
    if constexpr (sizeof(T) == 2) {
      v2 = (sq[0] + sq[1]) + (sq[2] + sq[3]);
    } else {
      // squares about the thread's own mean
      int own = 0;
      row = tm, i = first = anew(ln);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        apart();
        int pos, shift;
        own += slot(row, i, pos, shift) ? V - shift : 0;
        i += t;
        if (i - first >= ic * t) { i = first; row += teams; }
      }
      const float mean = all / (float)max(own, 1);
      float v = 0.f;
      row = tm, i = first = anew(ln);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        apart();
        int pos, shift;
        const bool ok = slot(row, i, pos, shift);
        i += t;
        if (i - first >= ic * t) { i = first; row += teams; }
        float f[V];
        q[u].get(f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float d = ok && j >= shift ? f[j] - mean : 0.f;
          v = __builtin_fmaf(d, d, v);
        }
      }
      v2 = (double)v + (double)mean * (2.0 * (double)all - (double)own * (double)mean);  // as above
    }
    block_sums(v1, v2, (double*)lds);
    v2 -= v1 * v1 * inv_count;
    m = (float)(v1 * inv_count);
    m2 = v2 < 0.0 ? 0.f : (float)v2;  // a NaN stays
  };
  if (MODE == kNormWhole) {
    float m2;
    statistics(mean, m2);
    rstd = 1.f / __builtin_sqrtf(m2 / ((float)a.s * (float)a.per) + a.eps);
    if (threadIdx.x == 0) {
      a.mean[ng] = mean;
      a.rstd[ng] = rstd;
    }
  } else if (MODE == kNormStats) {
    float m2;
    statistics(mean, m2);
    if (threadIdx.x == 0) ((float2*)a.part)[(size_t)ng * a.slices + k] = make_float2(mean, m2);
    return;
  } else if (MODE == kNormApply) {
    mean = a.mean[ng];
    rstd = a.rstd[ng];
    __syncthreads();
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
        ok = combine_joint(a, DEFT_CHANNELS_FIRST, jt, 1, 0, mean, rstd);
        if (threadIdx.x == 0) { got[0] = mean; got[1] = rstd; }
      }
      ok = __syncthreads_and(ok);
      mean = got[0];
      rstd = got[1];
      return ok;
    };
    for (int slice = k, alone = 0;;) {
      float m2;
      statistics(mean, m2);
      if (threadIdx.x == 0) jt.publish(slice, 1, 0, mean, m2);
      if (alone == 2) {
        if (!join()) mean = rstd = __builtin_nanf("");
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
    if (k == 0 && threadIdx.x == 0) {
      a.mean[ng] = mean;
      a.rstd[ng] = rstd;
    }
  }
  T* yp = (T*)a.out + base;
  with_act(a.act, [&](auto act) {
    const int first = anew(ln);
    int row = tm, i = first;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      apart();
      int pos, shift;
      const bool ok = slot(row, i, pos, shift);
      if (u < rounds && ok) {
        const float ga = gam[row] * rstd, be = bet[row];
        float f[V];
        q[u].keep();
        q[u].get(f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          f[j] = act_of<T, decltype(act)::value>(__builtin_fmaf(f[j] - mean, ga, be));
        }
        Chunk<T, V>::store(yp + (size_t)row * a.s + pos, f);
      }
      i += t;
      if (i - first >= ic * t) { i = first; row += teams; }
    }
  });
}

// mean and rstd of each group of each image from its slices.
__global__ __launch_bounds__(256) void k_norm_combine(const NormArgs a, int layout) {
  __shared__ double lds[8];
  const int ng = blockIdx.x;
  const float2* p = (const float2*)a.part + (size_t)ng * a.slices;
  Combine c;
#pragma unroll 4
  for (int k = threadIdx.x; k < a.slices; k += 256) c.add(slice_count(a, layout, k), p[k].x, p[k].y);
  block_sums(c.sum, c.squares, lds);
  float mean, rstd;
  c.finish(a, mean, rstd);
  if (threadIdx.x == 0) {
    a.mean[ng] = mean;
    a.rstd[ng] = rstd;
  }
}

template <typename T, int V, int U, int MODE>
hipError_t launch(const NormArgs& a, const NormPlan& p, int layout, hipStream_t st) {
  const dim3 grid(p.blocks), block(p.threads);
  if (layout == DEFT_CHANNELS_LAST)
    DEFT_LAUNCH("norm_fwd", (k_norm_fwd_last<T, V, U, MODE>), grid, block, p.lds, st, a);
  else
    DEFT_LAUNCH("norm_fwd", (k_norm_fwd_first<T, V, U, MODE>), grid, block, p.lds, st, a);
  return hipGetLastError();
}

template <typename T, int V, int U>
hipError_t launch_mode(const NormArgs& a, const NormPlan& p, int layout, int mode, hipStream_t st) {
  if (mode == kNormWhole) return launch<T, V, U, kNormWhole>(a, p, layout, st);
  if constexpr (U <= 8 || V == 1) {  // slices have no more
    if (mode == kNormJoint) return launch<T, V, U, kNormJoint>(a, p, layout, st);
    if (mode == kNormStats) return launch<T, V, U, kNormStats>(a, p, layout, st);
    if (mode == kNormApply) return launch<T, V, U, kNormApply>(a, p, layout, st);
  }
  return hipErrorInvalidValue;
}

template <typename T>
hipError_t launch_t(const NormArgs& a, const NormPlan& p, int layout, int mode, hipStream_t st) {
  constexpr int V = Elem<T>::VEC;
  if (p.vec == 1) return launch_mode<T, 1, 16>(a, p, layout, mode, st);
  if (p.u <= 4) return launch_mode<T, V, 4>(a, p, layout, mode, st);
  if (p.u <= 8) return launch_mode<T, V, 8>(a, p, layout, mode, st);
  if (p.u <= 16) return launch_mode<T, V, 16>(a, p, layout, mode, st);
  return launch_mode<T, V, 32>(a, p, layout, mode, st);
}

}  // namespace

hipError_t launch_norm_fwd(const NormArgs& a, const NormPlan& p, int layout, int dtype, int mode, hipStream_t st) {
  if (p.u > (p.vec == 1 ? 16 : 32)) return hipErrorInvalidValue;
  return dtype == DEFT_BF16 ? launch_t<bf16_t>(a, p, layout, mode, st) : launch_t<float>(a, p, layout, mode, st);
}

hipError_t launch_norm_combine(const NormArgs& a, int layout, hipStream_t st) {
  DEFT_LAUNCH("norm_combine", k_norm_combine, dim3((unsigned)(a.n * a.g)), dim3(256), 0, st, a, layout);
  return hipGetLastError();
}

}  // namespace deft
