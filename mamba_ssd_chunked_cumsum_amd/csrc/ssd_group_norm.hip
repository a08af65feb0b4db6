// Group norm with its activation, channels last: n = (x - mean) rstd over each sequence's tokens and a
// group's channels, v = n w + b, y = v / (1 + exp(-v)); forward and backward.
//
// A few operations for each element: bound by memory. Where a sequence's tokens fit a thread's
// registers (up to 8 of them), a block holds whole groups of them and each element is loaded once.
// Longer sequences are cut into strips of rows: one kernel leaves each strip's mean and squared
// deviations (backward: sums of dv and dv n) of every channel, so that a group may have any number of
// channels; one adds them up, one applies them. The second pass over x (and dy) finds what the last-
// level cache kept.
//
// Squared deviations are taken from a value of the strip itself (its first row, channel by channel):
// their sum about that value is at most n + 1 times the sum about the mean for n rows, so the
// difference keeps all but a few bits wherever the mean lies.
#include "ssd_recurrent.h"
#include "ssd_rows.h"

namespace ssd {

namespace {

constexpr int V = 8, kStrip = 64, kTile = 64 * V, kThreads = 256, kWaves = kThreads / 64;
constexpr int kHeld = 8;       // tokens that a thread holds
constexpr int kBlockC = 2048;  // channels of a block that holds whole groups

__device__ __forceinline__ float act_slope(float v) {  // of v sigmoid(v)
  const float s = sigmoid(v);
  return s * fmaf(v, 1.f - s, 1.f);
}

// A strip of one sequence, or of all rows (packed: the part of each sequence in it has a slot of
// its own, strip + sequence, which grows by one from each part to the next).
struct Strips {
  int per, n;     // strips of a sequence (dense), strips
  int64_t slots;  // partial results
};
Strips strips_of(const Rows& q) {
  Strips t;
  const int64_t rows = q.starts ? q.R : q.L;
  t.per = (int)((rows + kStrip - 1) / kStrip);
  t.n = q.starts ? t.per : (int)((int64_t)t.per * q.S);
  t.slots = q.starts ? (int64_t)t.n + q.S : t.n;
  return t;
}

// f(sequence, slot, first row, rows) for each part of a sequence in a strip; uniform over the block.
template <typename F>
__device__ __forceinline__ void parts(const Rows& q, int per, int strip, F f) {
  if (!q.starts) {
    const int s = strip / per, at = strip % per * kStrip;
    f(s, (int64_t)strip, s * q.L + at, min(q.L - at, kStrip));
    return;
  }
  const int stop = min(q.R - strip * kStrip, kStrip) + strip * kStrip;
  for (int r = strip * kStrip; r < stop;) {
    const int s = seq_of(q, r);
    if (s < 0) {
      r = after_gap(q, r);
      continue;
    }
    const int end = min(seq_end(q, s), stop);
    f(s, (int64_t)strip + s, r, end - r);
    r = end;
  }
}

// Slots of sequence s: n of them from the first; rows of the i-th.
struct Slots {
  int begin, end, strip0, n;
  int64_t first;
  __device__ __forceinline__ Slots(const Rows& q, int per, int s) {
    begin = seq_begin(q, s);
    end = max(seq_end(q, s), begin);
    if (q.starts) {
      strip0 = begin / kStrip;
      first = (int64_t)strip0 + s;
      n = end > begin ? (end - 1) / kStrip - strip0 + 1 : 0;
    } else {
      strip0 = 0;
      first = (int64_t)s * per;
      n = per;
    }
  }
  __device__ __forceinline__ int rows(const Rows& q, int i) const {
    if (!q.starts) return min(q.L - i * kStrip, kStrip);
    const int at = (strip0 + i) * kStrip;
    return min(end, q.R - at > kStrip ? at + kStrip : q.R) - max(begin, at);
  }
};

// Sums over the waves of a block, in order, in wave 0. red: [waves][64 * 2 V].
template <int N>
__device__ __forceinline__ void add_waves(float (&v)[N], float (&red)[kWaves][N][64]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) red[wave][i][lane] = v[i];
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = ((v[i] + red[1][i][lane]) + red[2][i][lane]) + red[3][i][lane];
  }
}

__device__ __forceinline__ double block_sum(double v, double (&red)[kWaves]) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, kWave);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return ((red[0] + red[1]) + red[2]) + red[3];
}

// ---- strips: forward ---------------------------------------------------------------------------------
// part [slots, 2, C]: means, sums of squared deviations.
template <typename IO>
__global__ __launch_bounds__(kThreads) void k_gn_parts(GroupArgs q, int per, int tiles, float* part) {
  __shared__ float red[kWaves][2 * V][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c0 = (int)(blockIdx.x % tiles) * kTile + lane * V;
  const bool live = c0 < q.C;
  const int c = live ? c0 : q.C - V;
  const IO* x = (const IO*)q.x + c;
  parts(q.rows, per, (int)(blockIdx.x / tiles), [&](int, int64_t slot, int r, int n) {
    Vec<IO, V> first, v;
    float sum[2 * V];
    first.load(x + r * q.xs);
#pragma unroll
    for (int j = 0; j < 2 * V; ++j) sum[j] = 0.f;
#pragma unroll 4
    for (int i = wave; i < n; i += kWaves) {
      v.load(x + (int64_t)(r + i) * q.xs);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = v.get(j) - first.get(j);
        sum[j] += d;
        sum[V + j] = fmaf(d, d, sum[V + j]);
      }
    }
    add_waves(sum, red);
    if (wave == 0 && live) {
      float mean[V], dev[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = sum[j] / n;
        mean[j] = first.get(j) + d;
        dev[j] = fmaxf(fmaf(-d, sum[j], sum[V + j]), 0.f);
      }
      store_vec<float, V>(part + slot * 2 * q.C + c, mean);
      store_vec<float, V>(part + (slot * 2 + 1) * q.C + c, dev);
    }
  });
}

// A block a sequence and group: stats [S, G, 2], mean and 1 / sqrt(variance + eps); (0, 1 / sqrt(eps))
// of a sequence without tokens. Sums in 64 bits: a thread adds as many values as the sequence is long.
__global__ __launch_bounds__(kThreads) void k_gn_stats(GroupArgs q, int per, const float* part,
                                                       float* stats) {
  __shared__ double red[kWaves];
  const int s = (int)(blockIdx.x / q.G), g = (int)(blockIdx.x % q.G), cg = q.C / q.G;
  const Slots at(q.rows, per, s);
  const double count = (double)(at.end - at.begin) * cg;
  const int64_t all = (int64_t)at.n * cg;
  double sum = 0.;
  for (int64_t i = threadIdx.x; i < all; i += kThreads) {
    const int slot = (int)(i / cg), c = g * cg + (int)(i % cg);
    sum += (double)at.rows(q.rows, slot) * part[(at.first + slot) * 2 * q.C + c];
  }
  const double mean = at.n ? block_sum(sum, red) / count : 0.;
  double dev = 0.;
  for (int64_t i = threadIdx.x; i < all; i += kThreads) {
    const int slot = (int)(i / cg), c = g * cg + (int)(i % cg);
    const float* p = part + (at.first + slot) * 2 * q.C + c;
    const double d = p[0] - mean;
    dev += at.rows(q.rows, slot) * d * d + p[q.C];
  }
  const double var = at.n ? block_sum(dev, red) / count : 0.;
  if (threadIdx.x == 0) {
    stats[2 * (int64_t)blockIdx.x] = (float)mean;
    stats[2 * (int64_t)blockIdx.x + 1] = (float)(1. / sqrt(var + q.eps));
  }
}

// w rstd, mean and b of a thread's channels in sequence s.
struct Affine {
  float w[V], b[V];
  __device__ __forceinline__ Affine(const GroupArgs& q, int c) {
#pragma unroll
    for (int j = 0; j < V; ++j) w[j] = 1.f, b[j] = 0.f;
    if (q.w) load_f32<V>(q.w + c, w);
    if (q.b) load_f32<V>(q.b + c, b);
  }
};
__device__ __forceinline__ void load_stats(const GroupArgs& q, const float* stats, int s, int c,
                                           float (&mean)[V], float (&rstd)[V]) {
  const int cg = q.C / q.G;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const float2 st = reinterpret_cast<const float2*>(stats)[(int64_t)s * q.G + (c + j) / cg];
    mean[j] = st.x;
    rstd[j] = st.y;
  }
}

template <typename IO>
__global__ __launch_bounds__(kThreads) void k_gn_apply(GroupArgs q, int per, int tiles,
                                                       const float* stats, IO* y) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = (int)(blockIdx.x % tiles) * kTile + lane * V;
  if (c >= q.C) return;
  const IO* x = (const IO*)q.x + c;
  const Affine af(q, c);
  parts(q.rows, per, (int)(blockIdx.x / tiles), [&](int s, int64_t, int r, int n) {
    float mean[V], rstd[V], o[V];
    load_stats(q, stats, s, c, mean, rstd);
#pragma unroll 4
    for (int i = wave; i < n; i += kWaves) {
      Vec<IO, V> v;
      v.load(x + (int64_t)(r + i) * q.xs);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        o[j] = fmaf((v.get(j) - mean[j]) * rstd[j], af.w[j], af.b[j]);
        if (q.act) o[j] *= sigmoid(o[j]);
      }
      store_vec<IO, V>(y + (int64_t)(r + i) * q.C + c, o);
    }
  });
}

// ---- strips: backward --------------------------------------------------------------------------------
// part [slots, 2, C]: sums of dv and of dv n over a part's rows.
template <typename IO>
__global__ __launch_bounds__(kThreads) void k_gn_bwd_parts(GroupArgs q, int per, int tiles,
                                                           const float* stats, const IO* dy,
                                                           float* part) {
  __shared__ float red[kWaves][2 * V][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c0 = (int)(blockIdx.x % tiles) * kTile + lane * V;
  const bool live = c0 < q.C;
  const int c = live ? c0 : q.C - V;
  const IO* x = (const IO*)q.x + c;
  const Affine af(q, c);
  parts(q.rows, per, (int)(blockIdx.x / tiles), [&](int s, int64_t slot, int r, int n) {
    float mean[V], rstd[V], sum[2 * V];
    load_stats(q, stats, s, c, mean, rstd);
#pragma unroll
    for (int j = 0; j < 2 * V; ++j) sum[j] = 0.f;
#pragma unroll 4
    for (int i = wave; i < n; i += kWaves) {
      Vec<IO, V> v, d;
      v.load(x + (int64_t)(r + i) * q.xs);
      d.load(dy + (int64_t)(r + i) * q.C + c);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float nv = (v.get(j) - mean[j]) * rstd[j];
        float dv = d.get(j);
        if (q.act) dv *= act_slope(fmaf(nv, af.w[j], af.b[j]));
        sum[j] += dv;
        sum[V + j] = fmaf(dv, nv, sum[V + j]);
      }
    }
    add_waves(sum, red);
    if (wave == 0 && live) {
      float a[V], b[V];
#pragma unroll
      for (int j = 0; j < V; ++j) a[j] = sum[j], b[j] = sum[V + j];
      store_vec<float, V>(part + slot * 2 * q.C + c, a);
      store_vec<float, V>(part + (slot * 2 + 1) * q.C + c, b);
    }
  });
}

// Sums over a sequence's slots, in 64 bits: total [S, 2, C]. 64 columns a block, four groups of slots.
__global__ __launch_bounds__(kThreads) void k_gn_bwd_total(GroupArgs q, int per, int cols,
                                                           const float* part, float* total) {
  __shared__ double red[kWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int s = (int)(blockIdx.x / cols);
  const int64_t m = (int64_t)(blockIdx.x % cols) * 64 + lane, M = 2 * (int64_t)q.C;
  const Slots at(q.rows, per, s);
  double sum = 0.;
  if (m < M) {
#pragma unroll 4
    for (int i = wave; i < at.n; i += kWaves) sum += part[(at.first + i) * M + m];
  }
  red[wave][lane] = sum;
  __syncthreads();
  if (wave == 0 && m < M)
    total[s * M + m] = (float)(((sum + red[1][lane]) + red[2][lane]) + red[3][lane]);
}

// Means over each sequence and group of g = dv w and of g n: mid [S, G, 2]. A wave each.
__global__ __launch_bounds__(kThreads) void k_gn_bwd_means(GroupArgs q, const float* total, float* mid) {
  const int64_t u = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (u >= (int64_t)q.rows.S * q.G) return;
  const int s = (int)(u / q.G), g = (int)(u % q.G), cg = q.C / q.G;
  float a = 0.f, b = 0.f;
  for (int i = threadIdx.x & 63; i < cg; i += 64) {
    const int c = g * cg + i;
    const float w = q.w ? q.w[c] : 1.f;
    const float* t = total + (int64_t)s * 2 * q.C + c;
    a = fmaf(w, t[0], a);
    b = fmaf(w, t[q.C], b);
  }
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
    a += __shfl_xor(a, m, kWave);
    b += __shfl_xor(b, m, kWave);
  }
  const float count = (float)max(seq_end(q.rows, s) - seq_begin(q.rows, s), 1) * cg;
  if ((threadIdx.x & 63) == 0)
    reinterpret_cast<float2*>(mid)[u] = make_float2(a / count, b / count);
}

// dx = rstd (g - mean(g) - n mean(g n)); zero in rows of no sequence.
template <typename IO>
__global__ __launch_bounds__(kThreads) void k_gn_bwd_apply(GroupArgs q, int per, int tiles,
                                                           const float* stats, const float* mid,
                                                           const IO* dy, IO* dx) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = (int)(blockIdx.x % tiles) * kTile + lane * V;
  if (c >= q.C) return;
  const IO* x = (const IO*)q.x + c;
  const Affine af(q, c);
  const int strip = (int)(blockIdx.x / tiles);
  float o[V];
  if (q.rows.starts) {
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = 0.f;
    const int stop = min(q.rows.R - strip * kStrip, kStrip);
    for (int i = wave; i < stop; i += kWaves)
      if (seq_of(q.rows, strip * kStrip + i) < 0)
        store_vec<IO, V>(dx + (int64_t)(strip * kStrip + i) * q.C + c, o);
  }
  parts(q.rows, per, strip, [&](int s, int64_t, int r, int n) {
    float mean[V], rstd[V], m1[V], m2[V];
    load_stats(q, stats, s, c, mean, rstd);
    load_stats(q, mid, s, c, m1, m2);
#pragma unroll 4
    for (int i = wave; i < n; i += kWaves) {
      Vec<IO, V> v, d;
      v.load(x + (int64_t)(r + i) * q.xs);
      d.load(dy + (int64_t)(r + i) * q.C + c);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float nv = (v.get(j) - mean[j]) * rstd[j];
        float g = d.get(j) * af.w[j];
        if (q.act) g *= act_slope(fmaf(nv, af.w[j], af.b[j]));
        o[j] = rstd[j] * (g - m1[j] - nv * m2[j]);
      }
      store_vec<IO, V>(dx + (int64_t)(r + i) * q.C + c, o);
    }
  });
}

// ---- sequences of a few tokens -----------------------------------------------------------------------
// Dense sequences of up to kHeld tokens, groups of a multiple of 8 up to kBlockC channels: a block
// takes `groups` whole groups of `seqs` sequences at a time, a thread eight channels and all tokens.
struct Few {
  int groups, slices, width, seqs;  // slices of a sequence; threads of a slice
};
bool few_tokens(const GroupArgs& a) {
  const int cg = a.C / a.G;
  return !a.rows.starts && a.rows.L <= kHeld && cg % V == 0 && cg <= kBlockC;
}
Few few_of(const GroupArgs& a) {
  Few f;
  const int cg = a.C / a.G;
  f.groups = kBlockC / cg < a.G ? kBlockC / cg : a.G;
  f.slices = (a.G + f.groups - 1) / f.groups;
  f.groups = (a.G + f.slices - 1) / f.slices;  // even slices
  f.width = f.groups * cg / V;
  f.seqs = kThreads / f.width;
  return f;
}

// Sum over a group, whose threads are neighbours: from one value of each.
__device__ __forceinline__ float group_sum(float v, float* red, int first, int n) {
  __syncthreads();
  red[threadIdx.x] = v;
  __syncthreads();
  float sum = 0.f;
  for (int i = 0; i < n; ++i) sum += red[first + i];
  return sum;
}

template <typename IO>
__global__ __launch_bounds__(kThreads) void k_gn_few(GroupArgs q, Few f, float* stats, IO* y) {
  __shared__ float red[kThreads];
  const int cg = q.C / q.G, vg = cg / V, L = q.rows.L;
  const int t = threadIdx.x % f.width, at = threadIdx.x / f.width;
  const int slice = (int)(blockIdx.x % f.slices);
  const int64_t s = (int64_t)(blockIdx.x / f.slices) * f.seqs + at;
  const int c = slice * f.groups * cg + t * V;
  const bool live = at < f.seqs && s < q.rows.S && c < q.C;
  const int first = threadIdx.x - t % vg;
  Vec<IO, V> v[kHeld];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (i < L) {
      v[i].zero();
      if (live) v[i].load((const IO*)q.x + (s * L + i) * q.xs + c);
#pragma unroll
      for (int j = 0; j < V; ++j) sum += v[i].get(j);
    }
  // (threads past the last slice's groups, and of no sequence, add up zeros of their own)
  const int n = min(vg, kThreads - first);
  const float mean = group_sum(sum, red, first, n) / (float)(L * cg);
  float dev = 0.f;
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (i < L) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = v[i].get(j) - mean;
        dev = fmaf(d, d, dev);
      }
    }
  const float rstd = 1.f / sqrtf(group_sum(dev, red, first, n) / (float)(L * cg) + q.eps);
  if (!live) return;
  if (stats && t % vg == 0)
    reinterpret_cast<float2*>(stats)[s * q.G + c / cg] = make_float2(mean, rstd);
  const Affine af(q, c);
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (i < L) {
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        o[j] = fmaf((v[i].get(j) - mean) * rstd, af.w[j], af.b[j]);
        if (q.act) o[j] *= sigmoid(o[j]);
      }
      store_vec<IO, V>(y + (s * L + i) * q.C + c, o);
    }
}

// Backward: a block walks sequences and keeps the sums for dw and db of its channels in registers.
// part [walkers, 2, C]: db, dw.
template <typename IO>
__global__ __launch_bounds__(kThreads) void k_gn_few_bwd(GroupArgs q, Few f, int walkers,
                                                         const float* stats, const IO* dy, IO* dx,
                                                         float* part) {
  __shared__ float red[2][kThreads];
  const int cg = q.C / q.G, vg = cg / V, L = q.rows.L;
  const int t = threadIdx.x % f.width, at = threadIdx.x / f.width;
  const int slice = (int)(blockIdx.x % f.slices), walker = (int)(blockIdx.x / f.slices);
  const int c = slice * f.groups * cg + t * V;
  const bool mine = at < f.seqs && c < q.C;
  const int first = threadIdx.x - t % vg, n = min(vg, kThreads - first);
  const Affine af(q, mine ? c : 0);
  float dw[V], db[V];
#pragma unroll
  for (int j = 0; j < V; ++j) dw[j] = db[j] = 0.f;
  for (int64_t s0 = (int64_t)walker * f.seqs; s0 < q.rows.S; s0 += (int64_t)walkers * f.seqs) {
    const int64_t s = s0 + at;
    const bool live = mine && s < q.rows.S;
    Vec<IO, V> v[kHeld], d[kHeld];
    float2 st = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (i < L) {
        v[i].zero();
        d[i].zero();
        if (live) {
          v[i].load((const IO*)q.x + (s * L + i) * q.xs + c);
          d[i].load(dy + (s * L + i) * q.C + c);
        }
      }
    if (live) st = reinterpret_cast<const float2*>(stats)[s * q.G + c / cg];
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (i < L) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float nv = (v[i].get(j) - st.x) * st.y;
          float dv = d[i].get(j);
          if (q.act) dv *= act_slope(fmaf(nv, af.w[j], af.b[j]));
          db[j] += dv;
          dw[j] = fmaf(dv, nv, dw[j]);
          a = fmaf(dv, af.w[j], a);
          b = fmaf(dv * af.w[j], nv, b);
        }
      }
    const float m1 = group_sum(a, red[0], first, n) / (float)(L * cg);
    const float m2 = group_sum(b, red[1], first, n) / (float)(L * cg);
    if (live) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i)
        if (i < L) {
          float o[V];
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float nv = (v[i].get(j) - st.x) * st.y;
            float g = d[i].get(j) * af.w[j];
            if (q.act) g *= act_slope(fmaf(nv, af.w[j], af.b[j]));
            o[j] = st.y * (g - m1 - nv * m2);
          }
          store_vec<IO, V>(dx + (s * L + i) * q.C + c, o);
        }
    }
  }
  if (mine) {
    float* p = part + ((int64_t)walker * f.seqs + at) * 2 * q.C + c;
    store_vec<float, V>(p, db);
    store_vec<float, V>(p + q.C, dw);
  }
}

// Blocks of a slice that walk the sequences: at most 1024 in all, at least 4 turns each.
int walkers_of(const GroupArgs& a, const Few& f) {
  const int64_t turns = ((int64_t)a.rows.S + f.seqs - 1) / f.seqs;
  const int64_t want = (turns + 3) / 4, most = 1024 / f.slices;
  return (int)(want < most ? want : most < 1 ? 1 : most);
}

int tiles_of(const GroupArgs& a) { return (a.C + kTile - 1) / kTile; }

int64_t up64(int64_t floats) { return (floats + 63) / 64 * 64; }

}  // namespace

int64_t group_norm_bytes(const GroupArgs& a) {
  if (few_tokens(a)) return 0;
  const Strips t = strips_of(a.rows);
  return 4 * (up64(t.slots * 2 * a.C) + (int64_t)a.rows.S * a.G * 2);
}

bool group_norm_fits(const GroupArgs& a) {
  auto fits = [](double blocks) { return blocks * kThreads < 4294967296.0; };
  if (few_tokens(a)) {
    const Few f = few_of(a);
    return fits((double(a.rows.S) / f.seqs + 1) * f.slices);
  }
  const double strips = a.rows.starts ? double(a.rows.R) / kStrip + 1
                                      : (double(a.rows.L) / kStrip + 1) * a.rows.S;
  const double slots = strips + (a.rows.starts ? a.rows.S : 0);
  return fits(strips * tiles_of(a)) && fits(double(a.rows.S) * a.G) &&
         fits(double(a.rows.S) * (a.C / 32 + 1)) && slots * 2 * a.C < 1099511627776.0;
}

hipError_t launch_group_norm(const GroupArgs& a, void* y, float* stats, float* ws, hipStream_t s) {
  auto run = [&](auto io) {
    using IO = decltype(io);
    if (few_tokens(a)) {
      const Few f = few_of(a);
      const int64_t blocks = ((int64_t)a.rows.S + f.seqs - 1) / f.seqs * f.slices;
      hipLaunchKernelGGL((k_gn_few<IO>), dim3((unsigned)blocks), dim3(kThreads), 0, s, a, f, stats,
                         (IO*)y);
      return hipGetLastError();
    }
    const Strips t = strips_of(a.rows);
    const int tiles = tiles_of(a);
    if (!stats) stats = ws + up64(t.slots * 2 * a.C);
    const dim3 grid((unsigned)((int64_t)t.n * tiles));
    hipLaunchKernelGGL((k_gn_parts<IO>), grid, dim3(kThreads), 0, s, a, t.per, tiles, ws);
    hipLaunchKernelGGL(k_gn_stats, dim3((unsigned)((int64_t)a.rows.S * a.G)), dim3(kThreads), 0, s, a,
                       t.per, ws, stats);
    hipLaunchKernelGGL((k_gn_apply<IO>), grid, dim3(kThreads), 0, s, a, t.per, tiles, stats, (IO*)y);
    return hipGetLastError();
  };
  return a.io == kIoBf16 ? run(u16{}) : run(float{});
}

int64_t group_norm_backward_bytes(const GroupArgs& a) {
  if (few_tokens(a)) {
    const Few f = few_of(a);
    return 4 * (int64_t)walkers_of(a, f) * f.seqs * 2 * a.C;
  }
  const Strips t = strips_of(a.rows);
  return 4 * (up64(t.slots * 2 * a.C) + up64((int64_t)a.rows.S * 2 * a.C) +
              (int64_t)a.rows.S * a.G * 2);
}

hipError_t launch_group_norm_backward(const GroupArgs& a, const float* stats, const void* dy, void* dx,
                                      float* dw, float* db, float* ws, hipStream_t s) {
  auto run = [&](auto io) {
    using IO = decltype(io);
    if (few_tokens(a)) {
      const Few f = few_of(a);
      const int w = walkers_of(a, f);
      hipLaunchKernelGGL((k_gn_few_bwd<IO>), dim3((unsigned)((int64_t)w * f.slices)), dim3(kThreads), 0,
                         s, a, f, w, stats, (const IO*)dy, (IO*)dx, ws);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess || !(dw || db)) return e;
      return launch_column_sums(ws, w * f.seqs, 0, nullptr, 1, 0, 0, a.C, db, a.C, dw, s);
    }
    const Strips t = strips_of(a.rows);
    const int tiles = tiles_of(a), cols = (2 * a.C + 63) / 64;
    float* total = ws + up64(t.slots * 2 * a.C);
    float* mid = total + up64((int64_t)a.rows.S * 2 * a.C);
    const dim3 grid((unsigned)((int64_t)t.n * tiles));
    hipLaunchKernelGGL((k_gn_bwd_parts<IO>), grid, dim3(kThreads), 0, s, a, t.per, tiles, stats,
                       (const IO*)dy, ws);
    hipLaunchKernelGGL(k_gn_bwd_total, dim3((unsigned)((int64_t)a.rows.S * cols)), dim3(kThreads), 0, s,
                       a, t.per, cols, ws, total);
    hipLaunchKernelGGL(k_gn_bwd_means,
                       dim3((unsigned)(((int64_t)a.rows.S * a.G + kWaves - 1) / kWaves)),
                       dim3(kThreads), 0, s, a, total, mid);
    hipLaunchKernelGGL((k_gn_bwd_apply<IO>), grid, dim3(kThreads), 0, s, a, t.per, tiles, stats, mid,
                       (const IO*)dy, (IO*)dx);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !(dw || db)) return e;
    return launch_column_sums(total, a.rows.S, 0, nullptr, 1, 0, 0, a.C, db, a.C, dw, s);
  };
  return a.io == kIoBf16 ? run(u16{}) : run(float{});
}

}  // namespace ssd
