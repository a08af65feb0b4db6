// Group norm with its activation, channels last: n = (x - mean) rstd over each sequence's tokens and a
// group's channels, v = n w + b, y = v / (1 + exp(-v)); forward and backward.
//
// A few operations for each element: bound by memory. Where a sequence's tokens fit the registers of a
// group's threads (up to 8 tokens a thread) or of a block, each element is loaded once.
// Longer sequences are cut into strips of rows and tiles of channels: one kernel leaves the mean and
// squared deviations (backward: sums of g and g n, and what dw and db need) of every group's piece in
// every strip; the second adds up those of its groups and finds what the last-level cache kept of x
// (and dy). A group may have any number of channels. 2 x 8192 x 2560 bf16 in 32 groups: 47 us in all
// (reading x twice and writing y at a copy's rate takes 47), backward 89 (84).
//
// Squared deviations are taken from a value of the strip itself (its first row, channel by channel):
// their sum about that value is at most n + 1 times the sum about the mean for n rows, so the
// difference keeps all but a few bits wherever the mean lies. A group's channels are put together as distances
// from one of its values, too, and pieces in 64 bits from that value and the mean's distance to it.
#include <type_traits>

#include "ssd_recurrent.h"
#include "ssd_selective.h"

namespace ssd {

namespace {

constexpr int V = 8, kTile = 64 * V, kThreads = 256, kWaves = kThreads / 64;
constexpr int kBlocks = 512;   // two for each of the card's 256 compute units
constexpr int kAhead = 4;      // rows of a wave that are loaded together (2, 3, 8: no faster)
constexpr int kHeld = 8;       // tokens that a thread holds

__device__ __forceinline__ float act_slope(float v) {  // of v sigmoid(v)
  const float s = sigmoid(v);
  return s * fmaf(v, 1.f - s, 1.f);
}

// 1 / sqrt(v), to a unit in the last place (below 2^-126 the instruction would take v as zero).
__device__ __forceinline__ float inverse_root(float v) {
  return v < 0x1p-126f ? 1.f / sqrtf(v) : __builtin_amdgcn_rsqf(v);
}

// ---- how a problem is cut --------------------------------------------------------------------------
// Strips of `rows` rows, of each sequence or (packed) of all rows, where the part of each sequence in a
// strip has a slot of its own: strip + sequence, which grows by one from each part to the next. In the
// same way the piece of a group in a tile of channels is piece tile + group. In the backward pass dense
// sequences of which several fit a strip share it, `seqs` whole ones, each with its slot: what the strips leave
// of every channel for dw and db is then small beside x and soon added up (2^20 single tokens x 1000 in groups
// of 20: 0.1 GB where x has 2, not 8; 16384 x 2600 in groups of 650 1645 -> 1057 us). The forward leaves
// nothing of the kind, and the loop over sequences costs it registers (20000 x 12 tokens x 1024 387 -> 434 us).
struct Cut {
  int rows, per, strips;  // rows of a strip; strips of a sequence (packed: of all rows); strips
  int seqs;               // sequences of a strip, where several may share one
  int tiles, pieces;
  int64_t slots;
};
Cut cut_of(const GroupArgs& a, bool back) {
  Cut t;
  t.tiles = (a.C + kTile - 1) / kTile;
  t.pieces = t.tiles + a.G;
  const int64_t rows = a.rows.starts ? a.rows.R : a.rows.L, seqs = a.rows.starts ? 1 : a.rows.S;
  t.rows = 64;  // (32, 128: slower) shorter where that leaves compute units without blocks
  while (t.rows > 16 && (rows + t.rows - 1) / t.rows * seqs * t.tiles < kBlocks) t.rows /= 2;
  t.per = (int)((rows + t.rows - 1) / t.rows);
  t.seqs = !back || a.rows.starts || t.per > 1 ? 1 : t.rows / a.rows.L;
  // (as many blocks as run at once, eight a unit)
  while (t.seqs > 1 && (seqs + t.seqs - 1) / t.seqs * t.tiles < 4 * kBlocks) --t.seqs;
  t.strips = (int)(t.per * ((seqs + t.seqs - 1) / t.seqs));
  t.slots = a.rows.starts ? t.strips + (int64_t)a.rows.S : t.per * seqs;
  return t;
}

__device__ __forceinline__ int offset(const Rows& q, int i) {
  typedef const __attribute__((address_space(4))) int* Words;  // read through scalar loads
  return ((Words)(uintptr_t)q.starts)[__builtin_amdgcn_readfirstlane(i)];
}

// f(sequence, slot, first row, rows) for each part of a sequence in a strip; uniform over the block.
// SHARED: strips of several dense sequences.
template <bool SHARED, typename F>
__device__ __forceinline__ void parts(const Rows& q, const Cut& t, int strip, F f) {
  if (!q.starts) {
    if constexpr (!SHARED) {
      const int s = strip / t.per, at = strip % t.per * t.rows;
      f(s, (int64_t)strip, s * q.L + at, min(q.L - at, t.rows));
    } else {
      const int s0 = strip / t.per * t.seqs, at = strip % t.per * t.rows, stop = min(s0 + t.seqs, q.S);
      for (int s = s0; s < stop; ++s)
        f(s, (int64_t)s * t.per + strip % t.per, s * q.L + at, min(q.L - at, t.rows));
    }
    return;
  }
  const int front = offset(q, 0), begin = strip * t.rows, stop = min(q.R - begin, t.rows) + begin;
  for (int r = begin; r < stop;) {
    if (r < front) {
      r = min(front, stop);
      continue;
    }
    int lo = 0, hi = q.S;  // as seq_of
    while (hi - lo > 1) {
      const int m = lo + ((hi - lo) >> 1);
      if (offset(q, m) <= r) lo = m; else hi = m;
    }
    const int end = min(offset(q, lo + 1), stop);
    if (end <= r) return;  // behind the last
    f(lo, (int64_t)strip + lo, r, end - r);
    r = end;
  }
}

// Slots of sequence s: n of them from the first; rows of the i-th.
struct Slots {
  int begin, end, strip0, n;
  int64_t first;
  __device__ __forceinline__ Slots(const Rows& q, const Cut& t, int s) {
    begin = seq_begin(q, s);
    end = max(seq_end(q, s), begin);
    if (q.starts) {
      strip0 = begin / t.rows;
      first = (int64_t)strip0 + s;
      n = end > begin ? (end - 1) / t.rows - strip0 + 1 : 0;
    } else {
      strip0 = 0;
      first = (int64_t)s * t.per;
      n = t.per;
    }
  }
  __device__ __forceinline__ int rows(const Rows& q, const Cut& t, int i) const {
    if (!q.starts) return min(q.L - i * t.rows, t.rows);
    const int at = (strip0 + i) * t.rows;
    return min(end, q.R - at > t.rows ? at + t.rows : q.R) - max(begin, at);
  }
};

// Rows [r, r + n) of a wave's share (every kWaves-th), kAhead at a time: load(k, row) for each, then
// work(k, row); k is known at compile time.
template <typename L, typename W>
__device__ __forceinline__ void walk(int r, int n, L load, W work) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int i = wave;
  for (; i + (kAhead - 1) * kWaves < n; i += kAhead * kWaves) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) load(k, r + i + k * kWaves);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) work(k, r + i + k * kWaves);
  }
  if (i < n) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i + k * kWaves < n) load(k, r + i + k * kWaves);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i + k * kWaves < n) work(k, r + i + k * kWaves);
  }
}

// Sums over the waves of a block, in order: column c of value i to out[i][c] in LDS, from where every
// thread may take it.
struct Columns {
  float red[kWaves][2][kTile];
  __device__ __forceinline__ void add(const float (&a)[V], const float (&b)[V]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __syncthreads();  // what was here has been read
    store_vec<float, V>(&red[wave][0][lane * V], a);
    store_vec<float, V>(&red[wave][1][lane * V], b);
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * kTile; i += kThreads) {
      float* p = &red[0][0][i];
      *p = ((p[0] + p[2 * kTile]) + p[4 * kTile]) + p[6 * kTile];
    }
    __syncthreads();
  }
};

// f(group, first channel, channels, lane of K) for every group with channels in the tile, K threads
// each: f adds up what it finds over the group's channels in this tile. K goes by the most groups that a tile
// may hold, not by this one's: every tile of a group forms its sums in one order.
template <typename F>
__device__ __forceinline__ void groups_of_tile(const GroupArgs& q, int tile, F f) {
  const int cg = q.C / q.G, c0 = tile * kTile, c1 = min(c0 + kTile, q.C);
  const int g0 = c0 / cg, g1 = (c1 - 1) / cg + 1;
  const int n = min(q.G, kTile % cg ? (kTile - 2) / cg + 2 : kTile / cg);
  const int per = n <= 4 ? 64 : n <= 8 ? 32 : n <= 16 ? 16 : n <= 32 ? 8 : n <= 64 ? 4 : 1;
  for (int g = g0 + (int)threadIdx.x / per; g < g1; g += kThreads / per) {
    const int a = max(g * cg, c0), b = min((g + 1) * cg, c1);
    f(g, a - c0, b - a, (int)threadIdx.x % per, per);
  }
}
template <typename F>
__device__ __forceinline__ F sum_of(F v, int per) {  // over neighbouring threads, in each of them
  for (int m = per >> 1; m >= 1; m >>= 1) v += __shfl_xor(v, m, kWave);
  return v;
}

// ---- sums over a sequence and group ------------------------------------------------------------------
// What is left of a group's piece: a value of it, the mean's distance to that, the sum of squared deviations
// from the mean; or (BACK) sums of g and of g n.
struct Moments {
  float value, mean, dev;
};
template <bool BACK>
using Piece = std::conditional_t<BACK, float2, Moments>;

// Mean and 1 / sqrt(variance + eps) of a group from its pieces, or (BACK) the means of g and g n. `per` threads
// share it; sums in 64 bits, in a fixed order.
template <bool BACK>
__device__ __forceinline__ float2 total_of(const GroupArgs& q, const Cut& t, const Piece<BACK>* part, int s,
                                           int g, int lane, int per) {
  const int cg = q.C / q.G, t0 = g * cg / kTile, n = ((g + 1) * cg - 1) / kTile - t0 + 1;
  const Slots at(q.rows, t, s);
  double a = 0., b = 0., dev = 0.;
  const int64_t all = (int64_t)at.n * n;
  constexpr int U = 4;  // loads issued together
  for (int64_t i0 = lane; i0 < all; i0 += U * per) {
    Piece<BACK> v[U];
    int slot[U], tile[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = min(i0 + u * per, all - 1);
      slot[u] = (int)(n == 1 ? i : i / n);
      tile[u] = t0 + (n == 1 ? 0 : (int)(i - (int64_t)slot[u] * n));
      v[u] = part[(at.first + slot[u]) * t.pieces + tile[u] + g];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * per >= all) break;
      if constexpr (BACK) {
        a += v[u].x;
        b += v[u].y;
      } else {
        const int width = min((g + 1) * cg, (tile[u] + 1) * kTile) - max(g * cg, tile[u] * kTile);
        const double m = (double)v[u].value + v[u].mean, k = (double)at.rows(q.rows, t, slot[u]) * width;
        a += k * m;
        b += k * m * m;  // (in 64 bits the difference below loses nothing that 32 hold)
        dev += v[u].dev;
      }
    }
  }
  a = sum_of(a, per);
  b = sum_of(b, per);
  const double count = (double)max(at.end - at.begin, 1) * cg;
  if (BACK) return make_float2((float)(a / count), (float)(b / count));
  dev = sum_of(dev, per);
  const double mean = a / count, var = (dev + fmax(b - a * mean, 0.)) / count;
  return make_float2((float)mean, (float)(1. / sqrt(var + q.eps)));
}

// out [S, G]: where a block of the second pass would have too much to add up, or stats are asked for
// of sequences without tokens (0 and 1 / sqrt(eps)). A wave each.
template <bool BACK>
__global__ __launch_bounds__(kThreads) void k_gn_totals(GroupArgs q, Cut t, const Piece<BACK>* part,
                                                        float2* out) {
  const int64_t u = (int64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  if (u >= (int64_t)q.rows.S * q.G) return;
  const float2 v = total_of<BACK>(q, t, part, (int)(u / q.G), (int)(u % q.G), threadIdx.x & 63, 64);
  if ((threadIdx.x & 63) == 0) out[u] = v;
}

// ---- forward -----------------------------------------------------------------------------------------
// part [slots, pieces].
template <typename IO>
__global__ __launch_bounds__(kThreads) void k_gn_parts(GroupArgs q, Cut t, Moments* part) {
  __shared__ Columns col;
  const int lane = threadIdx.x & 63, tile = (int)(blockIdx.x % t.tiles);
  const int c = min(tile * kTile + lane * V, q.C - V);  // idle lanes load the last channels again
  const IO* x = (const IO*)q.x + c;
  parts<false>(q.rows, t, (int)(blockIdx.x / t.tiles), [&](int, int64_t slot, int r, int n) {
    Vec<IO, V> first, v[kAhead];
    float sum[V], sq[V];
    first.load(x + r * q.xs);
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] = sq[j] = 0.f;
    walk(r, n, [&](int k, int row) { v[k].load(x + row * q.xs); },
         [&](int k, int) {
#pragma unroll
           for (int j = 0; j < V; ++j) {
             const float d = v[k].get(j) - first.get(j);
             sum[j] += d;
             sq[j] = fmaf(d, d, sq[j]);
           }
         });
    col.add(sum, sq);
    // each channel's mean and deviations, from its first row's value
    const float rows = (float)n;
    const IO* top = (const IO*)q.x + r * q.xs + tile * kTile;
    groups_of_tile(q, tile, [&](int g, int c0, int width, int me, int per) {
      const float value = Io<IO>::load(top, c0);
      float mean = 0.f, dev = 0.f;
      for (int i = c0 + me; i < c0 + width; i += per) {
        const float d = col.red[0][0][i] / rows;
        mean += (Io<IO>::load(top, i) - value) + d;
        dev += fmaxf(fmaf(-d, col.red[0][0][i], col.red[0][1][i]), 0.f);
      }
      mean = sum_of(mean, per) / width;
      for (int i = c0 + me; i < c0 + width; i += per) {
        const float d = (Io<IO>::load(top, i) - value) + col.red[0][0][i] / rows - mean;
        dev = fmaf(rows * d, d, dev);
      }
      dev = sum_of(dev, per);
      if (me == 0) part[slot * t.pieces + tile + g] = Moments{value, mean, dev};
    });
  });
}

struct Affine {
  float w[V], b[V];
  __device__ __forceinline__ Affine(const GroupArgs& q, int c) {
#pragma unroll
    for (int j = 0; j < V; ++j) w[j] = 1.f, b[j] = 0.f;
    if (q.w) load_f32<V>(q.w + c, w);
    if (q.b) load_f32<V>(q.b + c, b);
  }
};

// A pair for each of a thread's channels, or (ONE: groups of a multiple of 8 channels) one for all.
template <bool ONE>
struct Pair {
  float2 v[ONE ? 1 : V];
  __device__ __forceinline__ float2 operator[](int j) const { return v[ONE ? 0 : j]; }
  __device__ __forceinline__ void load(const GroupArgs& q, const float2* from, int s, int c) {
#pragma unroll
    for (int j = 0; j < (ONE ? 1 : V); ++j) v[j] = from[(int64_t)s * q.G + (c + j) / (q.C / q.G)];
  }
};

// A pair a group of the tile (statistics, or means of the backward pass), of sequence s: read, or added
// up here; to v of this thread's channels.
struct Pairs {
  float2 of[kTile];
  template <bool BACK, bool ONE>
  __device__ __forceinline__ void get(const GroupArgs& q, const Cut& t, const Piece<BACK>* part,
                                      const float2* ready, int s, int tile, int c, Pair<ONE>& v,
                                      float2* out) {
    const int cg = q.C / q.G;
    if (ready) {
      v.load(q, ready, s, c);
      return;
    }
    const int g0 = tile * kTile / cg;
    __syncthreads();  // what was here has been read
    groups_of_tile(q, tile, [&](int g, int, int, int me, int per) {
      const float2 p = total_of<BACK>(q, t, part, s, g, me, per);
      if (me == 0) {
        of[g - g0] = p;
        if (out) out[(int64_t)s * q.G + g] = p;
      }
    });
    __syncthreads();
#pragma unroll
    for (int j = 0; j < (ONE ? 1 : V); ++j) v.v[j] = of[(c + j) / cg - g0];
  }
};

// stats: written where given and not `ready` (by each strip and each tile of a group alike: the same bits).
template <typename IO, bool ONE>
__global__ __launch_bounds__(kThreads) void k_gn_apply(GroupArgs q, Cut t, const Moments* part,
                                                       const float2* ready, float2* stats, IO* y) {
  __shared__ Pairs pairs;
  const int lane = threadIdx.x & 63, tile = (int)(blockIdx.x % t.tiles);
  const int c0 = tile * kTile + lane * V, c = min(c0, q.C - V);
  const bool live = c0 < q.C;
  const IO* x = (const IO*)q.x + c;
  const Affine af(q, c);
  parts<false>(q.rows, t, (int)(blockIdx.x / t.tiles), [&](int s, int64_t, int r, int n) {
    Pair<ONE> st;
    float o[V];
    Vec<IO, V> v[kAhead];
    pairs.get<false>(q, t, part, ready, s, tile, c, st, stats);
    walk(r, n, [&](int k, int row) { v[k].load(x + row * q.xs); },
         [&](int k, int row) {
#pragma unroll
           for (int j = 0; j < V; ++j) {
             o[j] = fmaf((v[k].get(j) - st[j].x) * st[j].y, af.w[j], af.b[j]);
             if (q.act) o[j] *= sigmoid(o[j]);
           }
           if (live) store_vec<IO, V>(y + (int64_t)row * q.C + c, o, q.stream);
         });
  });
}

// ---- backward ----------------------------------------------------------------------------------------
// part [slots, pieces]: sums of g = w dv and of g n. chan [strips, 2, C]: sums of dv (db), of dv n (dw).
template <typename IO, bool ONE, bool SHARED>
__global__ __launch_bounds__(kThreads) void k_gn_bwd_parts(GroupArgs q, Cut t, const float2* stats,
                                                           const IO* dy, float2* part, float* chan) {
  __shared__ Columns col;
  const int lane = threadIdx.x & 63, tile = (int)(blockIdx.x % t.tiles);
  const int strip = (int)(blockIdx.x / t.tiles);
  const int c = min(tile * kTile + lane * V, q.C - V);
  const IO* x = (const IO*)q.x + c;
  const IO* d = dy + c;
  const Affine af(q, c);
  float db[kTile / kThreads], dw[kTile / kThreads];  // of channels tile * kTile + threadIdx.x + i 256
#pragma unroll
  for (int i = 0; i < kTile / kThreads; ++i) db[i] = dw[i] = 0.f;
  parts<SHARED>(q.rows, t, strip, [&](int s, int64_t slot, int r, int n) {
    Pair<ONE> st;
    float a[V], b[V];
    Vec<IO, V> v[kAhead], e[kAhead];
    st.load(q, stats, s, c);
#pragma unroll
    for (int j = 0; j < V; ++j) a[j] = b[j] = 0.f;
    walk(r, n,
         [&](int k, int row) {
           v[k].load(x + row * q.xs);
           e[k].load(d + (int64_t)row * q.C);
         },
         [&](int k, int) {
#pragma unroll
           for (int j = 0; j < V; ++j) {
             const float nv = (v[k].get(j) - st[j].x) * st[j].y;
             float dv = e[k].get(j);
             if (q.act) dv *= act_slope(fmaf(nv, af.w[j], af.b[j]));
             a[j] += dv;
             b[j] = fmaf(dv, nv, b[j]);
           }
         });
    col.add(a, b);
    groups_of_tile(q, tile, [&](int g, int c0, int width, int me, int per) {
      float m1 = 0.f, m2 = 0.f;
      for (int i = c0 + me; i < c0 + width; i += per) {
        const float w = q.w ? q.w[tile * kTile + i] : 1.f;
        m1 = fmaf(w, col.red[0][0][i], m1);
        m2 = fmaf(w, col.red[0][1][i], m2);
      }
      m1 = sum_of(m1, per);
      m2 = sum_of(m2, per);
      if (me == 0) part[slot * t.pieces + tile + g] = make_float2(m1, m2);
    });
#pragma unroll
    for (int i = 0; i < kTile / kThreads; ++i) {
      db[i] += col.red[0][0][threadIdx.x + i * kThreads];
      dw[i] += col.red[0][1][threadIdx.x + i * kThreads];
    }
  });
  if (!chan) return;
#pragma unroll
  for (int i = 0; i < kTile / kThreads; ++i) {
    const int at = tile * kTile + threadIdx.x + i * kThreads;
    if (at < q.C) {
      chan[(int64_t)strip * 2 * q.C + at] = db[i];
      chan[((int64_t)strip * 2 + 1) * q.C + at] = dw[i];
    }
  }
}

// dx = rstd (g - mean(g) - n mean(g n)); zero in rows of no sequence. The blocks behind the strips' add
// up the columns of chan, 64 each, in a fixed order.
template <typename IO, bool ONE, bool SHARED>
__global__ __launch_bounds__(kThreads) void k_gn_bwd_apply(GroupArgs q, Cut t, const float2* stats,
                                                           const float2* part, const float2* ready,
                                                           const float* chan, const IO* dy, IO* dx,
                                                           float* dw, float* db) {
  __shared__ Pairs pairs;
  const int64_t main_blocks = (int64_t)t.strips * t.tiles;
  const int lane = threadIdx.x & 63;
  if (blockIdx.x >= main_blocks) {
    double* red = reinterpret_cast<double*>(&pairs);
    const int64_t m = (blockIdx.x - main_blocks) * 64 + lane, M = 2 * (int64_t)q.C;
    double sum = 0.;
    if (m < M) {
#pragma unroll 8
      for (int i = threadIdx.x >> 6; i < t.strips; i += kWaves) sum += chan[i * M + m];
    }
    red[threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.x < 64 && m < M) {
      const float v = (float)(((sum + red[64 + lane]) + red[128 + lane]) + red[192 + lane]);
      if (m < q.C) {
        if (db) db[m] = v;
      } else if (dw) {
        dw[m - q.C] = v;
      }
    }
    return;
  }
  const int tile = (int)(blockIdx.x % t.tiles), strip = (int)(blockIdx.x / t.tiles);
  const int c0 = tile * kTile + lane * V, c = min(c0, q.C - V);
  const bool live = c0 < q.C;
  const IO* x = (const IO*)q.x + c;
  const IO* d = dy + c;
  const Affine af(q, c);
  float o[V];
  int done = strip * t.rows;  // packed: rows up to here are in a sequence or have been cleared
  const int wave = threadIdx.x >> 6;
  auto clear = [&](int to) {
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = 0.f;
    if (live)
      for (int i = done + wave; i < to; i += kWaves) store_vec<IO, V>(dx + (int64_t)i * q.C + c, o);
  };
  parts<SHARED>(q.rows, t, strip, [&](int s, int64_t, int r, int n) {
    Pair<ONE> st, m;
    Vec<IO, V> v[kAhead], e[kAhead];
    if (q.rows.starts) {
      clear(r);
      done = r + n;
    }
    st.load(q, stats, s, c);
    pairs.get<true>(q, t, part, ready, s, tile, c, m, nullptr);
    walk(r, n,
         [&](int k, int row) {
           v[k].load(x + row * q.xs);
           e[k].load(d + (int64_t)row * q.C);
         },
         [&](int k, int row) {
#pragma unroll
           for (int j = 0; j < V; ++j) {
             const float nv = (v[k].get(j) - st[j].x) * st[j].y;
             float g = e[k].get(j) * af.w[j];
             if (q.act) g *= act_slope(fmaf(nv, af.w[j], af.b[j]));
             o[j] = st[j].y * (g - m[j].x - nv * m[j].y);
           }
           if (live) store_vec<IO, V>(dx + (int64_t)row * q.C + c, o);
         });
  });
  if (q.rows.starts) clear(min(q.rows.R - strip * t.rows, t.rows) + strip * t.rows);
}

// ---- sequences of a few tokens -----------------------------------------------------------------------
// Dense sequences of up to kHeld tokens, groups of a multiple of 8 channels. A group's vectors of eight
// have lanes of their own, `per` of them: the next power of two within a wave, or whole waves, which are
// then a block; the lanes behind the group's vectors idle. Sums run over lanes, without LDS within a
// wave, and what a thread needs of weight and bias serves all its tokens. One read and one write: 80
// groups of 64 channels at 16384 single tokens in bf16 take 62 us (5.4 TB/s), backward 109 (4.6); one
// group of 5120 takes 84 and 134, of 2048 25 and 46. (A thread for each vector without gaps, and sums
// over neighbours in LDS: 118 and 335 us for the last.)
constexpr int kWide = 1024;  // lanes of a group, at most
struct Lanes {
  int per, block;
};
Lanes lanes_of(const GroupArgs& a) {
  const int vg = a.C / a.G / V;
  Lanes l = {1, kThreads};
  if (vg > kWave)
    l.per = l.block = (vg + kWave - 1) / kWave * kWave;
  else
    while (l.per < vg) l.per *= 2;
  return l;
}

// The n-th of this launch's threads as (row, group, vector of the group).
struct Place {
  int64_t row;
  int g, at, c;
  bool live;
  __device__ __forceinline__ Place(const GroupArgs& q, int per) {
    const int64_t first = (int64_t)blockIdx.x * blockDim.x;
    const unsigned width = (unsigned)q.G * per, rest = (unsigned)(first % width) + threadIdx.x;
    row = first / width + rest / width;
    g = (int)(rest % width / per);
    at = (int)(rest % width % per);
    const int cg = q.C / q.G;
    live = at * V < cg;
    c = g * cg + (live ? at * V : 0);
  }
};

__device__ __forceinline__ float lanes_sum(float v, int per) {  // per: uniform
  if (per >= 2) v = add_dpp<0xB1>(v);    // quad_perm [1,0,3,2]
  if (per >= 4) v = add_dpp<0x4E>(v);    // quad_perm [2,3,0,1]
  if (per >= 8) v = add_dpp<0x141>(v);   // row_half_mirror
  if (per >= 16) v = add_dpp<0x140>(v);  // row_mirror
  if (per >= 32) v += __shfl_xor(v, 16, kWave);
  if (per >= 64) v += __shfl_xor(v, 32, kWave);
  return v;
}

// Sums of N values over a group's lanes, in each of them. Across waves through LDS, in two halves in
// turn: who writes one again has passed the other's barrier, behind all that read the first.
template <bool WIDE, int N>
struct Group {
  float of[WIDE ? 2 : 1][WIDE ? kWide / kWave : 1][N];
  __device__ __forceinline__ void add(float (&v)[N], int per, int half) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes_sum(v[i], WIDE ? kWave : per);
    if (!WIDE) return;
    const int waves = per / kWave;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((threadIdx.x & 63) == 0) of[half][threadIdx.x / kWave][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.f;
    for (int w = 0; w < waves; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += of[half][w][i];
  }
};

// NV sequences of one token a thread. A block of a wide group is one row, so that all of it returns or reaches a barrier.
template <typename IO, int NV, bool WIDE>
__global__ __launch_bounds__(WIDE ? kWide : kThreads) void k_gn_tokens(GroupArgs q, int per, float2* stats,
                                                                       IO* y) {
  __shared__ Group<WIDE, NV> group;
  const Place p(q, per);
  const int64_t s0 = p.row * NV;
  if (s0 >= q.rows.S) return;  // whole groups
  const float share = 1.f / (q.C / q.G);
  Vec<IO, V> v[NV];
  float mean[NV], rstd[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i)
    v[i].load((const IO*)q.x + min(s0 + i, (int64_t)q.rows.S - 1) * q.xs + p.c);
  const Affine af(q, p.c);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    mean[i] = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) mean[i] += v[i].get(j);
    if (!p.live) mean[i] = 0.f;
  }
  group.add(mean, per, 0);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    mean[i] *= share;
    rstd[i] = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float d = v[i].get(j) - mean[i];
      rstd[i] = fmaf(d, d, rstd[i]);
    }
    if (!p.live) rstd[i] = 0.f;
  }
  group.add(rstd, per, 1);
  if (!p.live) return;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (s0 + i >= q.rows.S) break;
    const float r = inverse_root(fmaf(rstd[i], share, q.eps));
    if (stats && p.at == 0) stats[(s0 + i) * q.G + p.g] = make_float2(mean[i], r);
    float o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      o[j] = fmaf((v[i].get(j) - mean[i]) * r, af.w[j], af.b[j]);
      if (q.act) o[j] *= sigmoid(o[j]);
    }
    store_vec<IO, V>(y + (s0 + i) * q.C + p.c, o, q.stream);
  }
}

template <typename IO, bool WIDE>
__global__ __launch_bounds__(WIDE ? kWide : kThreads) void k_gn_few(GroupArgs q, int per, float2* stats,
                                                                    IO* y) {
  __shared__ Group<WIDE, 1> group;
  const Place p(q, per);
  const int64_t s = p.row;
  if (s >= q.rows.S) return;
  const int L = q.rows.L;
  const float count = (float)(L * (q.C / q.G));
  Vec<IO, V> v[kHeld];
  float mean[1] = {0.f}, rstd[1] = {0.f};
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (i < L) v[i].load((const IO*)q.x + (s * L + i) * q.xs + p.c);
  const Affine af(q, p.c);
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (i < L && p.live) {
#pragma unroll
      for (int j = 0; j < V; ++j) mean[0] += v[i].get(j);
    }
  group.add(mean, per, 0);
  mean[0] /= count;
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (i < L && p.live) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = v[i].get(j) - mean[0];
        rstd[0] = fmaf(d, d, rstd[0]);
      }
    }
  group.add(rstd, per, 1);
  if (!p.live) return;
  const float r = inverse_root(rstd[0] / count + q.eps);
  if (stats && p.at == 0) stats[s * q.G + p.g] = make_float2(mean[0], r);
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (i < L) {
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        o[j] = fmaf((v[i].get(j) - mean[0]) * r, af.w[j], af.b[j]);
        if (q.act) o[j] *= sigmoid(o[j]);
      }
      store_vec<IO, V>(y + (s * L + i) * q.C + p.c, o, q.stream);
    }
}

// Backward: a thread walks every walkers-th sequence and keeps the sums for dw and db of its channels in
// registers. part [walkers, 2, C]: sums of dv (db) and of dv n (dw).
template <typename IO, int NV, bool WIDE>
__global__ __launch_bounds__(WIDE ? kWide : kThreads) void k_gn_tokens_bwd(GroupArgs q, int per,
                                                                           int walkers,
                                                                           const float2* stats,
                                                                           const IO* dy, IO* dx,
                                                                           float* part) {
  __shared__ Group<WIDE, 2 * NV> group;
  const Place p(q, per);
  if (p.row >= walkers) return;
  const float share = 1.f / (q.C / q.G);
  const Affine af(q, p.c);
  float dw[V], db[V];
#pragma unroll
  for (int j = 0; j < V; ++j) dw[j] = db[j] = 0.f;
  int half = 0;
  for (int64_t s0 = p.row; s0 < q.rows.S; s0 += (int64_t)NV * walkers) {
    Vec<IO, V> v[NV], d[NV];
    float2 st[NV];
    float m[2 * NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t s = min(s0 + (int64_t)i * walkers, (int64_t)q.rows.S - 1);
      v[i].load((const IO*)q.x + s * q.xs + p.c);
      d[i].load(dy + s * q.C + p.c);
      st[i] = stats[s * q.G + p.g];
    }
    // the gradient of n, and n: once for the sums and once for dx
    auto each = [&](int i, auto f) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float n = (v[i].get(j) - st[i].x) * st[i].y;
        float e = d[i].get(j);
        if (q.act) e *= act_slope(fmaf(n, af.w[j], af.b[j]));
        f(j, n, e);
      }
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      m[2 * i] = m[2 * i + 1] = 0.f;
      if (!p.live || s0 + (int64_t)i * walkers >= q.rows.S) continue;
      each(i, [&](int j, float n, float e) {
        db[j] += e;
        dw[j] = fmaf(e, n, dw[j]);
        e *= af.w[j];
        m[2 * i] += e;
        m[2 * i + 1] = fmaf(e, n, m[2 * i + 1]);
      });
    }
    group.add(m, per, half);
    half ^= 1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t s = s0 + (int64_t)i * walkers;
      if (!p.live || s >= q.rows.S) continue;
      float o[V];
      each(i, [&](int j, float n, float e) {
        o[j] = st[i].y * (e * af.w[j] - m[2 * i] * share - n * (m[2 * i + 1] * share));
      });
      store_vec<IO, V>(dx + s * q.C + p.c, o);
    }
  }
  if (!p.live) return;
  float* to = part + p.row * 2 * q.C + p.c;
  store_vec<float, V>(to, db);
  store_vec<float, V>(to + q.C, dw);
}

template <typename IO, bool WIDE>
__global__ __launch_bounds__(WIDE ? kWide / 2 : kThreads) void k_gn_few_bwd(GroupArgs q, int per,
                                                                            int walkers,
                                                                            const float2* stats,
                                                                            const IO* dy, IO* dx,
                                                                            float* part) {
  __shared__ Group<WIDE, 2> group;
  const Place p(q, per);
  if (p.row >= walkers) return;
  const int L = q.rows.L;
  const float count = (float)(L * (q.C / q.G));
  const Affine af(q, p.c);
  float dw[V], db[V];
#pragma unroll
  for (int j = 0; j < V; ++j) dw[j] = db[j] = 0.f;
  int half = 0;
  for (int64_t s = p.row; s < q.rows.S; s += walkers) {
    Vec<IO, V> v[kHeld], d[kHeld];
    float m[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (i < L) {
        v[i].load((const IO*)q.x + (s * L + i) * q.xs + p.c);
        d[i].load(dy + (s * L + i) * q.C + p.c);
      }
    const float2 st = stats[s * q.G + p.g];
    auto each = [&](int i, auto f) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float n = (v[i].get(j) - st.x) * st.y;
        float e = d[i].get(j);
        if (q.act) e *= act_slope(fmaf(n, af.w[j], af.b[j]));
        f(j, n, e);
      }
    };
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (i < L && p.live)
        each(i, [&](int j, float n, float e) {
          db[j] += e;
          dw[j] = fmaf(e, n, dw[j]);
          e *= af.w[j];
          m[0] += e;
          m[1] = fmaf(e, n, m[1]);
        });
    group.add(m, per, half);
    half ^= 1;
    const float m1 = m[0] / count, m2 = m[1] / count;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (i < L && p.live) {
        float o[V];
        each(i, [&](int j, float n, float e) { o[j] = st.y * (e * af.w[j] - m1 - n * m2); });
        store_vec<IO, V>(dx + (s * L + i) * q.C + p.c, o);
      }
  }
  if (!p.live) return;
  float* to = part + p.row * 2 * q.C + p.c;
  store_vec<float, V>(to, db);
  store_vec<float, V>(to + q.C, dw);
}

bool few_tokens(const GroupArgs& a) {
  const int cg = a.C / a.G;
  return !a.rows.starts && a.rows.L <= kHeld && cg % V == 0 &&
         cg <= V * (a.rows.L == 1 ? kWide : kWide / 2);
}

// Sequences side by side in the backward pass: 131072 threads, two waves a SIMD (twice as many cost up to
// 19% more where groups are wide), and at least four tokens each.
int walkers_of(const GroupArgs& a) {
  const int64_t turn = 4 / a.rows.L > 1 ? 4 / a.rows.L : 1;
  const int64_t want = ((int64_t)a.rows.S + turn - 1) / turn;
  const int64_t most = 131072 / ((int64_t)a.G * lanes_of(a).per);
  return (int)(want < most ? want : most < 1 ? 1 : most);
}

// ---- whole sequences in a block ----------------------------------------------------------------------
// Where the tokens of a sequence (packed: all rows, since any may be the longest) and a group's channels (a
// multiple of 8) fit a block's registers: a block takes `groups` whole groups of one sequence, a thread
// eight channels of every par-th token. One launch, and each element is loaded once: calls of 300 packed
// x 768 fp32 17 -> 11 us, 2 x 100 x 1024 bf16 15 -> 10 us against the strips. (Blocks that load longer
// sequences again for each of their passes: 26 us at 3001 x 768, where the strips take 19.)
constexpr int kWhole = 512;
template <typename IO>
constexpr int kRows = sizeof(IO) == 2 ? 8 : 4;  // tokens of a thread
struct Whole {
  int groups, slices, width, par;  // slices of a sequence; threads of a token; tokens side by side
  bool deep;
};
// Deep blocks hold twice as many tokens a thread: in the forward, where no more of them than compute units
// take the call (235 packed in 19 sequences x 832 fp32 28 -> 10 us, 8 x 700 x 2560 bf16 22 -> 21; 16 x 800 x
// 2560 without that limit 41 -> 43; backward, 1 x 700 x 2560 bf16, 18 -> 28).
bool whole_of(const GroupArgs& a, bool forward, Whole* w) {
  const int cg = a.C / a.G, vg = cg / V;
  int held = a.io == kIoBf16 ? kRows<u16> : kRows<float>;
  if (cg % V || vg > kWhole) return false;
  const int64_t fit = a.rows.starts ? a.rows.R : a.rows.L, seqs = a.rows.S;
  w->deep = forward && fit > (int64_t)held * (kWhole / vg) && seqs * a.G <= 256;
  if (w->deep) held *= 2;
  if (fit > (int64_t)held * (kWhole / vg) || seqs * a.G > 65536) return false;
  int64_t groups = (int64_t)held * kWhole / (fit * vg);  // of a block, at most
  const int64_t most = kWhole / vg, spread = (seqs * a.G + 255) / 256;  // a block each compute unit
  if (groups > most) groups = most;
  if (groups > spread) groups = spread;
  if (groups > a.G) groups = a.G;
  for (; groups > 1; --groups)
    if (fit <= (int64_t)held * (kWhole / (groups * vg))) break;
  w->slices = (int)((a.G + groups - 1) / groups);
  w->groups = (a.G + w->slices - 1) / w->slices;
  w->width = w->groups * vg;
  w->par = kWhole / w->width;
  return true;
}

// Where a thread stands: its sequence's rows [begin, end), of which it takes begin + at, + par .., and
// its channels.
struct Part {
  int s, t, at, c, c_slice;
  int begin, end;
  bool mine;
  __device__ __forceinline__ Part(const GroupArgs& q, const Whole& w) {
    s = (int)(blockIdx.x / w.slices);
    t = threadIdx.x % w.width;
    at = threadIdx.x / w.width;
    c_slice = (int)(blockIdx.x % w.slices) * w.groups * (q.C / q.G);
    c = c_slice + t * V;
    begin = q.rows.starts ? min(max(offset(q.rows, s), 0), q.rows.R) : s * q.rows.L;
    end = q.rows.starts ? max(min(offset(q.rows, s + 1), q.rows.R), begin) : begin + q.rows.L;
    mine = at < w.par && c < q.C;
    if (!mine) c = 0;
  }
  // f(k, row) for this thread's rows; k < K at compile time
  template <int K, typename F>
  __device__ __forceinline__ void rows(const Whole& w, F f) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t r = (int64_t)begin + at + k * w.par;
      if (mine && r < end) f(k, r);
    }
  }
};

// Sums over a group of the block (its vg threads of every token side by side) of two values of each
// thread, in every one of them.
struct Shares {
  float2 of[kWhole], total[kWhole];
  __device__ __forceinline__ float2 add(const Whole& w, int vg, float a, float b) {
    __syncthreads();
    of[threadIdx.x] = make_float2(a, b);
    __syncthreads();
    int per = 64;  // threads that add up one group
    while (per > 1 && per * w.groups > kWhole) per >>= 1;
    const int me = threadIdx.x % per, all = w.par * vg;
    for (int g = threadIdx.x / per; g < w.groups; g += kWhole / per) {
      float x = 0.f, y = 0.f;
      for (int i = me; i < all; i += per) {
        const float2 v = of[i / vg * w.width + g * vg + i % vg];
        x += v.x;
        y += v.y;
      }
      x = sum_of(x, per);
      y = sum_of(y, per);
      if (me == 0) total[g] = make_float2(x, y);
    }
    __syncthreads();
    return total[threadIdx.x % w.width / vg];
  }
};

template <typename IO, int K>
__global__ __launch_bounds__(kWhole) void k_gn_whole(GroupArgs q, Whole w, float2* stats, IO* y) {
  __shared__ Shares shares;
  const int cg = q.C / q.G, vg = cg / V;
  const Part p(q, w);
  const float count = (float)max(p.end - p.begin, 1) * cg;
  const IO* x = (const IO*)q.x + p.c;
  Vec<IO, V> v[K];
  const Affine af(q, p.c);
  p.rows<K>(w, [&](int k, int64_t r) { v[k].load(x + r * q.xs); });
  float sum = 0.f, dev = 0.f;
  p.rows<K>(w, [&](int k, int64_t) {
#pragma unroll
    for (int j = 0; j < V; ++j) sum += v[k].get(j);
  });
  const float mean = shares.add(w, vg, sum, 0.f).x / count;
  p.rows<K>(w, [&](int k, int64_t) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float d = v[k].get(j) - mean;
      dev = fmaf(d, d, dev);
    }
  });
  const float rstd = 1.f / sqrtf(shares.add(w, vg, dev, 0.f).x / count + q.eps);
  if (stats && p.mine && p.at == 0 && p.t % vg == 0)
    stats[(int64_t)p.s * q.G + p.c / cg] = make_float2(mean, rstd);
  p.rows<K>(w, [&](int k, int64_t r) {
    float o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      o[j] = fmaf((v[k].get(j) - mean) * rstd, af.w[j], af.b[j]);
      if (q.act) o[j] *= sigmoid(o[j]);
    }
    store_vec<IO, V>(y + r * q.C + p.c, o, q.stream);
  });
}

// Sums of dv and of dv n of sequence s to db + s step and dw + s step (each null: not wanted).
template <typename IO>
__global__ __launch_bounds__(kWhole) void k_gn_whole_bwd(GroupArgs q, Whole w, const float2* stats,
                                                         const IO* dy, IO* dx, float* db_out,
                                                         float* dw_out, int64_t step) {
  constexpr int K = kRows<IO>;
  __shared__ Shares shares;
  __shared__ __attribute__((aligned(16))) float cols[kWhole * V];
  const int cg = q.C / q.G, vg = cg / V;
  const Part p(q, w);
  const float count = (float)max(p.end - p.begin, 1) * cg;
  const IO *x = (const IO*)q.x + p.c, *d = dy + p.c;
  Vec<IO, V> v[K], e[K];
  const Affine af(q, p.c);
  p.rows<K>(w, [&](int k, int64_t r) {
    v[k].load(x + r * q.xs);
    e[k].load(d + r * q.C);
  });
  const float2 st = stats[(int64_t)p.s * q.G + p.c / cg];
  float dw[V], db[V], a = 0.f, b = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) dw[j] = db[j] = 0.f;
  p.rows<K>(w, [&](int k, int64_t) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float n = (v[k].get(j) - st.x) * st.y;
      float dv = e[k].get(j);
      if (q.act) dv *= act_slope(fmaf(n, af.w[j], af.b[j]));
      db[j] += dv;
      dw[j] = fmaf(dv, n, dw[j]);
      a = fmaf(dv, af.w[j], a);
      b = fmaf(dv * af.w[j], n, b);
    }
  });
  const float2 m = shares.add(w, vg, a, b);
  const float m1 = m.x / count, m2 = m.y / count;
  p.rows<K>(w, [&](int k, int64_t r) {
    float o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float n = (v[k].get(j) - st.x) * st.y;
      float g = e[k].get(j) * af.w[j];
      if (q.act) g *= act_slope(fmaf(n, af.w[j], af.b[j]));
      o[j] = st.y * (g - m1 - n * m2);
    }
    store_vec<IO, V>(dx + r * q.C + p.c, o);
  });
  if (q.rows.starts) {  // rows in front of the first sequence and behind the last
    float o[V];
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = 0.f;
    const int64_t from = p.s == 0 ? 0 : p.begin, to = p.s == q.rows.S - 1 ? q.rows.R : p.end;
    for (int64_t r = from + p.at; p.mine && r < p.begin; r += w.par) store_vec<IO, V>(dx + r * q.C + p.c, o);
    for (int64_t r = (int64_t)p.end + p.at; p.mine && r < to; r += w.par)
      store_vec<IO, V>(dx + r * q.C + p.c, o);
  }
  const int rows = min(w.par, p.end - p.begin);  // threads of a channel that took any
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* to = which ? dw_out : db_out;
    if (!to) continue;
    __syncthreads();
    store_vec<float, V>(cols + threadIdx.x * V, which ? dw : db);
    __syncthreads();
    for (int i = threadIdx.x; i < w.width * V && p.c_slice + i < q.C; i += kWhole) {
      float sum = 0.f;
#pragma unroll 8
      for (int r = 0; r < rows; ++r) sum += cols[r * w.width * V + i];
      to[p.s * step + p.c_slice + i] = sum;
    }
  }
}

int64_t up64(int64_t floats) { return (floats + 63) / 64 * 64; }

// A block of the second pass adds up its groups' pieces by itself up to 16 values a thread. (Sums of
// sequences without tokens have no block, so packed stats are always written by a kernel of their own.)
bool adds_itself(const GroupArgs& a, const Cut& t, bool stats) {
  if (stats && a.rows.starts) return false;
  const int cg = a.C / a.G;
  const int64_t groups = kTile / cg + 2, pieces = cg / kTile + 2;
  return groups * pieces * t.per <= 16 * kThreads;
}

}  // namespace

bool group_norm_fits(const GroupArgs& a) {
  auto fits = [](double blocks) { return blocks * kThreads < 4294967296.0; };
  if (few_tokens(a)) return fits(double(a.rows.S) * a.G * lanes_of(a).per / kThreads + 1);
  Whole w;
  if (whole_of(a, false, &w)) return true;
  const Cut t = cut_of(a, true), f = cut_of(a, false);
  // (k_gn_totals is launched where the second pass does not add up by itself)
  return fits(double(t.strips) * t.tiles + (2 * a.C + 63) / 64) && fits(double(f.strips) * f.tiles + 1) &&
         (fits(double(a.rows.S) * a.G / kWaves + 1) || (!a.rows.starts && adds_itself(a, t, false))) &&
         double(t.slots) * t.pieces < 1099511627776.0;
}

int64_t group_norm_bytes(const GroupArgs& a) {
  Whole w;
  if (few_tokens(a) || whole_of(a, true, &w)) return 0;
  const Cut t = cut_of(a, false);
  return 4 * up64(3 * t.slots * t.pieces) + 8 * (int64_t)a.rows.S * a.G;
}

hipError_t launch_group_norm(const GroupArgs& given, void* y, float* stats, float* ws,
                             hipStream_t s) {
  GroupArgs a = given;
  a.stream = past_caches((double)a.rows.R * a.C * (a.io == kIoBf16 ? 2 : 4));
  auto run = [&](auto io) {
    using IO = decltype(io);
    if (few_tokens(a)) {
      const Lanes l = lanes_of(a);
      const int64_t lanes = (int64_t)a.G * l.per;
      // Sequences of one token: four a thread once that leaves four waves a SIMD; two of a wide group
      // (16384 x 5120 in one group: 84 us; four 100, one 118).
      const int nv = a.rows.L > 1 || a.rows.S * lanes < 4 * 262144 ? 1 : l.per > kWave ? 2 : 4;
      const int64_t n = ((int64_t)a.rows.S + nv - 1) / nv * lanes;
      auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)((n + l.block - 1) / l.block)), dim3(l.block), 0, s, a,
                           l.per, (float2*)stats, (IO*)y);
        return hipGetLastError();
      };
      if (a.rows.L > 1) return l.per > kWave ? go(k_gn_few<IO, true>) : go(k_gn_few<IO, false>);
      if (nv > 1) return l.per > kWave ? go(k_gn_tokens<IO, 2, true>) : go(k_gn_tokens<IO, 4, false>);
      return l.per > kWave ? go(k_gn_tokens<IO, 1, true>) : go(k_gn_tokens<IO, 1, false>);
    }
    Whole w;
    if (whole_of(a, true, &w)) {
      auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)(a.rows.S * w.slices)), dim3(kWhole), 0, s, a, w,
                           (float2*)stats, (IO*)y);
        return hipGetLastError();
      };
      return w.deep ? go(k_gn_whole<IO, 2 * kRows<IO>>) : go(k_gn_whole<IO, kRows<IO>>);
    }
    const Cut t = cut_of(a, false);
    Moments* part = (Moments*)ws;
    float2* ready = nullptr;
    const dim3 grid((unsigned)((int64_t)t.strips * t.tiles));
    hipLaunchKernelGGL((k_gn_parts<IO>), grid, dim3(kThreads), 0, s, a, t, part);
    if (!adds_itself(a, t, stats != nullptr)) {
      ready = stats ? (float2*)stats : (float2*)(ws + up64(3 * t.slots * t.pieces));
      hipLaunchKernelGGL((k_gn_totals<false>),
                         dim3((unsigned)(((int64_t)a.rows.S * a.G + kWaves - 1) / kWaves)),
                         dim3(kThreads), 0, s, a, t, part, ready);
    }
    auto apply = [&](auto one) {
      hipLaunchKernelGGL((k_gn_apply<IO, decltype(one)::value>), grid, dim3(kThreads), 0, s, a, t, part,
                         ready, (float2*)stats, (IO*)y);
      return hipGetLastError();
    };
    return a.C / a.G % V ? apply(std::false_type{}) : apply(std::true_type{});
  };
  return a.io == kIoBf16 ? run(u16{}) : run(float{});
}

int64_t group_norm_backward_bytes(const GroupArgs& a) {
  if (few_tokens(a)) return 4 * (int64_t)walkers_of(a) * 2 * a.C;
  Whole w;
  if (whole_of(a, false, &w)) return a.rows.S > 1 ? 8 * (int64_t)a.rows.S * a.C : 0;
  const Cut t = cut_of(a, true);
  return 8 * (up64(t.slots * t.pieces) + up64((int64_t)a.rows.S * a.G) + (int64_t)t.strips * a.C);
}

hipError_t launch_group_norm_backward(const GroupArgs& a, const float* stats, const void* dy, void* dx,
                                      float* dw, float* db, float* ws, hipStream_t s) {
  auto run = [&](auto io) {
    using IO = decltype(io);
    if (few_tokens(a)) {
      const Lanes l = lanes_of(a);
      const int w = walkers_of(a);
      const int64_t n = (int64_t)w * a.G * l.per;
      auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)((n + l.block - 1) / l.block)), dim3(l.block), 0, s, a,
                           l.per, w, (const float2*)stats, (const IO*)dy, (IO*)dx, ws);
        return hipGetLastError();
      };
      const hipError_t e =
          a.rows.L > 1 ? l.per > kWave ? go(k_gn_few_bwd<IO, true>) : go(k_gn_few_bwd<IO, false>)
                       : l.per > kWave ? go(k_gn_tokens_bwd<IO, 2, true>) : go(k_gn_tokens_bwd<IO, 4, false>);
      if (e != hipSuccess || !(dw || db)) return e;
      return launch_column_sums(ws, w, 0, nullptr, 1, 0, 0, a.C, db, a.C, dw, s);
    }
    Whole whole;
    if (whole_of(a, false, &whole)) {
      const bool add = a.rows.S > 1 && (dw || db);  // else they are the only sequence's
      hipLaunchKernelGGL((k_gn_whole_bwd<IO>), dim3((unsigned)(a.rows.S * whole.slices)), dim3(kWhole),
                         0, s, a, whole, (const float2*)stats, (const IO*)dy, (IO*)dx, add ? ws : db,
                         add ? ws + a.C : dw, 2 * (int64_t)a.C);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess || !add) return e;
      return launch_column_sums(ws, a.rows.S, 0, nullptr, 1, 0, 0, a.C, db, a.C, dw, s);
    }
    const Cut t = cut_of(a, true);
    float2 *part = (float2*)ws, *ready = nullptr, *mid = part + up64(t.slots * t.pieces);
    float* chan = dw || db ? (float*)(mid + up64((int64_t)a.rows.S * a.G)) : nullptr;
    const unsigned blocks = (unsigned)((int64_t)t.strips * t.tiles);
    const unsigned more = chan ? (2 * a.C + 63) / 64 : 0;
    auto passes = [&](auto one, auto shared) {
      constexpr bool ONE = decltype(one)::value, SHARED = decltype(shared)::value;
      hipLaunchKernelGGL((k_gn_bwd_parts<IO, ONE, SHARED>), dim3(blocks), dim3(kThreads), 0, s, a, t,
                         (const float2*)stats, (const IO*)dy, part, chan);
      if (!adds_itself(a, t, false)) {
        ready = mid;
        hipLaunchKernelGGL((k_gn_totals<true>),
                           dim3((unsigned)(((int64_t)a.rows.S * a.G + kWaves - 1) / kWaves)),
                           dim3(kThreads), 0, s, a, t, part, ready);
      }
      hipLaunchKernelGGL((k_gn_bwd_apply<IO, ONE, SHARED>), dim3(blocks + more), dim3(kThreads), 0, s, a, t,
                         (const float2*)stats, part, ready, chan, (const IO*)dy, (IO*)dx, dw, db);
      return hipGetLastError();
    };
    auto by_strip = [&](auto one) {
      return t.seqs > 1 ? passes(one, std::true_type{}) : passes(one, std::false_type{});
    };
    return a.C / a.G % V ? by_strip(std::false_type{}) : by_strip(std::true_type{});
  };
  return a.io == kIoBf16 ? run(u16{}) : run(float{});
}

}  // namespace ssd
