// Gated linear recurrence, one state entry a channel: forward, backward and single token.
//
//   h_t = a_t h_{t-1} + m_t v_t,  v = sigmoid(input_gate) x  (x without an input gate)
//   with a decay parameter:  u = sharpness softplus(decay) sigmoid(gate), a = exp(-u),
//                            m = sqrt(1 - a^2)
//   without:                 a = sigmoid(gate), m = 1 - a
//
// A few dozen operations for each element read once: bound by memory if the rows are read once and
// the exponentials evaluated once. The tokens of a sequence are sequential, but the recurrence is
// linear, so a run of rows is summed up by two numbers a channel, the product P of its a and its
// end state H from a zero state: h_end = P h_in + H. The adjoint runs the same way backwards
// (l_t = dy_t + a_{t+1} l_{t+1}; what leaves the run to the left is P c_in + G with the same P).
//
// A lane holds the channels of four bytes (two bf16, one fp32), a wave 64 lanes and T rows, all of
// whose loads are issued at once; the waves of a block take consecutive rows (a chunk) and combine
// their (P, H) through LDS. Chunks are chained by a kernel between two passes over the rows.
#include <cmath>

#include "ssd_recurrent.h"
#include "ssd_selective.h"

namespace ssd {

namespace {

constexpr int T = 16;      // rows of a wave
constexpr int kWaves = 8;  // most waves of a block
template <typename IO>
constexpr int kV = 4 / (int)sizeof(IO);  // channels of a lane

// How the rows are cut. Dense: `chunks` of each sequence, of `waves` waves each; where a sequence is
// one chunk, a block takes `seqs` of them. Packed: chunks of all rows, wherever sequences begin.
struct Plan {
  int waves, seqs, chunks, units;  // units: blocks of one channel tile
};
Plan plan(const Rows& q) {
  Plan p;
  const int64_t rows = q.starts ? q.R : q.L;
  const int64_t need = (rows + T - 1) / T;
  p.waves = (int)(need < kWaves ? need : kWaves);
  p.chunks = (int)((need + kWaves - 1) / kWaves);
  p.seqs = q.starts || p.chunks > 1 ? 1 : kWaves / p.waves;
  if (!q.starts && p.seqs > q.S) p.seqs = q.S;
  p.units = q.starts ? p.chunks
                     : (int)(p.chunks > 1 ? (int64_t)p.chunks * q.S : ((int64_t)q.S + p.seqs - 1) / p.seqs);
  return p;
}
int threads_of(const Plan& p) { return 64 * p.waves * p.seqs; }

// ---- one element -----------------------------------------------------------------------------------
struct Sig {
  float p, n;  // sigmoid(v), sigmoid(-v), each exact to a few roundings where it is small too
};
__device__ __forceinline__ Sig both_sides(float v) {
  const float e = exp2_fast(-fabsf(v) * kLog2e), big = __builtin_amdgcn_rcpf(1.f + e), small = e * big;
  return v >= 0.f ? Sig{big, small} : Sig{small, big};
}

// 1 - exp(-2u) from u >= 0 and a = exp(-u): the series where the difference would cancel (below
// 2u = 1/4, where the term left out is under 2^-24 of the sum).
__device__ __forceinline__ float one_minus_square(float u, float a) {
  const float v = 2.f * u;
  float s = fmaf(v, -1.f / 6.f, 1.f);
  s = fmaf(v * s, -1.f / 5.f, 1.f);
  s = fmaf(v * s, -1.f / 4.f, 1.f);
  s = fmaf(v * s, -1.f / 3.f, 1.f);
  s = fmaf(v * s, -1.f / 2.f, 1.f);
  return v < 0.25f ? v * s : fmaf(-a, a, 1.f);
}

// What a token does to a channel's state. k = sharpness softplus(decay).
template <bool DECAY>
struct Gate {
  float a, m;
  Sig r;
  float u, inv;  // with a decay: u and 1 / m (at most 2^63, so that u / m is 0 where u is)
  __device__ __forceinline__ Gate(float g, float k) {
    r = both_sides(g);
    if constexpr (DECAY) {
      u = k * r.p;
      a = exp2_fast(-u * kLog2e);
      const float sq = one_minus_square(u, a);
      inv = __builtin_amdgcn_rsqf(fmaxf(sq, 1.17549435e-38f));
      m = sq * inv;
    } else {
      a = r.p;
      m = r.n;
    }
  }
};

__device__ __forceinline__ float decay_rate(const RecArgs& q, int c) {
  const float d = q.decay[c];
  return q.sharp * (d > 20.f ? d : log1pf(expf(d)));
}

// P of a run with a sequence's start in it is -0 (products of decays are never negative): what
// enters the run does not reach its end, not even as NaN.
__device__ __forceinline__ bool cut(float P) { return __float_as_uint(P) == 0x80000000u; }
__device__ __forceinline__ float enter(float P, float H, float h) { return cut(P) ? H : fmaf(P, h, H); }
__device__ __forceinline__ float join(float P, float Q) { return cut(P) || cut(Q) ? -0.f : P * Q; }

// ---- rows of a wave --------------------------------------------------------------------------------
// Value j of the raw word of a lane's channels.
template <typename IO>
__device__ __forceinline__ float word(uint32_t u, int j) {
  if constexpr (sizeof(IO) == 4) return __uint_as_float(u);
  else return __uint_as_float(j ? u & 0xffff0000u : u << 16);
}
template <typename IO>
__device__ __forceinline__ void store_word(IO* row, unsigned off, const float (&v)[kV<IO>]) {
  uint32_t u;
  if constexpr (sizeof(IO) == 4) u = __float_as_uint(v[0]);
  else u = pack_bf16(v[0], v[1]);
  *(uint32_t*)((char*)row + off) = u;
}

// T rows of n at row r0 of a tensor (null: zeros); the rows past n are not read.
template <typename IO>
__device__ __forceinline__ void load_rows(uint32_t (&u)[T], const void* t, int64_t stride, int r0,
                                          int n, unsigned off) {
  const char* p = (const char*)((const IO*)t + r0 * stride);
  if (n == T) {
#pragma unroll
    for (int i = 0; i < T; ++i) {
      u[i] = *(const uint32_t*)(p + off);
      p += stride * sizeof(IO);
    }
  } else {
#pragma unroll
    for (int i = 0; i < T; ++i) {
      u[i] = 0;
      if (i < n) u[i] = *(const uint32_t*)(p + off);
      p += stride * sizeof(IO);
    }
  }
}

// Where a block's waves stand.
struct Place {
  int unit, wave, first, n;  // block of a tile; wave; its rows [first, first + n)
  int s, part;               // dense: its sequence; its place among the sequence's waves here
  bool last;                 // dense: the sequence ends in these rows
  int lo, hi;                // waves whose runs this one's joins
  __device__ __forceinline__ Place(const Rows& q, const Plan& p, int unit_) {
    unit = unit_;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    part = wave;
    lo = 0;
    hi = p.waves;
    if (q.starts) {
      s = 0;
      last = false;
      const int64_t at = ((int64_t)unit * p.waves + wave) * T;
      first = at < q.R ? (int)at : q.R;
      n = min(q.R - first, T);
      return;
    }
    int chunk = 0;
    if (p.chunks > 1) {
      s = unit / p.chunks;
      chunk = unit % p.chunks;
    } else {
      const int at = wave / p.waves;
      const int64_t s_ = (int64_t)unit * p.seqs + at;
      part = wave % p.waves;
      lo = at * p.waves;
      hi = lo + p.waves;
      if (s_ >= q.S) {
        s = 0, first = 0, n = 0, last = false;
        return;
      }
      s = (int)s_;
    }
    const int64_t at = ((int64_t)chunk * p.waves + part) * T;  // row of the sequence
    n = at < q.L ? min((int)(q.L - at), T) : 0;
    first = n ? s * q.L + (int)at : 0;
    last = n && at + n == q.L;
  }
};

// Sequence boundaries among a wave's rows (packed).
struct Marks {
  uint64_t starts = 0, ends = 0, inside = 0;
  int seq = -1;  // of row i, in lane i
  bool plain = true;
  __device__ __forceinline__ void find(const Rows& q, int first, int n) {
    mark_rows(q, first, first + n, starts, ends, inside, seq);
    const uint64_t all = n >= 64 ? ~0ull : (1ull << n) - 1;
    plain = !starts && !ends && inside == all;
  }
};

// States of the sequences without rows pass through; the blocks behind the tiles' do it.
__device__ __forceinline__ void pass_empty(const Rows& q, int C, int block, int blocks,
                                           const float* from, float* to) {
  const int64_t all = (int64_t)q.S * C, step = (int64_t)blocks * blockDim.x;
  for (int64_t i = (int64_t)block * blockDim.x + threadIdx.x; i < all; i += step) {
    const int s = (int)(i / C);
    if (seq_end(q, s) <= seq_begin(q, s)) to[i] = from ? from[i] : 0.f;
  }
}
int empty_blocks(const RecArgs& a, const Plan& p, const float* to) {
  if (!to || !a.rows.starts) return 0;
  const int64_t n = ((int64_t)a.rows.S * a.C + 8 * threads_of(p) - 1) / (8 * threads_of(p));
  return (int)(n < 4096 ? n : 4096);
}

// Sums of the runs, [units, C] each.
struct Sums {
  float *P, *H, *G;
};

// ---- forward ---------------------------------------------------------------------------------------
// ENDS: only the runs' sums, for the chain. Otherwise y and the final states; `chained`: the states
// entering the chunks are in sums.H.
template <typename IO, bool DECAY, bool GATED, bool PACKED, bool ENDS>
__global__ __launch_bounds__(64 * kWaves) void k_rec(RecArgs q, Plan pl, int tiles, Sums sums,
                                                     int chained, IO* __restrict__ y,
                                                     float* __restrict__ fin) {
  constexpr int V = kV<IO>;
  __shared__ float2 runs[kWaves][V][64];
  const int64_t main_blocks = (int64_t)tiles * pl.units;
  if (PACKED && blockIdx.x >= main_blocks) {
    pass_empty(q.rows, q.C, (int)(blockIdx.x - main_blocks), (int)(gridDim.x - main_blocks), q.h0, fin);
    return;
  }
  const int tile = (int)(blockIdx.x % tiles), lane = threadIdx.x & 63;
  const Place at(q.rows, pl, (int)(blockIdx.x / tiles));
  const int c0 = (tile * 64 + lane) * V;
  const bool live = c0 < q.C;
  const int c = live ? c0 : q.C - V;  // idle lanes compute the last channels again
  const unsigned off = (unsigned)c * sizeof(IO);
  uint32_t rx[T], rg[T], ri[T];
  load_rows<IO>(rg, q.g, q.gs, at.first, at.n, off);
  if (GATED) load_rows<IO>(ri, q.gi, q.is, at.first, at.n, off);
  load_rows<IO>(rx, q.x, q.xs, at.first, at.n, off);
  Marks mk;
  if (PACKED && at.n > 0) mk.find(q.rows, at.first, at.n);
  float k[V];
#pragma unroll
  for (int j = 0; j < V; ++j) k[j] = DECAY ? decay_rate(q, c + j) : 0.f;

  float P[T][V], H[T][V];  // of the rows up to each
  float p[V], h[V];
#pragma unroll
  for (int j = 0; j < V; ++j) p[j] = 1.f, h[j] = 0.f;
  auto row = [&](int i) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const Gate<DECAY> t(word<IO>(rg[i], j), k[j]);
      float v = word<IO>(rx[i], j);
      if (GATED) v *= both_sides(word<IO>(ri[i], j)).p;
      if (PACKED && !mk.plain) {
        if (mk.starts >> i & 1) {
          const float h0 = q.h0 ? q.h0[(int64_t)seq_at(mk.seq, i) * q.C + c + j] : 0.f;
          p[j] = -0.f;
          h[j] = fmaf(t.a, h0, t.m * v);
        } else if (mk.inside >> i & 1) {
          p[j] = join(p[j], t.a);
          h[j] = fmaf(t.a, h[j], t.m * v);
        } else {
          p[j] = -0.f;
          h[j] = 0.f;
        }
      } else {
        p[j] *= t.a;
        h[j] = fmaf(t.a, h[j], t.m * v);
      }
      if (!ENDS) P[i][j] = p[j], H[i][j] = h[j];
    }
  };
  if (at.n == T && (!PACKED || mk.plain)) {
#pragma unroll
    for (int i = 0; i < T; ++i) row(i);
  } else {
#pragma unroll
    for (int i = 0; i < T; ++i)
      if (i < at.n) row(i);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) runs[at.wave][j][lane] = make_float2(p[j], h[j]);
  __syncthreads();
  if (ENDS) {
    if (at.wave == 0 && live) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        for (int w = 1; w < pl.waves; ++w) {
          const float2 r = runs[w][j][lane];
          h[j] = enter(r.x, r.y, h[j]);
          p[j] = join(p[j], r.x);
        }
        sums.P[(int64_t)at.unit * q.C + c + j] = p[j];
        sums.H[(int64_t)at.unit * q.C + c + j] = h[j];
      }
    }
    return;
  }
  if (at.n <= 0) return;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float e = 0.f;
    if (chained) e = sums.H[(int64_t)at.unit * q.C + c + j];
    else if (!PACKED && q.h0) e = q.h0[(int64_t)at.s * q.C + c + j];
    for (int w = at.lo; w < at.wave; ++w) {
      const float2 r = runs[w][j][lane];
      e = enter(r.x, r.y, e);
    }
#pragma unroll
    for (int i = 0; i < T; ++i) H[i][j] = PACKED ? enter(P[i][j], H[i][j], e) : fmaf(P[i][j], e, H[i][j]);
  }
  if (!live) return;
  IO* out = y + (int64_t)at.first * q.C;
  if (at.n == T && (!PACKED || mk.plain)) {
#pragma unroll
    for (int i = 0; i < T; ++i) store_word<IO>(out + (int64_t)i * q.C, off, H[i]);
  } else {
#pragma unroll
    for (int i = 0; i < T; ++i)
      if (i < at.n && (!PACKED || (mk.inside >> i & 1)))
        store_word<IO>(out + (int64_t)i * q.C, off, H[i]);
  }
  if (!fin) return;
  if (PACKED) {
    if (mk.ends) {
#pragma unroll
      for (int i = 0; i < T; ++i)
        if (mk.ends >> i & 1) {
#pragma unroll
          for (int j = 0; j < V; ++j) fin[(int64_t)seq_at(mk.seq, i) * q.C + c + j] = H[i][j];
        }
    }
  } else if (at.last) {
#pragma unroll
    for (int i = 0; i < T; ++i)
      if (i == at.n - 1) {
#pragma unroll
        for (int j = 0; j < V; ++j) fin[(int64_t)at.s * q.C + c + j] = H[i][j];
      }
  }
}

// Chain over the chunks, in place: sums.H from a chunk's end state to the state entering it
// (blockIdx.y 0), sums.G from what leaves the chunk to the left to what enters it from the right
// (blockIdx.y 1). Bound by the latency of its loads, which are issued kAhead chunks at a time.
__global__ __launch_bounds__(256) void k_rec_chain(RecArgs q, Plan pl, Sums sums,
                                                   const float* __restrict__ dfinal) {
  constexpr int kAhead = 16;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= (q.rows.starts ? 1 : (int64_t)q.rows.S) * q.C) return;
  const int64_t s = id / q.C;
  const int c = (int)(id % q.C);
  const bool back = blockIdx.y;
  const float* start = q.rows.starts ? nullptr : back ? dfinal : q.h0;
  float h = start ? start[id] : 0.f;
  const int64_t base = s * pl.chunks * q.C + c;
  float* io = back ? sums.G : sums.H;
  for (int u = 0; u < pl.chunks; u += kAhead) {
    float P[kAhead], H[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int v = min(u + i, pl.chunks - 1);
      const int64_t o = base + (int64_t)(back ? pl.chunks - 1 - v : v) * q.C;
      P[i] = sums.P[o];
      H[i] = io[o];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (u + i < pl.chunks) io[base + (int64_t)(back ? pl.chunks - 1 - u - i : u + i) * q.C] = h;
      h = enter(P[i], H[i], h);
    }
  }
}

// ---- backward --------------------------------------------------------------------------------------
// With l_t = dL/dh_t = dy_t + a_{t+1} l_{t+1}, c_t = a_t l_t (what goes on to the left):
//   dx = l m s, dinput_gate = l m v (1 - s), s = sigmoid(input_gate);
//   dlog a = l (a h_{t-1} - a^2 / m v), dgate = -dlog a u (1 - r), ddecay = -sum dlog a r times
//   sharpness sigmoid(decay); without a decay dgate = l (h_{t-1} - v) a (1 - a).
// ENDS: the runs' sums in both directions. Otherwise the gradients; part [units, C]: each block's
// sums for ddecay.
template <typename IO, bool DECAY, bool GATED, bool PACKED, bool ENDS>
__global__ __launch_bounds__(64 * kWaves) void k_rec_bwd(
    RecArgs q, Plan pl, int tiles, Sums sums, int chained, const IO* __restrict__ dy,
    const float* __restrict__ dfinal, IO* __restrict__ dx, IO* __restrict__ dg,
    IO* __restrict__ dgi, float* __restrict__ dh0, float* __restrict__ part) {
  constexpr int V = kV<IO>;
  __shared__ float2 runs[kWaves][V][64];
  __shared__ float left[kWaves][V][64];  // G of each wave; then the waves' sums for ddecay
  const int64_t main_blocks = (int64_t)tiles * pl.units;
  if (PACKED && blockIdx.x >= main_blocks) {
    pass_empty(q.rows, q.C, (int)(blockIdx.x - main_blocks), (int)(gridDim.x - main_blocks), dfinal,
               dh0);
    return;
  }
  const int tile = (int)(blockIdx.x % tiles), lane = threadIdx.x & 63;
  const Place at(q.rows, pl, (int)(blockIdx.x / tiles));
  const int c0 = (tile * 64 + lane) * V;
  const bool live = c0 < q.C;
  const int c = live ? c0 : q.C - V;
  const unsigned off = (unsigned)c * sizeof(IO);
  uint32_t rx[T], rg[T], ri[T], rd[T];
  load_rows<IO>(rg, q.g, q.gs, at.first, at.n, off);
  if (GATED) load_rows<IO>(ri, q.gi, q.is, at.first, at.n, off);
  load_rows<IO>(rx, q.x, q.xs, at.first, at.n, off);
  load_rows<IO>(rd, dy, q.C, at.first, at.n, off);
  Marks mk;
  if (PACKED && at.n > 0) mk.find(q.rows, at.first, at.n);
  float k[V];
#pragma unroll
  for (int j = 0; j < V; ++j) k[j] = DECAY ? decay_rate(q, c + j) : 0.f;
  auto start_state = [&](int i, int j) {
    return q.h0 ? q.h0[(int64_t)seq_at(mk.seq, i) * q.C + c + j] : 0.f;
  };
  auto end_grad = [&](int i, int j) {
    return dfinal ? dfinal[(int64_t)seq_at(mk.seq, i) * q.C + c + j] : 0.f;
  };

  float P[T][V], H[T][V];  // of the rows before each
  float p[V], h[V], g[V];
#pragma unroll
  for (int j = 0; j < V; ++j) p[j] = 1.f, h[j] = 0.f, g[j] = 0.f;
  auto row = [&](int i) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (!ENDS) P[i][j] = p[j], H[i][j] = h[j];
      const Gate<DECAY> t(word<IO>(rg[i], j), k[j]);
      float v = word<IO>(rx[i], j);
      if (GATED) v *= both_sides(word<IO>(ri[i], j)).p;
      float d = word<IO>(rd[i], j);
      if (PACKED && !mk.plain) {
        if (!(mk.inside >> i & 1)) {
          p[j] = -0.f;
          h[j] = 0.f;
          continue;
        }
        if (mk.ends >> i & 1) d += end_grad(i, j);
        if (mk.starts >> i & 1) {
          p[j] = -0.f;
          h[j] = fmaf(t.a, start_state(i, j), t.m * v);
          continue;
        }
      }
      p[j] = PACKED ? join(p[j], t.a) : p[j] * t.a;
      h[j] = fmaf(t.a, h[j], t.m * v);
      // (behind a start nothing reaches the left end)
      if (!PACKED || !cut(p[j])) g[j] = fmaf(p[j], d, g[j]);
    }
  };
  if (at.n == T && (!PACKED || mk.plain)) {
#pragma unroll
    for (int i = 0; i < T; ++i) row(i);
  } else {
#pragma unroll
    for (int i = 0; i < T; ++i)
      if (i < at.n) row(i);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    runs[at.wave][j][lane] = make_float2(p[j], h[j]);
    left[at.wave][j][lane] = g[j];
  }
  __syncthreads();
  if (ENDS) {
    if (at.wave == 0 && live) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        for (int w = 1; w < pl.waves; ++w) {
          const float2 r = runs[w][j][lane];
          if (!cut(p[j])) g[j] = fmaf(p[j], left[w][j][lane], g[j]);
          h[j] = enter(r.x, r.y, h[j]);
          p[j] = join(p[j], r.x);
        }
        const int64_t o = (int64_t)at.unit * q.C + c + j;
        sums.P[o] = p[j];
        sums.H[o] = h[j];
        sums.G[o] = g[j];
      }
    }
    return;
  }
  float sum[V];
#pragma unroll
  for (int j = 0; j < V; ++j) sum[j] = 0.f;
  if (at.n > 0) {
    float cl[V];  // c of the row to the right
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int64_t o = (int64_t)at.unit * q.C + c + j, so = (int64_t)at.s * q.C + c + j;
      float e = 0.f, r = 0.f;
      if (chained) e = sums.H[o], r = sums.G[o];
      else if (!PACKED) e = q.h0 ? q.h0[so] : 0.f, r = dfinal ? dfinal[so] : 0.f;
      for (int w = at.lo; w < at.wave; ++w) {
        const float2 t = runs[w][j][lane];
        e = enter(t.x, t.y, e);
      }
      for (int w = at.hi - 1; w > at.wave; --w) r = enter(runs[w][j][lane].x, left[w][j][lane], r);
#pragma unroll
      for (int i = 0; i < T; ++i)
        H[i][j] = PACKED ? enter(P[i][j], H[i][j], e) : fmaf(P[i][j], e, H[i][j]);
      cl[j] = r;
    }
    auto row_back = [&](int i) {
      float ox[V], og[V], oi[V];
      bool in = true;
      if (PACKED && !mk.plain) in = mk.inside >> i & 1;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const Gate<DECAY> t(word<IO>(rg[i], j), k[j]);
        const float x = word<IO>(rx[i], j);
        Sig s{1.f, 0.f};
        if (GATED) s = both_sides(word<IO>(ri[i], j));
        const float v = GATED ? x * s.p : x;
        float before = H[i][j];
        if (PACKED && !mk.plain) {
          if (!in) {
            ox[j] = og[j] = oi[j] = 0.f;
            cl[j] = 0.f;
            continue;
          }
          if (mk.ends >> i & 1) cl[j] = end_grad(i, j);
          if (mk.starts >> i & 1) before = start_state(i, j);
        }
        const float l = word<IO>(rd[i], j) + cl[j], lm = l * t.m;
        ox[j] = GATED ? lm * s.p : lm;
        oi[j] = lm * v * s.n;
        if constexpr (DECAY) {
          const float av = t.a * t.a * v, ah = t.a * before;
          og[j] = l * t.r.n * fmaf(av, t.u * t.inv, -t.u * ah);
          sum[j] = fmaf(l, fmaf(av, t.r.p * t.inv, -t.r.p * ah), sum[j]);
        } else {
          og[j] = l * (before - v) * (t.a * t.m);
        }
        cl[j] = t.a * l;
        if (PACKED && !mk.plain && (mk.starts >> i & 1)) {
          if (dh0 && live) dh0[(int64_t)seq_at(mk.seq, i) * q.C + c + j] = cl[j];
          cl[j] = 0.f;
        }
      }
      if (live) {
        const int64_t o = (int64_t)(at.first + i) * q.C;
        store_word<IO>(dx + o, off, ox);
        store_word<IO>(dg + o, off, og);
        if (GATED) store_word<IO>(dgi + o, off, oi);
      }
    };
    if (at.n == T && (!PACKED || mk.plain)) {
#pragma unroll
      for (int i = T - 1; i >= 0; --i) row_back(i);
    } else {
#pragma unroll
      for (int i = T - 1; i >= 0; --i)
        if (i < at.n) row_back(i);
    }
    if (!PACKED && dh0 && live && at.part == 0 && (pl.chunks == 1 || at.unit % pl.chunks == 0)) {
#pragma unroll
      for (int j = 0; j < V; ++j) dh0[(int64_t)at.s * q.C + c + j] = cl[j];
    }
  }
  if constexpr (DECAY) {
    __syncthreads();  // `left` has been read
#pragma unroll
    for (int j = 0; j < V; ++j) left[at.wave][j][lane] = sum[j];
    __syncthreads();
    if (at.wave == 0 && live) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float t = sum[j];
        for (int w = 1; w < (int)blockDim.x / 64; ++w) t += left[w][j][lane];
        part[(int64_t)at.unit * q.C + c + j] = t * (q.sharp * both_sides(q.decay[c + j]).p);
      }
    }
  }
}

// ---- single token ----------------------------------------------------------------------------------
// Four channels of a sequence a thread: bound by the launch and, for large batches, by the state read
// and written once.
template <typename IO, bool DECAY, bool GATED>
__global__ __launch_bounds__(256) void k_rec_step(RecArgs q, float* state_out, IO* y) {
  const int per = q.C / 4;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= (int64_t)q.rows.R * per) return;
  const int64_t b = id / per;
  const int c = (int)(id % per) * 4;
  Vec<IO, 4> x, g, gi;
  x.load((const IO*)q.x + b * q.xs + c);
  g.load((const IO*)q.g + b * q.gs + c);
  if (GATED) gi.load((const IO*)q.gi + b * q.is + c);
  float h[4], o[4];
  load_f32<4>(q.h0 + b * q.C + c, h);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const Gate<DECAY> t(g.get(j), DECAY ? decay_rate(q, c + j) : 0.f);
    float v = x.get(j);
    if (GATED) v *= both_sides(gi.get(j)).p;
    o[j] = fmaf(t.a, h[j], t.m * v);
  }
  store_vec<float, 4>(state_out + b * q.C + c, o);
  store_vec<IO, 4>(y + b * q.C + c, o);
}

template <typename F>
hipError_t by_kind(const RecArgs& a, F f) {
  auto gated = [&](auto io, auto decay) {
    return a.gi ? f(io, decay, std::true_type{}) : f(io, decay, std::false_type{});
  };
  auto decays = [&](auto io) {
    return a.decay ? gated(io, std::true_type{}) : gated(io, std::false_type{});
  };
  return a.io == kIoBf16 ? decays(u16{}) : decays(float{});
}

int tiles_of(const RecArgs& a) {
  const int v = a.io == kIoBf16 ? 2 : 1;
  return (a.C / v + 63) / 64;
}
int64_t sum_floats(const RecArgs& a, const Plan& p) {
  return ((int64_t)p.units * a.C + 63) / 64 * 64;
}
dim3 chain_grid(const RecArgs& a, int directions) {
  const int64_t n = (a.rows.starts ? 1 : (int64_t)a.rows.S) * a.C;
  return dim3((unsigned)((n + 255) / 256), directions);
}

}  // namespace

bool recurrence_fits(const RecArgs& a) {
  auto fits = [](double blocks, int threads) { return blocks * threads < 4294967296.0; };
  const Plan p = plan(a.rows);
  return fits(double(tiles_of(a)) * p.units + 4096, threads_of(p)) &&
         fits(double(a.rows.starts ? 1 : a.rows.S) * a.C / 256 + 1, 256);
}

int64_t recurrence_bytes(const RecArgs& a) {
  const Plan p = plan(a.rows);
  return p.chunks > 1 ? 8 * sum_floats(a, p) : 0;
}

hipError_t launch_recurrence(const RecArgs& a, void* y, float* fin, float* ws, hipStream_t s) {
  const Plan p = plan(a.rows);
  const int tiles = tiles_of(a), chained = p.chunks > 1;
  const Sums sums{ws, ws ? ws + sum_floats(a, p) : nullptr, nullptr};
  const unsigned blocks = (unsigned)((int64_t)tiles * p.units), more = empty_blocks(a, p, fin);
  return by_kind(a, [&](auto io, auto decay, auto gated) {
    using IO = decltype(io);
    constexpr bool D = decltype(decay)::value, G = decltype(gated)::value;
    auto run = [&](auto packed) {
      constexpr bool K = decltype(packed)::value;
      if (chained) {
        hipLaunchKernelGGL((k_rec<IO, D, G, K, true>), dim3(blocks), dim3(threads_of(p)), 0, s, a, p,
                           tiles, sums, 0, (IO*)nullptr, (float*)nullptr);
        hipLaunchKernelGGL(k_rec_chain, chain_grid(a, 1), dim3(256), 0, s, a, p, sums,
                           (const float*)nullptr);
      }
      hipLaunchKernelGGL((k_rec<IO, D, G, K, false>), dim3(blocks + more), dim3(threads_of(p)), 0, s,
                         a, p, tiles, sums, chained, (IO*)y, fin);
      return hipGetLastError();
    };
    return a.rows.starts ? run(std::true_type{}) : run(std::false_type{});
  });
}

hipError_t launch_recurrence_step(const RecArgs& a, float* state_out, void* y, hipStream_t s) {
  const unsigned blocks = (unsigned)(((int64_t)a.rows.R * (a.C / 4) + 255) / 256);
  return by_kind(a, [&](auto io, auto decay, auto gated) {
    using IO = decltype(io);
    hipLaunchKernelGGL((k_rec_step<IO, decltype(decay)::value, decltype(gated)::value>),
                       dim3(blocks), dim3(256), 0, s, a, state_out, (IO*)y);
    return hipGetLastError();
  });
}

int64_t recurrence_backward_bytes(const RecArgs& a) {
  const Plan p = plan(a.rows);
  return 4 * sum_floats(a, p) * ((p.chunks > 1 ? 3 : 0) + (a.decay ? 1 : 0));
}

hipError_t launch_recurrence_backward(const RecArgs& a, const void* dy, const float* dfinal,
                                      const RecGrads& g, float* ws, hipStream_t s) {
  const Plan p = plan(a.rows);
  const int tiles = tiles_of(a), chained = p.chunks > 1;
  const int64_t n = sum_floats(a, p);
  Sums sums{nullptr, nullptr, nullptr};
  float* part = ws;
  if (chained) {
    sums = Sums{ws, ws + n, ws + 2 * n};
    part = ws + 3 * n;
  }
  const unsigned blocks = (unsigned)((int64_t)tiles * p.units), more = empty_blocks(a, p, g.dh0);
  const hipError_t e = by_kind(a, [&](auto io, auto decay, auto gated) {
    using IO = decltype(io);
    constexpr bool D = decltype(decay)::value, G = decltype(gated)::value;
    auto run = [&](auto packed) {
      constexpr bool K = decltype(packed)::value;
      if (chained) {
        hipLaunchKernelGGL((k_rec_bwd<IO, D, G, K, true>), dim3(blocks), dim3(threads_of(p)), 0, s, a,
                           p, tiles, sums, 0, (const IO*)dy, dfinal, (IO*)nullptr, (IO*)nullptr,
                           (IO*)nullptr, (float*)nullptr, (float*)nullptr);
        hipLaunchKernelGGL(k_rec_chain, chain_grid(a, 2), dim3(256), 0, s, a, p, sums, dfinal);
      }
      hipLaunchKernelGGL((k_rec_bwd<IO, D, G, K, false>), dim3(blocks + more), dim3(threads_of(p)), 0,
                         s, a, p, tiles, sums, chained, (const IO*)dy, dfinal, (IO*)g.dx, (IO*)g.dg,
                         (IO*)g.dgi, g.dh0, part);
      return hipGetLastError();
    };
    return a.rows.starts ? run(std::true_type{}) : run(std::false_type{});
  });
  if (e != hipSuccess || !a.decay) return e;
  return launch_column_sums(part, p.units, a.C, g.ddecay, a.C, 0, 1, 0, nullptr, 0, nullptr, s);
}

}  // namespace ssd
