// Gated linear recurrence, one state entry a channel: forward, backward and single token.
//
//   h_t = a_t h_{t-1} + m_t v_t,  v = sigmoid(input_gate) x  (x without an input gate)
//   with a decay parameter:  u = sharpness softplus(decay) sigmoid(gate), a = exp(-u),
//                            m = sqrt(1 - a^2)
//   without:                 a = sigmoid(gate), m = 1 - a
//
// About 30 vector operations for each element read once: bound by memory if the rows are read once and
// the exponentials evaluated once, and not by much. The tokens of a sequence are sequential, but the
// recurrence is linear, so a run of rows is summed up by two numbers a channel, the product P of its a
// and its end state H from a zero state: h_end = P h_in + H. The adjoint runs the same way backwards
// (l_t = dy_t + a_{t+1} l_{t+1}; what leaves the run to the left is P c_in + G with the same P).
//
// A lane holds the channels of four bytes (two bf16, one fp32), a wave 64 lanes and T rows, all of
// whose loads are issued at once; the waves of a block take consecutive rows (a chunk) and combine
// their (P, H) through LDS.
#include <cmath>

#include "ssd_recurrent.h"
#include "ssd_selective.h"

namespace ssd {

namespace {

constexpr int kGroup = 8;  // chunks between those that hand on their end state
constexpr float kLn2 = 0.6931471805599453f;

// Rows of a wave (at most 31), waves of a block, bytes of a lane: of the forward, and of the backward's
// two passes (bf16, fp32).
struct Fwd { static constexpr int T = 16, W = 8, B = 4; };
struct Tall { static constexpr int T = 16, W = 16, B = 4; };  // forward: see tall()
// As many rows as fit 128 registers (eight of bf16 would take 134).
struct Bwd { static constexpr int T = 7, W = 4, B = 4; };
struct Bwd32 { static constexpr int T = 12, W = 4, B = 4; };
struct BwdTall { static constexpr int T = 7, W = 16, B = 4; };  // where that is one chunk a sequence
struct BwdTall32 { static constexpr int T = 12, W = 16, B = 4; };
template <typename IO, typename X>
constexpr int kV = X::B / (int)sizeof(IO);  // channels of a lane

// How the rows are cut. Dense: `chunks` of each sequence, of `waves` waves each; where a sequence is
// one chunk, a block takes `seqs` of them. Packed: chunks of all rows, wherever sequences begin.
struct Plan {
  int waves, seqs, chunks, units;  // units: blocks of one channel tile
};
template <typename X>
Plan plan(const Rows& q) {
  Plan p;
  const int64_t rows = q.starts ? q.R : q.L;
  const int64_t need = (rows + X::T - 1) / X::T;
  p.waves = (int)(need < X::W ? need : X::W);
  p.chunks = (int)((need + X::W - 1) / X::W);
  p.seqs = q.starts || p.chunks > 1 ? 1 : X::W / p.waves;
  if (!q.starts && p.seqs > q.S) p.seqs = q.S;
  p.units = q.starts ? p.chunks
                     : (int)(p.chunks > 1 ? (int64_t)p.chunks * q.S : ((int64_t)q.S + p.seqs - 1) / p.seqs);
  return p;
}
int threads_of(const Plan& p) { return 64 * p.waves * p.seqs; }

// ---- one element -----------------------------------------------------------------------------------
// 1 / (1 + exp(-v)), exact to a few roundings where it is small too (0 below -88).
__device__ __forceinline__ float one_side(float v) {
  return __builtin_amdgcn_rcpf(1.f + exp2_fast(-v * kLog2e));
}
// exp(-v), at most 2^126 (the minimum keeps NaN), and from it sigmoid(v), at least 2^-126, and
// sigmoid(-v), both to a few roundings of themselves.
__device__ __forceinline__ float exp_minus(float v) {
  return __builtin_elementwise_minimum(exp2_fast(-v * kLog2e), 0x1p126f);
}
struct Sig {
  float p, n;
  __device__ __forceinline__ explicit Sig(float e) : p(__builtin_amdgcn_rcpf(1.f + e)), n(e * p) {}
};

// 1 - a^2 from a = 2^-t, t >= 0: where the difference would cancel (below t = 0.36, that is a^2 = 0.61)
// the polynomial t c(t) of degree 5 that is nearest, to 9e-8 relative.
__device__ __forceinline__ float one_minus_square(float t, float a) {
  float s = fmaf(t, 0.03472883999347687f, -0.15147662162780762f);
  s = fmaf(t, s, 0.44372719526290894f);
  s = fmaf(t, s, -0.960892379283905f);
  s = fmaf(t, s, 1.3862942457199097f);
  return t < 0.36f ? t * s : fmaf(-a, a, 1.f);
}

// What a token does to a channel's state; rate = sharpness softplus(decay) log2(e).
struct Step {
  float a, m;
};
__device__ __forceinline__ Step decayed(float r, float rate) {
  const float t = rate * r, a = exp2_fast(-t);
  return Step{a, __builtin_amdgcn_sqrtf(one_minus_square(t, a))};
}
template <bool DECAY>
__device__ __forceinline__ Step step_of(float g, float rate) {
  if constexpr (DECAY) return decayed(one_side(g), rate);
  const Sig r(exp_minus(g));
  return Step{r.p, r.n};
}

// sharpness softplus(decay) log2(e), to a few roundings: exp(-|d|) with the product's rounding made
// good, log(1 + e) by its series where e is small, else from the hardware's log2 of the rounded sum and
// what the rounding lost. Finite for an infinite decay (at most 2^126), so that nothing times it is NaN;
// the minima keep NaN.
__device__ __forceinline__ float decay_rate(const RecArgs& q, int c) {
  const float d = q.decay[c], v = -__builtin_elementwise_minimum(fabsf(d), 200.f), hi = v * kLog2e;
  const float lo = fmaf(v, kLog2e, -hi) + v * 1.9259629911e-8f;  // log2(e) is 1.9e-8 above kLog2e
  const float e = exp2_fast(hi), x = fmaf(e, lo * kLn2, e), w = 1.f + x;
  const float small = x * fmaf(x, fmaf(x, fmaf(x, -0.25f, 1.f / 3.f), -0.5f), 1.f);
  const float large = fmaf(__builtin_amdgcn_logf(w), kLn2, x - (w - 1.f));
  const float rate = q.sharp * (fmaxf(d, 0.f) + (x < 0x1p-6f ? small : large)) * kLog2e;
  return __builtin_elementwise_minimum(rate, 0x1p126f);
}

// P of a run with a sequence's start in it is -0 (products of decays are never negative): what
// enters the run does not reach its end, not even as NaN.
__device__ __forceinline__ bool cut(float P) { return __float_as_uint(P) == 0x80000000u; }
__device__ __forceinline__ float enter(float P, float H, float h) { return cut(P) ? H : fmaf(P, h, H); }
__device__ __forceinline__ float join(float P, float Q) { return cut(P) || cut(Q) ? -0.f : P * Q; }

// ---- rows of a wave --------------------------------------------------------------------------------
// The channels of a lane, B bytes of a row, as loaded.
template <typename IO, int B>
struct Word {
  uint32_t u[B / 4];
  __device__ __forceinline__ float operator[](int j) const {
    if constexpr (sizeof(IO) == 4) return __uint_as_float(u[j]);
    else return __uint_as_float(j & 1 ? u[j / 2] & 0xffff0000u : u[j / 2] << 16);
  }
};

template <typename IO, int B, int V>
__device__ __forceinline__ void store_word(IO* row, unsigned off, const float (&v)[V], int stream) {
  typedef uint32_t words __attribute__((ext_vector_type(B / 4)));
  words u;
#pragma unroll
  for (int i = 0; i < B / 4; ++i) {
    if constexpr (sizeof(IO) == 4) u[i] = __float_as_uint(v[i]);
    else u[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  }
  store_words((words*)((char*)row + off), u, stream);
}

// Rows of several tensors, one after another, so that the first rows can be worked on while the others
// arrive.
template <typename IO, int B>
struct Source {
  const char* p;
  int64_t step;
  __device__ __forceinline__ Source(const void* t, int64_t stride, int r0)
      : p((const char*)((const IO*)t + r0 * stride)), step(stride * sizeof(IO)) {}
  __device__ __forceinline__ void next(Word<IO, B>& w, unsigned off) {
    typedef uint32_t words __attribute__((ext_vector_type(B / 4)));
    const words v = *(const words*)(p + off);
#pragma unroll
    for (int i = 0; i < B / 4; ++i) w.u[i] = v[i];
    p += step;
  }
};
template <int T, typename F>
__device__ __forceinline__ void for_rows(bool all, int n, F f) {
  if (all) {
#pragma unroll
    for (int i = 0; i < T; ++i) f(i);
  } else {
#pragma unroll
    for (int i = 0; i < T; ++i)
      if (i < n) f(i);
  }
}
template <int T, typename F>
__device__ __forceinline__ void for_rows_back(bool all, int n, F f) {
  if (all) {
#pragma unroll
    for (int i = T - 1; i >= 0; --i) f(i);
  } else {
#pragma unroll
    for (int i = T - 1; i >= 0; --i)
      if (i < n) f(i);
  }
}

// Where a block's waves stand.
struct Place {
  int unit, wave, first, n;  // block of a tile; wave; its rows [first, first + n)
  int s, part;               // dense: its sequence; its place among the sequence's waves here
  bool last;                 // dense: the sequence ends in these rows
  int lo, hi;                // waves whose runs this one's joins
  __device__ __forceinline__ Place(const Rows& q, const Plan& p, int T, int unit_) {
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

// Channels of a lane.
template <int V>
struct Lane {
  int c, lane;
  bool live;
  __device__ __forceinline__ Lane(const RecArgs& q, int tile) {
    lane = threadIdx.x & 63;
    const int c0 = (tile * 64 + lane) * V;
    live = c0 < q.C;
    c = live ? c0 : q.C - V;  // idle lanes compute the last channels again
  }
};

// Sequence boundaries among a wave's rows (packed), found by the scalar unit beside the rows' loads.
struct Marks {
  uint32_t starts = 0, ends = 0, inside = 0;  // a bit a row
  int seq = -1;                               // of row i, in lane i
  bool plain = true;
  static __device__ __forceinline__ int offset(const Rows& q, int i) {
    typedef const __attribute__((address_space(4))) int* Words;  // read through scalar loads
    return ((Words)(uintptr_t)q.starts)[__builtin_amdgcn_readfirstlane(i)];
  }
  __device__ __forceinline__ void find(const Rows& q, int first, int n) {
    const int lane = threadIdx.x & 63, stop = first + n;
    const uint32_t all = (1u << n) - 1;
    const int front = offset(q, 0);
    for (int r = first; r < stop;) {
      if (r < front) {  // in front of the first sequence
        r = min(front, stop);
        continue;
      }
      int lo = 0, hi = q.S;  // as seq_of
      while (hi - lo > 1) {
        const int m = lo + ((hi - lo) >> 1);
        if (offset(q, m) <= r) lo = m; else hi = m;
      }
      const int begin = max(offset(q, lo), 0), end = min(offset(q, lo + 1), q.R);
      if (end <= r) break;  // behind the last
      const int to = min(end, stop);
      if (begin == r) starts |= 1u << (r - first);
      if (to == end) ends |= 1u << (to - 1 - first);
      inside |= ((1u << (to - first)) - 1) & ~((1u << (r - first)) - 1);
      seq = lane >= r - first && lane < to - first ? lo : seq;
      r = to;
    }
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

// ---- forward ---------------------------------------------------------------------------------------
// Chunks of one call hand on what follows them needs through `slots` [units, C], one 64-bit word a
// channel: (P, H) of the chunk, or of every kGroup-th chunk its end state, as a run with P = -0. A word
// is written once, as a whole, so it needs no flag beside it: `kEmpty` until then.
constexpr uint64_t kEmpty = ~0ull;
struct Chain {
  uint64_t* slots;
  uint32_t* tickets;  // a counter a tile and sequence (packed: a tile), kApart words apart
  int counters;
};
constexpr int kApart = 16;
// Looks at the words of the chunks in front, each at least a load that passes the caches (over half a
// microsecond): half a second or more where an ordinary wait is some microseconds. It runs out only where
// another call uses the same workspace at the same time; what has not come then counts as NaN.
constexpr int kLooks = 1 << 20;
__device__ __forceinline__ void publish(uint64_t* slot, float P, float H) {
  uint32_t h = __float_as_uint(H);
  if (h == ~0u) h = 0x7fc00000u;  // (a NaN of a caller's, which would look empty)
  __hip_atomic_store(slot, (uint64_t)__float_as_uint(P) << 32 | h, __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
__global__ __launch_bounds__(256) void k_rec_clear(Chain chain, int64_t n) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id < chain.counters) chain.tickets[id * kApart] = 0;
  if (id < n) chain.slots[id] = kEmpty;
}

// One pass: each element is read once. 2 x 8192 x 5120 bf16 with gates and decay takes 160 us (4.2 TB/s; the
// bytes alone 129 at a large copy's rate, the same loads and stores without the arithmetic 138, which
// keeps the vector units busy for 90 of them); 5003 packed x 1536 takes 25. Two passes over the rows with
// a chain between took 319 and 53. Without gain: 8, 10 or 12 rows a wave, 8 bytes a lane, chunks of one
// sequence next to one another in the grid, end states handed on every 4 (16 or 32: more registers,
// slower), and rows of the tensors loaded in turn.
// CHAIN: sequences of several chunks. A block belongs to a tile and sequence and takes the next chunk of
// them by a ticket. It waits only for chunks before its own, whose blocks have lower tickets: those are
// running or done, and the first of them waits for none, so every wait ends. (Calls that share a workspace
// and overlap, against the contract, take tickets from one counter and clear each other's words: a ticket
// past the last chunk is no work, and a wait ends after kLooks.)
template <typename X, typename IO, bool DECAY, bool GATED, bool PACKED, bool CHAIN>
__global__ __launch_bounds__(64 * X::W) void k_rec(RecArgs q, Plan pl, int tiles, Chain chain,
                                                   IO* __restrict__ y, float* __restrict__ fin) {
  constexpr int V = kV<IO, X>, T = X::T, B = X::B;
  __shared__ float2 runs[X::W][V][64];
  __shared__ float entry[V][64];
  __shared__ uint32_t place;
  const int64_t main_blocks = (int64_t)tiles * pl.units;
  if (PACKED && blockIdx.x >= main_blocks) {
    pass_empty(q.rows, q.C, (int)(blockIdx.x - main_blocks), (int)(gridDim.x - main_blocks), q.h0, fin);
    return;
  }
  const int tile = (int)(blockIdx.x % tiles);
  int unit = (int)(blockIdx.x / tiles);
  const int s = PACKED ? 0 : unit % q.rows.S;
  uint32_t ticket = 0;
  if (CHAIN && threadIdx.x == 0)
    ticket = __hip_atomic_fetch_add(chain.tickets + ((int64_t)s * tiles + tile) * kApart, 1u,
                                    __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const Lane<V> me(q, tile);
  const int c = me.c, lane = me.lane;
  const unsigned off = (unsigned)c * sizeof(IO);
  float k[V];
#pragma unroll
  for (int j = 0; j < V; ++j) k[j] = DECAY ? decay_rate(q, c + j) : 0.f;
  if (CHAIN) {
    if (threadIdx.x == 0) place = ticket;
    __syncthreads();
    const unsigned turn = __builtin_amdgcn_readfirstlane(place);
    if (turn >= (unsigned)pl.chunks) return;
    unit = s * pl.chunks + (int)turn;
  }
  const Place at(q.rows, pl, T, unit);
  Word<IO, B> rx[T], rg[T], ri[T];
  Source<IO, B> sg(q.g, q.gs, at.first), si(q.gi, q.is, at.first), sx(q.x, q.xs, at.first);
  for_rows<T>(at.n == T, at.n, [&](int i) {
    sg.next(rg[i], off);
    if (GATED) si.next(ri[i], off);
    sx.next(rx[i], off);
  });
  Marks mk;
  if (PACKED && at.n > 0) mk.find(q.rows, at.first, at.n);
  const bool plain = at.n == T && (!PACKED || mk.plain);

  float P[T][V], H[T][V];  // of the rows up to each
  float p[V], h[V];
#pragma unroll
  for (int j = 0; j < V; ++j) p[j] = 1.f, h[j] = 0.f;
  for_rows<T>(plain, at.n, [&](int i) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const Step t = step_of<DECAY>(rg[i][j], k[j]);
      float v = rx[i][j];
      if (GATED) v *= one_side(ri[i][j]);
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
      P[i][j] = p[j], H[i][j] = h[j];
    }
  });
#pragma unroll
  for (int j = 0; j < V; ++j) runs[at.wave][j][lane] = make_float2(p[j], h[j]);
  __syncthreads();
  // the run of the waves in front of this one; of wave 0 with a chain: of all the block's
  const int to = CHAIN && at.wave == 0 ? pl.waves : at.wave;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float2 r[X::W];
#pragma unroll
    for (int w = 0; w < X::W; ++w) r[w] = runs[w][j][lane];
    p[j] = 1.f, h[j] = 0.f;
#pragma unroll
    for (int w = 0; w < X::W; ++w)
      if (w >= at.lo && w < to) {
        h[j] = enter(r[w].x, r[w].y, h[j]);
        p[j] = join(p[j], r[w].x);
      }
  }
  float e[V];  // the state that enters
  if (CHAIN) {
    const int chunk = PACKED ? at.unit : at.unit % pl.chunks;
    if (at.wave == 0) {
      uint64_t* slot = chain.slots + (int64_t)at.unit * q.C + c;
      const bool hands_on = chunk % kGroup == kGroup - 1, needed = chunk + 1 < pl.chunks;
      if (needed && !hands_on && me.live) {
#pragma unroll
        for (int j = 0; j < V; ++j) publish(slot + j, p[j], h[j]);
      }
      const int from = max(chunk / kGroup * kGroup - 1, 0);
#pragma unroll
      for (int j = 0; j < V; ++j)
        e[j] = !PACKED && q.h0 ? q.h0[(int64_t)at.s * q.C + c + j] : 0.f;
      uint64_t got[kGroup][V];
      bool all;
      int looks = 0;
      do {
        all = true;
#pragma unroll
        for (int i = 0; i < kGroup; ++i)
          if (from + i < chunk) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
              got[i][j] = __hip_atomic_load(slot + (int64_t)(from + i - chunk) * q.C + j,
                                            __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
              all = all && got[i][j] != kEmpty;
            }
          }
      } while (!__all(all) && ++looks < kLooks);
#pragma unroll
      for (int i = 0; i < kGroup; ++i)
        if (from + i < chunk) {
#pragma unroll
          for (int j = 0; j < V; ++j)
            e[j] = enter(__uint_as_float((uint32_t)(got[i][j] >> 32)),
                         __uint_as_float((uint32_t)got[i][j]), e[j]);
        }
      if (needed && hands_on && me.live) {
#pragma unroll
        for (int j = 0; j < V; ++j) publish(slot + j, -0.f, enter(p[j], h[j], e[j]));
      }
#pragma unroll
      for (int j = 0; j < V; ++j) entry[j][lane] = e[j];
    }
    __syncthreads();
    if (at.n <= 0) return;
#pragma unroll
    for (int j = 0; j < V; ++j) e[j] = entry[j][lane];
  } else {
    if (at.n <= 0) return;
#pragma unroll
    for (int j = 0; j < V; ++j)
      e[j] = !PACKED && q.h0 ? q.h0[(int64_t)at.s * q.C + c + j] : 0.f;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (!CHAIN || at.wave) e[j] = enter(p[j], h[j], e[j]);
#pragma unroll
    for (int i = 0; i < T; ++i)
      H[i][j] = PACKED ? enter(P[i][j], H[i][j], e[j]) : fmaf(P[i][j], e[j], H[i][j]);
  }
  if (!me.live) return;
  IO* out = y + (int64_t)at.first * q.C;
  for_rows<T>(plain, at.n, [&](int i) {
    if (!PACKED || (mk.inside >> i & 1))
      store_word<IO, B>(out + (int64_t)i * q.C, off, H[i], q.stream);
  });
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

// Sums of the runs, [units, C] each.
struct Sums {
  float *P, *H, *G;
};

// Chain over the chunks, in place: sums.H from a chunk's end state to the state entering it
// (blockIdx.y 0), sums.G from what leaves the chunk to the left to what enters it from the right
// (blockIdx.y 1). Bound by the latency of its loads: the kParts waves of a block take a run of chunks of
// the same 64 channels each, up to kAhead of them, whose loads are issued together, and join their runs
// through LDS (147 chunks of 2 x 5120 channels: 15 -> 11 us against one thread for all of a channel's).
constexpr int kParts = 8, kAhead = 32;
__global__ __launch_bounds__(64 * kParts) void k_rec_chain(RecArgs q, Plan pl, Sums sums,
                                                           const float* __restrict__ dfinal) {
  __shared__ float2 runs[kParts][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t all = (q.rows.starts ? 1 : (int64_t)q.rows.S) * q.C;
  const bool live = (int64_t)blockIdx.x * 64 + lane < all, back = blockIdx.y;
  const int64_t id = live ? (int64_t)blockIdx.x * 64 + lane : all - 1;
  const int64_t base = id / q.C * pl.chunks * q.C + id % q.C;
  const float* start = q.rows.starts ? nullptr : back ? dfinal : q.h0;
  float* io = back ? sums.G : sums.H;
  float carry = start ? start[id] : 0.f;
  const int each = min((pl.chunks + kParts - 1) / kParts, kAhead);
  for (int u0 = 0; u0 < pl.chunks; u0 += kParts * each) {
    const int first = u0 + wave * each, n = min(pl.chunks - first, each);
    auto place = [&](int i) { return base + (int64_t)(back ? pl.chunks - 1 - first - i : first + i) * q.C; };
    float P[kAhead], H[kAhead], p = 1.f, h = 0.f;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i < n) P[i] = sums.P[place(i)], H[i] = io[place(i)];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i < n) {
        h = enter(P[i], H[i], h);
        p = join(p, P[i]);
      }
    __syncthreads();  // what was here has been read
    runs[wave][lane] = make_float2(p, h);
    __syncthreads();
    float e = carry;
#pragma unroll
    for (int w = 0; w < kParts; ++w) {
      const float2 r = runs[w][lane];
      if (w == wave) e = carry;
      carry = enter(r.x, r.y, carry);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i < n) {
        if (live) io[place(i)] = e;
        e = enter(P[i], H[i], e);
      }
  }
}

// ---- backward --------------------------------------------------------------------------------------
// With l_t = dL/dh_t = dy_t + a_{t+1} l_{t+1}, c_t = a_t l_t (what goes on to the left):
//   dx = l m s, dinput_gate = l m v (1 - s), s = sigmoid(input_gate);
//   dlog a = l (a h_{t-1} - a^2 / m v), dgate = -dlog a u (1 - r), ddecay = -sum dlog a r times
//   sharpness sigmoid(decay); without a decay dgate = l (h_{t-1} - v) a (1 - a).
// Two passes and a chain between them: what enters a chunk from the left needs all before it, what enters
// from the right all behind it. First pass: the chunks' sums in both directions.
template <typename X, typename IO, bool DECAY, bool GATED, bool PACKED>
__global__ __launch_bounds__(64 * X::W) void k_rec_sums(RecArgs q, Plan pl, int tiles, Sums sums,
                                                        const IO* __restrict__ dy,
                                                        const float* __restrict__ dfinal) {
  constexpr int V = kV<IO, X>, T = X::T, B = X::B;
  __shared__ float2 runs[X::W][V][64];
  __shared__ float left[X::W][V][64];
  const Lane<V> me(q, (int)(blockIdx.x % tiles));
  const Place at(q.rows, pl, T, (int)(blockIdx.x / tiles));
  const int c = me.c, lane = me.lane;
  const unsigned off = (unsigned)c * sizeof(IO);
  Word<IO, B> rx[T], rg[T], ri[T], rd[T];
  Source<IO, B> sg(q.g, q.gs, at.first), si(q.gi, q.is, at.first), sx(q.x, q.xs, at.first),
      sd(dy, q.C, at.first);
  for_rows<T>(at.n == T, at.n, [&](int i) {
    sg.next(rg[i], off);
    if (GATED) si.next(ri[i], off);
    sx.next(rx[i], off);
    sd.next(rd[i], off);
  });
  Marks mk;
  if (PACKED && at.n > 0) mk.find(q.rows, at.first, at.n);
  float p[V], h[V], g[V], k[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    k[j] = DECAY ? decay_rate(q, c + j) : 0.f;
    p[j] = 1.f, h[j] = 0.f, g[j] = 0.f;
  }
  for_rows<T>(at.n == T && (!PACKED || mk.plain), at.n, [&](int i) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const Step t = step_of<DECAY>(rg[i][j], k[j]);
      float v = rx[i][j], d = rd[i][j];
      if (GATED) v *= one_side(ri[i][j]);
      if (PACKED && !mk.plain) {
        const int64_t o = (int64_t)max(seq_at(mk.seq, i), 0) * q.C + c + j;
        if (!(mk.inside >> i & 1)) {
          p[j] = -0.f;
          h[j] = 0.f;
          continue;
        }
        if ((mk.ends >> i & 1) && dfinal) d += dfinal[o];
        if (mk.starts >> i & 1) {
          p[j] = -0.f;
          h[j] = fmaf(t.a, q.h0 ? q.h0[o] : 0.f, t.m * v);
          continue;
        }
      }
      p[j] = PACKED ? join(p[j], t.a) : p[j] * t.a;
      h[j] = fmaf(t.a, h[j], t.m * v);
      // (behind a start nothing reaches the left end)
      if (!PACKED || !cut(p[j])) g[j] = fmaf(p[j], d, g[j]);
    }
  });
#pragma unroll
  for (int j = 0; j < V; ++j) {
    runs[at.wave][j][lane] = make_float2(p[j], h[j]);
    left[at.wave][j][lane] = g[j];
  }
  __syncthreads();
  if (at.wave || !me.live) return;
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

// How a chunk of the second pass finds what enters it: it is the only one; from the chain; or from the sums
// of the others.
enum { kAlone, kJoined, kSingly };

// Second pass (or the only one): the gradients; part [units, C]: each block's sums for ddecay. Forward
// through the rows, then back; what the way back needs of the way forward stays in registers, the
// gates by their exponentials, from which both sides of a sigmoid come exactly. 2 x 4096 x 5120 bf16 with
// gates and decay: first pass 72 us, chain 10, this one 115 to 120, sums for ddecay 5; the bytes read and
// written once take 113, and this pass alone moves them all. 4 x 2048 x 768 fp32 without: 15, 4, 20.
template <typename X, typename IO, bool DECAY, bool GATED, bool PACKED>
__global__ __launch_bounds__(64 * X::W, 4) void k_rec_bwd(
    RecArgs q, Plan pl, int tiles, Sums sums, int chained, const IO* __restrict__ dy,
    const float* __restrict__ dfinal, IO* __restrict__ dx, IO* __restrict__ dg,
    IO* __restrict__ dgi, float* __restrict__ dh0, float* __restrict__ part) {
  constexpr int V = kV<IO, X>, T = X::T, B = X::B;
  __shared__ float2 runs[X::W][V][64];
  __shared__ float left[X::W][V][64];  // G of each wave; then the waves' sums for ddecay
  const int64_t main_blocks = (int64_t)tiles * pl.units;
  if (PACKED && blockIdx.x >= main_blocks) {
    pass_empty(q.rows, q.C, (int)(blockIdx.x - main_blocks), (int)(gridDim.x - main_blocks), dfinal,
               dh0);
    return;
  }
  const Lane<V> me(q, (int)(blockIdx.x % tiles));
  // from the end, where the first pass left what it read in the last-level cache
  const Place at(q.rows, pl, T, pl.units - 1 - (int)(blockIdx.x / tiles));
  const int c = me.c, lane = me.lane;
  const unsigned off = (unsigned)c * sizeof(IO);
  Word<IO, B> rx[T], rg[T], ri[T], rd[T];
  Source<IO, B> sg(q.g, q.gs, at.first), si(q.gi, q.is, at.first), sx(q.x, q.xs, at.first),
      sd(dy, q.C, at.first);
  for_rows<T>(at.n == T, at.n, [&](int i) {
    sg.next(rg[i], off);
    if (GATED) si.next(ri[i], off);
    sx.next(rx[i], off);
    sd.next(rd[i], off);
  });
  float cl[V], e[V];  // c of the row to the right; the state that enters
  auto alone = [&](int j) {
    const int64_t so = (int64_t)at.s * q.C + c + j;
    e[j] = !PACKED && q.h0 ? q.h0[so] : 0.f, cl[j] = !PACKED && dfinal ? dfinal[so] : 0.f;
  };
  const int64_t o = (int64_t)at.unit * q.C + c;
  if (chained == kSingly) {
    const int chunk = PACKED ? at.unit : at.unit % pl.chunks;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      alone(j);
#pragma unroll 4
      for (int u = -chunk; u < 0; ++u) e[j] = enter(sums.P[o + u * q.C + j], sums.H[o + u * q.C + j], e[j]);
#pragma unroll 4
      for (int u = pl.chunks - 1 - chunk; u > 0; --u)
        cl[j] = enter(sums.P[o + u * q.C + j], sums.G[o + u * q.C + j], cl[j]);
    }
  }
  Marks mk;
  if (PACKED && at.n > 0) mk.find(q.rows, at.first, at.n);
  const bool plain = at.n == T && (!PACKED || mk.plain);
  float k[V];
#pragma unroll
  for (int j = 0; j < V; ++j) k[j] = DECAY ? decay_rate(q, c + j) : 0.f;
  auto start_state = [&](int i, int j) {
    return q.h0 ? q.h0[(int64_t)seq_at(mk.seq, i) * q.C + c + j] : 0.f;
  };
  auto end_grad = [&](int i, int j) {
    return dfinal ? dfinal[(int64_t)seq_at(mk.seq, i) * q.C + c + j] : 0.f;
  };

  float eg[T][V], es[T][V], ka[T][V], km[T][V];  // exp(-gate), exp(-input_gate), a, m
  float b[T][V];                                 // m v, then the state before each row
  float p[V], h[V], g[V];
#pragma unroll
  for (int j = 0; j < V; ++j) p[j] = 1.f, h[j] = 0.f, g[j] = 0.f;
  for_rows<T>(plain, at.n, [&](int i) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      eg[i][j] = exp_minus(rg[i][j]);
      const Sig r(eg[i][j]);
      Step t{r.p, r.n};
      if constexpr (DECAY) t = decayed(r.p, k[j]);
      ka[i][j] = t.a;
      km[i][j] = t.m;
      float v = rx[i][j], d = rd[i][j];
      if (GATED) {
        es[i][j] = exp_minus(ri[i][j]);
        v *= Sig(es[i][j]).p;
      }
      b[i][j] = t.m * v;
      if (PACKED && !mk.plain) {
        if (!(mk.inside >> i & 1)) {
          p[j] = -0.f;
          h[j] = 0.f;
          continue;
        }
        if (mk.ends >> i & 1) d += end_grad(i, j);
        if (mk.starts >> i & 1) {
          p[j] = -0.f;
          h[j] = fmaf(t.a, start_state(i, j), b[i][j]);
          continue;
        }
      }
      p[j] = PACKED ? join(p[j], t.a) : p[j] * t.a;
      h[j] = fmaf(t.a, h[j], b[i][j]);
      if (!PACKED || !cut(p[j])) g[j] = fmaf(p[j], d, g[j]);
    }
  });
#pragma unroll
  for (int j = 0; j < V; ++j) {
    runs[at.wave][j][lane] = make_float2(p[j], h[j]);
    left[at.wave][j][lane] = g[j];
  }
  __syncthreads();
  float sum[V];
#pragma unroll
  for (int j = 0; j < V; ++j) sum[j] = 0.f;
  if (at.n > 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (chained == kJoined) e[j] = sums.H[o + j], cl[j] = sums.G[o + j];
      if (chained == kAlone) alone(j);
      for (int w = at.lo; w < at.wave; ++w) {
        const float2 t = runs[w][j][lane];
        e[j] = enter(t.x, t.y, e[j]);
      }
      for (int w = at.hi - 1; w > at.wave; --w)
        cl[j] = enter(runs[w][j][lane].x, left[w][j][lane], cl[j]);
    }
    for_rows<T>(plain, at.n, [&](int i) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (PACKED && !mk.plain) {
          if (mk.starts >> i & 1) e[j] = start_state(i, j);
          if (!(mk.inside >> i & 1)) e[j] = 0.f;
        }
        const float before = e[j];
        e[j] = fmaf(ka[i][j], e[j], b[i][j]);
        b[i][j] = before;
      }
    });
    for_rows_back<T>(plain, at.n, [&](int i) {
      float ox[V], og[V], oi[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (PACKED && !mk.plain) {
          if (!(mk.inside >> i & 1)) {
            ox[j] = og[j] = oi[j] = 0.f;
            cl[j] = 0.f;
            continue;
          }
          if (mk.ends >> i & 1) cl[j] = end_grad(i, j);
        }
        const Sig r(eg[i][j]);
        const float a = ka[i][j], m = km[i][j], before = b[i][j];
        const float l = rd[i][j] + cl[j], lm = l * m;
        float v = rx[i][j];
        ox[j] = lm;
        if (GATED) {
          const Sig s(es[i][j]);
          v *= s.p;
          ox[j] = lm * s.p;
          oi[j] = lm * (v * s.n);
        }
        if constexpr (DECAY) {
          // 1 / m at most 2^63, so that u / m is 0 where u is
          const float inv = __builtin_amdgcn_rcpf(fmaxf(m, 0x1p-63f));
          const float d = l * fmaf(a * a, v * inv, -a * before);  // -dL/dlog a
          og[j] = d * (r.n * (k[j] * kLn2 * r.p));
          sum[j] = fmaf(d, r.p, sum[j]);
        } else {
          og[j] = l * (before - v) * (a * m);
        }
        cl[j] = a * l;
        if (PACKED && !mk.plain && (mk.starts >> i & 1)) {
          if (dh0 && me.live) dh0[(int64_t)seq_at(mk.seq, i) * q.C + c + j] = cl[j];
          cl[j] = 0.f;
        }
      }
      if (me.live) {
        const int64_t o = (int64_t)(at.first + i) * q.C;
        store_word<IO, B>(dx + o, off, ox, q.stream);
        store_word<IO, B>(dg + o, off, og, q.stream);
        if (GATED) store_word<IO, B>(dgi + o, off, oi, q.stream);
      }
    });
    if (!PACKED && dh0 && me.live && at.part == 0 && (pl.chunks == 1 || at.unit % pl.chunks == 0)) {
#pragma unroll
      for (int j = 0; j < V; ++j) dh0[(int64_t)at.s * q.C + c + j] = cl[j];
    }
  }
  if constexpr (DECAY) {
    __syncthreads();  // `left` has been read
#pragma unroll
    for (int j = 0; j < V; ++j) left[at.wave][j][lane] = sum[j];
    __syncthreads();
    if (at.wave == 0 && me.live) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float t = sum[j];
        for (int w = 1; w < (int)blockDim.x / 64; ++w) t += left[w][j][lane];
        part[(int64_t)at.unit * q.C + c + j] = t * (q.sharp * one_side(q.decay[c + j]));
      }
    }
  }
}

// ---- single token ----------------------------------------------------------------------------------
// Four channels of a sequence a thread: bound by the launch (64 x 2560 bf16: 3 us) and, for large batches,
// by the state read and written once.
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
    const Step t = step_of<DECAY>(g.get(j), DECAY ? decay_rate(q, c + j) : 0.f);
    float v = x.get(j);
    if (GATED) v *= one_side(gi.get(j));
    o[j] = fmaf(t.a, h[j], t.m * v);
  }
  store_vec<float, 4>(state_out + b * q.C + c, o);
  store_vec<IO, 4>(y + b * q.C + c, o);
}

template <typename F>
hipError_t by_kind(const RecArgs& a, F f) {
  auto packed = [&](auto io, auto decay, auto gated) {
    return a.rows.starts ? f(io, decay, gated, std::true_type{}) : f(io, decay, gated, std::false_type{});
  };
  auto gated = [&](auto io, auto decay) {
    return a.gi ? packed(io, decay, std::true_type{}) : packed(io, decay, std::false_type{});
  };
  auto decays = [&](auto io) {
    return a.decay ? gated(io, std::true_type{}) : gated(io, std::false_type{});
  };
  return a.io == kIoBf16 ? decays(u16{}) : decays(float{});
}

// The backward's shape and plan: f(shape, plan). Sixteen waves where they hold a whole sequence (packed:
// all rows) and four do not: the rows are read once, and there is no first pass and no chain; and where they
// hold the whole call, whose sums for ddecay then need no launch of their own (8 x 3 x 280 bf16 23 -> 19 us; 87 x 104 bf16 28 -> 18 us,
// 64 x 100 x 5120 222 -> 141, 256 x 30 x 5120 421 -> 151).
template <typename Low, typename High, typename F>
auto by_height(const RecArgs& a, F f) {
  const Plan low = plan<Low>(a.rows), high = plan<High>(a.rows);
  const bool one = high.units == 1 && low.units > 1;
  return high.chunks == 1 && (low.chunks > 1 || one) ? f(High{}, high) : f(Low{}, low);
}
template <typename F>
auto by_shape(const RecArgs& a, F f) {
  return a.io == kIoBf16 ? by_height<Bwd, BwdTall>(a, f) : by_height<Bwd32, BwdTall32>(a, f);
}

template <typename X>
int tiles_of(const RecArgs& a) {
  const int width = 64 * X::B / (a.io == kIoBf16 ? 2 : 4);
  return (a.C + width - 1) / width;
}
int64_t sum_floats(const RecArgs& a, const Plan& p) {
  return ((int64_t)p.units * a.C + 63) / 64 * 64;
}
int64_t counters_of(const RecArgs& a) {
  return (int64_t)tiles_of<Fwd>(a) * (a.rows.starts ? 1 : a.rows.S);
}
// Blocks of sixteen waves where they hold a whole sequence and eight do not (200 x 104 bf16 18 -> 14 us,
// 64 x 256 x 5120 157 -> 148), and where all of them run at once, one a compute unit: half as many chunks
// wait for one another (5003 packed x 1536 bf16: 28 -> 25 us; with more blocks than that, 2 x 8192 x 5120,
// two of eight waves a unit overlap better: 160 against 187 us).
bool tall(const RecArgs& a) {
  const Plan p = plan<Tall>(a.rows), f = plan<Fwd>(a.rows);
  if (f.chunks == 1 || p.chunks == 1) return f.chunks > 1;
  return (int64_t)tiles_of<Tall>(a) * p.units <= 256 && (int64_t)tiles_of<Fwd>(a) * f.units > 256;
}
dim3 chain_grid(const RecArgs& a) {  // both directions
  const int64_t n = (a.rows.starts ? 1 : (int64_t)a.rows.S) * a.C;
  return dim3((unsigned)((n + 63) / 64), 2);
}

// (The backward's first pass finds more of its inputs there: 2 x 4096 x 5120 88 -> 72 us; the forward of
// 2 x 8192 x 5120 166 -> 160 us.)
int stream_of(const RecArgs& a) {
  return past_caches((double)a.rows.R * a.C * (a.io == kIoBf16 ? 2 : 4));
}

}  // namespace

bool recurrence_fits(const RecArgs& a) {
  auto fits = [](double blocks, int threads) { return blocks * threads < 4294967296.0; };
  const Plan f = plan<Fwd>(a.rows), b = by_shape(a, [](auto, Plan p) { return p; });
  return fits(double(tiles_of<Fwd>(a)) * f.units + 4096, threads_of(f)) &&
         fits(double(tiles_of<Bwd>(a)) * b.units + 4096, threads_of(b)) &&
         (b.chunks == 1 || fits(double(a.rows.starts ? 1 : a.rows.S) * a.C / 64 + 1, 2 * 64 * kParts));
}

// Chained: the tickets, then the slots.
int64_t recurrence_bytes(const RecArgs& a) {
  const Plan p = tall(a) ? plan<Tall>(a.rows) : plan<Fwd>(a.rows);
  return p.chunks > 1 ? 4 * kApart * counters_of(a) + 8 * (int64_t)p.units * a.C : 0;
}

hipError_t launch_recurrence(const RecArgs& given, void* y, float* fin, float* ws, hipStream_t s) {
  RecArgs a = given;
  a.stream = stream_of(a);
  const bool high = tall(a);
  const Plan p = high ? plan<Tall>(a.rows) : plan<Fwd>(a.rows);
  const int tiles = tiles_of<Fwd>(a);
  const unsigned blocks = (unsigned)((int64_t)tiles * p.units), more = empty_blocks(a, p, fin);
  const int64_t counters = counters_of(a);
  const Chain chain{ws ? (uint64_t*)(ws + kApart * counters) : nullptr, (uint32_t*)ws, (int)counters};
  if (p.chunks > 1) {
    const int64_t n = (int64_t)p.units * a.C;  // more than counters
    hipLaunchKernelGGL(k_rec_clear, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, chain, n);
  }
  return by_kind(a, [&](auto io, auto decay, auto gated, auto packed) {
    using IO = decltype(io);
    auto run = [&](auto shape, auto chained) {
      hipLaunchKernelGGL((k_rec<decltype(shape), IO, decltype(decay)::value, decltype(gated)::value,
                                decltype(packed)::value, decltype(chained)::value>),
                         dim3(blocks + more), dim3(threads_of(p)), 0, s, a, p, tiles, chain, (IO*)y,
                         fin);
      return hipGetLastError();
    };
    if (p.chunks > 1) return high ? run(Tall{}, std::true_type{}) : run(Fwd{}, std::true_type{});
    return high ? run(Tall{}, std::false_type{}) : run(Fwd{}, std::false_type{});
  });
}

hipError_t launch_recurrence_step(const RecArgs& a, float* state_out, void* y, hipStream_t s) {
  const unsigned blocks = (unsigned)(((int64_t)a.rows.R * (a.C / 4) + 255) / 256);
  return by_kind(a, [&](auto io, auto decay, auto gated, auto) {
    using IO = decltype(io);
    hipLaunchKernelGGL((k_rec_step<IO, decltype(decay)::value, decltype(gated)::value>),
                       dim3(blocks), dim3(256), 0, s, a, state_out, (IO*)y);
    return hipGetLastError();
  });
}

int64_t recurrence_backward_bytes(const RecArgs& a) {
  const Plan p = by_shape(a, [](auto, Plan b) { return b; });
  return 4 * sum_floats(a, p) * ((p.chunks > 1 ? 3 : 0) + (a.decay && p.units > 1 ? 1 : 0));
}

hipError_t launch_recurrence_backward(const RecArgs& given, const void* dy, const float* dfinal,
                                      const RecGrads& g, float* ws, hipStream_t s) {
  RecArgs a = given;
  a.stream = stream_of(a);
  const Plan p = by_shape(a, [](auto, Plan b) { return b; });
  const int tiles = tiles_of<Bwd>(a);
  // Chunks that look up the others' sums by themselves: few of them (32 x 128 x 5120 bf16 138 -> 119 us), or
  // some more where all run at once and a launch counts (400 x 1536 28 -> 24; with 24 chunks and more
  // blocks, 8 x 670 x 5120, 147 -> 191). The borders lie between these sizes, no nearer to either.
  const bool few = p.chunks <= 8 || (p.chunks <= 24 && (int64_t)tiles * p.units <= 1024);
  const int chained = p.chunks == 1 ? kAlone : few ? kSingly : kJoined;
  const int64_t n = sum_floats(a, p);
  Sums sums{nullptr, nullptr, nullptr};
  float* part = p.units > 1 ? ws : g.ddecay;  // of a single unit its sums are all
  if (chained) {
    sums = Sums{ws, ws + n, ws + 2 * n};
    part = ws + 3 * n;
  }
  const unsigned blocks = (unsigned)((int64_t)tiles * p.units), more = empty_blocks(a, p, g.dh0);
  const hipError_t e = by_kind(a, [&](auto io, auto decay, auto gated, auto packed) {
    using IO = decltype(io);
    constexpr bool D = decltype(decay)::value, G = decltype(gated)::value, K = decltype(packed)::value;
    constexpr bool half = sizeof(IO) == 2;
    using Low = std::conditional_t<half, Bwd, Bwd32>;
    using High = std::conditional_t<half, BwdTall, BwdTall32>;
    return by_height<Low, High>(a, [&](auto shape, Plan) {
      using X = decltype(shape);
      if constexpr (std::is_same_v<X, Low>) {
        if (chained) {
          hipLaunchKernelGGL((k_rec_sums<X, IO, D, G, K>), dim3(blocks), dim3(threads_of(p)), 0, s, a, p,
                             tiles, sums, (const IO*)dy, dfinal);
          if (chained == kJoined)
            hipLaunchKernelGGL(k_rec_chain, chain_grid(a), dim3(64 * kParts), 0, s, a, p, sums, dfinal);
        }
      }
      hipLaunchKernelGGL((k_rec_bwd<X, IO, D, G, K>), dim3(blocks + more), dim3(threads_of(p)), 0, s, a,
                         p, tiles, sums, chained, (const IO*)dy, dfinal, (IO*)g.dx, (IO*)g.dg,
                         (IO*)g.dgi, g.dh0, part);
      return hipGetLastError();
    });
  });
  if (e != hipSuccess || !a.decay || p.units == 1) return e;
  return launch_column_sums(part, p.units, a.C, g.ddecay, a.C, 0, 1, 0, nullptr, 0, nullptr, s);
}

}  // namespace ssd
