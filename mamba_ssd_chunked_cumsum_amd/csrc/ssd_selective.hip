// Selective scan with a decay of its own for every channel d and state entry n: forward and single
// token.
//
//   delta = softplus(dt + bias);  h <- exp(delta A[d,n]) h + delta x B[n];  y = sum_n h C[n] + D x
//
// For each (token, channel, state entry) one exponential, two products and two fused
// multiply-adds. With a different decay for every state entry no matrix product covers several
// tokens, so the vector units bound it: 8 cycles of a SIMD for the exponential and 4 for each of the
// others (from counters), 24 for 64 entries of a token, 214 us at 2 x 8192 tokens x 5120 channels x
// 16 entries if nothing else were done.
//
// A lane holds one channel with all its states in registers and a wave 64 neighbouring channels, so
// the sum over n needs no exchange between lanes, and B and C of a token are the same for the whole
// wave: they come through scalar loads and are unpacked by the scalar unit, beside the vector
// work. There is no LDS and no barrier. The tokens of a sequence are sequential; parallel are only
// channels and sequences, and where those do not fill the card the rows are cut into chunks (split
// variant): one kernel computes each chunk's end state from a zero state and the sum of its delta,
// one chains the chunks (the decay of a whole chunk is exp(A sum delta)), and the scan starts every
// chunk from the state entering it. That evaluates the exponentials twice. At the size above (bf16,
// gated): 250 us the end states, 10 the chain, 330 the scan, with the vector units busy 90 to 95% of
// the time; 565 us a call. 64 x 5120 x 16 single tokens: 11 us, 4.1 TB/s. (Four lanes a channel with
// tiles in LDS and one wave on most SIMDs, the first version, took 2031 us.)
#include <cmath>

#include "ssd_selective.h"

namespace ssd {

namespace {

constexpr int kWaves = 4;  // of a block, on neighbouring channel tiles: they share B and C

// How the rows are divided: a wave takes sequence u (len 0), or chunk u of `len` rows.
struct Plan {
  int len, chunks;
  float* state;  // [chunks, C, N]: end states, then the states entering the chunks
  float* sums;   // [chunks, C]: sums of delta; NaN where a sequence begins in the chunk
};

// STATES: only the end state and sum of delta of each chunk.
template <typename IO, int NT, bool EXACT, bool STATES>
__global__ __launch_bounds__(64 * kWaves) void k_scan(SelArgs q, Plan pl, int units,
                                                      IO* __restrict__ y, float* __restrict__ fin) {
  constexpr int GR = 8, U = 4;  // tokens whose loads are in flight while the U before them are computed
  const int cg = q.C / q.G, tiles = (cg + 63) / 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t id = (int64_t)blockIdx.x * kWaves + wave;
  const int ct = (int)(id % (tiles * q.G)), u = (int)(id / (tiles * q.G));
  if (u >= units) return;
  const int g = ct / tiles, c0 = g * cg + ct % tiles * 64, c1 = (g + 1) * cg;
  const bool live = c0 + (threadIdx.x & 63) < c1;
  const int c = live ? c0 + (threadIdx.x & 63) : c1 - 1;  // idle lanes compute the last one again
  int r0, r1;
  if (pl.len && u < pl.chunks) {
    r0 = u * pl.len;
    r1 = q.rows.R - r0 > pl.len ? r0 + pl.len : q.rows.R;  // (r0 + len may pass 31 bits)
  } else {
    const int s = pl.len ? u - pl.chunks : u;
    r0 = seq_begin(q.rows, s);
    r1 = seq_end(q.rows, s);
    if (r1 <= r0) {  // an empty sequence: its state passes through
      if (!STATES && fin && live) {
        const int64_t at = ((int64_t)s * q.C + c) * q.N;
        for (int n = 0; n < q.N; ++n) fin[at + n] = q.h0 ? q.h0[at + n] : 0.f;
      }
      return;
    }
    if (pl.len) return;
  }
  if (STATES) {  // only what follows the last sequence start in the chunk reaches its end, and only
                 // a sequence that goes on behind the chunk needs it
    const int s = seq_of(q.rows, r1 - 1);
    if (s < 0 || seq_end(q.rows, s) <= r1) {
      if (live) {
        for (int n = 0; n < q.N; ++n) pl.state[((int64_t)u * q.C + c) * q.N + n] = 0.f;
        pl.sums[(int64_t)u * q.C + c] = __builtin_nanf("");
      }
      return;
    }
    r0 = max(r0, seq_begin(q.rows, s));
  }
  float A[NT], h[NT], sum = 0.f;
  load_all<NT>(q.A + (int64_t)c * q.N, q.N, A);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    A[n] *= kLog2e;
    h[n] = 0.f;
  }
  if (!STATES && pl.len) load_all<NT>(pl.state + ((int64_t)u * q.C + c) * q.N, q.N, h);
  const float bias = q.dt_bias ? q.dt_bias[c] : 0.f, D = q.D ? q.D[c] : 0.f;
  const unsigned off = (unsigned)c * sizeof(IO);
  const IO *B = (const IO*)q.B + g * q.N, *C = (const IO*)q.Cm + g * q.N;
  bool began = false;
  const void* zp = q.z ? q.z : q.x;  // (without a gate the values read are not used)
  const int64_t zs = q.z ? q.zs : q.xs;
  for (int r = r0; r < r1;) {  // sequence by sequence
    const int s = seq_of(q.rows, r);
    if (s < 0) {
      r = after_gap(q.rows, r);
      continue;
    }
    const int end = seq_end(q.rows, s), b = min(end, r1);
    if (r == seq_begin(q.rows, s)) {
      began = true;
#pragma unroll
      for (int n = 0; n < NT; ++n) h[n] = 0.f;
      if (q.h0) load_all<NT>(q.h0 + ((int64_t)s * q.C + c) * q.N, q.N, h);
    }
    // rows that are read next: a row's address is scalar, the channel the lane's offset
    const char *px = row_at((const IO*)q.x, r * q.xs), *pt = row_at((const IO*)q.dt, r * q.dts),
               *pz = row_at((const IO*)zp, r * zs), *pb = row_at(B, r * q.bs),
               *pc = row_at(C, r * q.cs);
    int ahead = r, ahead_bc = r;  // their indices, held at the last row of the run
    struct Rows2 {
      Row<IO, NT, EXACT> B, C;
    };
    auto rows = [&] {
      Rows2 w;
      w.B.load((const IO*)pb, q.N);
      if (!STATES) w.C.load((const IO*)pc, q.N);
      if (++ahead_bc < b) {
        pb += q.bs * sizeof(IO);
        if (!STATES) pc += q.cs * sizeof(IO);
      }
      return w;
    };
    uint32_t rx[U], rt[U], rz[U];
    auto fetch = [&] {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        rx[i] = load_raw<IO>(px, off);
        rt[i] = load_raw<IO>(pt, off);
        if (!STATES) rz[i] = load_raw<IO>(pz, off);
        if (++ahead < b) {
          px += q.xs * sizeof(IO);
          pt += q.dts * sizeof(IO);
          if (!STATES) pz += zs * sizeof(IO);
        }
      }
    };
    fetch();
    Rows2 w = rows();
#pragma unroll 1
    for (; r < b; r += U) {
      float x[U], dl[U], gate[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        x[i] = raw_value<IO>(rx[i]);
        dl[i] = raw_value<IO>(rt[i]) + bias;
        if (!STATES) gate[i] = raw_value<IO>(rz[i]);
      }
      fetch();
      if (q.softplus) {
#pragma unroll
        for (int i = 0; i < U; ++i) dl[i] = softplus(dl[i]);
      }
      if (!STATES) {
        if (q.z) {
#pragma unroll
          for (int i = 0; i < U; ++i) gate[i] *= sigmoid(gate[i]);
        } else {
#pragma unroll
          for (int i = 0; i < U; ++i) gate[i] = 1.f;
        }
      }
      auto token = [&](int i) {
        const Rows2 wn = rows();  // a token ahead
        const float du = dl[i] * x[i];
        float acc[2] = {0.f, 0.f};
        if (STATES) sum += dl[i];
        // in groups of GR state entries, so that no instruction waits for the one before it
#pragma unroll
        for (int n = 0; n < NT; n += GR) {
          float a[GR], v[GR];
#pragma unroll
          for (int j = 0; j < GR; ++j) a[j] = dl[i] * A[n + j];
#pragma unroll
          for (int j = 0; j < GR; ++j) a[j] = exp2_fast(a[j]);
#pragma unroll
          for (int j = 0; j < GR; ++j) v[j] = du * w.B.get(n + j);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int j = 0; j < GR; ++j) h[n + j] = fmaf(a[j], h[n + j], v[j]);
          if (!STATES) {
#pragma unroll
            for (int j = 0; j < GR; ++j) acc[j & 1] = fmaf(h[n + j], w.C.get(n + j), acc[j & 1]);
          }
        }
        w = wn;
        // (idle lanes write the last channel's value once more)
        if (!STATES)
          store_io((IO*)((char*)(y + (int64_t)(r + i) * q.C) + off), 0,
                   fmaf(D, x[i], acc[0] + acc[1]) * gate[i]);
      };
      if (r + U <= b) {
#pragma unroll
        for (int i = 0; i < U; ++i) token(i);
      } else {
#pragma unroll
        for (int i = 0; i < U - 1; ++i)
          if (r + i < b) token(i);
      }
    }
    r = b;
    if (!STATES && fin && b == end && live)
      store_all<NT>(fin + ((int64_t)s * q.C + c) * q.N, q.N, h);
  }
  if (STATES && live) {
    store_all<NT>(pl.state + ((int64_t)u * q.C + c) * q.N, q.N, h);
    pl.sums[(int64_t)u * q.C + c] = began ? __builtin_nanf("") : sum;
  }
}

// Chain over the chunks, in place: state[u] from chunk u's end state to the state entering it. Where
// a sequence begins in a chunk (its sum is NaN, as is the end state where delta was NaN) nothing
// passes through it. The loads of kAhead chunks are issued together.
__global__ __launch_bounds__(256) void k_scan_chain(SelArgs q, Plan pl) {
  constexpr int kAhead = 32;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, CN = (int64_t)q.C * q.N;
  if (id >= CN) return;
  const int c = (int)(id / q.N);
  const float A = q.A[id] * kLog2e;
  float h = 0.f;
  for (int u = 0; u < pl.chunks; u += kAhead) {
    float e[kAhead], d[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int v = min(u + i, pl.chunks - 1);
      e[i] = pl.state[v * CN + id];
      d[i] = pl.sums[(int64_t)v * q.C + c];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (u + i < pl.chunks) pl.state[(u + i) * CN + id] = h;
      h = d[i] == d[i] ? fmaf(exp2_fast(A * d[i]), h, e[i]) : e[i];
    }
  }
}

// ---- single token ----------------------------------------------------------------------------------
// L lanes a channel with four states each, as the SSD step: bound by the state, read and written
// once past the caches. A thread takes NB sequences of its channel, whose states it loads together
// and which share A, D and the bias.
template <typename IO, int L, int NB>
__global__ __launch_bounds__(256) void k_sel_step(SelArgs q, float* state_out, IO* y) {
  const int64_t id = ((int64_t)blockIdx.x * 256 + threadIdx.x) / L;
  const int n = (threadIdx.x % L) * 4, groups = (q.rows.R + NB - 1) / NB;
  if (id >= (int64_t)groups * q.C) return;
  const int b0 = (int)(id / q.C) * NB, c = (int)(id % q.C), g = c / (q.C / q.G);
  const bool on = n < q.N;
  const int nc = on ? n : 0;
  f32x4 h[NB];
  Vec<IO, 4> B[NB], Cv[NB];
  float x[NB], dl[NB], z[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int64_t b = min(b0 + i, q.rows.R - 1);
    h[i] = __builtin_nontemporal_load(
        reinterpret_cast<const f32x4*>(q.h0 + (b * q.C + c) * q.N + nc));
    B[i].load((const IO*)q.B + b * q.bs + g * q.N + nc);
    Cv[i].load((const IO*)q.Cm + b * q.cs + g * q.N + nc);
    x[i] = Io<IO>::load((const IO*)q.x, b * q.xs + c);
    dl[i] = Io<IO>::load((const IO*)q.dt, b * q.dts + c);
    if (q.z) z[i] = Io<IO>::load((const IO*)q.z, b * q.zs + c);
  }
  const float4 Av = *reinterpret_cast<const float4*>(q.A + (int64_t)c * q.N + nc);
  const float a[4] = {Av.x, Av.y, Av.z, Av.w};
  const float bias = q.dt_bias ? q.dt_bias[c] : 0.f, D = q.D ? q.D[c] : 0.f;
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    if (b0 + i >= q.rows.R) break;
    const int64_t at = (int64_t)(b0 + i) * q.C + c;
    float d = dl[i] + bias;
    if (q.softplus) d = softplus(d);
    const float du = d * x[i], d2 = d * kLog2e;
    f32x4 o;
    float acc = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[j] = fmaf(exp2_fast(d2 * a[j]), h[i][j], du * B[i].get(j));
      acc = fmaf(o[j], Cv[i].get(j), acc);
    }
    if (on)
      __builtin_nontemporal_store(o, reinterpret_cast<f32x4*>(state_out + at * q.N + n));
    else
      acc = 0.f;
#pragma unroll
    for (int m = L / 2; m >= 1; m >>= 1) acc += __shfl_xor(acc, m, kWave);
    if (n == 0) {
      acc = fmaf(D, x[i], acc);
      if (q.z) acc *= z[i] * sigmoid(z[i]);
      Io<IO>::store(y, at, acc);
    }
  }
}

constexpr int kMinLen = 32;  // rows of a chunk with several waves a SIMD

int64_t tiles_of(const SelArgs& a) { return (int64_t)((a.C / a.G + 63) / 64) * a.G; }

// Direct or split, in cycles of a SIMD. A wave alone on its SIMD issues about half of what several
// together do; a row costs about 28 cycles a state entry with the SIMD full, as much again for the
// split's first pass, whose chain and extra launches cost about 15 us more. The chunks make the
// largest number of waves up to four a SIMD that leaves them 32 rows or more: just over a whole
// number of waves a SIMD would leave most of the card idle for the last of them. Where even one wave a
// SIMD leaves fewer, time goes by the rows of a wave, and chunks go down to 8. (Four waves fit up to 16
// states; registers leave two above that and one above 32, which this does not count: 2 x 4096 x 2048
// bf16 takes 133 us with 16 states, 416 with 32, 1513 with 64.)
Plan plan(const SelArgs& a, int n_cu) {
  Plan pl{0, 0, nullptr, nullptr};
  const double simds = 4.0 * n_cu, row = 28.0 * (a.N < 8 ? 8 : a.N);
  const int64_t tiles = tiles_of(a);
  const double longest = a.rows.starts ? a.rows.R : a.rows.L;
  const double waves = std::ceil(double(tiles) * a.rows.S / simds);
  const double direct = longest * row * (waves < 2 ? 2 : waves);
  const double split = double(a.rows.R) * tiles * row * 2 / simds + 36000;
  if (direct <= split) return pl;
  for (int w = 4; w >= 1; --w) {
    const int64_t chunks = (int64_t)(w * simds) / tiles;
    if (chunks < 2) break;
    const int64_t len = ((a.rows.R + chunks - 1) / chunks + 3) / 4 * 4;
    if (len < kMinLen && w > 1) continue;
    pl.len = (int)(len < 8 ? 8 : len);
    pl.chunks = (int)(((int64_t)a.rows.R + pl.len - 1) / pl.len);
    break;
  }
  if (pl.chunks < 2) pl.len = pl.chunks = 0;
  return pl;
}

int64_t state_floats(const SelArgs& a, const Plan& pl) {
  return ((int64_t)pl.chunks * a.C * a.N + 63) / 64 * 64;
}

}  // namespace

int64_t selective_bytes(const SelArgs& a, int n_cu) {
  const Plan pl = plan(a, n_cu);
  return pl.len ? 4 * (state_floats(a, pl) + (int64_t)pl.chunks * a.C) : 0;
}

hipError_t launch_selective(const SelArgs& a, void* y, float* fin, float* ws, int n_cu,
                            hipStream_t s) {
  Plan pl = plan(a, n_cu);
  pl.state = ws;
  pl.sums = ws ? ws + state_floats(a, pl) : nullptr;
  auto blocks = [&](int64_t units) { return dim3((unsigned)((tiles_of(a) * units + kWaves - 1) / kWaves)); };
  auto run = [&](auto io, auto size, auto exact) {
    using IO = decltype(io);
    constexpr int NT = decltype(size)::value;
    constexpr bool EX = decltype(exact)::value;
    if (pl.len) {
      hipLaunchKernelGGL((k_scan<IO, NT, EX, true>), blocks(pl.chunks), dim3(64 * kWaves), 0, s, a,
                         pl, pl.chunks, (IO*)nullptr, (float*)nullptr);
      hipLaunchKernelGGL(k_scan_chain, dim3((unsigned)(((int64_t)a.C * a.N + 255) / 256)),
                         dim3(256), 0, s, a, pl);
    }
    // the units behind the chunks pass on the states of empty sequences
    const int64_t units = pl.len ? pl.chunks + (fin && a.rows.starts ? a.rows.S : 0) : a.rows.S;
    hipLaunchKernelGGL((k_scan<IO, NT, EX, false>), blocks(units), dim3(64 * kWaves), 0, s, a, pl,
                       (int)units, (IO*)y, fin);
    return hipGetLastError();
  };
  auto sizes = [&](auto io) {
    return by_size(a.N, [&](auto size, auto exact) { return run(io, size, exact); });
  };
  return a.io == kIoBf16 ? sizes(u16{}) : sizes(float{});
}

hipError_t launch_selective_step(const SelArgs& a, float* state_out, void* y, hipStream_t s) {
  auto run = [&](auto io, auto lanes, auto seqs) {
    using IO = decltype(io);
    constexpr int L = decltype(lanes)::value, NB = decltype(seqs)::value;
    const int64_t threads = (int64_t)((a.rows.R + NB - 1) / NB) * a.C * L;
    hipLaunchKernelGGL((k_sel_step<IO, L, NB>), dim3((unsigned)((threads + 255) / 256)), dim3(256),
                       0, s, a, state_out, (IO*)y);
    return hipGetLastError();
  };
  auto seqs = [&](auto io, auto lanes) {
    // four sequences a thread once that leaves four waves a SIMD
    using std::integral_constant;
    if ((int64_t)a.rows.R * a.C * decltype(lanes)::value >= 4 * 262144)
      return run(io, lanes, integral_constant<int, 4>{});
    return run(io, lanes, integral_constant<int, 1>{});
  };
  auto lanes = [&](auto io) {
    using std::integral_constant;
    if (a.N <= 4) return seqs(io, integral_constant<int, 1>{});
    if (a.N <= 8) return seqs(io, integral_constant<int, 2>{});
    if (a.N <= 16) return seqs(io, integral_constant<int, 4>{});
    if (a.N <= 32) return seqs(io, integral_constant<int, 8>{});
    return seqs(io, integral_constant<int, 16>{});
  };
  return a.io == kIoBf16 ? lanes(u16{}) : lanes(float{});
}

}  // namespace ssd
