// Backward of the selective scan.
//
// With e = dy silu(z), a_t = exp(delta_t A) and G_t = e_t C_t + a_{t+1} G_{t+1} (plus the final
// state's gradient at a sequence's last token), for every (token, channel, state entry):
//   dC_t[n] = sum_d e h_t      dB_t[n] = sum_d G delta x      q = sum_n G B
//   w = G a h_{t-1}            dx = D e + delta q             ddelta = x q + sum_n w A
//   dA = sum_t w delta         dz = dy (sum_n h C + D x) silu'(z)
//   dD = sum_t e x             ddt = ddelta softplus'         dh0 = a_0 G_0
// h runs forward and G backward. Rows are cut into chunks of 64. A first kernel (a channel a lane)
// computes for every chunk both its end state from a zero state, with the states after each quarter
// of it, and the gradient of its entering state from a zero gradient at its end, in one pass forward
// (the second as sum_t (a_0 .. a_t) C_t e_t: the exponentials are shared); a second kernel chains both
// over the chunks. Then every chunk is independent: the main kernel (four lanes a channel) takes its
// quarters from the last to the first, forward from the quarter's entering state, keeping h and a
// of its 16 tokens in registers, and back. So each exponential is evaluated twice and nothing of size
// tokens x channels x dstate goes to memory; the vector units bound it. At 2 x 4096 tokens x 5120
// channels x 16 entries (bf16, gated): 190 us the first kernel, 38 the chain, 635 the main kernel
// (vector units busy 76%: two waves a SIMD, by the registers that h and a take and by the LDS of the
// staged chunk, 80 KiB a block), 18 + 11 the sums; 850 us a call.
//
// dB and dC sum over channels, i.e. over lanes: sums over the 16 channels of a wave are formed 16
// values at a time, each step adding two lanes' values and merging two registers into one, so
// that they cost under two instructions a value; the four waves' sums meet in LDS and the blocks'
// in memory, added by another kernel in a fixed order.
#include "ssd_selective.h"

namespace ssd {

namespace {

// States a lane; rows a chunk and a quarter of it, so that a quarter's h and a take 128 registers.
constexpr int NPL = 4, kQuarter = 16, kChunk = 4 * kQuarter;
constexpr int kOneLaunch = 12;  // waves of k_bwd_ends a SIMD, up to which it is launched once
constexpr int kFours = 2;       // the same, up to which its lanes hold four state entries

struct Work {
  int chunks;
  float* state;  // [chunks, 4, C, N]: states after each quarter from a zero state at the chunk's
                 // start; the last, chained, becomes the state entering the chunk
  float* adj;    // [chunks, C, N]: gradients of the entering states; then those from later chunks
  float* sums;   // [chunks, 4, C]: sums of delta up to there, NaN where the entering state has no part
  float* back;   // [chunks, C]: the whole chunk's, NaN where no gradient passes
  float* bc;     // [tiles, R, 2, N]: dB and dC over a block's channels
  float* part;   // [chunks, C N + 2 C]: dA, dD, ddt_bias of a chunk
};

struct Tile {  // the channels of a block
  int ct, g, base, stop;
  __device__ __forceinline__ Tile(const SelArgs& q, int ch, int id) {
    const int cg = q.C / q.G, tiles = (cg + ch - 1) / ch;
    ct = id;
    g = id / tiles;
    base = g * cg + id % tiles * ch;
    stop = (g + 1) * cg;
  }
};

// T rows from r on in LDS: delta, delta x and e (zero outside every sequence), B and C.
template <typename IO, int T, int CH, int NP>
__device__ __forceinline__ void stage(const SelArgs& q, const IO* dy, const Tile& b, int r, int r1,
                                      uint64_t inside, float (&s_dl)[T][CH], float (&s_du)[T][CH],
                                      float (&s_e)[T][CH], float (&s_b)[T][NP],
                                      float (&s_c)[T][NP]) {
  constexpr int V = 8, NV = T * CH / V;
#pragma unroll
  for (int i = 0; i < (NV + kSelThreads - 1) / kSelThreads; ++i) {
    const int v = threadIdx.x + i * kSelThreads, t = v / (CH / V), cl = v % (CH / V) * V;
    if (v < NV) {
      const int64_t row = r + t;
      const int c = b.base + cl;
      float dl[V], du[V], e[V];
#pragma unroll
      for (int j = 0; j < V; ++j) dl[j] = du[j] = e[j] = 0.f;
      if (((inside >> t) & 1) && c < b.stop) {
        Vec<IO, V> xr, tr, dr, zr;
        xr.load((const IO*)q.x + row * q.xs + c);
        tr.load((const IO*)q.dt + row * q.dts + c);
        dr.load(dy + row * q.C + c);
        if (q.z) zr.load((const IO*)q.z + row * q.zs + c);
        if (q.dt_bias) load_f32<V>(q.dt_bias + c, dl);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          dl[j] += tr.get(j);
          if (q.softplus) dl[j] = softplus(dl[j]);
          du[j] = dl[j] * xr.get(j);
          e[j] = dr.get(j);
          if (q.z) e[j] *= zr.get(j) * sigmoid(zr.get(j));
        }
      }
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        *reinterpret_cast<float4*>(&s_dl[t][cl + j]) = make_float4(dl[j], dl[j + 1], dl[j + 2], dl[j + 3]);
        *reinterpret_cast<float4*>(&s_du[t][cl + j]) = make_float4(du[j], du[j + 1], du[j + 2], du[j + 3]);
        *reinterpret_cast<float4*>(&s_e[t][cl + j]) = make_float4(e[j], e[j + 1], e[j + 2], e[j + 3]);
      }
    }
  }
  constexpr int BV = T * NP / 4;
#pragma unroll
  for (int i = 0; i < (BV + kSelThreads - 1) / kSelThreads; ++i) {
    const int v = threadIdx.x + i * kSelThreads, t = v / (NP / 4), n = v % (NP / 4) * 4;
    if (v < BV) {
      Vec<IO, 4> br, cr;
      br.zero();
      cr.zero();
      if (((inside >> t) & 1) && n < q.N) {
        br.load((const IO*)q.B + (r + t) * q.bs + b.g * q.N + n);
        cr.load((const IO*)q.Cm + (r + t) * q.cs + b.g * q.N + n);
      }
      *reinterpret_cast<float4*>(&s_b[t][n]) = make_float4(br.get(0), br.get(1), br.get(2), br.get(3));
      *reinterpret_cast<float4*>(&s_c[t][n]) = make_float4(cr.get(0), cr.get(1), cr.get(2), cr.get(3));
    }
  }
}

__device__ __forceinline__ void seq_states(const SelArgs& q, const float* p, int s, int c, int k,
                                           bool live, float (&h)[NPL]) {
#pragma unroll
  for (int j = 0; j < NPL; ++j) h[j] = 0.f;
  if (p && live) {
    load_states<NPL>(p + ((int64_t)s * q.C + c) * q.N, k, q.N, h);
  }
}

// ---- chunk ends ----------------------------------------------------------------------------------
// As the forward's chunk states: a lane holds a channel, B and C come through scalar loads. NT: up to
// 16 states; of more (4 where the launch is small) other waves take the others.
// EVENTS: the chunks in which a sequence begins after the first row or ends before the last; the
// others take a launch of their own, whose waves need fewer registers (122 against 145: four of them
// on a SIMD against three). `all`: every chunk in the one launch. Two follow one another, and the
// second is a chunk's latency however few chunks it has; the fewer registers pay only over many
// rounds of waves (the whole backward, two launches and one: 1536 channels x 2041 tokens 161 and 130
// us, x 5497 255 and 225, x 24569, 9200 waves, 830 and 822; 5120 x 16377, 20500 waves, 1695 and 1724;
// the limit of kOneLaunch waves a SIMD, 12288 on 256 compute units, lies between the last two, where
// the two ways are level).
template <typename IO, int NT, bool EXACT, bool EVENTS>
__global__ __launch_bounds__(256) void k_bwd_ends(SelArgs q, Work w, const IO* dy,
                                                  const float* dfinal, int all) {
  constexpr int U = 4;  // tokens whose loads are in flight
  const int cg = q.C / q.G, tiles = (cg + 63) / 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t id = (int64_t)blockIdx.x * 4 + wave;
  const int parts = (q.N + NT - 1) / NT, n0 = (int)(id % parts) * NT, N = min(NT, q.N - n0);
  const int ct = (int)(id / parts % (tiles * q.G)), u = (int)(id / parts / (tiles * q.G));
  if (u >= w.chunks) return;
  const int g = ct / tiles, c0 = g * cg + ct % tiles * 64, c1 = (g + 1) * cg;
  const bool live = c0 + (threadIdx.x & 63) < c1;
  const int c = live ? c0 + (threadIdx.x & 63) : c1 - 1;  // idle lanes compute the last one again
  const unsigned off = (unsigned)c * sizeof(IO);
  const int r0 = u * kChunk, r1 = min(r0 + kChunk, q.rows.R);
  const int s0 = seq_of(q.rows, r0);
  const bool quiet = r1 - r0 == kChunk && s0 >= 0 && seq_end(q.rows, s0) >= r1;
  if (quiet == EVENTS && !(EVENTS && all)) return;
  const int64_t CN = (int64_t)q.C * q.N, at = (int64_t)c * q.N + n0;
  float A[NT], h[NT], p[NT], gl[NT], sum = 0.f;
  load_all<NT>(q.A + at, N, A);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    A[n] *= kLog2e;
    h[n] = gl[n] = 0.f;
    p[n] = 1.f;
  }
  const float bias = q.dt_bias ? q.dt_bias[c] : 0.f, none = __builtin_nanf("");
  const IO *B = (const IO*)q.B + g * q.N + n0, *C = (const IO*)q.Cm + g * q.N + n0;
  const void* zp = q.z ? q.z : q.x;  // (without a gate the values read are not used)
  const int64_t zs = q.z ? q.zs : q.xs;
  // rows that are read next: a row's address is scalar, the channel the lane's offset
  const char *px = row_at((const IO*)q.x, r0 * q.xs), *pt = row_at((const IO*)q.dt, r0 * q.dts),
             *py = row_at(dy, (int64_t)r0 * q.C), *pz = row_at((const IO*)zp, r0 * zs),
             *pb = row_at(B, r0 * q.bs), *pc = row_at(C, r0 * q.cs);
  int ahead = r0, ahead_bc = r0;  // their indices, held at the last row
  uint32_t rx[U], rt[U], ry[U], rz[U];
  auto fetch = [&] {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      rx[i] = load_raw<IO>(px, off);
      rt[i] = load_raw<IO>(pt, off);
      ry[i] = load_raw<IO>(py, off);
      rz[i] = load_raw<IO>(pz, off);
      if (++ahead < r1) {
        px += q.xs * sizeof(IO);
        pt += q.dts * sizeof(IO);
        py += (int64_t)q.C * sizeof(IO);
        pz += zs * sizeof(IO);
      }
    }
  };
  struct Rows2 {
    Row<IO, NT, EXACT> B, C;
  };
  auto rows = [&] {
    Rows2 m;
    m.B.load((const IO*)pb, N);
    m.C.load((const IO*)pc, N);
    if (++ahead_bc < r1) {
      pb += q.bs * sizeof(IO);
      pc += q.cs * sizeof(IO);
    }
    return m;
  };
  float x[U], dl[U], e[U];
  auto unpack = [&] {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      x[i] = raw_value<IO>(rx[i]);
      dl[i] = raw_value<IO>(rt[i]) + bias;
      e[i] = raw_value<IO>(ry[i]);
    }
    if (q.softplus) {
#pragma unroll
      for (int i = 0; i < U; ++i) dl[i] = softplus(dl[i]);
    }
    if (q.z) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const float zv = raw_value<IO>(rz[i]);
        e[i] *= zv * sigmoid(zv);
      }
    }
  };
  // open: no boundary so far, so the rows still reach the state that entered the chunk. (A flag, not
  // p = 0: a NaN of the next sequence would pass through that.)
  bool began = false, open = true;
  Rows2 bc = rows();
  auto token = [&](int i) {
    const Rows2 next = rows();  // a token ahead
    const float du = dl[i] * x[i];
    sum += dl[i];
    constexpr int GR = NT < 8 ? NT : 8;
#pragma unroll
    for (int n = 0; n < NT; n += GR) {
      float a[GR], v[GR];
#pragma unroll
      for (int j = 0; j < GR; ++j) a[j] = dl[i] * A[n + j];
#pragma unroll
      for (int j = 0; j < GR; ++j) a[j] = exp2_fast(a[j]);
#pragma unroll
      for (int j = 0; j < GR; ++j) v[j] = du * bc.B.get(n + j);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < GR; ++j) h[n + j] = fmaf(a[j], h[n + j], v[j]);
      if (!EVENTS || open) {
#pragma unroll
        for (int j = 0; j < GR; ++j) {
          p[n + j] *= a[j];
          gl[n + j] = fmaf(p[n + j], e[i] * bc.C.get(n + j), gl[n + j]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);  // (registers)
    }
    bc = next;
  };
  auto begin = [&](int s) {  // what came before belongs to another sequence
    began = true;
    open = false;
#pragma unroll
    for (int n = 0; n < NT; ++n) h[n] = 0.f;
    if (q.h0) load_all<NT>(q.h0 + (int64_t)s * CN + at, N, h);
  };
  auto finish = [&](int s) {
    if (open && dfinal) {
      float d[NT];
      load_all<NT>(dfinal + (int64_t)s * CN + at, N, d);
#pragma unroll
      for (int n = 0; n < NT; ++n) gl[n] = fmaf(p[n], d[n], gl[n]);
    }
    open = false;
  };
  auto write_quarter = [&](int i) {
    if (!live) return;
    const int64_t slot = (int64_t)u * 4 + i;
    store_all<NT>(w.state + slot * CN + at, N, h);
    if (n0 == 0) w.sums[slot * q.C + c] = began ? none : sum;
  };
  uint64_t starts = 0, ends = 0, inside = ~uint64_t(0);
  int seq = -1;
  if (EVENTS) mark_rows(q.rows, r0, r1, starts, ends, inside, seq);
  else if (seq_begin(q.rows, s0) == r0) begin(s0);
  fetch();
#pragma unroll 1
  for (int t = 0; t < (inside ? r1 - r0 : 0); t += U) {
    if (t && t % kQuarter == 0) write_quarter(t / kQuarter - 1);
    unpack();
    fetch();
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (EVENTS) {
        if (!((inside >> (t + i)) & 1)) {  // decays nothing, adds nothing, whatever lies there
          dl[i] = x[i] = e[i] = 0.f;
          bc.B.zero();
          bc.C.zero();
        }
        if ((starts >> (t + i)) & 1) begin(seq_at(seq, t + i));
      }
      token(i);
      if (EVENTS && ((ends >> (t + i)) & 1)) finish(seq_at(seq, t + i));
    }
  }
  if (!EVENTS && seq_end(q.rows, s0) == r1) finish(s0);
  if (!EVENTS && began) {  // nothing entered
#pragma unroll
    for (int n = 0; n < NT; ++n) gl[n] = 0.f;
  }
  if (live) {
    store_all<NT>(w.state + ((int64_t)u * 4 + 3) * CN + at, N, h);
    store_all<NT>(w.adj + (int64_t)u * CN + at, N, gl);
    // what passes: the state through rows of one sequence that began before the chunk, its gradient
    // if that sequence also goes on behind it
    const int s = seq_of(q.rows, r1 - 1);
    const bool fwd = s >= 0 && seq_begin(q.rows, s) < r0;
    const bool bwd = fwd && seq_end(q.rows, s) > r1;
    if (n0 == 0) {
      w.sums[((int64_t)u * 4 + 3) * q.C + c] = fwd ? sum : none;
      w.back[(int64_t)u * q.C + c] = bwd ? sum : none;
    }
  }
}

// Chains both ways, in place: state[u] becomes the state entering chunk u, adj[u] the gradient of
// the state after its last row that comes from later rows of the same sequence. blockIdx.y 0:
// states, 1: gradients. Where the chunk's rows are not all of one sequence that goes on across it
// (sums: NaN), nothing passes through. The loads of kAhead chunks are issued together.
__global__ __launch_bounds__(256) void k_bwd_chain(SelArgs q, Work w) {
  constexpr int kAhead = 16;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, CN = (int64_t)q.C * q.N;
  if (id >= CN) return;
  const int c = (int)(id / q.N), back = blockIdx.y;
  const float A = q.A[id] * kLog2e;
  // (states and sums of a chunk's last quarter)
  const int64_t step = back ? 1 : 4;
  const float* sums = back ? w.back : w.sums + 3 * q.C;
  float* state = back ? w.adj : w.state + 3 * CN;
  float h = 0.f;
  for (int i0 = 0; i0 < w.chunks; i0 += kAhead) {
    float e[kAhead], d[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int v = min(i0 + i, w.chunks - 1), u = back ? w.chunks - 1 - v : v;
      e[i] = state[u * step * CN + id];
      d[i] = sums[u * step * q.C + c];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int v = i0 + i, u = back ? w.chunks - 1 - v : v;
      if (v < w.chunks) state[u * step * CN + id] = h;
      h = d[i] == d[i] ? fmaf(exp2_fast(A * d[i]), h, e[i]) : e[i];
    }
  }
}

// ---- sums over the channels of a wave --------------------------------------------------------------
// Four registers to one: sums over the four channels of each row of 16 lanes; quads 1, 3, 0, 2 of
// the row hold those of v0, v1, v2, v3. Each instruction adds a lane's value and a rotated one, the
// masked ones only in the quads that take the other register's sum. (The waits in front of a
// rotated read of a register just written are inside: the assembler does not add them.)
__device__ __forceinline__ float merge4(float v0, float v1, float v2, float v3) {
  float o, a, b;
  asm("s_nop 1\n\t"
      "v_add_f32_dpp %1, %3, %3 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
      "v_add_f32_dpp %2, %5, %5 row_ror:8 row_mask:0xf bank_mask:0xf\n\t"
      "v_add_f32_dpp %1, %4, %4 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %2, %6, %6 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "s_nop 1\n\t"
      "v_add_f32_dpp %0, %1, %1 row_ror:4 row_mask:0xf bank_mask:0xa\n\t"
      "v_add_f32_dpp %0, %2, %2 row_ror:12 row_mask:0xf bank_mask:0x5\n\t"
      "s_nop 1"
      : "=&v"(o), "=&v"(a), "=&v"(b)
      : "v"(v0), "v"(v1), "v"(v2), "v"(v3));
  return o;
}

// Two registers to one: sums over the two channels of each row; quads 0 and 1 hold v0's, 2 and 3
// v1's.
__device__ __forceinline__ float merge2(float v0, float v1) {
  float o;
  asm("s_nop 1\n\t"
      "v_add_f32_dpp %0, %1, %1 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %0, %2, %2 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "s_nop 1"
      : "=&v"(o)
      : "v"(v0), "v"(v1));
  return o;
}

// 64 / K registers to one: lane (row p of 16 lanes, K lanes of a channel b in the row, k) holds the
// sum over the wave's channels of the value with index merged_value().
template <int K>
__device__ __forceinline__ float merge(const float (&v)[64 / K]) {
  float r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (K == 4) r[i] = merge4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    else if constexpr (K == 8) r[i] = merge2(v[2 * i], v[2 * i + 1]);
    else r[i] = v[i];
  }
  auto add32 = [](float x, float y) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false,
                                                    false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
  };
  const float lo = add32(r[0], r[1]), hi = add32(r[2], r[3]);
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(lo), __float_as_uint(hi), false,
                                                  false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}
template <int K>
__device__ __forceinline__ int merged_value() {
  const int p = (threadIdx.x >> 4) & 3, r = p == 1 ? 2 : p == 2 ? 1 : p;  // r of merge()
  const int b = (threadIdx.x & 15) / K;
  if constexpr (K == 4) return 4 * r + (b == 0 ? 2 : b == 1 ? 0 : b == 2 ? 3 : 1);
  else if constexpr (K == 8) return 2 * r + b;
  else return r;
}

// Gradients of a row of no sequence, 8 channels.
template <typename IO>
__device__ __forceinline__ void zero_row(const SelArgs& q, const SelGrads& o, int64_t row, int c) {
  const float zero[8] = {};
  store_vec<IO, 8>((IO*)o.dx + row * q.C + c, zero);
  store_vec<IO, 8>((IO*)o.ddt + row * q.C + c, zero);
  if (q.z) store_vec<IO, 8>((IO*)o.dz + row * q.C + c, zero);
}

// A chunk that holds no row of a sequence: zero gradients, nothing to the sums.
template <typename IO, int K>
__device__ __forceinline__ void leave_empty(const SelArgs& q, const SelGrads& o, const Tile& b,
                                            int r0, int r1, float* part) {
  constexpr int CH = kSelThreads / K, PER = CH / 8;
  const int c = b.base + threadIdx.x % PER * 8;
  for (int row = r0 + threadIdx.x / PER; row < r1; row += kSelThreads / PER)
    if (c < b.stop) zero_row<IO>(q, o, row, c);
  const int ch = min(CH, b.stop - b.base);
  for (int i = threadIdx.x; i < ch * q.N; i += kSelThreads) part[(int64_t)b.base * q.N + i] = 0.f;
  for (int i = threadIdx.x; i < 2 * ch; i += kSelThreads)
    part[(int64_t)q.C * q.N + (int64_t)(i / ch) * q.C + b.base + i % ch] = 0.f;
}

// ---- main ----------------------------------------------------------------------------------------
template <typename IO, int K>
__global__ __launch_bounds__(kSelThreads, 2) void k_bwd_main(SelArgs q, Work w, SelGrads o,
                                                             const IO* dy, const float* dfinal,
                                                             int tiles) {
  constexpr int T = kQuarter, TC = kChunk, NP = NPL * K, CH = kSelThreads / K;
  constexpr int MV = 64 / K;  // values of a merge
  __shared__ __attribute__((aligned(16))) float s_dl[TC][CH], s_du[TC][CH], s_e[TC][CH];
  __shared__ __attribute__((aligned(16))) float s_y[TC][CH];
  __shared__ __attribute__((aligned(16))) float s_b[TC][NP], s_c[TC][NP];
  __shared__ float s_bc[kSelThreads / 64][T][2][NP];
  const Tile b(q, CH, blockIdx.x % tiles);
  const int u = blockIdx.x / tiles, k = threadIdx.x % K, ch = threadIdx.x / K, c = b.base + ch;
  const int wave = threadIdx.x >> 6;
  const bool live = c < b.stop;
  const int r0 = u * TC, r1 = min(r0 + TC, q.rows.R);
  uint64_t starts, ends, inside;
  int seq;
  mark_rows(q.rows, r0, r1, starts, ends, inside, seq);
  float* part = w.part + (int64_t)u * q.C * (q.N + 2);
  if (!inside) {  // rows of no sequence
    leave_empty<IO, K>(q, o, b, r0, r1, part);
    return;
  }
  stage<IO, TC, CH, NP>(q, dy, b, r0, r1, inside, s_dl, s_du, s_e, s_b, s_c);
  float A[NPL], h[4][NPL], g[NPL], dA[NPL];
#pragma unroll
  for (int j = 0; j < NPL; ++j) A[j] = h[0][j] = h[1][j] = h[2][j] = h[3][j] = g[j] = dA[j] = 0.f;
  const int64_t CN = (int64_t)q.C * q.N, at = (int64_t)c * q.N;
  if (live) {
    load_states<NPL>(q.A + at, k, q.N, A);
    load_states<NPL>(w.state + ((int64_t)u * 4 + 3) * CN + at, k, q.N, h[0]);
    load_states<NPL>(w.adj + (int64_t)u * CN + at, k, q.N, g);
#pragma unroll
    for (int s = 0; s < 3; ++s)
      load_states<NPL>(w.state + ((int64_t)u * 4 + s) * CN + at, k, q.N, h[s + 1]);
  }
#pragma unroll
  for (int j = 0; j < NPL; ++j) A[j] *= kLog2e;
#pragma unroll
  for (int s = 0; s < 3; ++s) {  // the entering state's part in the quarters'
    const float d = live ? w.sums[((int64_t)u * 4 + s) * q.C + c] : 0.f;
#pragma unroll
    for (int j = 0; j < NPL; ++j)
      h[s + 1][j] = d == d ? fmaf(exp2_fast(d * A[j]), h[0][j], h[s + 1][j]) : h[s + 1][j];
  }
  __syncthreads();
  const int mine = merged_value<K>();
  // events: a sequence begins or ends in the chunk. Where none does (`quiet`), no branch separates
  // the tokens and the loads and products of several overlap.
  struct Token {
    float dl, du, e, b[NPL], c[NPL];
  };
  auto staged = [&](int t) {
    Token m;
    m.dl = s_dl[t][ch];
    m.du = s_du[t][ch];
    m.e = s_e[t][ch];
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
      m.b[j] = s_b[t][k * NPL + j];
      m.c[j] = s_c[t][k * NPL + j];
    }
    return m;
  };
  auto walk = [&](auto quiet) {
    constexpr bool EV = !decltype(quiet)::value;
#pragma unroll
    for (int s = 3; s >= 0; --s) {
      if (EV && s * T >= r1 - r0) continue;  // of a short last chunk
      float hn[T][NPL], a[T][NPL];  // h after each token, its decay
#pragma unroll
      for (int i = 0; i < T; ++i) {
        const int t = s * T + i;
        float prev[NPL];
#pragma unroll
        for (int j = 0; j < NPL; ++j) prev[j] = i ? hn[i - 1][j] : h[s][j];
        if (EV && ((starts >> t) & 1)) seq_states(q, q.h0, seq_at(seq, t), c, k, live, prev);
        const float dl = s_dl[t][ch], du = s_du[t][ch];
        float y = 0.f;
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
          a[i][j] = exp2_fast(dl * A[j]);
          hn[i][j] = fmaf(a[i][j], prev[j], du * s_b[t][k * NPL + j]);
          y = fmaf(hn[i][j], s_c[t][k * NPL + j], y);
        }
        // (without a gate y has no use, but leaving it out took more registers; the K lanes write
        // the same value)
        s_y[t][ch] = sum_lanes<K>(y);
        if (EV || i % 4 == 3)
          __builtin_amdgcn_sched_barrier(0);  // loads of later tokens would cost registers here
      }
      asm volatile("" ::: "memory");  // and so would what was loaded above, kept for its reuse below
      Token next = staged(s * T + T - 1);
      float vals[MV < 8 ? 8 : MV];  // dB of the four entries, then dC; K 4: of two tokens
#pragma unroll
      for (int i = T - 1; i >= 0; --i) {
        const int t = s * T + i;
        if (EV && ((ends >> t) & 1)) {
          seq_states(q, dfinal, seq_at(seq, t), c, k, live, g);
          if (inside >> t == 1) {  // what lies behind is of no sequence: its `prev` was this one's
                                   // last state, which infinite or NaN does not vanish with delta = 0
#pragma unroll
            for (int j = 0; j < NPL; ++j) dA[j] = 0.f;
          }
        }
        float prev[NPL];
#pragma unroll
        for (int j = 0; j < NPL; ++j) prev[j] = i ? hn[i - 1][j] : h[s][j];
        const bool start = EV && ((starts >> t) & 1);
        if (start) seq_states(q, q.h0, seq_at(seq, t), c, k, live, prev);
        const Token m = next;
        if (i) next = staged(t - 1);  // a token ahead
        const float dl = m.dl, du = m.du, e = m.e;
        float qs = 0.f, sa = 0.f;
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
          const float G = fmaf(m.c[j], e, g[j]);
          const float aG = a[i][j] * G, wv = aG * prev[j];
          qs = fmaf(G, m.b[j], qs);
          sa = fmaf(wv, A[j], sa);
          dA[j] = fmaf(wv, dl, dA[j]);
          g[j] = aG;
          const int slot = K == 4 ? (i & 1) * 8 + j : j;
          vals[slot] = G * du;
          vals[slot + 4] = hn[i][j] * e;
        }
        if constexpr (K == 4) {
          if ((i & 1) == 0)
            s_bc[wave][i + (mine >> 3)][(mine >> 2) & 1][k * NPL + (mine & 3)] = merge<K>(vals);
        } else if constexpr (K == 8) {
          s_bc[wave][i][mine >> 2][k * NPL + (mine & 3)] = merge<K>(vals);
        } else {
          const float vb[4] = {vals[0], vals[1], vals[2], vals[3]};
          const float vc[4] = {vals[4], vals[5], vals[6], vals[7]};
          s_bc[wave][i][0][k * NPL + mine] = merge<K>(vb);
          s_bc[wave][i][1][k * NPL + mine] = merge<K>(vc);
        }
        qs = sum_lanes<K>(qs);
        sa = sum_lanes<K>(sa);
        // this token's delta x and e have no further reader: q and sum w A take their places
        (k & 1 ? s_e : s_du)[t][ch] = k & 1 ? sa : qs;
        if (start) {
          if (o.dh0 && live) {
            store_states<NPL>(o.dh0 + ((int64_t)seq_at(seq, t) * q.C + c) * q.N, k, q.N, g);
          }
#pragma unroll
          for (int j = 0; j < NPL; ++j) g[j] = 0.f;
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      __syncthreads();
      for (int v = threadIdx.x; v < T * 2 * NP; v += kSelThreads) {
        const int i = v / (2 * NP), rest = v % (2 * NP), which = rest / NP, n = rest % NP;
        const int row = r0 + s * T + i;
        if (row < r1 && n < q.N) {
          float m = s_bc[0][i][which][n];
#pragma unroll
          for (int x = 1; x < kSelThreads / 64; ++x) m += s_bc[x][i][which][n];
          w.bc[(((int64_t)b.ct * q.rows.R + row) * 2 + which) * q.N + n] = m;
        }
      }
      __syncthreads();
    }
  };
  if (starts | ends) walk(std::false_type{});
  else walk(std::true_type{});
  if (live) store_states<NPL>(part + (int64_t)c * q.N, k, q.N, dA);
  // outputs of the chunk: a thread takes 8 channels of every 32nd row; e x and ddt are summed over
  // its rows, then over the threads of the same channels
  constexpr int V = 8, TR = kSelThreads / (CH / V);
  const int cl = threadIdx.x % (CH / V) * V, cc = b.base + cl;
  float sd[V], sb[V];
#pragma unroll
  for (int j = 0; j < V; ++j) sd[j] = sb[j] = 0.f;
  if (cc < b.stop) {
    float D[V], bias[V];
#pragma unroll
    for (int j = 0; j < V; ++j) D[j] = bias[j] = 0.f;
    if (q.D) load_f32<V>(q.D + cc, D);
    if (q.dt_bias) load_f32<V>(q.dt_bias + cc, bias);
    for (int t = threadIdx.x / (CH / V); t < TC; t += TR) {
      const int64_t row = r0 + t;
      if (!((inside >> t) & 1)) {
        if (row < r1) zero_row<IO>(q, o, row, cc);
        continue;
      }
      Vec<IO, V> xr, tr, dr, zr;
      xr.load((const IO*)q.x + row * q.xs + cc);
      tr.load((const IO*)q.dt + row * q.dts + cc);
      dr.load(dy + row * q.C + cc);
      if (q.z) zr.load((const IO*)q.z + row * q.zs + cc);
      float ox[V], ot[V], oz[V], vq[V], va[V], vy[V], vd[V];
      load_f32<V>(&s_du[t][cl], vq);
      load_f32<V>(&s_e[t][cl], va);
      load_f32<V>(&s_y[t][cl], vy);
      load_f32<V>(&s_dl[t][cl], vd);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float x = xr.get(j), qv = vq[j], sa = va[j] * 0.6931471805599453f;
        float e = dr.get(j);
        if (q.z) {
          const float zv = zr.get(j), sg = sigmoid(zv);
          oz[j] = e * fmaf(D[j], x, vy[j]) * (sg * fmaf(zv, 1.f - sg, 1.f));
          e *= zv * sg;
        }
        ox[j] = fmaf(vd[j], qv, D[j] * e);
        float dd = fmaf(x, qv, sa);
        if (q.softplus) dd *= sigmoid(tr.get(j) + bias[j]);
        ot[j] = dd;
        sd[j] = fmaf(e, x, sd[j]);
        sb[j] += dd;
      }
      store_vec<IO, V>((IO*)o.dx + row * q.C + cc, ox);
      store_vec<IO, V>((IO*)o.ddt + row * q.C + cc, ot);
      if (q.z) store_vec<IO, V>((IO*)o.dz + row * q.C + cc, oz);
    }
  }
  __syncthreads();
  float* red = &s_dl[0][0];  // [wave][dD, ddt_bias][CH]: the staged rows are done with
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int m = CH / V; m < 64; m <<= 1) {
      sd[j] += __shfl_xor(sd[j], m, kWave);
      sb[j] += __shfl_xor(sb[j], m, kWave);
    }
    if ((threadIdx.x & 63) < CH / V) {
      red[(wave * 2 + 0) * CH + cl + j] = sd[j];
      red[(wave * 2 + 1) * CH + cl + j] = sb[j];
    }
  }
  __syncthreads();
  if (threadIdx.x < 2 * CH) {
    const int which = threadIdx.x / CH, x = threadIdx.x % CH;
    if (b.base + x < b.stop) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < kSelThreads / 64; ++i) m += red[(i * 2 + which) * CH + x];
      part[(int64_t)q.C * q.N + (int64_t)which * q.C + b.base + x] = m;
    }
  }
}

// dB and dC: the sums over the tiles of a group, rounded once.
template <typename IO>
__global__ __launch_bounds__(256) void k_bwd_bc(SelArgs q, Work w, SelGrads o, int per_group) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t RN = (int64_t)q.rows.R * 2 * q.N;
  if (id >= RN * q.G) return;
  const int g = (int)(id / RN);
  const int64_t at = id % RN, row = at / (2 * q.N);
  const int which = (int)(at / q.N) & 1, n = (int)(at % q.N);
  const float* p = w.bc + (int64_t)g * per_group * RN + at;
  float m = 0.f;
  if (seq_of(q.rows, (int)row) >= 0) {
#pragma unroll 4
    for (int i = 0; i < per_group; ++i) m += p[i * RN];
  }
  Io<IO>::store((IO*)(which ? o.dC : o.dB), (row * q.G + g) * q.N + n, m);
}

// Gradients of the initial states of empty sequences: the final states' own.
__global__ __launch_bounds__(256) void k_bwd_empty(SelArgs q, const float* dfinal, float* dh0) {
  const int64_t CN = (int64_t)q.C * q.N, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= CN * q.rows.S) return;
  const int s = (int)(id / CN);
  if (seq_end(q.rows, s) <= seq_begin(q.rows, s)) dh0[id] = dfinal ? dfinal[id] : 0.f;
}

int64_t round64(int64_t v) { return (v + 63) / 64 * 64; }

int tiles_of(const SelArgs& a) {  // channel tiles of a group
  const int ch = kSelThreads / (a.N <= 16 ? 4 : a.N <= 32 ? 8 : 16), cg = a.C / a.G;
  return (cg + ch - 1) / ch;
}

// The workspace's parts from `ws` on; its floats.
int64_t lay_out(const SelArgs& a, float* ws, Work* w) {
  w->chunks = (a.rows.R + kChunk - 1) / kChunk;
  const int64_t tiles = (int64_t)tiles_of(a) * a.G, n = w->chunks;
  const int64_t st = round64(n * a.C * a.N), sm = round64(n * a.C);
  const int64_t bc = round64(tiles * a.rows.R * 2 * a.N), pt = round64(n * a.C * (a.N + 2));
  w->state = ws;
  w->adj = w->state + 4 * st;
  w->sums = w->adj + st;
  w->back = w->sums + 4 * sm;
  w->bc = w->back + sm;
  w->part = w->bc + bc;
  return 5 * (st + sm) + bc + pt;
}

}  // namespace

int64_t selective_backward_bytes(const SelArgs& a) {
  Work w;
  return 4 * lay_out(a, nullptr, &w);
}

hipError_t launch_selective_backward(const SelArgs& a, const void* dy, const float* dfinal,
                                     const SelGrads& g, float* ws, int n_cu, hipStream_t s) {
  Work w;
  lay_out(a, ws, &w);
  const int cg = a.C / a.G, per_group = tiles_of(a), tiles = per_group * a.G;
  const unsigned blocks = (unsigned)((int64_t)tiles * w.chunks);
  const int64_t CN = (int64_t)a.C * a.N, simds = 4 * (int64_t)n_cu;
  auto run = [&](auto io) {
    using IO = decltype(io);
    auto ends = [&](auto size, auto exact) {
      constexpr int NT = decltype(size)::value;
      const int64_t waves = (int64_t)((cg + 63) / 64) * a.G * w.chunks * ((a.N + NT - 1) / NT);
      constexpr bool EX = decltype(exact)::value;
      const dim3 grid((unsigned)((waves + 3) / 4));
      const bool events = a.rows.starts || a.rows.L % kChunk, all = events && waves <= kOneLaunch * simds;
      if (!all && (a.rows.starts || a.rows.L >= kChunk))
        hipLaunchKernelGGL((k_bwd_ends<IO, NT, EX, false>), grid, dim3(256), 0, s, a, w,
                           (const IO*)dy, dfinal, 0);
      if (events)
        hipLaunchKernelGGL((k_bwd_ends<IO, NT, EX, true>), grid, dim3(256), 0, s, a, w,
                           (const IO*)dy, dfinal, all ? 1 : 0);
      return hipGetLastError();
    };
    using std::integral_constant;
    // four entries a lane where that still fits the card at once: shorter for each token
    const int64_t fours = (int64_t)((cg + 63) / 64) * a.G * w.chunks * (a.N / 4);
    hipError_t e = fours <= kFours * simds ? ends(integral_constant<int, 4>{}, std::true_type{})
                   : a.N % 16 == 0 ? ends(integral_constant<int, 16>{}, std::true_type{})
                   : a.N <= 8      ? ends(integral_constant<int, 8>{}, std::false_type{})
                                   : ends(integral_constant<int, 16>{}, std::false_type{});
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(k_bwd_chain, dim3((unsigned)((CN + 255) / 256), 2), dim3(256), 0, s, a, w);
    e = by_states(a.N, [&](auto lanes) {
      hipLaunchKernelGGL((k_bwd_main<IO, decltype(lanes)::value>), dim3(blocks), dim3(kSelThreads),
                         0, s, a, w, g, (const IO*)dy, dfinal, tiles);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
    const int64_t n = (int64_t)a.rows.R * 2 * a.N * a.G;
    hipLaunchKernelGGL((k_bwd_bc<IO>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a, w, g,
                       per_group);
    return hipGetLastError();
  };
  const hipError_t e = a.io == kIoBf16 ? run(u16{}) : run(float{});
  if (e != hipSuccess) return e;
  if (g.dh0 && a.rows.starts) {
    hipLaunchKernelGGL(k_bwd_empty, dim3((unsigned)((CN * a.rows.S + 255) / 256)), dim3(256), 0, s,
                       a, dfinal, g.dh0);
    const hipError_t e2 = hipGetLastError();
    if (e2 != hipSuccess) return e2;
  }
  return launch_column_sums(w.part, w.chunks, CN, g.dA, (int)CN, 0, 1, a.C, g.dD, a.C, g.ddtb, s);
}

}  // namespace ssd
