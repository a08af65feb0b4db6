// Selective scan with a decay of its own for every channel d and state entry n: forward and single
// token.
//
//   delta = softplus(dt + bias);  h <- exp(delta A[d,n]) h + delta x B[n];  y = sum_n h C[n] + D x
//
// For each (token, channel, state entry) one exponential, two products and two fused
// multiply-adds. With a different decay for every state entry no matrix product covers several
// tokens, so the vector units and their transcendental rate bound it: 16 + 4 * 4 cycles of a SIMD
// for 64 entries. The tokens of a sequence are sequential; parallel are the channels, the states of
// a channel over K lanes, and, where those do not fill the card, chunks of rows (split variant): one
// kernel computes each chunk's end state from a zero state and the sum of its delta, one chains the
// chunks (the decay of a whole chunk is exp(A sum delta)), and the scan itself starts every chunk
// from the state entering it.
//
// A block stages a tile of kTile rows in LDS in fp32 (delta and delta x for its channels, B and C),
// scans it and writes its outputs with D, gate and rounding applied. The loads of the next tile are
// issued before the scan of the current one.
#include "ssd_selective.h"

namespace ssd {

namespace {

constexpr int kTile = 32;

// The rows a block walks. direct: sequence u, or with the split variant chunk u of `len` rows.
struct Split2 {
  int len;      // rows of a chunk; 0: direct
  int chunks;   // number of chunks
  float* state; // [chunks, C, N]: end states, then the states entering the chunks
  float* sums;  // [chunks, C]: sums of delta
};

template <typename IO, int NPL, int K, bool STATES>
__global__ __launch_bounds__(kSelThreads) void k_scan(SelArgs q, Split2 sp, IO* __restrict__ y,
                                                      float* __restrict__ fin) {
  constexpr int CH = kSelThreads / K, NP = NPL * K;
  constexpr int VS = 8, NV = kTile * CH / VS, PV = (NV + kSelThreads - 1) / kSelThreads;
  constexpr int BV = kTile * NP / 4, PB = (BV + kSelThreads - 1) / kSelThreads;
  __shared__ float s_dl[kTile][CH], s_du[kTile][CH];
  __shared__ float s_y[STATES ? 1 : kTile][CH];
  __shared__ __attribute__((aligned(16))) float s_b[kTile][NP];
  __shared__ __attribute__((aligned(16))) float s_c[STATES ? 1 : kTile][NP];
  const int cg = q.C / q.G, tiles = (cg + CH - 1) / CH;
  const int ct = blockIdx.x % (tiles * q.G), u = blockIdx.x / (tiles * q.G);
  const int g = ct / tiles, base = g * cg + (ct % tiles) * CH, stop_c = (g + 1) * cg;
  const int tid = threadIdx.x, k = tid % K, ch = tid / K, c = base + ch;
  const bool live = c < stop_c;
  int r0, r1;
  if (sp.len && u < sp.chunks) {
    r0 = u * sp.len;
    r1 = min(r0 + sp.len, q.rows.R);
  } else {
    const int s = sp.len ? u - sp.chunks : u;
    r0 = seq_begin(q.rows, s);
    r1 = seq_end(q.rows, s);
    if (r1 <= r0) {  // an empty sequence: its state passes through
      if (!STATES && fin && live) {
        float h[NPL];
        const int64_t at = ((int64_t)s * q.C + c) * q.N;
#pragma unroll
        for (int j = 0; j < NPL; ++j) h[j] = 0.f;
        if (q.h0) load_states<NPL>(q.h0 + at, k, q.N, h);
        store_states<NPL>(fin + at, k, q.N, h);
      }
      return;
    }
    if (sp.len) return;
  }
  float A[NPL], h[NPL], sum = 0.f;
#pragma unroll
  for (int j = 0; j < NPL; ++j) A[j] = h[j] = 0.f;
  if (live) {
    load_states<NPL>(q.A + (int64_t)c * q.N, k, q.N, A);
    if (!STATES && sp.len) load_states<NPL>(sp.state + ((int64_t)u * q.C + c) * q.N, k, q.N, h);
  }
#pragma unroll
  for (int j = 0; j < NPL; ++j) A[j] *= kLog2e;

  // tile loads: vectors of 8 channels of a row, of 4 state entries of a row's B and C
  Vec<IO, VS> xr[PV], dr[PV];
  Vec<IO, 4> br[PB], cr[PB];
  auto fetch = [&](int r) {
#pragma unroll
    for (int i = 0; i < PV; ++i) {
      const int v = tid + i * kSelThreads, row = r + v / (CH / VS), cc = base + v % (CH / VS) * VS;
      xr[i].zero();
      dr[i].zero();
      if (v < NV && row < r1 && cc < stop_c) {
        xr[i].load((const IO*)q.x + row * q.xs + cc);
        dr[i].load((const IO*)q.dt + row * q.dts + cc);
      }
    }
#pragma unroll
    for (int i = 0; i < PB; ++i) {
      const int v = tid + i * kSelThreads, row = r + v / (NP / 4), n = v % (NP / 4) * 4;
      br[i].zero();
      cr[i].zero();
      if (v < BV && row < r1 && n < q.N) {
        br[i].load((const IO*)q.B + row * q.bs + g * q.N + n);
        if (!STATES) cr[i].load((const IO*)q.Cm + row * q.cs + g * q.N + n);
      }
    }
  };
  fetch(r0);
  for (int r = r0; r < r1; r += kTile) {
    uint64_t starts, ends, inside;
    mark_rows(q.rows, r, min(r + kTile, r1), starts, ends, inside);
    float xk[PV][VS];
#pragma unroll
    for (int i = 0; i < PV; ++i) {
      const int v = tid + i * kSelThreads, t = v / (CH / VS), cl = v % (CH / VS) * VS;
      if (v < NV) {
        float dl[VS], bias[VS];
        xr[i].get(xk[i]);
#pragma unroll
        for (int j = 0; j < VS; ++j) bias[j] = 0.f;
        if (q.dt_bias && base + cl < stop_c) load_f32<VS>(q.dt_bias + base + cl, bias);
        const bool in = (inside >> t) & 1;
#pragma unroll
        for (int j = 0; j < VS; ++j) {
          float d = dr[i].get(j) + bias[j];
          if (q.softplus) d = softplus(d);
          dl[j] = in ? d : 0.f;
        }
        *reinterpret_cast<float4*>(&s_dl[t][cl]) = make_float4(dl[0], dl[1], dl[2], dl[3]);
        *reinterpret_cast<float4*>(&s_dl[t][cl + 4]) = make_float4(dl[4], dl[5], dl[6], dl[7]);
#pragma unroll
        for (int j = 0; j < VS; ++j) dl[j] = in ? dl[j] * xk[i][j] : 0.f;
        *reinterpret_cast<float4*>(&s_du[t][cl]) = make_float4(dl[0], dl[1], dl[2], dl[3]);
        *reinterpret_cast<float4*>(&s_du[t][cl + 4]) = make_float4(dl[4], dl[5], dl[6], dl[7]);
      }
    }
#pragma unroll
    for (int i = 0; i < PB; ++i) {
      const int v = tid + i * kSelThreads, t = v / (NP / 4), n = v % (NP / 4) * 4;
      if (v < BV) {
        *reinterpret_cast<float4*>(&s_b[t][n]) =
            make_float4(br[i].get(0), br[i].get(1), br[i].get(2), br[i].get(3));
        if (!STATES)
          *reinterpret_cast<float4*>(&s_c[t][n]) =
              make_float4(cr[i].get(0), cr[i].get(1), cr[i].get(2), cr[i].get(3));
      }
    }
    __syncthreads();
    if (r + kTile < r1) fetch(r + kTile);
#pragma unroll 4
    for (int t = 0; t < kTile; ++t) {
      if ((starts >> t) & 1) {  // a sequence begins: its state replaces the one before
#pragma unroll
        for (int j = 0; j < NPL; ++j) h[j] = 0.f;
        sum = 0.f;
        if (q.h0 && live) {
          const int s = seq_of(q.rows, r + t);
          load_states<NPL>(q.h0 + ((int64_t)s * q.C + c) * q.N, k, q.N, h);
        }
      }
      const float dl = s_dl[t][ch], du = s_du[t][ch];
      float acc = 0.f;
      if (STATES) sum += dl;
#pragma unroll
      for (int j = 0; j < NPL; ++j) {
        const float a = exp2_fast(dl * A[j]);
        h[j] = fmaf(a, h[j], du * s_b[t][k * NPL + j]);
        if (!STATES) acc = fmaf(h[j], s_c[t][k * NPL + j], acc);
      }
      if (!STATES) {
        acc = sum_lanes<K>(acc);
        if (k == t % K) s_y[t][ch] = acc;
        if (fin && ((ends >> t) & 1) && live) {
          const int s = seq_of(q.rows, r + t);
          store_states<NPL>(fin + ((int64_t)s * q.C + c) * q.N, k, q.N, h);
        }
      }
    }
    __syncthreads();
    if (!STATES) {
#pragma unroll
      for (int i = 0; i < PV; ++i) {
        const int v = tid + i * kSelThreads, t = v / (CH / VS), cl = v % (CH / VS) * VS;
        if (v < NV && ((inside >> t) & 1) && base + cl < stop_c) {
          float o[VS], d[VS];
#pragma unroll
          for (int j = 0; j < VS; ++j) {
            o[j] = s_y[t][cl + j];
            d[j] = 0.f;
          }
          if (q.D) load_f32<VS>(q.D + base + cl, d);
#pragma unroll
          for (int j = 0; j < VS; ++j) o[j] = fmaf(d[j], xk[i][j], o[j]);
          if (q.z) {
            Vec<IO, VS> zr;
            zr.load((const IO*)q.z + (int64_t)(r + t) * q.zs + base + cl);
#pragma unroll
            for (int j = 0; j < VS; ++j) {
              const float zv = zr.get(j);
              o[j] *= zv * sigmoid(zv);
            }
          }
          store_vec<IO, VS>(y + (int64_t)(r + t) * q.C + base + cl, o);
        }
      }
    }
  }
  if (STATES && live) {
    store_states<NPL>(sp.state + ((int64_t)u * q.C + c) * q.N, k, q.N, h);
    if (k == 0) sp.sums[(int64_t)u * q.C + c] = sum;
  }
}

// Chain over the chunks, in place: state[u] from chunk u's end state (from zero, or from the last
// sequence that begins in it) to the state entering it. A chunk in which a sequence begins after its
// first row passes nothing on; at a first row that begins a sequence the scan itself starts anew.
__global__ __launch_bounds__(256) void k_scan_chain(SelArgs q, Split2 sp) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t CN = (int64_t)q.C * q.N;
  if (id >= CN) return;
  const int c = (int)(id / q.N);
  const float A = q.A[id] * kLog2e;
  float h = 0.f;
  for (int u = 0; u < sp.chunks; ++u) {
    const int r0 = u * sp.len, r1 = min(r0 + sp.len, q.rows.R);
    const float e = sp.state[u * CN + id], d = sp.sums[(int64_t)u * q.C + c];
    sp.state[u * CN + id] = h;
    // the sequence of the chunk's last row (-1: none) and whether it began before the chunk
    const int s = seq_of(q.rows, r1 - 1);
    const bool through = s >= 0 && seq_begin(q.rows, s) < r0;
    h = through ? fmaf(exp2_fast(A * d), h, e) : e;
  }
}

// ---- single token ----------------------------------------------------------------------------------
// L lanes a channel with four states each, as the SSD step: bound by the state, read and written
// once past the caches.
template <typename IO, int L>
__global__ __launch_bounds__(256) void k_sel_step(SelArgs q, float* state_out, IO* y) {
  const int64_t id = ((int64_t)blockIdx.x * 256 + threadIdx.x) / L;
  const int n = (threadIdx.x % L) * 4;
  if (id >= (int64_t)q.rows.R * q.C) return;
  const int b = (int)(id / q.C), c = (int)(id % q.C), g = c / (q.C / q.G);
  const bool on = n < q.N;
  const int nc = on ? n : 0;
  const f32x4 h = __builtin_nontemporal_load(
      reinterpret_cast<const f32x4*>(q.h0 + id * q.N + nc));
  const float4 A = *reinterpret_cast<const float4*>(q.A + (int64_t)c * q.N + nc);
  Vec<IO, 4> B, Cv;
  B.load((const IO*)q.B + b * q.bs + g * q.N + nc);
  Cv.load((const IO*)q.Cm + b * q.cs + g * q.N + nc);
  const float x = Io<IO>::load((const IO*)q.x, b * q.xs + c);
  float dl = Io<IO>::load((const IO*)q.dt, b * q.dts + c) + (q.dt_bias ? q.dt_bias[c] : 0.f);
  if (q.softplus) dl = softplus(dl);
  const float du = dl * x, dl2 = dl * kLog2e;
  const float a[4] = {A.x, A.y, A.z, A.w};
  f32x4 o;
  float acc = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    o[j] = fmaf(exp2_fast(dl2 * a[j]), h[j], du * B.get(j));
    acc = fmaf(o[j], Cv.get(j), acc);
  }
  if (on)
    __builtin_nontemporal_store(o, reinterpret_cast<f32x4*>(state_out + id * q.N + n));
  else
    acc = 0.f;
#pragma unroll
  for (int m = L / 2; m >= 1; m >>= 1) acc += __shfl_xor(acc, m, kWave);
  if (n == 0) {
    if (q.D) acc = fmaf(q.D[c], x, acc);
    if (q.z) {
      const float zv = Io<IO>::load((const IO*)q.z, b * q.zs + c);
      acc *= zv * sigmoid(zv);
    }
    Io<IO>::store(y, id, acc);
  }
}

// The split that a scan takes.
Split2 plan(const SelArgs& a, int n_cu) {
  const int K = a.N <= 16 ? 4 : a.N <= 32 ? 8 : 16;
  Split2 sp{0, 0, nullptr, nullptr};
  const int ch = kSelThreads / K, cg = a.C / a.G;
  const int64_t tiles = (int64_t)((cg + ch - 1) / ch) * a.G;
  const int64_t direct = tiles * a.rows.S;
  if (direct >= n_cu / 2 || a.rows.R < 512) return sp;
  // about two blocks a compute unit, chunks of at least 128 rows
  int64_t chunks = (2 * (int64_t)n_cu + tiles - 1) / tiles;
  int64_t len = (a.rows.R + chunks - 1) / chunks;
  len = len < 128 ? 128 : (len + kTile - 1) / kTile * kTile;
  sp.len = (int)len;
  sp.chunks = (int)((a.rows.R + len - 1) / len);
  if (sp.chunks < 3) sp.len = sp.chunks = 0;
  return sp;
}

int64_t state_floats(const SelArgs& a, const Split2& sp) {
  return ((int64_t)sp.chunks * a.C * a.N + 63) / 64 * 64;
}

}  // namespace

int64_t selective_bytes(const SelArgs& a, int n_cu) {
  const Split2 sp = plan(a, n_cu);
  return sp.len ? 4 * (state_floats(a, sp) + (int64_t)sp.chunks * a.C) : 0;
}

hipError_t launch_selective(const SelArgs& a, void* y, float* fin, float* ws, int n_cu,
                            hipStream_t s) {
  Split2 sp = plan(a, n_cu);
  sp.state = ws;
  sp.sums = ws ? ws + state_floats(a, sp) : nullptr;
  return by_states(a.N, [&](auto lanes) {
    constexpr int NPL = 4, K = decltype(lanes)::value;
    const int ch = kSelThreads / K, cg = a.C / a.G;
    const int64_t tiles = (int64_t)((cg + ch - 1) / ch) * a.G;
    auto run = [&](auto io) {
      using IO = decltype(io);
      if (!sp.len) {
        hipLaunchKernelGGL((k_scan<IO, NPL, K, false>), dim3((unsigned)(tiles * a.rows.S)),
                           dim3(kSelThreads), 0, s, a, sp, (IO*)y, fin);
        return hipGetLastError();
      }
      hipLaunchKernelGGL((k_scan<IO, NPL, K, true>), dim3((unsigned)(tiles * sp.chunks)),
                         dim3(kSelThreads), 0, s, a, sp, (IO*)nullptr, (float*)nullptr);
      hipLaunchKernelGGL(k_scan_chain, dim3((unsigned)(((int64_t)a.C * a.N + 255) / 256)),
                         dim3(256), 0, s, a, sp);
      // the units behind the chunks pass on the states of empty sequences
      const int64_t units = sp.chunks + (fin && a.rows.starts ? a.rows.S : 0);
      hipLaunchKernelGGL((k_scan<IO, NPL, K, false>), dim3((unsigned)(tiles * units)),
                         dim3(kSelThreads), 0, s, a, sp, (IO*)y, fin);
      return hipGetLastError();
    };
    return a.io == kIoBf16 ? run(u16{}) : run(float{});
  });
}

hipError_t launch_selective_step(const SelArgs& a, float* state_out, void* y, hipStream_t s) {
  const int64_t ch = (int64_t)a.rows.R * a.C;
  auto run = [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    const unsigned nb = (unsigned)((ch * L + 255) / 256);
    if (a.io == kIoBf16)
      hipLaunchKernelGGL((k_sel_step<u16, L>), dim3(nb), dim3(256), 0, s, a, state_out, (u16*)y);
    else
      hipLaunchKernelGGL((k_sel_step<float, L>), dim3(nb), dim3(256), 0, s, a, state_out,
                         (float*)y);
    return hipGetLastError();
  };
  if (a.N <= 4) return run(std::integral_constant<int, 1>{});
  if (a.N <= 8) return run(std::integral_constant<int, 2>{});
  if (a.N <= 16) return run(std::integral_constant<int, 4>{});
  if (a.N <= 32) return run(std::integral_constant<int, 8>{});
  return run(std::integral_constant<int, 16>{});
}

}  // namespace ssd
