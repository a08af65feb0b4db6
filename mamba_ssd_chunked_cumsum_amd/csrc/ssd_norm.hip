// RMS norms of a state space block: behind the scan with its gate, and before a block with the
// residual sum; forward and backward.
//
// A few operations for each element read and written once: bound by memory. A row (gated: one group
// of a row) is held in registers, NT threads with NV vectors of 8 each, so each element is loaded
// once whatever the direction; the row's sums go over the wave by shuffles and, where a row takes
// more than a wave, over the block through LDS. Short rows take a wave each, four to a block (of a row
// of 64 channels 8 lanes: 16384 x 80 groups of 64 bf16 456 us, backward 646, 1.1 and 1.3 TB/s).
// Backward, a block walks rows and keeps the sums for the weight (and scale) gradients of its own
// columns in registers, writing one partial at the end; a second kernel adds the partials in a
// fixed order. Measured: gated backward of 16384 x 8 groups of 1024 bf16 250 us (5.3 TB/s, the copy
// rate), residual norm of 16384 x 2560 (bf16, fp32 residual) 94 us (5.3 TB/s), its backward at 8192 x
// 768 fp32 18 us (5.6 TB/s) and 4 us for the sums.
#include "ssd_rows.h"

namespace ssd {

namespace {

constexpr int V = 8;

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, kWave);
  return v;
}

// Sum over the NT threads that share a row; every one of them gets it. `red`: one float a wave.
// `turn` flips between two halves of red, so that one barrier a sum is enough.
template <int NT>
__device__ __forceinline__ float row_sum(float v, float (&red)[2][16], int& turn) {
  v = wave_sum(v);
  if constexpr (NT > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[turn][wave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) v += red[turn][i];
    turn ^= 1;
  }
  return v;
}

// Threads a row, and rows (of groups) a block.
template <int NT>
struct Shape {
  static constexpr int kThreads = NT < 256 ? 256 : NT, kRows = kThreads / NT;
};

// A block's sums for n columns: of its one row walker, or of the four that its waves are, added in
// LDS.
template <int NT, int NV>
__device__ __forceinline__ void store_sums(float* part, int n, float (&v)[NV][V]) {
  const int t = threadIdx.x % NT;
  if constexpr (NT == 64) {
    __shared__ __attribute__((aligned(16))) float red[4][64 * V];
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      __syncthreads();
      store_vec<float, V>(&red[wave][t * V], v[i]);
      __syncthreads();
      const int c = (t + i * NT) * V + 2 * wave;  // two columns a thread
      if (c < n) {
        float o[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int at = t * V + 2 * wave + j;
          o[j] = ((red[0][at] + red[1][at]) + red[2][at]) + red[3][at];
        }
        *reinterpret_cast<float2*>(part + c) = make_float2(o[0], o[1]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * NT) * V;
      if (c < n) store_vec<float, V>(part + c, v[i]);
    }
  }
}

// ---- gated norm --------------------------------------------------------------------------------
// BEFORE: norm before gate. z null: no gate.
template <typename IO, int NT, int NV, bool BEFORE, bool GATE>
__global__ __launch_bounds__(Shape<NT>::kThreads) void k_gated(NormArgs q, const IO* x, int64_t xs,
                                                               const IO* z, int64_t zs, IO* y) {
  __shared__ float red[2][16];
  int turn = 0;
  const int n = q.C / q.G, t = threadIdx.x % NT;
  const int64_t unit = (int64_t)blockIdx.x * Shape<NT>::kRows + threadIdx.x / NT;
  if (unit >= (int64_t)q.R * q.G) return;  // whole waves (rows of a wave) or nothing
  const int64_t row = unit / q.G;
  const int c0 = (int)(unit % q.G) * n;
  Vec<IO, V> xr[NV], zr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + i * NT) * V;
    xr[i].zero();
    zr[i].zero();
    if (c < n) {
      xr[i].load(x + row * xs + c0 + c);
      if (GATE) zr[i].load(z + row * zs + c0 + c);
    }
  }
  float v[NV][V], g[NV][V], sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      v[i][j] = xr[i].get(j);
      if (GATE) {
        const float zv = zr[i].get(j);
        g[i][j] = zv * sigmoid(zv);
        if (!BEFORE) v[i][j] *= g[i][j];
      }
      sum = fmaf(v[i][j], v[i][j], sum);
    }
  const float r = rsqrtf(row_sum<NT>(sum, red, turn) / n + q.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + i * NT) * V;
    if (c < n) {
      float w[V];
      load_f32<V>(q.w + c0 + c, w);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float o = w[j] * (v[i][j] * r);
        if (GATE && BEFORE) o *= g[i][j];
        v[i][j] = o;
      }
      store_vec<IO, V>(y + row * q.C + c0 + c, v[i]);
    }
  }
}

// With n = v r (v normalised) and dn = w dy (times the gate, if it comes after):
// dv = r (dn - n mean(dn n)); dw = sum dy n (times the gate).
template <typename IO, int NT, int NV, bool BEFORE, bool GATE>
__global__ __launch_bounds__(Shape<NT>::kThreads) void k_gated_bwd(
    NormArgs q, const IO* x, int64_t xs, const IO* z, int64_t zs, const IO* dy, IO* dx, IO* dz,
    float* part, int walkers) {
  __shared__ float red[2][16];
  int turn = 0;
  const int n = q.C / q.G, t = threadIdx.x % NT;
  const int c0 = (int)(blockIdx.x % q.G) * n;
  const int walker = (int)(blockIdx.x / q.G) * Shape<NT>::kRows + threadIdx.x / NT;
  float w[NV][V], dw[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + i * NT) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) w[i][j] = dw[i][j] = 0.f;
    if (c < n) load_f32<V>(q.w + c0 + c, w[i]);
  }
  Vec<IO, V> xr[NV], zr[NV], dr[NV];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * NT) * V;
      xr[i].zero();
      zr[i].zero();
      dr[i].zero();
      if (c < n) {
        xr[i].load(x + row * xs + c0 + c);
        if (GATE) zr[i].load(z + row * zs + c0 + c);
        dr[i].load(dy + row * q.C + c0 + c);
      }
    }
  };
  if (walker < q.R) fetch(walker);
  for (int64_t row = walker; row < q.R; row += walkers) {
    float v[NV][V], sum = 0.f, dot = 0.f;  // v, and sum of dn v
    Vec<IO, V> xc[NV], zc[NV], dc[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      xc[i] = xr[i];
      zc[i] = zr[i];
      dc[i] = dr[i];
    }
    if (row + walkers < q.R) fetch(row + walkers);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float a = xc[i].get(j), d = w[i][j] * dc[i].get(j);
        if (GATE) {
          const float zv = zc[i].get(j), g = zv * sigmoid(zv);
          if (BEFORE) d *= g; else a *= g;
        }
        v[i][j] = a;
        sum = fmaf(a, a, sum);
        dot = fmaf(d, a, dot);
      }
    const float r = rsqrtf(row_sum<NT>(sum, red, turn) / n + q.eps);
    const float m = row_sum<NT>(dot, red, turn) / n * r * r;  // dv = r (dn - v m)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * NT) * V;
      float ox[V], oz[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = dc[i].get(j), nv = v[i][j] * r;
        if (GATE) {
          const float zv = zc[i].get(j), s = sigmoid(zv), g = zv * s;
          const float slope = s * fmaf(zv, 1.f - s, 1.f);
          if (BEFORE) {
            ox[j] = r * (w[i][j] * d * g - v[i][j] * m);
            oz[j] = d * w[i][j] * nv * slope;
            dw[i][j] = fmaf(d * g, nv, dw[i][j]);
          } else {
            const float dv = r * (w[i][j] * d - v[i][j] * m);
            ox[j] = dv * g;
            oz[j] = dv * xc[i].get(j) * slope;
            dw[i][j] = fmaf(d, nv, dw[i][j]);
          }
        } else {
          ox[j] = r * (w[i][j] * d - v[i][j] * m);
          dw[i][j] = fmaf(d, nv, dw[i][j]);
        }
      }
      if (c < n) {
        store_vec<IO, V>(dx + row * q.C + c0 + c, ox);
        if (GATE) store_vec<IO, V>(dz + row * q.C + c0 + c, oz);
      }
    }
  }
  store_sums<NT, NV>(part + (int64_t)(blockIdx.x / q.G) * q.C + c0, n, dw);
}

// ---- residual norm -----------------------------------------------------------------------------
template <typename IO, typename RES, int NT, int NV>
__global__ __launch_bounds__(Shape<NT>::kThreads) void k_residual(NormArgs q, const IO* x,
                                                                  int64_t xs, const RES* res,
                                                                  const float* scale, IO* y,
                                                                  RES* out) {
  __shared__ float red[2][16];
  int turn = 0;
  const int n = q.C, t = threadIdx.x % NT;
  const int64_t row = (int64_t)blockIdx.x * Shape<NT>::kRows + threadIdx.x / NT;
  if (row >= q.R) return;
  Vec<IO, V> xr[NV];
  Vec<RES, V> rr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + i * NT) * V;
    xr[i].zero();
    rr[i].zero();
    if (c < n) {
      xr[i].load(x + row * xs + c);
      if (res) rr[i].load(res + row * n + c);
    }
  }
  float v[NV][V], sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + i * NT) * V;
    float sc[V];
#pragma unroll
    for (int j = 0; j < V; ++j) sc[j] = 1.f;
    if (scale && c < n) load_f32<V>(scale + c, sc);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      v[i][j] = fmaf(sc[j], xr[i].get(j), rr[i].get(j));
      sum = fmaf(v[i][j], v[i][j], sum);
    }
  }
  const float r = rsqrtf(row_sum<NT>(sum, red, turn) / n + q.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + i * NT) * V;
    if (c < n) {
      float w[V], o[V];
      load_f32<V>(q.w + c, w);
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = w[j] * (v[i][j] * r);
      store_vec<RES, V>(out + row * n + c, v[i]);
      store_vec<IO, V>(y + row * n + c, o);
    }
  }
}

template <typename IO, typename RES, int NT, int NV, bool SCALE>
__global__ __launch_bounds__(Shape<NT>::kThreads) void k_residual_bwd(
    NormArgs q, const RES* rsum, const IO* x, int64_t xs, const float* scale, const IO* dy,
    const RES* dres, IO* dx, RES* dresid, float* part, int walkers) {
  __shared__ float red[2][16];
  int turn = 0;
  const int n = q.C, t = threadIdx.x % NT;
  const int walker = (int)(blockIdx.x * Shape<NT>::kRows + threadIdx.x / NT);
  float w[NV][V], dw[NV][V], ds[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + i * NT) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) w[i][j] = dw[i][j] = ds[i][j] = 0.f;
    if (c < n) load_f32<V>(q.w + c, w[i]);
  }
  Vec<RES, V> nr[NV], ng[NV];  // the next row, loaded while the current one is worked on
  Vec<IO, V> nd[NV], nx[NV];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * NT) * V;
      nr[i].zero();
      ng[i].zero();
      nd[i].zero();
      nx[i].zero();
      if (c < n) {
        nr[i].load(rsum + row * n + c);
        nd[i].load(dy + row * n + c);
        if (dres) ng[i].load(dres + row * n + c);
        if (SCALE) nx[i].load(x + row * xs + c);
      }
    }
  };
  if (walker < q.R) fetch(walker);
  for (int64_t row = walker; row < q.R; row += walkers) {
    Vec<RES, V> rr[NV], gr[NV];
    Vec<IO, V> dr[NV], xr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      rr[i] = nr[i];
      gr[i] = ng[i];
      dr[i] = nd[i];
      xr[i] = nx[i];
    }
    if (row + walkers < q.R) fetch(row + walkers);
    float sum = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float a = rr[i].get(j);
        sum = fmaf(a, a, sum);
        dot = fmaf(w[i][j] * dr[i].get(j), a, dot);
      }
    const float r = rsqrtf(row_sum<NT>(sum, red, turn) / n + q.eps);
    const float m = row_sum<NT>(dot, red, turn) / n * r * r;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * NT) * V;
      if (c < n) {
        float o[V], ox[V], sc[V];
        if (SCALE) load_f32<V>(scale + c, sc);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float a = rr[i].get(j), d = dr[i].get(j);
          o[j] = fmaf(r, w[i][j] * d - a * m, gr[i].get(j));
          dw[i][j] = fmaf(d, a * r, dw[i][j]);
          ox[j] = o[j];
          if (SCALE) {
            ox[j] = o[j] * sc[j];
            ds[i][j] = fmaf(o[j], xr[i].get(j), ds[i][j]);
          }
        }
        store_vec<IO, V>(dx + row * n + c, ox);
        if (dresid) store_vec<RES, V>(dresid + row * n + c, o);
      }
    }
  }
  float* p = part + (int64_t)blockIdx.x * n * (SCALE ? 2 : 1);
  store_sums<NT, NV>(p, n, dw);
  if (SCALE) store_sums<NT, NV>(p + n, n, ds);
}

// The smallest shape that holds n channels: a wave up to 1024, a block of 256 up to 6144, of 512 up
// to 8192. (Longer rows would need more registers a thread than the backward has.)
template <typename F>
hipError_t by_length(int n, F f) {
  using std::integral_constant;
  auto go = [&](auto nt, auto nv) { return f(nt, nv); };
  const int vecs = n / V;
  if (vecs <= 64) return go(integral_constant<int, 64>{}, integral_constant<int, 1>{});
  if (vecs <= 128) return go(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  if (vecs <= 256) return go(integral_constant<int, 256>{}, integral_constant<int, 1>{});
  if (vecs <= 512) return go(integral_constant<int, 256>{}, integral_constant<int, 2>{});
  if (vecs <= 768) return go(integral_constant<int, 256>{}, integral_constant<int, 3>{});
  return go(integral_constant<int, 512>{}, integral_constant<int, 2>{});
}

// How a backward pass is divided: row walkers, each of a wave (up to 1024 channels) or a block, and
// the partial sums they leave, one a block. At least 4 rows a walker (8 of a block), so that the
// partials are small beside the rows, and at most 8192 waves or 1024 blocks, a few for every SIMD.
struct Walk {
  int walkers, parts;  // of a group
};
Walk walk_of(int R, int G, int n) {
  const int per = n <= 1024 ? 4 : 1;  // walkers a block
  const int most = (n <= 1024 ? 8192 : 1024) / G, want = n <= 1024 ? (R + 3) / 4 : (R + 7) / 8;
  const int w = want < most ? want : most < 1 ? 1 : most;
  const int parts = (w + per - 1) / per;
  return Walk{parts * per, parts};
}

}  // namespace

hipError_t launch_gated_norm(const NormArgs& a, const void* x, int64_t xs, const void* z,
                             int64_t zs, int before, void* y, hipStream_t s) {
  return by_length(a.C / a.G, [&](auto nt, auto nv) {
    constexpr int NT = decltype(nt)::value, NV = decltype(nv)::value;
    const unsigned nb = (unsigned)(((int64_t)a.R * a.G + Shape<NT>::kRows - 1) / Shape<NT>::kRows);
    auto run = [&](auto io, auto bf, auto gt) {
      using IO = decltype(io);
      hipLaunchKernelGGL((k_gated<IO, NT, NV, decltype(bf)::value, decltype(gt)::value>), dim3(nb),
                         dim3(Shape<NT>::kThreads), 0, s, a, (const IO*)x, xs, (const IO*)z, zs,
                         (IO*)y);
      return hipGetLastError();
    };
    auto gates = [&](auto io) {
      if (!z) return run(io, std::false_type{}, std::false_type{});
      if (before) return run(io, std::true_type{}, std::true_type{});
      return run(io, std::false_type{}, std::true_type{});
    };
    return a.io == kIoBf16 ? gates(u16{}) : gates(float{});
  });
}

int64_t norm_backward_bytes(const NormArgs& a, int sums) {
  return (int64_t)walk_of(a.R, a.G, a.C / a.G).parts * a.C * sums * 4;
}

hipError_t launch_gated_norm_backward(const NormArgs& a, const void* x, int64_t xs, const void* z,
                                      int64_t zs, int before, const void* dy, void* dx, void* dz,
                                      float* dw, float* ws, hipStream_t s) {
  const Walk walk = walk_of(a.R, a.G, a.C / a.G);
  const hipError_t e = by_length(a.C / a.G, [&](auto nt, auto nv) {
    constexpr int NT = decltype(nt)::value, NV = decltype(nv)::value;
    const unsigned nb = (unsigned)((int64_t)walk.parts * a.G);
    auto run = [&](auto io, auto bf, auto gt) {
      using IO = decltype(io);
      hipLaunchKernelGGL((k_gated_bwd<IO, NT, NV, decltype(bf)::value, decltype(gt)::value>),
                         dim3(nb), dim3(Shape<NT>::kThreads), 0, s, a, (const IO*)x, xs,
                         (const IO*)z, zs, (const IO*)dy, (IO*)dx, (IO*)dz, ws,
                         walk.walkers);
      return hipGetLastError();
    };
    auto gates = [&](auto io) {
      if (!z) return run(io, std::false_type{}, std::false_type{});
      if (before) return run(io, std::true_type{}, std::true_type{});
      return run(io, std::false_type{}, std::true_type{});
    };
    return a.io == kIoBf16 ? gates(u16{}) : gates(float{});
  });
  if (e != hipSuccess) return e;
  return launch_column_sums(ws, walk.parts, a.C, dw, a.C, 0, 1, 0, nullptr, 0, nullptr, s);
}

hipError_t launch_residual_norm(const NormArgs& a, const void* x, int64_t xs, const void* res,
                                int res_io, const float* scale, void* y, void* res_out,
                                hipStream_t s) {
  return by_length(a.C, [&](auto nt, auto nv) {
    constexpr int NT = decltype(nt)::value, NV = decltype(nv)::value;
    const unsigned nb = (unsigned)((a.R + Shape<NT>::kRows - 1) / Shape<NT>::kRows);
    auto run = [&](auto io, auto re) {
      using IO = decltype(io);
      using RES = decltype(re);
      hipLaunchKernelGGL((k_residual<IO, RES, NT, NV>), dim3(nb), dim3(Shape<NT>::kThreads), 0, s,
                         a, (const IO*)x, xs, (const RES*)res, scale, (IO*)y, (RES*)res_out);
      return hipGetLastError();
    };
    if (a.io == kIoF32) return run(float{}, float{});
    return res_io == kIoF32 ? run(u16{}, float{}) : run(u16{}, u16{});
  });
}

hipError_t launch_residual_norm_backward(const NormArgs& a, const void* r, int res_io,
                                         const void* x, int64_t xs, const float* scale,
                                         const void* dy, const void* dres, void* dx, void* dresid,
                                         float* dw, float* dscale, float* ws, hipStream_t s) {
  const Walk walk = walk_of(a.R, 1, a.C);
  const hipError_t e = by_length(a.C, [&](auto nt, auto nv) {
    constexpr int NT = decltype(nt)::value, NV = decltype(nv)::value;
    const unsigned nb = (unsigned)walk.parts;
    auto run = [&](auto io, auto re, auto sc) {
      using IO = decltype(io);
      using RES = decltype(re);
      hipLaunchKernelGGL((k_residual_bwd<IO, RES, NT, NV, decltype(sc)::value>), dim3(nb),
                         dim3(Shape<NT>::kThreads), 0, s, a, (const RES*)r, (const IO*)x, xs, scale,
                         (const IO*)dy, (const RES*)dres, (IO*)dx, (RES*)dresid, ws,
                         walk.walkers);
      return hipGetLastError();
    };
    auto scales = [&](auto io, auto re) {
      return scale ? run(io, re, std::true_type{}) : run(io, re, std::false_type{});
    };
    if (a.io == kIoF32) return scales(float{}, float{});
    return res_io == kIoF32 ? scales(u16{}, float{}) : scales(u16{}, u16{});
  });
  if (e != hipSuccess) return e;
  return launch_column_sums(ws, walk.parts, a.C, dw, a.C, 0, 1, scale ? a.C : 0, dscale, 0,
                            nullptr, s);
}

}  // namespace ssd
