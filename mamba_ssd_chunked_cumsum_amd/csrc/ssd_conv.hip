// Short causal depthwise convolution (width 2 to 4) with bias and SiLU: forward, single token and
// backward.
//
//   v[t,c] = bias[c] + sum_k w[c,k] x[t - W + 1 + k, c];   y = v / (1 + exp(-v))
//
// About 2 W + 10 operations for each element read and written once: bound by memory. A thread
// holds 8 (backward: 4) neighbouring channels, their weights and the last W - 1 inputs in registers
// and walks a strip of token rows, so that every input is loaded once but for the W - 1 rows in
// front of a strip (and, backward, behind it); a wave covers 64 neighbouring vectors of a row.
// Each thread finds the sequence of its strip's first row and reloads the window from the initial
// state where the next sequence begins, so packed sequences need no padding. At 2 x 8192 x 5376 bf16
// the forward takes 74 to 78 us (4.6 TB/s; a copy of that size 5.4), the backward with fp32 dy 156 us
// (4.5 TB/s); 5003 packed tokens x 1792 channels 16 us, a token for 4 x 5376 4 us (a launch).
#include "ssd_rows.h"

namespace ssd {

namespace {

constexpr int kBlock = 256;

// The tensor of a split that holds channel c, its width and c's column in it.
__device__ __forceinline__ int split_of(const Split& s, int c, int* width, int* col) {
  const int i = (c >= s.first[1]) + (c >= s.first[2]);
  *width = s.first[i + 1] - s.first[i];
  *col = c - s.first[i];
  return i;
}

// Input at position p of sequence s (begin row a), p >= -(W - 1): the row, or the initial state.
template <typename IO, int V>
__device__ __forceinline__ void input_at(const ConvArgs& q, int s, int a, int p, int W, int c,
                                         float (&v)[V]) {
  Vec<IO, V> r;
  if (p >= 0)
    r.load((const IO*)q.x + (int64_t)(a + p) * q.xs + c);
  else if (q.init)
    r.load((const IO*)q.init + ((int64_t)s * (W - 1) + W - 1 + p) * q.C + c);
  else
    r.zero();
  r.get(v);
}

template <int V, int W>
__device__ __forceinline__ void load_weights(const float* w, const float* bias, int c,
                                             float (&wv)[W][V], float (&bv)[V]) {
  float t[V * W];  // [V, W] as stored
#pragma unroll
  for (int i = 0; i < V * W / 4; ++i)
    *reinterpret_cast<float4*>(t + 4 * i) = reinterpret_cast<const float4*>(w + (int64_t)c * W)[i];
#pragma unroll
  for (int k = 0; k < W; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) wv[k][i] = t[i * W + k];
#pragma unroll
  for (int i = 0; i < V; ++i) bv[i] = 0.f;
  if (bias) load_f32<V>(bias + c, bv);
}

// ---- forward -------------------------------------------------------------------------------------
template <typename IO, int W>
__global__ __launch_bounds__(kBlock) void k_conv(ConvArgs q, IO* fin, int strip) {
  constexpr int V = 8, U = 8;  // U rows are loaded before the first of them is used
  const int nvec = q.C / V;
  const int64_t id = (int64_t)blockIdx.x * kBlock + threadIdx.x;
  const int64_t unit = id / nvec;  // strips and sequences together may pass 31 bits
  const int c = (int)(id % nvec) * V;
  const int nstrip = (q.rows.R + strip - 1) / strip;
  if (unit >= nstrip) {  // the final state of sequence `unit - nstrip`
    if (!fin || unit - nstrip >= q.rows.S) return;
    const int s = (int)(unit - nstrip);
    const int a = seq_begin(q.rows, s), len = max(seq_end(q.rows, s) - a, 0);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      float v[V];
      input_at<IO, V>(q, s, a, len - (W - 1) + j, W, c, v);
      store_vec<IO, V>(fin + ((int64_t)s * (W - 1) + j) * q.C + c, v);
    }
    return;
  }
  const int r0 = (int)unit * strip, r1 = min(r0 + strip, q.rows.R);
  int width, col;
  const int part = split_of(q.y, c, &width, &col);
  IO* y = (IO*)(part == 0 ? q.y.p[0] : part == 1 ? q.y.p[1] : q.y.p[2]);
  const IO* x = (const IO*)q.x;
  float w[W][V], bias[V];
  load_weights<V, W>(q.w, q.bias, c, w, bias);
  // rows are loaded before it is known which sequence they are of; a sequence's start replaces the
  // window's rows in front of it
  Vec<IO, V> before[W - 1], nx[U];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) before[j].load(x + (int64_t)max(r0 - (W - 1) + j, 0) * q.xs + c);
  int at = r0;  // the first row of nx
  auto fetch = [&](int r) {
    at = r;
#pragma unroll
    for (int u = 0; u < U; ++u) nx[u].load(x + (int64_t)min(r + u, r1 - 1) * q.xs + c);
  };
  fetch(r0);
  float win[W - 1][V];  // the last W - 1 inputs, oldest first
  int s = -1, end = r0;
  for (int r = r0; r < r1;) {
    if (r >= end) {  // the next sequence (the first one: where the strip stands in it)
      s = seq_of(q.rows, r);
      if (s < 0) {  // rows of no sequence
        r = end = after_gap(q.rows, r);
        continue;
      }
      const int a = seq_begin(q.rows, s);
      end = min(seq_end(q.rows, s), r1);
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        const int p = r - a - (W - 1) + j;
        if (r == r0 && p >= 0) before[j].get(win[j]);
        else input_at<IO, V>(q, s, a, p, W, c, win[j]);
      }
    }
    if (at != r) fetch(r);
    Vec<IO, V> in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) in[u] = nx[u];
    if (r + U < r1) fetch(r + U);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (r + u >= end) break;
      float xv[V], o[V];
      in[u].get(xv);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float v = bias[i];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) v = fmaf(w[k][i], win[k][i], v);
        v = fmaf(w[W - 1][i], xv[i], v);
        o[i] = q.silu ? v * sigmoid(v) : v;
      }
      store_vec<IO, V>(y + (int64_t)(r + u) * width + col, o, q.stream);
#pragma unroll
      for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int k = 0; k + 1 < W - 1; ++k) win[k][i] = win[k + 1][i];
        win[W - 2][i] = xv[i];
      }
    }
    r = min(r + U, end);
  }
}

// ---- single token ----------------------------------------------------------------------------------
// Every load of a thread comes before its first store: the state may be updated in place.
template <typename IO, int W>
__global__ __launch_bounds__(kBlock) void k_conv_step(ConvArgs q, IO* state_out) {
  constexpr int V = 8;
  const int nvec = q.C / V;
  const int64_t id = (int64_t)blockIdx.x * kBlock + threadIdx.x;
  const int b = (int)(id / nvec), c = (int)(id % nvec) * V;
  if (b >= q.rows.R) return;
  float w[W][V], bias[V], in[W][V], o[V];
  Vec<IO, V> raw[W];
#pragma unroll
  for (int k = 0; k < W - 1; ++k)
    raw[k].load((const IO*)q.init + ((int64_t)b * (W - 1) + k) * q.C + c);
  raw[W - 1].load((const IO*)q.x + (int64_t)b * q.xs + c);
  load_weights<V, W>(q.w, q.bias, c, w, bias);
#pragma unroll
  for (int k = 0; k < W; ++k) raw[k].get(in[k]);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float v = bias[i];
#pragma unroll
    for (int k = 0; k < W; ++k) v = fmaf(w[k][i], in[k][i], v);
    o[i] = q.silu ? v * sigmoid(v) : v;
  }
  int width, col;
  const int part = split_of(q.y, c, &width, &col);
  IO* y = (IO*)(part == 0 ? q.y.p[0] : part == 1 ? q.y.p[1] : q.y.p[2]);
  store_vec<IO, V>(y + (int64_t)b * width + col, o);
#pragma unroll
  for (int k = 0; k < W - 1; ++k)
    store_vec<IO, V>(state_out + ((int64_t)b * (W - 1) + k) * q.C + c, in[k + 1]);
}

// ---- backward ------------------------------------------------------------------------------------
// dv[t] = dy[t] silu'(v[t]) with v recomputed from the window. A strip's thread walks its rows and
// the W - 1 behind them (to the end of the sequence), keeping the W gradients of inputs that are
// still incomplete: dv[t] adds w[W - 1 - i] dv[t] to the gradient of x[t - i]. Sums over rows (dw,
// db) are kept in registers for the strip's own rows, added over the block's four strips in LDS and
// written as one partial per block, which a second kernel sums in a fixed order.
constexpr int kBwdV = 4, kBwdWaves = 4;
static_assert(64 * kBwdWaves == kBlock, "the trailing blocks count threads in kBlock");

template <typename IO, typename DY, int W>
__device__ __forceinline__ void conv_dv(const ConvArgs& q, const float (&w)[W][kBwdV],
                                        const float (&bias)[kBwdV], const float (&win)[W - 1][kBwdV],
                                        const float (&xv)[kBwdV], const float (&dy)[kBwdV],
                                        float (&dv)[kBwdV]) {
#pragma unroll
  for (int i = 0; i < kBwdV; ++i) {
    float v = bias[i];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) v = fmaf(w[k][i], win[k][i], v);
    v = fmaf(w[W - 1][i], xv[i], v);
    if (q.silu) {
      const float g = sigmoid(v);
      dv[i] = dy[i] * (g * fmaf(v, 1.f - g, 1.f));
    } else {
      dv[i] = dy[i];
    }
  }
}

// Gradient of the initial state: position p < 0 of sequence s takes w[k] dv[t] for its taps
// t = p + W - 1 - k >= 0, and the final state's gradient where the sequence is shorter than it.
template <typename IO, typename DY, int W>
__device__ __forceinline__ void conv_dinit(const ConvArgs& q, const float* dfinal, float* dinit,
                                           int64_t id) {
  constexpr int V = kBwdV;
  const int nvec = q.C / V;
  const int s = (int)(id / nvec), c = (int)(id % nvec) * V;
  if (s >= q.rows.S) return;
  const int a = seq_begin(q.rows, s), len = max(seq_end(q.rows, s) - a, 0);
  int width, col;
  const int pi = split_of(q.y, c, &width, &col);
  const DY* dyp = (const DY*)(pi == 0 ? q.y.p[0] : pi == 1 ? q.y.p[1] : q.y.p[2]) + col;
  float w[W][V], bias[V], win[W - 1][V], g[W - 1][V];
  load_weights<V, W>(q.w, q.bias, c, w, bias);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    input_at<IO, V>(q, s, a, j - (W - 1), W, c, win[j]);
#pragma unroll
    for (int i = 0; i < V; ++i) g[j][i] = 0.f;
    if (dfinal && j >= len) load_f32<V>(dfinal + ((int64_t)s * (W - 1) + j - len) * q.C + c, g[j]);
  }
#pragma unroll
  for (int t = 0; t < W - 1; ++t) {
    if (t >= len) break;
    float xv[V], dy[V], dv[V];
    input_at<IO, V>(q, s, a, t, W, c, xv);
    Vec<DY, V> d;
    d.load(dyp + (int64_t)(a + t) * width);
    d.get(dy);
    conv_dv<IO, DY, W>(q, w, bias, win, xv, dy, dv);
    // state entry j is at position j - (W - 1): tap k = j - t of token t
#pragma unroll
    for (int j = t; j < W - 1; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) g[j][i] = fmaf(w[j - t][i], dv[i], g[j][i]);
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
      for (int k = 0; k + 1 < W - 1; ++k) win[k][i] = win[k + 1][i];
      win[W - 2][i] = xv[i];
    }
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
    store_vec<float, V>(dinit + ((int64_t)s * (W - 1) + j) * q.C + c, g[j]);
}

template <typename IO, typename DY, int W>
__global__ __launch_bounds__(64 * kBwdWaves) void k_conv_bwd(ConvArgs q, const float* dfinal,
                                                             IO* dx, float* part, float* dinit,
                                                             int nvb, int nsb, int strip) {
  constexpr int V = kBwdV, U = 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const unsigned block = blockIdx.x;
  const int vb = block % nvb, sb = block / nvb;
  if (sb >= nsb) {  // the blocks behind the strips take the initial states' gradients
    const int64_t id = (int64_t)(block - (unsigned)nvb * nsb) * kBlock + threadIdx.x;
    conv_dinit<IO, DY, W>(q, dfinal, dinit, id);
    return;
  }
  const int c = (vb * 64 + lane) * V;
  const bool live = c < q.C;
  float dw[W + 1][V];
#pragma unroll
  for (int k = 0; k <= W; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) dw[k][i] = 0.f;
  const int r0 = (sb * kBwdWaves + wave) * strip, r1 = min(r0 + strip, q.rows.R);
  if (live && r0 < r1) {
    int width, col;
    const int pi = split_of(q.y, c, &width, &col);
    const DY* dyp = (const DY*)(pi == 0 ? q.y.p[0] : pi == 1 ? q.y.p[1] : q.y.p[2]) + col;
    const IO* x = (const IO*)q.x + c;
    float w[W][V], bias[V];
    load_weights<V, W>(q.w, q.bias, c, w, bias);
    float win[W - 1][V], acc[W][V];  // acc[i]: gradient of x[r - i], incomplete but for i = W - 1
    for (int r = r0; r < r1;) {  // sequence by sequence
      const int s = seq_of(q.rows, r);
      if (s < 0) {  // rows of no sequence: no gradient
        const float zero[V] = {};
        const int to = min(after_gap(q.rows, r), r1);
        for (; r < to; ++r) store_vec<IO, V>(dx + (int64_t)r * q.C + c, zero);
        continue;
      }
      const int a = seq_begin(q.rows, s), b = seq_end(q.rows, s);
      const int own = min(b, r1), last = min(b, r1 + W - 1);
#pragma unroll
      for (int j = 0; j < W - 1; ++j) input_at<IO, V>(q, s, a, r - a - (W - 1) + j, W, c, win[j]);
#pragma unroll
      for (int k = 0; k < W; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[k][i] = 0.f;
      const int first = r;
      // the gradient of row t is complete: add the final state's part, round, write
      auto emit = [&](int t, const float (&v)[V]) {
        if (t < first || t >= own) return;
        float o[V];
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = v[i];
        const int m = t - b + W - 1;
        if (dfinal && m >= 0) {
          float d[V];
          load_f32<V>(dfinal + ((int64_t)s * (W - 1) + m) * q.C + c, d);
#pragma unroll
          for (int i = 0; i < V; ++i) o[i] += d[i];
        }
        store_vec<IO, V>(dx + (int64_t)t * q.C + c, o);
      };
      Vec<IO, V> nx[U];  // the next U rows, loaded while the current ones are worked on
      Vec<DY, V> ny[U];
      auto fetch = [&](int from) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t t = min(from + u, last - 1);
          nx[u].load(x + t * q.xs);
          ny[u].load(dyp + t * width);
        }
      };
      fetch(r);
      while (r < last) {
        Vec<IO, V> in[U];
        Vec<DY, V> din[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          in[u] = nx[u];
          din[u] = ny[u];
        }
        fetch(r + U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int t = r + u;
          if (t >= last) break;
          float xv[V], dy[V], dv[V];
          in[u].get(xv);
          din[u].get(dy);
          conv_dv<IO, DY, W>(q, w, bias, win, xv, dy, dv);
#pragma unroll
          for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int k = 0; k < W; ++k) acc[k][i] = fmaf(w[W - 1 - k][i], dv[i], acc[k][i]);
            if (t < own) {
#pragma unroll
              for (int k = 0; k < W - 1; ++k) dw[k][i] = fmaf(dv[i], win[k][i], dw[k][i]);
              dw[W - 1][i] = fmaf(dv[i], xv[i], dw[W - 1][i]);
              dw[W][i] += dv[i];
            }
          }
          emit(t - (W - 1), acc[W - 1]);
#pragma unroll
          for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int k = W - 1; k > 0; --k) acc[k][i] = acc[k - 1][i];
            acc[0][i] = 0.f;
#pragma unroll
            for (int k = 0; k + 1 < W - 1; ++k) win[k][i] = win[k + 1][i];
            win[W - 2][i] = xv[i];
          }
        }
        r = min(r + U, last);
      }
      // the sequence's end (or the last rows behind the strip): acc[k] is now the gradient of row
      // last - k, complete where no later row of the sequence follows
#pragma unroll
      for (int k = W - 1; k > 0; --k) emit(last - k, acc[k]);
      r = own;
    }
  }
  // one partial per block: the four waves' sums in order
  __shared__ float red[kBwdWaves][64][V + 1];
#pragma unroll
  for (int k = 0; k <= W; ++k) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) red[wave][lane][i] = dw[k][i];
    __syncthreads();
    if (wave == 0 && live) {
      float o[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        o[i] = red[0][lane][i];
#pragma unroll
        for (int j = 1; j < kBwdWaves; ++j) o[i] += red[j][lane][i];
      }
      store_vec<float, V>(part + ((int64_t)sb * (W + 1) + k) * q.C + c, o);
    }
  }
}

unsigned blocks_of(int64_t threads) { return (unsigned)((threads + kBlock - 1) / kBlock); }

// Rows a backward strip: 128, or as many fewer (8 at least) as it takes for 512 blocks, two a compute
// unit (5882 rows x 784 channels: 147 us with 48 blocks of 128-row strips).
int conv_bwd_strip(const ConvArgs& a) {
  const int64_t nvb = (a.C / kBwdV + 63) / 64;
  int strip = 128;
  while (strip > 8 && nvb * (a.rows.R / (strip * kBwdWaves)) < 512) strip /= 2;
  return strip;
}
int conv_bwd_blocks(const ConvArgs& a) {
  const int rows = conv_bwd_strip(a) * kBwdWaves;
  return (a.rows.R + rows - 1) / rows;
}

template <typename F>
hipError_t by_width(int W, F f) {
  switch (W) {
    case 2: return f(std::integral_constant<int, 2>{});
    case 3: return f(std::integral_constant<int, 3>{});
    default: return f(std::integral_constant<int, 4>{});
  }
}

}  // namespace

hipError_t launch_conv(const ConvArgs& given, void* fin, hipStream_t s) {
  ConvArgs a = given;
  // bf16 outputs larger than the last-level cache (256 MiB) go past it: 8 x 8192 x 5376 263 -> 256 us, with
  // the SSD scan that reads them 825 -> 814. What fits is left there for what reads it: 2 x 8192 x 5376 with
  // the selective scan behind it 585 us, past the caches 591 (the convolution alone 80 and 78).
  a.stream = (int64_t)a.rows.R * a.C * (a.io == kIoBf16 ? 2 : 4) > (int64_t(256) << 20);
  const int nvec = a.C / 8;
  // 16 rows a thread; 8 where that would leave fewer than four waves a SIMD
  const int strip = (int64_t)a.rows.R * nvec >= 16 * 262144 ? 16 : 8;
  const int64_t nstrip = (a.rows.R + strip - 1) / strip;
  const unsigned nb = blocks_of((nstrip + (fin ? a.rows.S : 0)) * nvec);
  return by_width(a.W, [&](auto w) {
    constexpr int W = decltype(w)::value;
    if (a.io == kIoBf16)
      hipLaunchKernelGGL((k_conv<u16, W>), dim3(nb), dim3(kBlock), 0, s, a, (u16*)fin, strip);
    else
      hipLaunchKernelGGL((k_conv<float, W>), dim3(nb), dim3(kBlock), 0, s, a, (float*)fin, strip);
    return hipGetLastError();
  });
}

hipError_t launch_conv_step(const ConvArgs& a, void* state_out, hipStream_t s) {
  const unsigned nb = blocks_of((int64_t)a.rows.R * (a.C / 8));
  return by_width(a.W, [&](auto w) {
    constexpr int W = decltype(w)::value;
    if (a.io == kIoBf16)
      hipLaunchKernelGGL((k_conv_step<u16, W>), dim3(nb), dim3(kBlock), 0, s, a, (u16*)state_out);
    else
      hipLaunchKernelGGL((k_conv_step<float, W>), dim3(nb), dim3(kBlock), 0, s, a,
                         (float*)state_out);
    return hipGetLastError();
  });
}

int64_t conv_backward_bytes(const ConvArgs& a) {
  return (int64_t)conv_bwd_blocks(a) * (a.W + 1) * a.C * 4;
}

template <typename IO, typename DY, int W>
static hipError_t conv_backward(const ConvArgs& a, const float* dfinal, void* dx, float* dw,
                                float* db, float* dinit, float* ws, hipStream_t s) {
  const int nvb = (a.C / kBwdV + 63) / 64, nsb = conv_bwd_blocks(a);
  const int64_t tail = dinit ? ((int64_t)a.rows.S * (a.C / kBwdV) + kBlock - 1) / kBlock : 0;
  hipLaunchKernelGGL((k_conv_bwd<IO, DY, W>), dim3((unsigned)((int64_t)nvb * nsb + tail)),
                     dim3(64 * kBwdWaves), 0, s, a, dfinal, (IO*)dx, ws, dinit, nvb, nsb,
                     conv_bwd_strip(a));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_column_sums(ws, nsb, (int64_t)W * a.C, dw, a.C, 1, W, a.C, db, 0, nullptr, s);
}

hipError_t launch_conv_backward(const ConvArgs& a, int dy_io, const float* dfinal, void* dx,
                                float* dw, float* db, float* dinit, float* ws, hipStream_t s) {
  return by_width(a.W, [&](auto w) {
    constexpr int W = decltype(w)::value;
    if (a.io == kIoF32) return conv_backward<float, float, W>(a, dfinal, dx, dw, db, dinit, ws, s);
    if (dy_io == kIoF32) return conv_backward<u16, float, W>(a, dfinal, dx, dw, db, dinit, ws, s);
    return conv_backward<u16, u16, W>(a, dfinal, dx, dw, db, dinit, ws, s);
  });
}

}  // namespace ssd
