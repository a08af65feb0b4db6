// Rotation of B and C by positions: entries (p, q) of frequency j become
//   (p cos t - q sin t, p sin t + q cos t),   t = position[axis of j] * frequency[j].
//
// A few operations for each element read and written once: bound by memory. A thread takes eight (or
// four) frequencies of a token, forms their sines and cosines once and turns the entries of all its
// heads, of B and of C. The angle is formed in 64 bits: position times frequency is exact there, and
// what a far position leaves of a turn keeps 2^-53 of the whole angle.
#include "ssd_recurrent.h"
#include "ssd_rows.h"

namespace ssd {

namespace {

constexpr int kHeads = 4;  // of a thread, at most; their loads are issued together

template <typename IO, int F>
__global__ __launch_bounds__(256) void k_rotate(RotArgs q, int units, int splits) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int u = (int)(id % units), part = (int)(id / units % splits);
  const int64_t row = id / units / splits;
  if (row >= q.rows) return;
  const int turns = q.nf / F;
  const int g1 = min(q.G, (part + 1) * kHeads);
  if (u >= turns) {  // entries behind the turned ones: as they are
    const int at = 2 * q.nf + (u - turns) * 8;
    for (int g = part * kHeads; g < g1; ++g) {
      Vec<IO, 8> v;
      float f[8];
      v.load((const IO*)q.b + row * q.bs + g * q.N + at);
      v.get(f);
      store_vec<IO, 8>((IO*)q.ob + (row * q.G + g) * q.N + at, f);
      if (!q.c) continue;
      v.load((const IO*)q.c + row * q.cs + g * q.N + at);
      v.get(f);
      store_vec<IO, 8>((IO*)q.oc + (row * q.G + g) * q.N + at, f);
    }
    return;
  }
  const int j0 = u * F;
  const int p0 = q.interleaved ? 2 * j0 : j0, p1 = q.interleaved ? 2 * j0 + F : q.nf + j0;
  Vec<IO, F> v[kHeads][2][2];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    const int g = part * kHeads + h;
    if (g < g1) {
      const IO* b = (const IO*)q.b + row * q.bs + g * q.N;
      v[h][0][0].load(b + p0);
      v[h][0][1].load(b + p1);
      if (q.c) {
        const IO* c = (const IO*)q.c + row * q.cs + g * q.N;
        v[h][1][0].load(c + p0);
        v[h][1][1].load(c + p1);
      }
    }
  }
  float cs[F], sn[F], freq[F];
  load_f32<F>(q.freq + j0, freq);
  int pos[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) pos[i] = i < q.axes ? q.pos[i * q.rows + row] : 0;
#pragma unroll
  for (int i = 0; i < F; ++i) {
    const int j = j0 + i;
    const int at = j < q.ends[0] ? pos[0] : j < q.ends[1] ? pos[1] : j < q.ends[2] ? pos[2] : pos[3];
    const double quarters = (double)at * (double)freq[i] * 0.63661977236758134;  // 2 / pi
    const double whole = rint(quarters);
    float s, c;
    sincospif(0.5f * (float)(quarters - whole), &s, &c);  // within an eighth of a turn
    const int k = (int)((int64_t)whole & 3);  // quarter turns
    const float s1 = k & 1 ? c : s, c1 = k & 1 ? s : c;
    sn[i] = k & 2 ? -s1 : s1;
    cs[i] = (k == 1 || k == 2) ? -c1 : c1;
    if (q.inverse) sn[i] = -sn[i];
  }
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    const int g = part * kHeads + h;
    if (g >= g1) break;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (t && !q.c) break;
      float o[2][F];
      if (q.interleaved) {
#pragma unroll
        for (int i = 0; i < F; ++i) {
          const float a = v[h][t][2 * i / F].get(2 * i % F), b = v[h][t][2 * i / F].get(2 * i % F + 1);
          o[2 * i / F][2 * i % F] = a * cs[i] - b * sn[i];
          o[2 * i / F][2 * i % F + 1] = a * sn[i] + b * cs[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < F; ++i) {
          const float a = v[h][t][0].get(i), b = v[h][t][1].get(i);
          o[0][i] = a * cs[i] - b * sn[i];
          o[1][i] = a * sn[i] + b * cs[i];
        }
      }
      IO* to = (IO*)(t ? q.oc : q.ob) + (row * q.G + g) * q.N;
      store_vec<IO, F>(to + p0, o[0], q.stream);
      store_vec<IO, F>(to + p1, o[1], q.stream);
    }
  }
}

}  // namespace

bool rotate_fits(const RotArgs& a) {
  return double(a.rows) * (a.nf / 4 + (a.N - 2 * a.nf) / 8) * ((a.G + kHeads - 1) / kHeads) + 256 <
         4294967296.0;
}

hipError_t launch_rotate(const RotArgs& given, hipStream_t s) {
  RotArgs a = given;
  a.stream = past_caches((double)a.rows * a.G * a.N * (a.io == kIoBf16 ? 2 : 4));
  auto run = [&](auto io, auto freqs) {
    using IO = decltype(io);
    constexpr int F = decltype(freqs)::value;
    const int units = a.nf / F + (a.N - 2 * a.nf) / 8, splits = (a.G + kHeads - 1) / kHeads;
    const int64_t n = a.rows * units * splits;
    hipLaunchKernelGGL((k_rotate<IO, F>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, a, units,
                       splits);
    return hipGetLastError();
  };
  // 16 bytes a load where the frequencies are a multiple of 8 (fp32: always)
  if (a.io == kIoF32) return run(float{}, std::integral_constant<int, 4>{});
  if (a.nf % 8) return run(u16{}, std::integral_constant<int, 4>{});
  return run(u16{}, std::integral_constant<int, 8>{});
}

}  // namespace ssd
