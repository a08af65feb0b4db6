// Rotation of B and C by positions: entries (p, q) of frequency j become
//   (p cos t - q sin t, p sin t + q cos t),   t = position[axis of j] * frequency[j].
//
// A few operations for each element read and written once: bound by memory. A thread takes some
// frequencies of a token, forms their sines and cosines once and turns the entries of up to kHeads heads,
// of B and of C. Every load and store is 16 bytes where the sizes allow it and neighbours take neighbouring
// ones: in halves that is two vectors of eight (fp32: four) frequencies each, in pairs one vector of four
// (two). The angle is formed in 64 bits: position times frequency is exact there up to 2^29 positions
// (29 and 24 bits), rounded to 53 bits beyond, and so is its product with 2 / pi, itself rounded: what a far
// position leaves of a turn is off by a few 2^-53 of the whole angle.
//
// B and C of 2 x 16384 x 8 x 256 bf16: 94 us (5.7 TB/s) in halves, 91 in pairs (with two vectors a thread
// there, whose stores leave every other 16 bytes to the next, 146; fp32 181, then 317).
#include "ssd_recurrent.h"
#include "ssd_rows.h"

namespace ssd {

namespace {

constexpr int kHeads = 4;  // of a thread, at most; their loads are issued together

// F frequencies a thread. PAIRS: entries 2 j and 2 j + 1 turn together, else j and nf + j.
template <typename IO, int F, bool PAIRS>
__global__ __launch_bounds__(256) void k_rotate(RotArgs q, int units, int splits) {
  constexpr int K = PAIRS ? 1 : 2, M = 2 * F / K;  // vectors of a head, their entries
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
  const int at[2] = {PAIRS ? 2 * j0 : j0, q.nf + j0};
  Vec<IO, M> v[kHeads][2][K];
#pragma unroll
  for (int h = 0; h < kHeads; ++h) {
    const int g = part * kHeads + h;
    if (g < g1) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        v[h][0][k].load((const IO*)q.b + row * q.bs + g * q.N + at[k]);
        if (q.c) v[h][1][k].load((const IO*)q.c + row * q.cs + g * q.N + at[k]);
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
    const int p = j < q.ends[0] ? pos[0] : j < q.ends[1] ? pos[1] : j < q.ends[2] ? pos[2] : pos[3];
    const double quarters = (double)p * (double)freq[i] * 0.63661977236758134;  // 2 / pi
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
      float o[K][M];
#pragma unroll
      for (int i = 0; i < F; ++i) {
        const int i0 = PAIRS ? 2 * i : i, i1 = PAIRS ? 2 * i + 1 : i;
        const float a = v[h][t][0].get(i0), b = v[h][t][K - 1].get(i1);
        o[0][i0] = a * cs[i] - b * sn[i];
        o[K - 1][i1] = a * sn[i] + b * cs[i];
      }
      IO* to = (IO*)(t ? q.oc : q.ob) + (row * q.G + g) * q.N;
#pragma unroll
      for (int k = 0; k < K; ++k) store_vec<IO, M>(to + at[k], o[k], q.stream);
    }
  }
}

}  // namespace

bool rotate_fits(const RotArgs& a) {
  const int least = a.interleaved && a.io == kIoF32 ? 2 : 4;  // frequencies of a thread
  return double(a.rows) * (a.nf / least + (a.N - 2 * a.nf) / 8) * ((a.G + kHeads - 1) / kHeads) + 256 <
         4294967296.0;
}

hipError_t launch_rotate(const RotArgs& given, hipStream_t s) {
  RotArgs a = given;
  a.stream = past_caches((double)a.rows * a.G * a.N * (a.io == kIoBf16 ? 2 : 4));
  auto run = [&](auto io, auto freqs, auto pairs) {
    using IO = decltype(io);
    constexpr int F = decltype(freqs)::value;
    const int units = a.nf / F + (a.N - 2 * a.nf) / 8, splits = (a.G + kHeads - 1) / kHeads;
    const int64_t n = a.rows * units * splits;
    hipLaunchKernelGGL((k_rotate<IO, F, decltype(pairs)::value>), dim3((unsigned)((n + 255) / 256)),
                       dim3(256), 0, s, a, units, splits);
    return hipGetLastError();
  };
  const std::integral_constant<int, 2> two;
  const std::integral_constant<int, 4> four;
  const std::integral_constant<int, 8> eight;
  // 16 bytes a load, but for bf16 in halves where the frequencies are no multiple of 8
  if (a.interleaved)
    return a.io == kIoF32 ? run(float{}, two, std::true_type{}) : run(u16{}, four, std::true_type{});
  if (a.io == kIoF32) return run(float{}, four, std::false_type{});
  return a.nf % 8 ? run(u16{}, four, std::false_type{}) : run(u16{}, eight, std::false_type{});
}

}  // namespace ssd
