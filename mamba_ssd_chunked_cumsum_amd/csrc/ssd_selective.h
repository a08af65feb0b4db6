// What the selective scan's forward and backward kernels share. Library-internal.
#pragma once
#include "ssd_rows.h"

namespace ssd {

// ---- work split ----------------------------------------------------------------------------------
// A block of 256 threads takes kCh channels of one group and a range of rows. K lanes share a
// channel, each with NPL of its states (lane = K * channel + k, states k NPL .. k NPL + NPL - 1;
// past dstate they are zero: A = 0, B = 0).
constexpr int kSelThreads = 256;

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// Sum over the K (4, 8 or 16) lanes that share a channel, in every one of them.
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(
                 __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int K>
__device__ __forceinline__ float sum_lanes(float v) {
  v = add_dpp<0xB1>(v);                      // quad_perm [1,0,3,2]
  v = add_dpp<0x4E>(v);                      // quad_perm [2,3,0,1]
  if constexpr (K >= 8) v = add_dpp<0x141>(v);   // row_half_mirror
  if constexpr (K >= 16) v = add_dpp<0x140>(v);  // row_mirror
  return v;
}

// Starts and ends of sequences among the rows [r, r + 64) of a wave, as bit masks; rows at or past
// `stop` count as neither.
__device__ __forceinline__ void mark_rows(const Rows& q, int r, int stop, uint64_t& starts,
                                          uint64_t& ends, uint64_t& inside) {
  const int row = r + (threadIdx.x & 63);
  bool st = false, en = false, in = false;
  if (row < stop) {
    const int s = seq_of(q, row);
    if (s >= 0) {
      in = true;
      st = row == seq_begin(q, s);
      en = row == seq_end(q, s) - 1;
    }
  }
  starts = __ballot(st);
  ends = __ballot(en);
  inside = __ballot(in);
}

template <int NPL>
__device__ __forceinline__ void load_states(const float* p, int k, int N, float (&h)[NPL]) {
#pragma unroll
  for (int j = 0; j < NPL; j += 4) {
    const int n = k * NPL + j;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (n < N) v = *reinterpret_cast<const float4*>(p + n);
    h[j] = v.x; h[j + 1] = v.y; h[j + 2] = v.z; h[j + 3] = v.w;
  }
}
template <int NPL>
__device__ __forceinline__ void store_states(float* p, int k, int N, const float (&h)[NPL]) {
#pragma unroll
  for (int j = 0; j < NPL; j += 4) {
    const int n = k * NPL + j;
    if (n < N) *reinterpret_cast<float4*>(p + n) = make_float4(h[j], h[j + 1], h[j + 2], h[j + 3]);
  }
}

// Lanes a channel, four states each, for dstate N.
template <typename F>
hipError_t by_states(int N, F f) {
  if (N <= 16) return f(std::integral_constant<int, 4>{});
  if (N <= 32) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}

}  // namespace ssd
