// What the selective scan's forward and backward kernels share. Library-internal.
#pragma once
#include "ssd_rows.h"

namespace ssd {

// The hardware's exponential, one unit in the last place; arguments are products with log2(e).
__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// ---- a channel a lane, all its states in registers -------------------------------------------------
// B or C of a token: N state entries at p, uniform over the wave. NT: N rounded up to a template's
// size; entries past N read the last ones again (never past the row) and are set to zero.
template <typename IO, int NT, bool EXACT>
struct Row {
  static constexpr int kW = 4 * sizeof(IO) / 4;  // words of four entries
  uint32_t u[NT / 4][kW];
  __device__ __forceinline__ void load(const IO* p, int N) {
    typedef const __attribute__((address_space(4))) uint32_t* Words;  // read through scalar loads
#pragma unroll
    for (int i = 0; i < NT / 4; ++i) {
      const Words w = (Words)(uintptr_t)(p + (EXACT ? 4 * i : min(4 * i, N - 4)));
#pragma unroll
      for (int j = 0; j < kW; ++j) u[i][j] = w[j];
      if (!EXACT && 4 * i >= N) {
#pragma unroll
        for (int j = 0; j < kW; ++j) u[i][j] = 0;
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < NT / 4; ++i)
#pragma unroll
      for (int j = 0; j < kW; ++j) u[i][j] = 0;
  }
  __device__ __forceinline__ float get(int n) const {
    if constexpr (sizeof(IO) == 4) return __uint_as_float(u[n / 4][n % 4]);
    else return __uint_as_float(n & 1 ? u[n / 4][n % 4 / 2] & 0xffff0000u : u[n / 4][n % 4 / 2] << 16);
  }
};

template <typename IO>
__device__ __forceinline__ const char* row_at(const IO* p, int64_t elements) {
  return (const char*)(p + elements);
}

// One value as loaded, in a register of its own (two 16-bit values in one would make the second
// load wait for the first), and as a float.
template <typename IO>
__device__ __forceinline__ uint32_t load_raw(const char* row, unsigned off) {
  if constexpr (sizeof(IO) == 4) return *(const uint32_t*)(row + off);
  else return *(const u16*)(row + off);
}
template <typename IO>
__device__ __forceinline__ float raw_value(uint32_t v) {
  return __uint_as_float(sizeof(IO) == 4 ? v : v << 16);
}

template <int NT>
__device__ __forceinline__ void load_all(const float* p, int N, float (&h)[NT]) {
#pragma unroll
  for (int i = 0; i < NT; i += 4) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < N) v = *reinterpret_cast<const float4*>(p + i);
    h[i] = v.x; h[i + 1] = v.y; h[i + 2] = v.z; h[i + 3] = v.w;
  }
}
template <int NT>
__device__ __forceinline__ void store_all(float* p, int N, const float (&h)[NT]) {
#pragma unroll
  for (int i = 0; i < NT; i += 4)
    if (i < N) *reinterpret_cast<float4*>(p + i) = make_float4(h[i], h[i + 1], h[i + 2], h[i + 3]);
}

// ---- K lanes a channel -----------------------------------------------------------------------------
// A block of 256 threads takes 256 / K channels of one group and a range of rows; K lanes share a
// channel, each with NPL of its states (lane = K * channel + k, states k NPL .. k NPL + NPL - 1; past
// dstate they are zero: A = 0, B = 0).
constexpr int kSelThreads = 256;

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

// Starts and ends of sequences among the rows [r, r + 64), as bit masks of the wave, which rows are
// in a sequence, and in which (a row a lane: seq_at); rows at or past `stop` are in none.
__device__ __forceinline__ void mark_rows(const Rows& q, int r, int stop, uint64_t& starts,
                                          uint64_t& ends, uint64_t& inside, int& seq) {
  const int row = r + (threadIdx.x & 63);
  seq = row < stop ? seq_of(q, row) : -1;
  starts = __ballot(seq >= 0 && row == seq_begin(q, max(seq, 0)));
  ends = __ballot(seq >= 0 && row == seq_end(q, max(seq, 0)) - 1);
  inside = __ballot(seq >= 0);
}
__device__ __forceinline__ int seq_at(int seq, int t) { return __builtin_amdgcn_readlane(seq, t); }

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

// Template sizes of a lane that holds all N states: f(size, whether N is that size).
template <typename F>
hipError_t by_size(int N, F f) {
  using std::integral_constant;
  if (N == 16) return f(integral_constant<int, 16>{}, std::true_type{});
  if (N <= 8) return f(integral_constant<int, 8>{}, std::false_type{});
  if (N <= 16) return f(integral_constant<int, 16>{}, std::false_type{});
  if (N <= 32) return f(integral_constant<int, 32>{}, std::false_type{});
  return f(integral_constant<int, 64>{}, std::false_type{});
}

// Lanes a channel, four states each, for dstate N.
template <typename F>
hipError_t by_states(int N, F f) {
  if (N <= 16) return f(std::integral_constant<int, 4>{});
  if (N <= 32) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}

}  // namespace ssd
