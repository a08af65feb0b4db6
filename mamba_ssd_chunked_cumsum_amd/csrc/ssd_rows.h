// Device helpers of the operators around the scan: sequences of token rows, vectors of channels,
// activations. Library-internal.
#pragma once
#include "ssd_block.h"
#include "ssd_device.h"

namespace ssd {

// Bounds of sequence s. Packed offsets are clamped to the rows, so that offsets that break the
// contract cannot move an access outside a tensor.
__device__ __forceinline__ int seq_begin(const Rows& q, int s) {
  return q.starts ? min(max(q.starts[s], 0), q.R) : s * q.L;
}
__device__ __forceinline__ int seq_end(const Rows& q, int s) {
  return q.starts ? min(max(q.starts[s + 1], 0), q.R) : (s + 1) * q.L;
}

// The sequence that holds row r (the last one that begins at or before it), -1 if none does.
__device__ __forceinline__ int seq_of(const Rows& q, int r) {
  if (!q.starts) return r / q.L;
  int lo = 0, hi = q.S;  // starts[lo] <= r < starts[hi], taking starts[S] as beyond
  if (q.starts[0] > r) return -1;
  while (hi - lo > 1) {
    const int m = lo + ((hi - lo) >> 1);  // (the sum may pass 31 bits)
    if (q.starts[m] <= r) lo = m; else hi = m;
  }
  return r < seq_end(q, lo) ? lo : -1;
}

// Where to go on from row r of no sequence: only rows before the first sequence and behind the last
// are in none.
__device__ __forceinline__ int after_gap(const Rows& q, int r) {
  return r < seq_begin(q, 0) ? seq_begin(q, 0) : q.R;
}

// ---- vectors of V consecutive channels (16-byte aligned for V = 8, 8-byte for bf16 V = 4) -------
template <typename IO, int V>
struct Vec {
  static constexpr int kWords = V * (int)sizeof(IO) / 4;
  uint32_t u[kWords];
  __device__ __forceinline__ void load(const IO* p) {
    if constexpr (kWords % 4 == 0) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 r = reinterpret_cast<const uint4*>(p)[i];
        u[4 * i] = r.x; u[4 * i + 1] = r.y; u[4 * i + 2] = r.z; u[4 * i + 3] = r.w;
      }
    } else {
      static_assert(kWords == 2, "vector of 8 or a multiple of 16 bytes");
      const uint2 r = *reinterpret_cast<const uint2*>(p);
      u[0] = r.x; u[1] = r.y;
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) u[i] = 0;
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(IO) == 4) return __uint_as_float(u[i]);
    else return __uint_as_float(i & 1 ? u[i / 2] & 0xffff0000u : u[i / 2] << 16);
  }
  __device__ __forceinline__ void get(float (&v)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = get(i);
  }
};

// Two floats rounded to bf16 (nearest even, NaN kept), the first in the low half. The hardware
// conversion instruction of gfx950.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  typedef float f2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, bf2));
}

// One value, rounded as pack_bf16 does.
__device__ __forceinline__ void store_io(float* p, int i, float v) { p[i] = v; }
__device__ __forceinline__ void store_io(u16* p, int i, float v) { p[i] = (u16)pack_bf16(v, v); }

// stream: past the caches, for outputs far larger than they are.
template <typename IO, int V>
__device__ __forceinline__ void store_vec(IO* p, const float (&v)[V], bool stream = false) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  uint32_t u[Vec<IO, V>::kWords];
  if constexpr (sizeof(IO) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] = __float_as_uint(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) u[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  }
  if constexpr (Vec<IO, V>::kWords % 4 == 0) {
#pragma unroll
    for (int i = 0; i < Vec<IO, V>::kWords / 4; ++i) {
      const u32x4 w = {u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]};
      if (stream) __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(p) + i);
      else reinterpret_cast<u32x4*>(p)[i] = w;
    }
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
  }
}

template <int V>
__device__ __forceinline__ void load_f32(const float* p, float (&v)[V]) {
  Vec<float, V> r;
  r.load(p);
  r.get(v);
}

// ---- activations -----------------------------------------------------------------------------
constexpr float kLog2e = 1.4426950408889634f;

// 1 / (1 + exp(-v)): exp overflows to infinity, whose reciprocal is 0, so every v is covered.
__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-v * kLog2e));
}

// log(1 + exp(v)) = max(v, 0) + log(1 + e), e = exp(-|v|) <= 1. With w = 1 + e rounded, what the
// rounding lost, e - (w - 1), is exact, and log(1 + e) = log(w) + that / w; the 1 / w is left out:
// where it is not near 1 the whole term is below the result's last place. (Measured against
// double over [-24, 24]: at most 6e-7 relative above -8, 1.7e-6 at -24, from the argument of exp.)
__device__ __forceinline__ float softplus(float v) {
  const float e = __builtin_amdgcn_exp2f(-fabsf(v) * kLog2e), w = 1.f + e;
  return fmaxf(v, 0.f) + fmaf(__builtin_amdgcn_logf(w), 0.6931471805599453f, e - (w - 1.f));
}

}  // namespace ssd
