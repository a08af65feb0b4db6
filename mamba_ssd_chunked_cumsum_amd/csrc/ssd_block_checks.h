// Host-side checks shared by the operators that work on token rows. Library-internal.
#pragma once
#include <cstdint>

#include "ssd_block.h"
#include "ssd_checks.h"

namespace ssd {

constexpr int64_t kMaxChannels = int64_t(1) << 20;
// Bytes of any tensor: 64-bit offsets reach further, memory does not.
constexpr double kMaxBytes = 4398046511104.0;

inline int64_t bytes_of(int32_t dtype) { return dtype == SSD_DTYPE_BF16 ? 2 : 4; }

inline bool is_dtype(int32_t d) { return d == SSD_DTYPE_F32 || d == SSD_DTYPE_BF16; }

inline ssd_status check_tokens(const ssd_tokens* t, bool sequences) {
  if (!t) return SSD_ERR_INVALID_ARGUMENT;
  if (t->batch <= 0 || t->seqlen <= 0 || t->channels <= 0 || t->reserved != 0 ||
      !is_dtype(t->io_dtype))
    return SSD_ERR_INVALID_ARGUMENT;
  if (t->seq_starts) {
    if (!sequences || t->batch != 1 || t->nseq <= 0) return SSD_ERR_INVALID_ARGUMENT;
  } else if (sequences && t->nseq != t->batch) {
    return SSD_ERR_INVALID_ARGUMENT;
  }
  if (t->channels % 8 || t->channels > kMaxChannels) return SSD_ERR_UNSUPPORTED;
  // one row below 2^31, so that a row index one past the last is an int too; the kernels add up
  // to a tile of rows to it
  if (double(t->batch) * double(t->seqlen) > double(kMaxIndex - 4096) || t->nseq > kMaxIndex - 4096)
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

inline int64_t rows_of(const ssd_tokens* t) { return t->batch * t->seqlen; }

// Effective row stride: 0 means dense. Negative where it is not acceptable.
inline int64_t stride_of(int64_t given, int64_t width, int64_t multiple = 8) {
  if (given == 0) return width;
  return given >= width && given % multiple == 0 && given < (int64_t(1) << 32) ? given : -1;
}

// Bytes of `rows` rows of `width` elements at `stride`.
inline int64_t span(int64_t rows, int64_t width, int64_t stride, int64_t e) {
  return ((rows - 1) * stride + width) * e;
}

inline Rows make_rows(const ssd_tokens* t) {
  return Rows{(int)rows_of(t), (int)t->seqlen, (int)(t->seq_starts ? t->nseq : t->batch),
                   t->seq_starts};
}

// The buffers of a call: alignment, and no output on an input or another output.
struct Buffers {
  enum { kMost = 32 };
  Range in[kMost], out[kMost];
  int n_in = 0, n_out = 0;
  bool ok = true;
  void input(const void* p, int64_t bytes, uintptr_t align = 16) {
    if (!p) return;
    ok = ok && reinterpret_cast<uintptr_t>(p) % align == 0;
    in[n_in++] = range_of(p, bytes);
  }
  void output(const void* p, int64_t bytes) {
    if (!p) return;
    ok = ok && aligned16(p);
    out[n_out++] = range_of(p, bytes);
  }
  bool fine() const {
    if (!ok) return false;
    for (int i = 0; i < n_out; ++i) {
      for (int j = 0; j < n_in; ++j)
        if (overlap(out[i], in[j])) return false;
      for (int j = 0; j < i; ++j)
        if (overlap(out[i], out[j])) return false;
    }
    return true;
  }
};

inline int64_t starts_bytes(const ssd_tokens* t) { return (t->nseq + 1) * 4; }

inline void starts_input(Buffers& b, const ssd_tokens* t) {
  b.input(t->seq_starts, starts_bytes(t), 4);
}

// Blocks of a launch: HIP counts a grid's threads in 32 bits.
inline bool grid_fits(double blocks, int threads) { return blocks * threads < 4294967296.0; }

inline ssd_status with_workspace(const void* ws, int64_t have, int64_t need) {
  if (need > 0 && (!ws || have < need || !aligned16(ws))) return SSD_ERR_INVALID_ARGUMENT;
  return SSD_OK;
}

}  // namespace ssd
