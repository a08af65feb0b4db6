// Launchers of the operators of layers of linear recurrence (library-internal). Every launcher
// assumes the host checks of ssd_recurrent_api.cpp have passed.
#pragma once
#include "ssd_block.h"

namespace ssd {

// Whether outputs of so many bytes are written past the caches: from a quarter of the last-level cache on,
// so that what a call reads twice stays there instead. What reads the outputs next then takes them from
// memory, which costs less than it gains but for the smallest of them: the recurrence's backward of 2 x 4096
// x 5120 bf16 196 us for 217, with the convolution's behind it 266 for 279; the recurrence of 2 x 8192 x 5120
// with the heads' norm behind it 224 for 229, of 2 x 4096 118 for 115; the group norm of 2 x 8192 x 2560 52
// for 53, with a residual norm behind it 114 for 109.
inline bool past_caches(double bytes) { return bytes > 67108864.; }

// ---- gated linear recurrence ---------------------------------------------------------------------
struct RecArgs {
  Rows rows;
  int C, io;
  const void *x, *g, *gi;  // gi null: no input gate
  int64_t xs, gs, is;
  const float* decay;  // null: the gate is the decay
  float sharp;
  const float* h0;
  int stream = 0;  // outputs are written past the caches
};
struct RecGrads {
  void *dx, *dg, *dgi;
  float *ddecay, *dh0;
};

bool recurrence_fits(const RecArgs& a);  // whether its launches do
int64_t recurrence_bytes(const RecArgs& a);
hipError_t launch_recurrence(const RecArgs& a, void* y, float* fin, float* ws, hipStream_t s);
hipError_t launch_recurrence_step(const RecArgs& a, float* state_out, void* y, hipStream_t s);
int64_t recurrence_backward_bytes(const RecArgs& a);
hipError_t launch_recurrence_backward(const RecArgs& a, const void* dy, const float* dfinal,
                                      const RecGrads& g, float* ws, hipStream_t s);

// ---- rotation of B and C -------------------------------------------------------------------------
struct RotArgs {
  int64_t rows;
  int G, N, nf, axes;  // heads, entries of each, frequencies (two entries each), axes
  int ends[4];         // frequencies up to ends[i] go by axis i
  int io, interleaved, inverse;
  const int* pos;  // [axes, rows]
  const float* freq;
  const void *b, *c;  // c null: b alone
  int64_t bs, cs;
  void *ob, *oc;
  int stream = 0;  // turned entries are written past the caches
};
bool rotate_fits(const RotArgs& a);
hipError_t launch_rotate(const RotArgs& a, hipStream_t s);

// ---- group norm ------------------------------------------------------------------------------------
struct GroupArgs {
  Rows rows;
  int C, G, io, act;
  float eps;
  const void* x;
  int64_t xs;
  const float *w, *b;  // null: 1, 0
  int stream = 0;      // outputs are written past the caches
};
bool group_norm_fits(const GroupArgs& a);  // whether its launches do
int64_t group_norm_bytes(const GroupArgs& a);
hipError_t launch_group_norm(const GroupArgs& a, void* y, float* stats, float* ws,
                             hipStream_t s);
int64_t group_norm_backward_bytes(const GroupArgs& a);
hipError_t launch_group_norm_backward(const GroupArgs& a, const float* stats, const void* dy, void* dx,
                                      float* dw, float* db, float* ws, hipStream_t s);

}  // namespace ssd
