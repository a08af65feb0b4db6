// Launchers of the operators around the scan (library-internal). Every launcher assumes the host
// checks of ssd_block_api.cpp have passed.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssd {

// Token rows and their sequences: rows [s L, (s + 1) L) of sequence s (starts null), or
// [starts[s], starts[s + 1]).
struct Rows {
  int R, L, S;
  const int* starts;
};

// The channels of an activation in up to three dense tensors; channel c of [first[i], first[i + 1])
// is in tensor i at column c - first[i].
struct Split {
  void* p[3];
  int first[4];
};

struct ConvArgs {
  Rows rows;
  int C, W, io, silu;
  const void* x;
  int64_t xs;
  const float *w, *bias;
  const void* init;
  Split y;  // forward: outputs; backward: their gradients
  int stream = 0;  // forward: outputs are written past the caches
};

hipError_t launch_conv(const ConvArgs& a, void* fin, hipStream_t s);
hipError_t launch_conv_step(const ConvArgs& a, void* state_out, hipStream_t s);
int64_t conv_backward_bytes(const ConvArgs& a);
hipError_t launch_conv_backward(const ConvArgs& a, int dy_io, const float* dfinal, void* dx,
                                float* dw, float* db, float* dinit, float* ws, hipStream_t s);

struct SelArgs {
  Rows rows;
  int C, N, G, io, softplus;
  const void *x, *dt, *B, *Cm, *z;
  int64_t xs, dts, bs, cs, zs;
  const float *A, *D, *dt_bias, *h0;
};
struct SelGrads {
  void *dx, *ddt, *dz, *dB, *dC;
  float *dA, *dD, *ddtb, *dh0;
};

int64_t selective_bytes(const SelArgs& a, int n_cu);
hipError_t launch_selective(const SelArgs& a, void* y, float* fin, float* ws, int n_cu,
                            hipStream_t s);
hipError_t launch_selective_step(const SelArgs& a, float* state_out, void* y, hipStream_t s);
int64_t selective_backward_bytes(const SelArgs& a);
hipError_t launch_selective_backward(const SelArgs& a, const void* dy, const float* dfinal,
                                     const SelGrads& g, float* ws, int n_cu, hipStream_t s);

struct NormArgs {
  int R, C, G, io;  // rows, channels, groups (each normalised by itself)
  float eps;
  const float* w;
};
hipError_t launch_gated_norm(const NormArgs& a, const void* x, int64_t xs, const void* z,
                             int64_t zs, int before, void* y, hipStream_t s);
int64_t norm_backward_bytes(const NormArgs& a, int sums);
hipError_t launch_gated_norm_backward(const NormArgs& a, const void* x, int64_t xs, const void* z,
                                      int64_t zs, int before, const void* dy, void* dx, void* dz,
                                      float* dw, float* ws, hipStream_t s);
hipError_t launch_residual_norm(const NormArgs& a, const void* x, int64_t xs, const void* res,
                                int res_io, const float* scale, void* y, void* res_out,
                                hipStream_t s);
hipError_t launch_residual_norm_backward(const NormArgs& a, const void* r, int res_io,
                                         const void* x, int64_t xs, const float* scale,
                                         const void* dy, const void* dres, void* dx, void* dresid,
                                         float* dw, float* dscale, float* ws, hipStream_t s);

// Column sums of partial results part [n, M1 + M2 + M3] in a fixed order: column m < M1 to
// out1[(m / inner) * so + (m % inner) * si], the next M2 to out2, the last M3 to out3 (each of
// those two dropped where null).
hipError_t launch_column_sums(const float* part, int n, int64_t M1, float* out1, int inner,
                              int64_t so, int64_t si, int64_t M2, float* out2, int64_t M3,
                              float* out3, hipStream_t s);

}  // namespace ssd
