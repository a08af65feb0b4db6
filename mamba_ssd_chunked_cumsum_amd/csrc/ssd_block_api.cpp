// C ABI of the operators around the scan: argument checks and launches. Every check runs on the
// host before the first HIP call, but for the selective scan's workspace, whose size depends on the
// device.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/ssd.h"
#include "ssd_block_checks.h"

namespace {

using namespace ssd;

// ---- convolution -----------------------------------------------------------------------------------

ssd_status conv_args(const ssd_tokens* t, const void* x, int64_t x_stride, const float* weight,
                     const float* bias, int32_t width, int32_t silu, const void* init,
                     const void* const y[3], const int64_t split[3], int64_t y_bytes, bool y_out,
                     ssd::ConvArgs* a, Buffers* b) {
  ssd_status st = check_tokens(t, true);
  if (st != SSD_OK) return st;
  if (!x || !weight || !y || !split) return SSD_ERR_INVALID_ARGUMENT;
  if (width <= 0) return SSD_ERR_INVALID_ARGUMENT;
  if (width < 2 || width > 4) return SSD_ERR_UNSUPPORTED;
  const int64_t C = t->channels, R = rows_of(t), e = bytes_of(t->io_dtype);
  const int64_t xs = stride_of(x_stride, C);
  if (xs < 0) return SSD_ERR_INVALID_ARGUMENT;
  if (double(R) * double(xs) * 4 > kMaxBytes || double(t->nseq) * 4 * C * 4 > kMaxBytes)
    return SSD_ERR_UNSUPPORTED;
  int64_t sum = 0;
  for (int i = 0; i < 3; ++i) {
    if (split[i] < 0 || split[i] % 8 || split[i] > C || (split[i] > 0) != (y[i] != nullptr))
      return SSD_ERR_INVALID_ARGUMENT;
    a->y.p[i] = const_cast<void*>(y[i]);
    a->y.first[i] = (int)sum;
    sum += split[i];
    const int64_t bytes = R * split[i] * y_bytes;
    if (y_out) b->output(y[i], bytes); else b->input(y[i], bytes);
  }
  if (sum != C) return SSD_ERR_INVALID_ARGUMENT;
  a->y.first[3] = (int)C;
  a->rows = make_rows(t);
  a->C = (int)C;
  a->W = width;
  a->io = t->io_dtype;
  a->silu = silu != 0;
  a->x = x;
  a->xs = xs;
  a->w = weight;
  a->bias = bias;
  a->init = init;
  b->input(x, span(R, C, xs, e));
  b->input(weight, C * width * 4);
  b->input(bias, C * 4);
  starts_input(*b, t);
  return SSD_OK;
}

int64_t conv_state_bytes(const ssd_tokens* t, int32_t width, int64_t e) {
  return t->nseq * (width - 1) * t->channels * e;
}

// ---- selective scan ----------------------------------------------------------------------------

ssd_status selective_args(const ssd_tokens* t, const ssd_selective* in, ssd::SelArgs* a,
                          Buffers* b) {
  ssd_status st = check_tokens(t, true);
  if (st != SSD_OK) return st;
  if (!in || in->reserved != 0 || in->dstate <= 0 || in->ngroups <= 0) return SSD_ERR_INVALID_ARGUMENT;
  const int64_t C = t->channels, N = in->dstate, G = in->ngroups, R = rows_of(t);
  if (C % G) return SSD_ERR_INVALID_ARGUMENT;
  if (C / G % 8 || N % 4 || N > 64) return SSD_ERR_UNSUPPORTED;
  if (!in->x || !in->dt || !in->A || !in->B || !in->C) return SSD_ERR_INVALID_ARGUMENT;
  const int64_t e = bytes_of(t->io_dtype);
  const int64_t xs = stride_of(in->x_stride, C), ts = stride_of(in->dt_stride, C),
                zs = stride_of(in->z_stride, C);
  // B and C are read four elements at a time
  const int64_t bs = stride_of(in->b_stride, G * N, 4), cs = stride_of(in->c_stride, G * N, 4);
  if (xs < 0 || ts < 0 || zs < 0 || bs < 0 || cs < 0) return SSD_ERR_INVALID_ARGUMENT;
  const int64_t widest = xs > ts ? (xs > zs ? xs : zs) : (ts > zs ? ts : zs);
  if (double(R) * double(widest) * 4 > kMaxBytes || double(R) * double(bs > cs ? bs : cs) * 4 > kMaxBytes ||
      double(t->nseq) * C * N * 4 > kMaxBytes)
    return SSD_ERR_UNSUPPORTED;
  *a = ssd::SelArgs{make_rows(t), (int)C, (int)N, (int)G, t->io_dtype, in->dt_softplus != 0,
                    in->x, in->dt, in->B, in->C, in->z, xs, ts, bs, cs, zs,
                    in->A, in->D, in->dt_bias, in->initial_state};
  b->input(in->x, span(R, C, xs, e));
  b->input(in->dt, span(R, C, ts, e));
  b->input(in->z, span(R, C, zs, e));
  b->input(in->B, span(R, G * N, bs, e), 4 * e);
  b->input(in->C, span(R, G * N, cs, e), 4 * e);
  b->input(in->A, C * N * 4);
  b->input(in->D, C * 4);
  b->input(in->dt_bias, C * 4);
  starts_input(*b, t);
  return SSD_OK;
}

int64_t sel_state_bytes(const ssd_tokens* t, const ssd_selective* in) {
  return t->nseq * t->channels * in->dstate * 4;
}

bool selective_grid_fits(const ssd::SelArgs& a) {
  const int width = a.N <= 16 ? 64 : a.N <= 32 ? 32 : 16;  // channels of the backward's tiles
  const double tiles = double(a.C) / width + a.G;
  const double units = double(a.rows.R) / 64 + a.rows.S + 1;
  return grid_fits(tiles * units, 256) && grid_fits(double(a.C) * a.N * a.rows.S / 256 + 1, 256) &&
         grid_fits(double(a.rows.R) * 2 * a.N * a.G / 256 + 1, 256);
}

int compute_units() {  // of the current device, asked for once
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 256;
  if (dev >= 0 && dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
    n = 256;
  if (dev >= 0 && dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// ---- norms ---------------------------------------------------------------------------------------

constexpr int64_t kMaxNorm = 8192;

ssd_status norm_args(const ssd_tokens* t, int64_t ngroups, float eps, const float* weight,
                     ssd::NormArgs* a) {
  ssd_status st = check_tokens(t, false);
  if (st != SSD_OK) return st;
  if (ngroups <= 0 || t->channels % ngroups || !(eps >= 0.f) || std::isinf(eps))
    return SSD_ERR_INVALID_ARGUMENT;
  const int64_t n = t->channels / ngroups;
  if (n % 8 || n > kMaxNorm) return SSD_ERR_UNSUPPORTED;
  if (!grid_fits(double(rows_of(t)) * ngroups, n <= 1024 ? 64 : 512)) return SSD_ERR_UNSUPPORTED;
  *a = ssd::NormArgs{(int)rows_of(t), (int)t->channels, (int)ngroups, t->io_dtype, eps, weight};
  return SSD_OK;
}

}  // namespace

extern "C" {

ssd_status ssd_conv(const ssd_tokens* t, const void* x, int64_t x_stride, const float* weight,
                    const float* bias, int32_t width, int32_t silu, const void* initial_state,
                    void* const y[3], const int64_t split[3], void* final_state, void* stream) {
  ssd::ConvArgs a;
  Buffers b;
  const int64_t e = t && is_dtype(t->io_dtype) ? bytes_of(t->io_dtype) : 4;
  ssd_status st = conv_args(t, x, x_stride, weight, bias, width, silu, initial_state, y, split, e,
                            true, &a, &b);
  if (st != SSD_OK) return st;
  b.input(initial_state, conv_state_bytes(t, width, e));
  b.output(final_state, conv_state_bytes(t, width, e));
  if (!b.fine()) return SSD_ERR_INVALID_ARGUMENT;
  if (!grid_fits((double(a.rows.R) / 8 + a.rows.S + 1) * (a.C / 8) / 256 + 1, 256))
    return SSD_ERR_UNSUPPORTED;
  st = device_ready();
  if (st != SSD_OK) return st;
  return from_hip(ssd::launch_conv(a, final_state, static_cast<hipStream_t>(stream)));
}

ssd_status ssd_conv_step(const ssd_tokens* t, const void* x, int64_t x_stride, const float* weight,
                         const float* bias, int32_t width, int32_t silu, const void* state_in,
                         void* state_out, void* const y[3], const int64_t split[3], void* stream) {
  ssd::ConvArgs a;
  Buffers b;
  const int64_t e = t && is_dtype(t->io_dtype) ? bytes_of(t->io_dtype) : 4;
  ssd_status st = conv_args(t, x, x_stride, weight, bias, width, silu, state_in, y, split, e, true,
                            &a, &b);
  if (st != SSD_OK) return st;
  if (t->seqlen != 1 || t->seq_starts || !state_in || !state_out) return SSD_ERR_INVALID_ARGUMENT;
  const int64_t n = conv_state_bytes(t, width, e);
  b.output(state_out, n);
  if (state_in == state_out) {  // in place: no overlap of its own
    if (!b.fine()) return SSD_ERR_INVALID_ARGUMENT;
  } else {
    b.input(state_in, n);
    if (!b.fine()) return SSD_ERR_INVALID_ARGUMENT;
  }
  if (!grid_fits(double(a.rows.R) * (a.C / 8) / 256 + 1, 256)) return SSD_ERR_UNSUPPORTED;
  st = device_ready();
  if (st != SSD_OK) return st;
  return from_hip(ssd::launch_conv_step(a, state_out, static_cast<hipStream_t>(stream)));
}

ssd_status ssd_conv_backward_workspace(const ssd_tokens* t, int32_t width, int64_t* bytes) {
  ssd_status st = check_tokens(t, true);
  if (st != SSD_OK) return st;
  if (!bytes || width <= 0) return SSD_ERR_INVALID_ARGUMENT;
  if (width < 2 || width > 4) return SSD_ERR_UNSUPPORTED;
  ssd::ConvArgs a{};
  a.rows = make_rows(t);
  a.C = (int)t->channels;
  a.W = width;
  *bytes = ssd::conv_backward_bytes(a);
  return SSD_OK;
}

ssd_status ssd_conv_backward(const ssd_tokens* t, const void* x, int64_t x_stride,
                             const float* weight, const float* bias, int32_t width, int32_t silu,
                             const void* initial_state, const void* const dy[3],
                             const int64_t split[3], int32_t dy_dtype, const float* dfinal,
                             void* dx, float* dweight, float* dbias, float* dinitial_state,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  ssd::ConvArgs a;
  Buffers b;
  if (!t) return SSD_ERR_INVALID_ARGUMENT;
  if (!is_dtype(dy_dtype) || (dy_dtype != SSD_DTYPE_F32 && dy_dtype != t->io_dtype))
    return SSD_ERR_INVALID_ARGUMENT;
  ssd_status st = conv_args(t, x, x_stride, weight, bias, width, silu, initial_state, dy, split,
                            bytes_of(dy_dtype), false, &a, &b);
  if (st != SSD_OK) return st;
  if (!dx || !dweight) return SSD_ERR_INVALID_ARGUMENT;
  const int64_t e = bytes_of(t->io_dtype), need = ssd::conv_backward_bytes(a);
  b.input(initial_state, conv_state_bytes(t, width, e));
  b.input(dfinal, conv_state_bytes(t, width, 4));
  b.output(dx, rows_of(t) * t->channels * e);
  b.output(dweight, t->channels * width * 4);
  b.output(dbias, t->channels * 4);
  b.output(dinitial_state, conv_state_bytes(t, width, 4));
  b.output(workspace, need);
  st = with_workspace(workspace, workspace_bytes, need);
  if (st != SSD_OK) return st;
  if (!b.fine()) return SSD_ERR_INVALID_ARGUMENT;
  if (!grid_fits((double(a.C) / 256 + 1) * (double(a.rows.R) / 512 + 1) + 1024 +
                     double(a.rows.S) * (a.C / 4) / 256 + 1, 256))
    return SSD_ERR_UNSUPPORTED;
  st = device_ready();
  if (st != SSD_OK) return st;
  return from_hip(ssd::launch_conv_backward(a, dy_dtype, dfinal, dx, dweight, dbias,
                                            dinitial_state, static_cast<float*>(workspace),
                                            static_cast<hipStream_t>(stream)));
}

ssd_status ssd_selective_scan_workspace(const ssd_tokens* t, const ssd_selective* in,
                                        int64_t* bytes) {
  ssd::SelArgs a;
  Buffers b;
  ssd_status st = selective_args(t, in, &a, &b);
  if (st != SSD_OK) return st;
  if (!bytes) return SSD_ERR_INVALID_ARGUMENT;
  st = device_ready();
  if (st != SSD_OK) return st;
  *bytes = ssd::selective_bytes(a, compute_units());
  return SSD_OK;
}

ssd_status ssd_selective_scan(const ssd_tokens* t, const ssd_selective* in, void* y,
                              float* final_state, void* workspace, int64_t workspace_bytes,
                              void* stream) {
  ssd::SelArgs a;
  Buffers b;
  ssd_status st = selective_args(t, in, &a, &b);
  if (st != SSD_OK) return st;
  if (!y) return SSD_ERR_INVALID_ARGUMENT;
  b.input(in->initial_state, sel_state_bytes(t, in));
  b.output(y, rows_of(t) * t->channels * bytes_of(t->io_dtype));
  b.output(final_state, sel_state_bytes(t, in));
  if (!b.fine()) return SSD_ERR_INVALID_ARGUMENT;
  if (!selective_grid_fits(a)) return SSD_ERR_UNSUPPORTED;
  st = device_ready();
  if (st != SSD_OK) return st;
  const int n_cu = compute_units();
  const int64_t need = ssd::selective_bytes(a, n_cu);
  st = with_workspace(workspace, workspace_bytes, need);
  if (st != SSD_OK) return st;
  if (need) {
    b.output(workspace, need);
    if (!b.fine()) return SSD_ERR_INVALID_ARGUMENT;
  }
  return from_hip(ssd::launch_selective(a, y, final_state, static_cast<float*>(workspace), n_cu,
                                        static_cast<hipStream_t>(stream)));
}

ssd_status ssd_selective_step(const ssd_tokens* t, const ssd_selective* in, float* state_out,
                              void* y, void* stream) {
  ssd::SelArgs a;
  Buffers b;
  ssd_status st = selective_args(t, in, &a, &b);
  if (st != SSD_OK) return st;
  if (t->seqlen != 1 || t->seq_starts || !in->initial_state || !state_out || !y)
    return SSD_ERR_INVALID_ARGUMENT;
  b.output(y, t->batch * t->channels * bytes_of(t->io_dtype));
  b.output(state_out, sel_state_bytes(t, in));
  if (in->initial_state != state_out) b.input(in->initial_state, sel_state_bytes(t, in));
  if (!b.fine()) return SSD_ERR_INVALID_ARGUMENT;
  if (!grid_fits(double(a.rows.R) * a.C * 16 / 256 + 1, 256)) return SSD_ERR_UNSUPPORTED;
  st = device_ready();
  if (st != SSD_OK) return st;
  return from_hip(ssd::launch_selective_step(a, state_out, y, static_cast<hipStream_t>(stream)));
}

ssd_status ssd_selective_backward_workspace(const ssd_tokens* t, const ssd_selective* in,
                                            int64_t* bytes) {
  ssd::SelArgs a;
  Buffers b;
  ssd_status st = selective_args(t, in, &a, &b);
  if (st != SSD_OK) return st;
  if (!bytes) return SSD_ERR_INVALID_ARGUMENT;
  *bytes = ssd::selective_backward_bytes(a);
  return SSD_OK;
}

ssd_status ssd_selective_backward(const ssd_tokens* t, const ssd_selective* in, const void* dy,
                                  const float* dfinal, const ssd_selective_grads* out,
                                  void* workspace, int64_t workspace_bytes, void* stream) {
  ssd::SelArgs a;
  Buffers b;
  ssd_status st = selective_args(t, in, &a, &b);
  if (st != SSD_OK) return st;
  if (!dy || !out || !out->dx || !out->ddt || !out->dB || !out->dC || !out->dA ||
      (in->z != nullptr) != (out->dz != nullptr))
    return SSD_ERR_INVALID_ARGUMENT;
  const int64_t R = rows_of(t), C = t->channels, N = in->dstate, e = bytes_of(t->io_dtype);
  const int64_t need = ssd::selective_backward_bytes(a);
  b.input(in->initial_state, sel_state_bytes(t, in));
  b.input(dy, R * C * e);
  b.input(dfinal, sel_state_bytes(t, in));
  b.output(out->dx, R * C * e);
  b.output(out->ddt, R * C * e);
  b.output(out->dz, R * C * e);
  b.output(out->dB, R * in->ngroups * N * e);
  b.output(out->dC, R * in->ngroups * N * e);
  b.output(out->dA, C * N * 4);
  b.output(out->dD, C * 4);
  b.output(out->ddt_bias, C * 4);
  b.output(out->dinitial_state, sel_state_bytes(t, in));
  b.output(workspace, need);
  st = with_workspace(workspace, workspace_bytes, need);
  if (st != SSD_OK) return st;
  if (!b.fine()) return SSD_ERR_INVALID_ARGUMENT;
  if (!selective_grid_fits(a)) return SSD_ERR_UNSUPPORTED;
  st = device_ready();
  if (st != SSD_OK) return st;
  const ssd::SelGrads g{out->dx, out->ddt, out->dz, out->dB, out->dC,
                        out->dA, out->dD, out->ddt_bias, out->dinitial_state};
  return from_hip(ssd::launch_selective_backward(a, dy, dfinal, g, static_cast<float*>(workspace),
                                                 compute_units(),
                                                 static_cast<hipStream_t>(stream)));
}

ssd_status ssd_gated_norm(const ssd_tokens* t, const void* x, int64_t x_stride, const void* z,
                          int64_t z_stride, const float* weight, int64_t ngroups, float eps,
                          int32_t norm_before_gate, void* y, void* stream) {
  ssd::NormArgs a;
  ssd_status st = norm_args(t, ngroups, eps, weight, &a);
  if (st != SSD_OK) return st;
  if (!x || !weight || !y) return SSD_ERR_INVALID_ARGUMENT;
  const int64_t R = rows_of(t), C = t->channels, e = bytes_of(t->io_dtype);
  const int64_t xs = stride_of(x_stride, C), zs = stride_of(z_stride, C);
  if (xs < 0 || zs < 0) return SSD_ERR_INVALID_ARGUMENT;
  Buffers b;
  b.input(x, span(R, C, xs, e));
  b.input(z, span(R, C, zs, e));
  b.input(weight, C * 4);
  b.output(y, R * C * e);
  if (!b.fine()) return SSD_ERR_INVALID_ARGUMENT;
  st = device_ready();
  if (st != SSD_OK) return st;
  return from_hip(ssd::launch_gated_norm(a, x, xs, z, zs, norm_before_gate != 0, y,
                                         static_cast<hipStream_t>(stream)));
}

ssd_status ssd_gated_norm_backward_workspace(const ssd_tokens* t, int64_t ngroups,
                                             int64_t* bytes) {
  ssd::NormArgs a;
  ssd_status st = norm_args(t, ngroups, 0.f, nullptr, &a);
  if (st != SSD_OK) return st;
  if (!bytes) return SSD_ERR_INVALID_ARGUMENT;
  *bytes = ssd::norm_backward_bytes(a, 1);
  return SSD_OK;
}

ssd_status ssd_gated_norm_backward(const ssd_tokens* t, const void* x, int64_t x_stride,
                                   const void* z, int64_t z_stride, const float* weight,
                                   int64_t ngroups, float eps, int32_t norm_before_gate,
                                   const void* dy, void* dx, void* dz, float* dweight,
                                   void* workspace, int64_t workspace_bytes, void* stream) {
  ssd::NormArgs a;
  ssd_status st = norm_args(t, ngroups, eps, weight, &a);
  if (st != SSD_OK) return st;
  if (!x || !weight || !dy || !dx || !dweight || (z != nullptr) != (dz != nullptr))
    return SSD_ERR_INVALID_ARGUMENT;
  const int64_t R = rows_of(t), C = t->channels, e = bytes_of(t->io_dtype);
  const int64_t xs = stride_of(x_stride, C), zs = stride_of(z_stride, C);
  if (xs < 0 || zs < 0) return SSD_ERR_INVALID_ARGUMENT;
  const int64_t need = ssd::norm_backward_bytes(a, 1);
  Buffers b;
  b.input(x, span(R, C, xs, e));
  b.input(z, span(R, C, zs, e));
  b.input(weight, C * 4);
  b.input(dy, R * C * e);
  b.output(dx, R * C * e);
  b.output(dz, R * C * e);
  b.output(dweight, C * 4);
  b.output(workspace, need);
  st = with_workspace(workspace, workspace_bytes, need);
  if (st != SSD_OK) return st;
  if (!b.fine()) return SSD_ERR_INVALID_ARGUMENT;
  st = device_ready();
  if (st != SSD_OK) return st;
  return from_hip(ssd::launch_gated_norm_backward(a, x, xs, z, zs, norm_before_gate != 0, dy, dx,
                                                  dz, dweight, static_cast<float*>(workspace),
                                                  static_cast<hipStream_t>(stream)));
}

ssd_status ssd_residual_norm(const ssd_tokens* t, const void* x, int64_t x_stride,
                             const void* residual, int32_t res_dtype, const float* scale,
                             const float* weight, float eps, void* y, void* residual_out,
                             void* stream) {
  ssd::NormArgs a;
  ssd_status st = norm_args(t, 1, eps, weight, &a);
  if (st != SSD_OK) return st;
  if (!x || !weight || !y || !residual_out || !is_dtype(res_dtype) ||
      (res_dtype != SSD_DTYPE_F32 && res_dtype != t->io_dtype))
    return SSD_ERR_INVALID_ARGUMENT;
  const int64_t R = rows_of(t), C = t->channels, e = bytes_of(t->io_dtype), re = bytes_of(res_dtype);
  const int64_t xs = stride_of(x_stride, C);
  if (xs < 0) return SSD_ERR_INVALID_ARGUMENT;
  Buffers b;
  b.input(x, span(R, C, xs, e));
  b.input(residual, R * C * re);
  b.input(scale, C * 4);
  b.input(weight, C * 4);
  b.output(y, R * C * e);
  b.output(residual_out, R * C * re);
  if (!b.fine()) return SSD_ERR_INVALID_ARGUMENT;
  st = device_ready();
  if (st != SSD_OK) return st;
  return from_hip(ssd::launch_residual_norm(a, x, xs, residual, res_dtype, scale, y, residual_out,
                                            static_cast<hipStream_t>(stream)));
}

ssd_status ssd_residual_norm_backward_workspace(const ssd_tokens* t, int64_t* bytes) {
  ssd::NormArgs a;
  ssd_status st = norm_args(t, 1, 0.f, nullptr, &a);
  if (st != SSD_OK) return st;
  if (!bytes) return SSD_ERR_INVALID_ARGUMENT;
  *bytes = ssd::norm_backward_bytes(a, 2);
  return SSD_OK;
}

ssd_status ssd_residual_norm_backward(const ssd_tokens* t, const void* residual_sum,
                                      int32_t res_dtype, const void* x, int64_t x_stride,
                                      const float* scale, const float* weight, float eps,
                                      const void* dy, const void* dres, void* dx, void* dresidual,
                                      float* dweight, float* dscale, void* workspace,
                                      int64_t workspace_bytes, void* stream) {
  ssd::NormArgs a;
  ssd_status st = norm_args(t, 1, eps, weight, &a);
  if (st != SSD_OK) return st;
  if (!residual_sum || !weight || !dy || !dx || !dweight || !is_dtype(res_dtype) ||
      (res_dtype != SSD_DTYPE_F32 && res_dtype != t->io_dtype) || (scale && !x) ||
      (scale != nullptr) != (dscale != nullptr))
    return SSD_ERR_INVALID_ARGUMENT;
  if (!scale) {  // x is not read, so nothing about it matters
    x = nullptr;
    x_stride = 0;
  }
  const int64_t R = rows_of(t), C = t->channels, e = bytes_of(t->io_dtype), re = bytes_of(res_dtype);
  const int64_t xs = stride_of(x_stride, C), need = ssd::norm_backward_bytes(a, scale ? 2 : 1);
  if (xs < 0) return SSD_ERR_INVALID_ARGUMENT;
  Buffers b;
  b.input(residual_sum, R * C * re);
  b.input(x, span(R, C, xs, e));
  b.input(scale, C * 4);
  b.input(weight, C * 4);
  b.input(dy, R * C * e);
  b.input(dres, R * C * re);
  b.output(dx, R * C * e);
  b.output(dresidual, R * C * re);
  b.output(dweight, C * 4);
  b.output(dscale, C * 4);
  b.output(workspace, need);
  st = with_workspace(workspace, workspace_bytes, need);
  if (st != SSD_OK) return st;
  if (!b.fine()) return SSD_ERR_INVALID_ARGUMENT;
  st = device_ready();
  if (st != SSD_OK) return st;
  return from_hip(ssd::launch_residual_norm_backward(a, residual_sum, res_dtype, x, xs, scale, dy,
                                                     dres, dx, dresidual, dweight, dscale,
                                                     static_cast<float*>(workspace),
                                                     static_cast<hipStream_t>(stream)));
}

}  // extern "C"
