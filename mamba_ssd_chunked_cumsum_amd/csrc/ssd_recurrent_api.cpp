// C ABI of the operators of layers of linear recurrence: argument checks and launches. Every check
// runs on the host before the first HIP call.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/ssd.h"
#include "ssd_block_checks.h"
#include "ssd_recurrent.h"

namespace {

using namespace ssd;

// ---- recurrence ------------------------------------------------------------------------------------

ssd_status recurrence_args(const ssd_tokens* t, const ssd_recurrent* in, RecArgs* a, Buffers* b) {
  ssd_status st = check_tokens(t, true);
  if (st != SSD_OK) return st;
  if (!in || in->reserved != 0 || !in->x || !in->gate) return SSD_ERR_INVALID_ARGUMENT;
  if (in->decay && (!(in->sharpness > 0.f) || std::isinf(in->sharpness)))
    return SSD_ERR_INVALID_ARGUMENT;
  const int64_t C = t->channels, R = rows_of(t), e = bytes_of(t->io_dtype);
  const int64_t xs = stride_of(in->x_stride, C), gs = stride_of(in->gate_stride, C),
                is = stride_of(in->input_gate_stride, C);
  if (xs < 0 || gs < 0 || is < 0) return SSD_ERR_INVALID_ARGUMENT;
  const int64_t widest = xs > gs ? (xs > is ? xs : is) : (gs > is ? gs : is);
  if (double(R) * double(widest) * 4 > kMaxBytes || double(t->nseq) * double(C) * 4 > kMaxBytes)
    return SSD_ERR_UNSUPPORTED;
  *a = RecArgs{make_rows(t), (int)C, t->io_dtype, in->x, in->gate, in->input_gate, xs, gs, is,
               in->decay, in->sharpness, in->initial_state};
  if (!recurrence_fits(*a)) return SSD_ERR_UNSUPPORTED;
  b->input(in->x, span(R, C, xs, e));
  b->input(in->gate, span(R, C, gs, e));
  b->input(in->input_gate, span(R, C, is, e));
  b->input(in->decay, C * 4);
  starts_input(*b, t);
  return SSD_OK;
}

int64_t state_bytes(const ssd_tokens* t) { return t->nseq * t->channels * 4; }

// The workspace as one more output.
ssd_status take_workspace(Buffers* b, void* workspace, int64_t have, int64_t need) {
  const ssd_status st = with_workspace(workspace, have, need);
  if (st != SSD_OK || !need) return st;
  b->output(workspace, need);
  return b->fine() ? SSD_OK : SSD_ERR_INVALID_ARGUMENT;
}

// ---- group norm ------------------------------------------------------------------------------------

ssd_status group_args(const ssd_tokens* t, const void* x, int64_t x_stride, const float* weight,
                      const float* bias, int64_t ngroups, float eps, int32_t silu, GroupArgs* a,
                      Buffers* b) {
  ssd_status st = check_tokens(t, true);
  if (st != SSD_OK) return st;
  if (ngroups <= 0 || t->channels % ngroups || !(eps >= 0.f) || std::isinf(eps))
    return SSD_ERR_INVALID_ARGUMENT;
  const int64_t C = t->channels, R = rows_of(t), xs = stride_of(x_stride, C);
  if (xs < 0) return SSD_ERR_INVALID_ARGUMENT;
  if (double(R) * double(xs) * 4 > kMaxBytes) return SSD_ERR_UNSUPPORTED;
  *a = GroupArgs{make_rows(t), (int)C, (int)ngroups, t->io_dtype, silu != 0, eps, x, xs, weight, bias};
  if (!group_norm_fits(*a)) return SSD_ERR_UNSUPPORTED;
  b->input(x, span(R, C, xs, bytes_of(t->io_dtype)));
  b->input(weight, C * 4);
  b->input(bias, C * 4);
  starts_input(*b, t);
  return SSD_OK;
}

}  // namespace

extern "C" {

ssd_status ssd_recurrence_workspace(const ssd_tokens* t, const ssd_recurrent* in, int64_t* bytes) {
  RecArgs a;
  Buffers b;
  ssd_status st = recurrence_args(t, in, &a, &b);
  if (st != SSD_OK) return st;
  if (!bytes) return SSD_ERR_INVALID_ARGUMENT;
  *bytes = recurrence_bytes(a);
  return SSD_OK;
}

ssd_status ssd_recurrence(const ssd_tokens* t, const ssd_recurrent* in, void* y, float* final_state,
                          void* workspace, int64_t workspace_bytes, void* stream) {
  RecArgs a;
  Buffers b;
  ssd_status st = recurrence_args(t, in, &a, &b);
  if (st != SSD_OK) return st;
  if (!y) return SSD_ERR_INVALID_ARGUMENT;
  const int64_t need = recurrence_bytes(a);
  b.input(in->initial_state, state_bytes(t));
  b.output(y, rows_of(t) * t->channels * bytes_of(t->io_dtype));
  b.output(final_state, state_bytes(t));
  if (!b.fine()) return SSD_ERR_INVALID_ARGUMENT;
  st = take_workspace(&b, workspace, workspace_bytes, need);
  if (st != SSD_OK) return st;
  st = device_ready();
  if (st != SSD_OK) return st;
  return from_hip(launch_recurrence(a, y, final_state, static_cast<float*>(workspace),
                                    static_cast<hipStream_t>(stream)));
}

ssd_status ssd_recurrence_step(const ssd_tokens* t, const ssd_recurrent* in, float* state_out,
                               void* y, void* stream) {
  RecArgs a;
  Buffers b;
  ssd_status st = recurrence_args(t, in, &a, &b);
  if (st != SSD_OK) return st;
  if (t->seqlen != 1 || t->seq_starts || !in->initial_state || !state_out || !y)
    return SSD_ERR_INVALID_ARGUMENT;
  b.output(y, t->batch * t->channels * bytes_of(t->io_dtype));
  b.output(state_out, state_bytes(t));
  if (in->initial_state != state_out) b.input(in->initial_state, state_bytes(t));
  if (!b.fine()) return SSD_ERR_INVALID_ARGUMENT;
  if (!grid_fits(double(t->batch) * (t->channels / 4) / 256 + 1, 256)) return SSD_ERR_UNSUPPORTED;
  st = device_ready();
  if (st != SSD_OK) return st;
  return from_hip(launch_recurrence_step(a, state_out, y, static_cast<hipStream_t>(stream)));
}

ssd_status ssd_recurrence_backward_workspace(const ssd_tokens* t, const ssd_recurrent* in,
                                             int64_t* bytes) {
  RecArgs a;
  Buffers b;
  ssd_status st = recurrence_args(t, in, &a, &b);
  if (st != SSD_OK) return st;
  if (!bytes) return SSD_ERR_INVALID_ARGUMENT;
  *bytes = recurrence_backward_bytes(a);
  return SSD_OK;
}

ssd_status ssd_recurrence_backward(const ssd_tokens* t, const ssd_recurrent* in, const void* dy,
                                   const float* dfinal, void* dx, void* dgate, void* dinput_gate,
                                   float* ddecay, float* dinitial_state, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
  RecArgs a;
  Buffers b;
  ssd_status st = recurrence_args(t, in, &a, &b);
  if (st != SSD_OK) return st;
  if (!dy || !dx || !dgate || (in->input_gate != nullptr) != (dinput_gate != nullptr) ||
      (in->decay != nullptr) != (ddecay != nullptr))
    return SSD_ERR_INVALID_ARGUMENT;
  const int64_t act = rows_of(t) * t->channels * bytes_of(t->io_dtype);
  const int64_t need = recurrence_backward_bytes(a);
  b.input(in->initial_state, state_bytes(t));
  b.input(dy, act);
  b.input(dfinal, state_bytes(t));
  b.output(dx, act);
  b.output(dgate, act);
  b.output(dinput_gate, act);
  b.output(ddecay, t->channels * 4);
  b.output(dinitial_state, state_bytes(t));
  if (!b.fine()) return SSD_ERR_INVALID_ARGUMENT;
  st = take_workspace(&b, workspace, workspace_bytes, need);
  if (st != SSD_OK) return st;
  st = device_ready();
  if (st != SSD_OK) return st;
  const RecGrads g{dx, dgate, dinput_gate, ddecay, dinitial_state};
  return from_hip(launch_recurrence_backward(a, dy, dfinal, g, static_cast<float*>(workspace),
                                             static_cast<hipStream_t>(stream)));
}

ssd_status ssd_rotate(const ssd_rotation* in, void* B_out, void* C_out, void* stream) {
  if (!in || in->rows <= 0 || in->ngroups <= 0 || in->dstate <= 0 || in->nfreq <= 0 ||
      in->naxes <= 0 || in->reserved != 0 || !is_dtype(in->io_dtype) || !in->positions ||
      !in->frequencies || !in->B || !B_out || (in->C != nullptr) != (C_out != nullptr) ||
      in->nfreq > in->dstate / 2)
    return SSD_ERR_INVALID_ARGUMENT;
  if (in->naxes > 4 || in->dstate % 8 || in->nfreq % 4 || in->dstate > kMaxChannels ||
      in->ngroups > kMaxChannels || in->ngroups * in->dstate > kMaxChannels ||
      in->rows > kMaxIndex - 4096)
    return SSD_ERR_UNSUPPORTED;
  const int64_t R = in->rows, W = in->ngroups * in->dstate, e = bytes_of(in->io_dtype);
  RotArgs a{R, (int)in->ngroups, (int)in->dstate, (int)in->nfreq, (int)in->naxes, {0, 0, 0, 0},
            in->io_dtype, in->interleaved != 0, in->inverse != 0, in->positions, in->frequencies,
            in->B, in->C, stride_of(in->b_stride, W), stride_of(in->c_stride, W), B_out, C_out};
  int64_t sum = 0;
  for (int i = 0; i < 4; ++i) {
    const int64_t n = in->sections[i];
    if (n < 0 || n > in->nfreq || (i >= in->naxes && n)) return SSD_ERR_INVALID_ARGUMENT;
    sum += n;
    a.ends[i] = (int)sum;
  }
  if (sum != in->nfreq || a.bs < 0 || a.cs < 0) return SSD_ERR_INVALID_ARGUMENT;
  if (double(R) * double(a.bs > a.cs ? a.bs : a.cs) * 4 > kMaxBytes || !rotate_fits(a))
    return SSD_ERR_UNSUPPORTED;
  Buffers b;
  b.input(in->positions, in->naxes * R * 4, 4);
  b.input(in->frequencies, in->nfreq * 4);
  b.input(in->B, span(R, W, a.bs, e));
  b.input(in->C, span(R, W, a.cs, e));
  b.output(B_out, R * W * e);
  b.output(C_out, R * W * e);
  if (!b.fine()) return SSD_ERR_INVALID_ARGUMENT;
  const ssd_status st = device_ready();
  if (st != SSD_OK) return st;
  return from_hip(launch_rotate(a, static_cast<hipStream_t>(stream)));
}

ssd_status ssd_group_norm_workspace(const ssd_tokens* t, int64_t ngroups, int64_t* bytes) {
  GroupArgs a;
  Buffers b;
  ssd_status st = group_args(t, nullptr, 0, nullptr, nullptr, ngroups, 0.f, 0, &a, &b);
  if (st != SSD_OK) return st;
  if (!bytes) return SSD_ERR_INVALID_ARGUMENT;
  *bytes = group_norm_bytes(a);
  return SSD_OK;
}

ssd_status ssd_group_norm(const ssd_tokens* t, const void* x, int64_t x_stride, const float* weight,
                          const float* bias, int64_t ngroups, float eps, int32_t silu, void* y,
                          float* stats, void* workspace, int64_t workspace_bytes, void* stream) {
  GroupArgs a;
  Buffers b;
  ssd_status st = group_args(t, x, x_stride, weight, bias, ngroups, eps, silu, &a, &b);
  if (st != SSD_OK) return st;
  if (!x || !y) return SSD_ERR_INVALID_ARGUMENT;
  b.output(y, rows_of(t) * t->channels * bytes_of(t->io_dtype));
  b.output(stats, t->nseq * ngroups * 8);
  if (!b.fine()) return SSD_ERR_INVALID_ARGUMENT;
  st = take_workspace(&b, workspace, workspace_bytes, group_norm_bytes(a));
  if (st != SSD_OK) return st;
  st = device_ready();
  if (st != SSD_OK) return st;
  return from_hip(launch_group_norm(a, y, stats, static_cast<float*>(workspace),
                                    static_cast<hipStream_t>(stream)));
}

ssd_status ssd_group_norm_backward_workspace(const ssd_tokens* t, int64_t ngroups, int64_t* bytes) {
  GroupArgs a;
  Buffers b;
  ssd_status st = group_args(t, nullptr, 0, nullptr, nullptr, ngroups, 0.f, 0, &a, &b);
  if (st != SSD_OK) return st;
  if (!bytes) return SSD_ERR_INVALID_ARGUMENT;
  *bytes = group_norm_backward_bytes(a);
  return SSD_OK;
}

ssd_status ssd_group_norm_backward(const ssd_tokens* t, const void* x, int64_t x_stride,
                                   const float* weight, const float* bias, int64_t ngroups,
                                   int32_t silu, const float* stats, const void* dy, void* dx,
                                   float* dweight, float* dbias, void* workspace,
                                   int64_t workspace_bytes, void* stream) {
  GroupArgs a;
  Buffers b;
  ssd_status st = group_args(t, x, x_stride, weight, bias, ngroups, 0.f, silu, &a, &b);
  if (st != SSD_OK) return st;
  if (!x || !stats || !dy || !dx || (weight != nullptr) != (dweight != nullptr) ||
      (bias != nullptr) != (dbias != nullptr))
    return SSD_ERR_INVALID_ARGUMENT;
  const int64_t act = rows_of(t) * t->channels * bytes_of(t->io_dtype);
  b.input(stats, t->nseq * ngroups * 8);
  b.input(dy, act);
  b.output(dx, act);
  b.output(dweight, t->channels * 4);
  b.output(dbias, t->channels * 4);
  if (!b.fine()) return SSD_ERR_INVALID_ARGUMENT;
  st = take_workspace(&b, workspace, workspace_bytes, group_norm_backward_bytes(a));
  if (st != SSD_OK) return st;
  st = device_ready();
  if (st != SSD_OK) return st;
  return from_hip(launch_group_norm_backward(a, stats, dy, dx, dweight, dbias,
                                             static_cast<float*>(workspace),
                                             static_cast<hipStream_t>(stream)));
}

}  // extern "C"
