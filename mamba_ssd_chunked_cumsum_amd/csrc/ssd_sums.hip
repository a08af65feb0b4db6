// Sums over the rows of partial results (gradients of parameters), in a fixed order.
#include "ssd_block.h"

namespace ssd {

// Bound by reading the partials (42 MB of a scan's dA: 11 us), or by the launch. 64 columns a block; 16 groups of rows, each in order, then the groups in order: the same sum
// whatever runs beside it.
namespace {
__global__ __launch_bounds__(1024) void k_column_sums(const float* __restrict__ part, int n,
                                                      int64_t M1, float* out1, int inner,
                                                      int64_t so, int64_t si, int64_t M2,
                                                      float* out2, int64_t M3, float* out3) {
  const int lane = threadIdx.x & 63, grp = threadIdx.x >> 6;
  const int64_t m = (int64_t)blockIdx.x * 64 + lane;
  const int64_t M = M1 + M2 + M3;
  __shared__ float red[16][64];
  float sum = 0.f;
  if (m < M) {
#pragma unroll 4
    for (int i = grp; i < n; i += 16) sum += part[(int64_t)i * M + m];
  }
  red[grp][lane] = sum;
  __syncthreads();
  if (grp == 0 && m < M) {
#pragma unroll
    for (int g = 1; g < 16; ++g) sum += red[g][lane];
    if (m < M1) out1[(m / inner) * so + (m % inner) * si] = sum;
    else if (m < M1 + M2) { if (out2) out2[m - M1] = sum; }
    else if (out3) out3[m - M1 - M2] = sum;
  }
}
}  // namespace

hipError_t launch_column_sums(const float* part, int n, int64_t M1, float* out1, int inner,
                              int64_t so, int64_t si, int64_t M2, float* out2, int64_t M3, float* out3,
                              hipStream_t s) {
  const int64_t M = M1 + M2 + M3;
  hipLaunchKernelGGL(k_column_sums, dim3((unsigned)((M + 63) / 64)), dim3(1024), 0, s, part, n, M1,
                     out1, inner, so, si, M2, out2, M3, out3);
  return hipGetLastError();
}

}  // namespace ssd
