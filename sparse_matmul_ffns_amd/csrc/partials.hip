// Sums of partial sums: the second step of reductions over rows (a bias's or a norm weight's gradient).
#include "common.hpp"
#include "launch.hpp"

namespace nms {
namespace {

// out[c] = sum over g of part[g][c], in fp32: 64 columns a workgroup, its 16 waves every 16th row each,
// then the waves' sums in their order.  The order does not depend on anything but G.  512 x 4096 and 64 x 8192 take 5 us,
// which is a launch behind another one (with every load in flight at once the same).
__global__ __launch_bounds__(1024) void sum_partials_kernel(const float* part, int64_t G, int64_t N, float* out) {
  __shared__ float sh[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float sum = 0.f;
  if (c < N) {
    float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
    int64_t g = wave;
    for (; g + 48 < G; g += 64) {
      s0 += part[g * N + c];
      s1 += part[(g + 16) * N + c];
      s2 += part[(g + 32) * N + c];
      s3 += part[(g + 48) * N + c];
    }
    for (; g < G; g += 16) s0 += part[g * N + c];
    sum = (s0 + s1) + (s2 + s3);
  }
  sh[wave][lane] = sum;
  __syncthreads();
  if (wave == 0 && c < N) {
#pragma unroll
    for (int w = 1; w < 16; ++w) sum += sh[w][lane];
    out[c] = sum;
  }
}

}  // namespace

hipError_t launch_sum_partials(const float* part, int64_t G, int64_t N, float* out, hipStream_t s) {
  hipLaunchKernelGGL(sum_partials_kernel, dim3((unsigned)((N + 63) / 64)), dim3(1024), 0, s, part, G, N, out);
  return hipGetLastError();
}

}  // namespace nms
