// The gradient of an activation, and of the bias in front of it.
#include "act.hpp"
#include "launch.hpp"
#include "rows8.hpp"

namespace nms {
namespace {

// dZ = dY act'(pre) and the sums of its columns before rounding.  A workgroup takes 256 columns (32 threads of eight)
// and every 8 gridDim.y-th row from its own eight on; its column sums are added over the eight in their order.
// Bound by bytes: 4096 x 8192 with GELU, 201 MB not in a cache, takes 43 us with the addition of the workgroups' sums (5), 16384
// x 16384 301 (5.4 TB/s); with four rows of a thread in flight 45 and 306.
__global__ __launch_bounds__(256) void linear_bwd_act_kernel(ActBwdArgs a, float* part) {
  __shared__ float sh[8][256];
  const int tc = threadIdx.x & 31, tr = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 256 + tc * 8;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (c < a.N) {
    with_act(a.act, [&](auto act) {
      constexpr int ACT = decltype(act)::value;
      for (int64_t r = (int64_t)blockIdx.y * 8 + tr; r < a.M; r += (int64_t)gridDim.y * 8) {
        float d[8];
        load8f((const uint16_t*)a.dY + r * a.lddy, c, a.N, d);
        if constexpr (ACT != ACT_NONE) {
          float z[8];
          load8f((const uint16_t*)a.pre + r * a.ldp, c, a.N, z);
#pragma unroll
          for (int q = 0; q < 8; ++q) d[q] = act_gate<ACT>(d[q], z[q]);
        }
        if (a.dZ) store8f((uint16_t*)a.dZ + r * a.lddz, c, a.N, d);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q] += d[q];
      }
    });
  }
  if (!part) return;
#pragma unroll
  for (int q = 0; q < 8; ++q) sh[tr][q * 32 + tc] = acc[q];
  __syncthreads();
  const int64_t col = (int64_t)blockIdx.x * 256 + (threadIdx.x & 31) * 8 + (threadIdx.x >> 5);
  float sum = sh[0][threadIdx.x];
#pragma unroll
  for (int w = 1; w < 8; ++w) sum += sh[w][threadIdx.x];
  if (col < a.N) part[blockIdx.y * a.N + col] = sum;
}

}  // namespace

// Rows of partial sums: workgroups for every CU eight times, at least 32 rows each.
int64_t act_bwd_groups(int64_t M, int64_t N) {
  const int64_t cols = (N + 255) / 256, fill = (2048 + cols - 1) / cols, rows = (M + 31) / 32;
  const int64_t g = fill < rows ? fill : rows;
  return g < 1 ? 1 : g;
}

hipError_t launch_linear_bwd_act(const ActBwdArgs& a, hipStream_t s) {
  const int64_t g = act_bwd_groups(a.M, a.N);
  const dim3 grid((unsigned)((a.N + 255) / 256), (unsigned)g);
  float* part = !a.db ? nullptr : g > 1 ? a.work : a.db;
  hipLaunchKernelGGL(linear_bwd_act_kernel, grid, dim3(256), 0, s, a, part);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || !a.db || g == 1 ? e : launch_sum_partials(a.work, g, a.N, a.db, s);
}

}  // namespace nms
