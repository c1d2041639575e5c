// The gradient of an activation, and of the bias in front of it.
#include "act.hpp"
#include "launch.hpp"
#include "rows8.hpp"

namespace nms {
namespace {

// dZ = dY act'(pre) and the sums of its columns before rounding.  A workgroup takes 256 columns (32 threads of eight)
// and every 8 gridDim.y-th row from its own eight on, DEPTH of a thread's rows in flight; its column sums are added over the
// eight in their order.  TAIL: N is not a multiple of eight.
// Bound by bytes: 4096 x 8192 with GELU (201 MB) takes 36 us (5.6 TB/s), and with one row in flight 44.6.
template <bool TAIL>
__global__ __launch_bounds__(256) void linear_bwd_act_kernel(ActBwdArgs a, float* part) {
  constexpr int DEPTH = 4;
  __shared__ float sh[8][256];
  const int tc = threadIdx.x & 31, tr = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 256 + tc * 8, step = (int64_t)gridDim.y * 8;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (c < a.N) {
    with_act(a.act, [&](auto act) {
      constexpr int ACT = decltype(act)::value;
      const uint16_t* dY = (const uint16_t*)a.dY;
      const uint16_t* pre = (const uint16_t*)a.pre;
      for (int64_t r0 = (int64_t)blockIdx.y * 8 + tr; r0 < a.M; r0 += DEPTH * step) {
        Row8<uint16_t> y[DEPTH], p[DEPTH];
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
          const int64_t r = r0 + i * step;
          if (r >= a.M) break;
          y[i].template load<TAIL>(dY + r * a.lddy, c, a.N);
          if constexpr (ACT != ACT_NONE) p[i].template load<TAIL>(pre + r * a.ldp, c, a.N);
        }
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
          const int64_t r = r0 + i * step;
          if (r >= a.M) break;
          float d[8];
          y[i].get(d);
          if constexpr (ACT != ACT_NONE) {
            float z[8];
            p[i].get(z);
#pragma unroll
            for (int q = 0; q < 8; ++q) d[q] = act_gate<ACT>(d[q], z[q]);
          }
          if (a.dZ) store8f<uint16_t, TAIL>((uint16_t*)a.dZ + r * a.lddz, c, a.N, d);
#pragma unroll
          for (int q = 0; q < 8; ++q) acc[q] += d[q];
        }
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
  if (a.N % 8) hipLaunchKernelGGL(linear_bwd_act_kernel<true>, grid, dim3(256), 0, s, a, part);
  else hipLaunchKernelGGL(linear_bwd_act_kernel<false>, grid, dim3(256), 0, s, a, part);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || !a.db || g == 1 ? e : launch_sum_partials(a.work, g, a.N, a.db, s);
}

}  // namespace nms
