// The norm of many tensors together, and their scaling to a largest norm.
//
// A launch takes the tensors' addresses and sizes by value (up to kTensors of them), so nothing has to be
// written to device memory first and a captured launch keeps them.  A tensor is cut into chunks of kChunk
// elements, numbered through all tensors of the launch; a workgroup takes every gridDim-th chunk.  Sums of
// squares are 64-bit: the square of an fp32 value neither overflows nor vanishes there, and the result is
// the norm of the values rounded once.  Partial sums are added in a fixed order.
#include "common.hpp"
#include "launch.hpp"
#include "rows8.hpp"

namespace nms {
namespace {

constexpr int kTensors = 96;
constexpr int64_t kChunk = 16384;
constexpr int kGroups = 1024;   // workgroups of a launch, at most: 4 a CU

struct Table {
  const void* in[kTensors];
  void* out[kTensors];
  int64_t count[kTensors];
  int64_t first[kTensors];    // its first chunk
  int64_t chunks;
  int n;
  uint32_t bf16_in[kTensors / 32], bf16_out[kTensors / 32];
};
__device__ __host__ inline bool bit(const uint32_t* b, int i) { return b[i / 32] >> (i % 32) & 1; }

// The tensor that chunk c belongs to: the last whose first chunk is at most c (tensors have one at least).
__device__ inline int tensor_of(const Table& t, int64_t c) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ inline double block_sum(double v, double* sh) {   // 256 threads; the sum in thread 0
#pragma unroll
  for (int d = 32; d >= 1; d /= 2) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  return threadIdx.x == 0 ? ((sh[0] + sh[1]) + sh[2]) + sh[3] : 0.0;
}

template <typename T>
__device__ inline double chunk_squares(const T* p, int64_t n) {
  double s0 = 0, s1 = 0;
  for (int64_t c = 8 * (int64_t)threadIdx.x; c < n; c += 8 * 256) {
    float v[8];
    load8f(p, c, n, v);
#pragma unroll
    for (int q = 0; q < 8; q += 2) {
      s0 = __builtin_fma((double)v[q], (double)v[q], s0);
      s1 = __builtin_fma((double)v[q + 1], (double)v[q + 1], s1);
    }
  }
  return s0 + s1;
}

__global__ __launch_bounds__(256) void grad_squares_kernel(Table t, double* part) {
  __shared__ double sh[4];
  double sum = 0;
  for (int64_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    const int64_t at = (c - t.first[i]) * kChunk, left = t.count[i] - at, n = left < kChunk ? left : kChunk;
    sum += bit(t.bf16_in, i) ? chunk_squares((const uint16_t*)t.in[i] + at, n)
                             : chunk_squares((const uint32_t*)t.in[i] + at, n);
  }
  sum = block_sum(sum, sh);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__global__ __launch_bounds__(256) void grad_norm_kernel(const double* part, int64_t n, float* norm) {
  __shared__ double sh[4];
  double sum = 0;
  for (int64_t i = threadIdx.x; i < n; i += 256) sum += part[i];
  sum = block_sum(sum, sh);
  if (threadIdx.x == 0) *norm = (float)sqrt(sum);
}

// min(1, max_norm / norm); 1 where the norm is not finite (the comparison with a NaN is false)
__device__ inline float factor_of(float norm, float max_norm) {
  return norm > max_norm && norm < __builtin_inff() ? (float)((double)max_norm / (double)norm) : 1.f;
}

template <typename T, typename O>
__device__ inline void chunk_scale(const T* p, O* o, int64_t n, float f) {
  for (int64_t c = 8 * (int64_t)threadIdx.x; c < n; c += 8 * 256) {
    float v[8];
    load8f(p, c, n, v);
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] *= f;
    store8f(o, c, n, v);
  }
}

__global__ __launch_bounds__(256) void grad_scale_kernel(Table t, const float* norm, float max_norm) {
  const float f = factor_of(*norm, max_norm);
  for (int64_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const int i = tensor_of(t, c);
    if (f == 1.f && t.in[i] == t.out[i]) continue;   // in place, and nothing changes
    const int64_t at = (c - t.first[i]) * kChunk, left = t.count[i] - at, n = left < kChunk ? left : kChunk;
    const bool bi = bit(t.bf16_in, i), bo = bit(t.bf16_out, i);
    if (bi) {
      const uint16_t* p = (const uint16_t*)t.in[i] + at;
      if (bo) chunk_scale(p, (uint16_t*)t.out[i] + at, n, f);
      else chunk_scale(p, (uint32_t*)t.out[i] + at, n, f);
    } else {
      const uint32_t* p = (const uint32_t*)t.in[i] + at;
      if (bo) chunk_scale(p, (uint16_t*)t.out[i] + at, n, f);
      else chunk_scale(p, (uint32_t*)t.out[i] + at, n, f);
    }
  }
}

// f(table, workgroups) for every launch's tensors, until one fails; tensors without elements are left out.
template <typename F>
hipError_t for_tables(const Grads& g, F f) {
  Table t;
  int64_t i = 0;
  while (i < g.n) {
    t.n = 0;
    t.chunks = 0;
    for (int w = 0; w < kTensors / 32; ++w) t.bf16_in[w] = t.bf16_out[w] = 0;
    for (; i < g.n && t.n < kTensors; ++i) {
      if (g.count[i] == 0) continue;
      t.in[t.n] = g.in[i];
      t.out[t.n] = g.out ? g.out[i] : nullptr;
      t.count[t.n] = g.count[i];
      t.first[t.n] = t.chunks;
      t.chunks += (g.count[i] + kChunk - 1) / kChunk;
      if (g.dt[i] == DT_BF16) t.bf16_in[t.n / 32] |= 1u << t.n % 32;
      if (g.out && g.odt[i] == DT_BF16) t.bf16_out[t.n / 32] |= 1u << t.n % 32;
      ++t.n;
    }
    if (t.n == 0) break;
    const hipError_t e = f(t, t.chunks < kGroups ? t.chunks : kGroups);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

int64_t grad_partials(const int64_t* count, int64_t n) {
  int64_t total = 0, chunks = 0;
  int held = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (count[i] == 0) continue;
    chunks += (count[i] + kChunk - 1) / kChunk;
    if (++held == kTensors) {
      total += chunks < kGroups ? chunks : kGroups;
      held = 0;
      chunks = 0;
    }
  }
  return total + (chunks < kGroups ? chunks : kGroups);
}

hipError_t launch_grad_norm(const Grads& g, float* norm, double* work, hipStream_t s) {
  int64_t parts = 0;
  const hipError_t e = for_tables(g, [&](const Table& t, int64_t groups) {
    hipLaunchKernelGGL(grad_squares_kernel, dim3((unsigned)groups), dim3(256), 0, s, t, work + parts);
    parts += groups;
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(256), 0, s, (const double*)work, parts, norm);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const Grads& g, const float* norm, float max_norm, hipStream_t s) {
  return for_tables(g, [&](const Table& t, int64_t groups) {
    hipLaunchKernelGGL(grad_scale_kernel, dim3((unsigned)groups), dim3(256), 0, s, t, norm, max_norm);
    return hipGetLastError();
  });
}

}  // namespace nms
