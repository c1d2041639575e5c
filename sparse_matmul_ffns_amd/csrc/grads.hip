// The norm of many tensors together, and their scaling to a largest norm.
//
// A launch takes the tensors' addresses and sizes by value (up to kTensors of them), so nothing has to be
// written to device memory first and a captured launch keeps them.  A tensor is cut into chunks of kChunk
// elements, numbered through all tensors of the launch; a workgroup takes every gridDim-th chunk.  Sums of
// squares are 64-bit: the square of an fp32 value neither overflows nor vanishes there, and the result is
// the norm of the values rounded once.  Partial sums are added in a fixed order.
//
// Bound by bytes: every value is read for the norm, read again and written.  537 MB that are not in a cache: the norm 95 us
// (5.6 TB/s; with 2048 workgroups 99, with four of a thread's loads in flight 97), clipped in place in bf16 243 (four in flight, 2048
// workgroups: 319), fp32 to other tensors 311; 537 MB of bf16 in 192 tensors to fp32
// 437.
#include "common.hpp"
#include "launch.hpp"

namespace nms {
namespace {

constexpr int kTensors = 160;
constexpr int kChunk = 16384;
constexpr int kGroups = 1024;      // workgroups of a launch, at most: 4 a CU
constexpr int64_t kOne = 65536;    // as many elements as one workgroup does by itself,
constexpr int kWaveChunk = 2048;   // in chunks that a wave loads at once

struct Table {
  const void* in[kTensors];
  void* out[kTensors];
  uint32_t first[kTensors];        // a tensor's first chunk
  uint16_t last[kTensors];         // the elements of its last chunk, less one
  uint32_t bf16_in[kTensors / 32], bf16_out[kTensors / 32];
  uint32_t chunks;
  int n;
};
static_assert(sizeof(Table) <= 3800, "a launch's arguments");
__device__ __host__ inline bool bit(const uint32_t* b, int i) { return b[i / 32] >> (i % 32) & 1; }

// A chunk: its tensor, its first element there, its elements.
struct Chunk {
  int i, n;
  int64_t at;
};
template <int CHUNK>
__device__ inline Chunk chunk_of(const Table& t, uint32_t c) {
  int lo = 0, hi = t.n - 1;   // the last tensor whose first chunk is at most c (each has one at least)
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= c) lo = mid;
    else hi = mid - 1;
  }
  const uint32_t end = lo + 1 < t.n ? t.first[lo + 1] : t.chunks;
  return Chunk{lo, c + 1 == end ? t.last[lo] + 1 : CHUNK, (int64_t)(c - t.first[lo]) * CHUNK};
}

// Four elements, whatever their address; 0 beyond n.
__device__ inline f32x4 four(const uint16_t* p, int c, int n) {
  uint16_t b[4] = {0, 0, 0, 0};
  if (c + 4 <= n) {
    __builtin_memcpy(b, p + c, 8);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (c + q < n) b[q] = p[c + q];
  }
  return f32x4{Elem<uint16_t>::to_f32(b[0]), Elem<uint16_t>::to_f32(b[1]), Elem<uint16_t>::to_f32(b[2]), Elem<uint16_t>::to_f32(b[3])};
}
__device__ inline f32x4 four(const float* p, int c, int n) {
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
  if (c + 4 <= n) {
    __builtin_memcpy(&v, p + c, 16);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (c + q < n) v[q] = p[c + q];
  }
  return v;
}
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
__device__ inline void put(uint16_t* p, int c, int n, const f32x4& v) {
  const bf16x4 h = __builtin_convertvector(v, bf16x4);   // nearest even
  uint16_t b[4];
  __builtin_memcpy(b, &h, 8);
  if (c + 4 <= n) {
    __builtin_memcpy(p + c, b, 8);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (c + q < n) p[c + q] = b[q];
  }
}
__device__ inline void put(float* p, int c, int n, const f32x4& v) {
  if (c + 4 <= n) {
    __builtin_memcpy(p + c, &v, 16);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (c + q < n) p[c + q] = v[q];
  }
}

// f(first element, values) over a chunk by NT threads (a wave or a workgroup), four elements each, DEPTH of a thread's
// loads in flight.
template <int NT, typename T, typename F>
__device__ inline void over(const T* p, int n, F f) {
  constexpr int DEPTH = 8, LINE = 4 * NT;
  int c = 4 * (threadIdx.x % NT);
  for (; c + LINE * (DEPTH - 1) + 4 <= n; c += LINE * DEPTH) {
    f32x4 v[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) v[d] = four(p, c + LINE * d, 1 << 30);
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) f(c + LINE * d, v[d]);
  }
  for (; c < n; c += LINE) f(c, four(p, c, n));
}

template <int NT, typename T>
__device__ inline double chunk_squares(const T* p, int n) {
  double s[2] = {0, 0};
  over<NT>(p, n, [&](int, const f32x4& v) {
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q & 1] = __builtin_fma((double)v[q], (double)v[q], s[q & 1]);
  });
  return s[0] + s[1];
}
template <int NT, int CHUNK>
__device__ inline double squares_of(const Table& t, uint32_t c) {
  const Chunk k = chunk_of<CHUNK>(t, c);
  return bit(t.bf16_in, k.i) ? chunk_squares<NT>((const uint16_t*)t.in[k.i] + k.at, k.n)
                             : chunk_squares<NT>((const float*)t.in[k.i] + k.at, k.n);
}

template <int NT, typename T, typename O>
__device__ inline void chunk_scale(const T* p, O* o, int n, float f) {
  over<NT>(p, n, [&](int c, const f32x4& v) { put(o, c, n, v * f); });
}
template <int NT, int CHUNK>
__device__ inline void scale_of(const Table& t, uint32_t c, float f) {
  const Chunk k = chunk_of<CHUNK>(t, c);
  if (f == 1.f && t.in[k.i] == t.out[k.i]) return;   // in place, and nothing changes
  const bool bi = bit(t.bf16_in, k.i), bo = bit(t.bf16_out, k.i);
  const uint16_t* h = (const uint16_t*)t.in[k.i] + k.at;
  const float* w = (const float*)t.in[k.i] + k.at;
  uint16_t* oh = (uint16_t*)t.out[k.i] + k.at;
  float* ow = (float*)t.out[k.i] + k.at;
  if (bi && bo) chunk_scale<NT>(h, oh, k.n, f);
  else if (bi) chunk_scale<NT>(h, ow, k.n, f);
  else if (bo) chunk_scale<NT>(w, oh, k.n, f);
  else chunk_scale<NT>(w, ow, k.n, f);
}

// The sum over NT threads, in every one of them: over a wave's lanes, then over the waves in their order.
template <int NT>
__device__ inline double block_sum(double v, double* sh) {
#pragma unroll
  for (int d = 32; d >= 1; d /= 2) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  v = sh[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) v += sh[w];
  return v;
}
// The norm from the partial sums, the same in every workgroup that computes it (256 threads).
__device__ inline float norm_of(const double* part, int64_t n, double* sh) {
  double sum = 0;
  for (int64_t i = threadIdx.x; i < n; i += 256) sum += part[i];
  return (float)sqrt(block_sum<256>(sum, sh));
}
// min(1, max_norm / norm); 1 where the norm is not finite (the comparison with a NaN is false)
__device__ inline float factor_of(float norm, float max_norm) {
  return norm > max_norm && norm < __builtin_inff() ? (float)((double)max_norm / (double)norm) : 1.f;
}

__global__ __launch_bounds__(256) void grad_squares_kernel(Table t, double* part) {
  __shared__ double sh[4];
  double sum = 0;
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) sum += squares_of<256, kChunk>(t, c);
  sum = block_sum<256>(sum, sh);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

__global__ __launch_bounds__(256) void grad_norm_kernel(const double* part, int64_t n, float* norm) {
  __shared__ double sh[4];
  const float v = norm_of(part, n, sh);
  if (threadIdx.x == 0) *norm = v;
}

// With the partial sums of all tensors (few enough that every workgroup adds them for itself, which costs less than a launch) or,
// without, the norm.  The chunks are taken from the last to the first: the last that the norm's pass read are
// still in the memory-side cache.
__global__ __launch_bounds__(256) void grad_scale_kernel(Table t, const double* part, int parts, float* norm, float max_norm) {
  __shared__ double sh[4];
  float v;
  if (part) {
    v = norm_of(part, parts, sh);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
  } else {
    v = *norm;
  }
  const float f = factor_of(v, max_norm);
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) scale_of<256, kChunk>(t, t.chunks - 1 - c, f);
}

// Few elements: the norm and, where max_norm is not negative, the scaling in one workgroup, whose waves take a
// chunk each.  2 matrices of 128 x 128 and a few vectors: 8 us on the GPU in one launch; in three 25 us a call, now 14.
__global__ __launch_bounds__(1024) void grad_one_kernel(Table t, float* norm, float max_norm) {
  __shared__ double sh[16];
  const uint32_t wave = threadIdx.x >> 6;
  double sum = 0;
  for (uint32_t c = wave; c < t.chunks; c += 16) sum += squares_of<64, kWaveChunk>(t, c);
  const float v = (float)sqrt(block_sum<1024>(sum, sh));
  if (threadIdx.x == 0) *norm = v;
  if (max_norm < 0.f) return;
  const float f = factor_of(v, max_norm);
  for (uint32_t c = wave; c < t.chunks; c += 16) scale_of<64, kWaveChunk>(t, c, f);
}

// The next launch's tensors from tensor i on; tensors without elements are left out.  False where none is left.
bool next_table(const Grads& g, int64_t& i, Table& t, int chunk = kChunk) {
  t.n = 0;
  t.chunks = 0;
  for (int w = 0; w < kTensors / 32; ++w) t.bf16_in[w] = t.bf16_out[w] = 0;
  for (; i < g.n && t.n < kTensors; ++i) {
    const int64_t count = g.count[i];
    if (count == 0) continue;
    const int64_t chunks = (count + chunk - 1) / chunk;
    if (t.n > 0 && t.chunks + chunks > UINT32_MAX) break;
    t.in[t.n] = g.in[i];
    t.out[t.n] = g.out ? g.out[i] : nullptr;
    t.first[t.n] = t.chunks;
    t.last[t.n] = (uint16_t)((count - 1) % chunk);
    t.chunks += (uint32_t)chunks;
    if (g.dt[i] == DT_BF16) t.bf16_in[t.n / 32] |= 1u << t.n % 32;
    if (g.out && g.odt[i] == DT_BF16) t.bf16_out[t.n / 32] |= 1u << t.n % 32;
    ++t.n;
  }
  return t.n > 0;
}
unsigned groups_of(const Table& t) { return t.chunks < (uint32_t)kGroups ? t.chunks : kGroups; }

// Whether one workgroup does it all: few elements, in one table.
bool one_group(const int64_t* count, int64_t n) {
  int64_t total = 0;
  if (n > kTensors) return false;
  for (int64_t i = 0; i < n; ++i) {
    if (count[i] > kOne) return false;
    total += count[i];
  }
  return total <= kOne;
}

}  // namespace

int64_t grad_partials(const int64_t* count, int64_t n) {
  if (one_group(count, n)) return 0;
  int64_t total = 0, chunks = 0;
  int held = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (count[i] == 0) continue;
    const int64_t c = (count[i] + kChunk - 1) / kChunk;
    if (held == kTensors || (held > 0 && chunks + c > UINT32_MAX)) {
      total += chunks < kGroups ? chunks : kGroups;
      held = 0;
      chunks = 0;
    }
    chunks += c;
    ++held;
  }
  return total + (chunks < kGroups ? chunks : kGroups);
}

// The norm, and with g.out the scaling (have_norm: *norm is given).
hipError_t launch_grads(const Grads& g, bool have_norm, float* norm, float max_norm, double* work, hipStream_t s) {
  Table t;
  if (!have_norm && one_group(g.count, g.n)) {
    int64_t i = 0;
    (void)next_table(g, i, t, kWaveChunk);
    hipLaunchKernelGGL(grad_one_kernel, dim3(1), dim3(1024), 0, s, t, norm, g.out ? max_norm : -1.f);
    return hipGetLastError();
  }
  int64_t parts = 0, tables = 0;
  if (!have_norm) {
    for (int64_t i = 0; next_table(g, i, t); ++tables) {
      hipLaunchKernelGGL(grad_squares_kernel, dim3(groups_of(t)), dim3(256), 0, s, t, work + parts);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
      parts += groups_of(t);
    }
  }
  const bool join = !have_norm && g.out && tables == 1;
  if (!have_norm && !join) {
    hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(256), 0, s, (const double*)work, parts, norm);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!g.out) return hipSuccess;
  for (int64_t i = 0; next_table(g, i, t);) {
    hipLaunchKernelGGL(grad_scale_kernel, dim3(groups_of(t)), dim3(256), 0, s, t, join ? (const double*)work : nullptr, (int)parts,
                       norm, max_norm);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace nms
