// Quantisation to 8-bit floating point in blocks of 128 with a power-of-two scale.
#include "fp8.hpp"
#include "launch.hpp"

namespace nms {
namespace {

// Eight consecutive elements of a row from column c, 0 beyond K.
template <typename T>
__device__ inline void load8(const T* p, int64_t c, int64_t K, bool vec, float (&x)[8]) {
  T b[8];
  if (vec && c + 8 <= K) {
    __builtin_memcpy(b, __builtin_assume_aligned(p + c, 16), sizeof(b));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = c + i < K ? p[c + i] : (T)0;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = Elem<T>::to_f32(b[i]);
}

// Eight elements of row r of the quantisers' input: gathered, and gated.
template <typename T>
__device__ inline void input8(const QuantArgs& a, int64_t r, int64_t c, bool vec, float (&x)[8]) {
  const T* X = (const T*)a.X;
  int64_t row = r;
  if (a.src) {
    const int sl = a.src[r];
    row = sl < 0 ? -1 : sl / a.div;
    if (row >= a.RX) row = -1;
  }
  if (row < 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    return;
  }
  load8(X + row * a.ldx, c, a.K, vec, x);
  if (a.gate) {
    float g[8];
    load8((const T*)a.gate + r * a.ldg, c, a.K, vec, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = g[i] > 0.f ? x[i] : 0.f;
  }
}

__device__ inline uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Rows: 16 lanes hold a block (8 elements a lane), a wave four consecutive blocks of one row, a
// workgroup 32 rows x 4 blocks; the scales leave through LDS so that a block's 32 are written
// together.  One pass over the data; bound by its bytes.
template <typename T, bool E5M2>
__global__ __launch_bounds__(256) void fp8_quantize_kernel(QuantArgs a, bool vec) {
  __shared__ float sc[4][32];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t r0 = (int64_t)blockIdx.x * 32;
  const int64_t kb0 = (int64_t)blockIdx.y * 4, nkb = (a.K + 127) / 128;
  const int64_t kb = kb0 + (lane >> 4);
  const int64_t c = kb * 128 + (lane & 15) * 8;
#pragma unroll 4
  for (int i = 0; i < 8; ++i) {
    const int rl = wave + 4 * i;
    const int64_t r = r0 + rl;
    const bool on = r < a.R && kb < nkb;
    float x[8];
    if (on) {
      input8<T>(a, r, c, vec, x);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = 0.f;
    }
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) m = umax(m, finite_bits(x[q]));
#pragma unroll
    for (int d = 8; d > 0; d /= 2) m = umax(m, __shfl_xor(m, d));
    const int e = block_exponent(m, E5M2);
    const float inv = power2(-e);
    const float lo[4] = {x[0], x[1], x[2], x[3]}, hi[4] = {x[4], x[5], x[6], x[7]};
    const u32x2 q = {pack4<E5M2>(lo, inv), pack4<E5M2>(hi, inv)};
    if (on) {
      uint8_t* dst = a.Q + r * a.ldq + c;
      if (((uintptr_t)dst & 7) == 0) {
        *reinterpret_cast<u32x2*>(dst) = q;
      } else {
#pragma unroll
        for (int b = 0; b < 8; ++b) dst[b] = (uint8_t)(q[b >> 2] >> (8 * (b & 3)));
      }
    }
    if ((lane & 15) == 0) sc[lane >> 4][rl] = power2(e);
  }
  __syncthreads();
  if (threadIdx.x < 128) {
    const int kq = threadIdx.x >> 5, rl = threadIdx.x & 31;
    if (kb0 + kq < nkb && r0 + rl < a.R) a.S[(kb0 + kq) * a.lds + r0 + rl] = sc[kq][rl];
  }
}

// A 128 x 128 tile held in registers: thread -> columns 8 (tid % 16) .. +7, rows 8 (tid / 16) .. +7.
// The bytes are transposed through LDS: column j's 128 bytes are 16 slots of 8 rows, slot s at
// s ^ (j / 8), so the 16 lanes of a row group write 16 different slots.
struct TileT {
  unsigned char b[128][128];
};
__device__ inline uint64_t* tile_slot(TileT& t, int col, int slot) {
  return reinterpret_cast<uint64_t*>(&t.b[col][((slot ^ (col >> 3)) & 15) * 8]);
}
// Columns k0 .. of the transposed matrix: 16-byte stores of 16 rows, r0 + 128 <= ld.
__device__ inline void store_transposed(TileT& t, uint8_t* Qt, int64_t ldqt, int64_t k0, int64_t K, int64_t r0) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int id = threadIdx.x + 256 * i, col = id >> 3, pair = id & 7;
    if (k0 + col >= K) continue;
    const uint64_t v[2] = {*tile_slot(t, col, 2 * pair), *tile_slot(t, col, 2 * pair + 1)};
    uint8_t* dst = Qt + (k0 + col) * ldqt + r0 + 16 * pair;
    if (((uintptr_t)dst & 15) == 0) {
      u32x4 w;
      __builtin_memcpy(&w, v, 16);
      *reinterpret_cast<u32x4*>(dst) = w;
    } else {
      for (int b = 0; b < 16; ++b) dst[b] = (uint8_t)(v[b >> 3] >> (8 * (b & 7)));
    }
  }
}

template <typename T, bool E5M2>
__global__ __launch_bounds__(256) void fp8_quantize_t_kernel(QuantArgs a, bool vec) {
  __shared__ __align__(16) TileT tile;
  __shared__ uint32_t cmax[4][128];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t r0 = (int64_t)blockIdx.x * 128, k0 = (int64_t)blockIdx.y * 128;
  const int cg = tid & 15, rg = tid >> 4;
  const int64_t c = k0 + cg * 8;
  float x[8][8];   // [row][column]
  uint32_t m[8] = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + rg * 8 + i;
    if (r < a.R && c < a.K) {
      input8<T>(a, r, c, vec, x[i]);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) x[i][q] = 0.f;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) m[q] = umax(m[q], finite_bits(x[i][q]));
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    m[q] = umax(m[q], __shfl_xor(m[q], 16));
    m[q] = umax(m[q], __shfl_xor(m[q], 32));
    if (lane < 16) cmax[wave][cg * 8 + q] = m[q];
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int col = cg * 8 + q;
    const int e = block_exponent(umax(umax(cmax[0][col], cmax[1][col]), umax(cmax[2][col], cmax[3][col])), E5M2);
    const float inv = power2(-e);
    const float lo[4] = {x[0][q], x[1][q], x[2][q], x[3][q]}, hi[4] = {x[4][q], x[5][q], x[6][q], x[7][q]};
    *tile_slot(tile, col, rg) = (uint64_t)pack4<E5M2>(lo, inv) | ((uint64_t)pack4<E5M2>(hi, inv) << 32);
    if (rg == 0 && k0 + col < a.K) a.S[(int64_t)blockIdx.x * a.lds + k0 + col] = power2(e);
  }
  __syncthreads();
  store_transposed(tile, a.Q, a.ldq, k0, a.K, r0);
}

// One 128 x 128 block of a weight: its bytes row by row, and the same bytes transposed.
template <typename T, bool E5M2>
__global__ __launch_bounds__(256) void fp8_quantize_weight_kernel(const T* W, int64_t ldw, int64_t N, int64_t K, uint8_t* Q,
                                                                  int64_t ldq, float* S, uint8_t* Qt, int64_t ldqt,
                                                                  float* St, bool vec) {
  __shared__ __align__(16) TileT tile;
  __shared__ uint32_t bmax[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t nb = (N + 127) / 128, kbn = (K + 127) / 128;
  // one block a workgroup, along a row of blocks first
  const int64_t ib = blockIdx.x / kbn, jb = blockIdx.x % kbn, ex = blockIdx.y;
  const int64_t n0 = ib * 128, k0 = jb * 128;
  const int cg = tid & 15, rg = tid >> 4;
  const int64_t c = k0 + cg * 8;
  W += ex * N * ldw;
  float x[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = n0 + rg * 8 + i;
    if (r < N && c < K) {
      load8(W + r * ldw, c, K, vec, x[i]);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) x[i][q] = 0.f;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) m = umax(m, finite_bits(x[i][q]));
  }
#pragma unroll
  for (int d = 32; d > 0; d /= 2) m = umax(m, __shfl_xor(m, d));
  if (lane == 0) bmax[wave] = m;
  __syncthreads();
  const int e = block_exponent(umax(umax(bmax[0], bmax[1]), umax(bmax[2], bmax[3])), E5M2);
  const float inv = power2(-e);
  if (tid == 0) {
    S[(ex * nb + ib) * kbn + jb] = power2(e);
    if (St) St[(ex * kbn + jb) * nb + ib] = power2(e);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = n0 + rg * 8 + i;
    if (r >= N) continue;
    const float lo[4] = {x[i][0], x[i][1], x[i][2], x[i][3]}, hi[4] = {x[i][4], x[i][5], x[i][6], x[i][7]};
    const u32x2 q = {pack4<E5M2>(lo, inv), pack4<E5M2>(hi, inv)};
    uint8_t* dst = Q + (ex * N + r) * ldq + c;
    if (((uintptr_t)dst & 7) == 0) {
      *reinterpret_cast<u32x2*>(dst) = q;
    } else {
#pragma unroll
      for (int b = 0; b < 8; ++b) dst[b] = (uint8_t)(q[b >> 2] >> (8 * (b & 3)));
    }
  }
  if (!Qt) return;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float lo[4] = {x[0][q], x[1][q], x[2][q], x[3][q]}, hi[4] = {x[4][q], x[5][q], x[6][q], x[7][q]};
    *tile_slot(tile, cg * 8 + q, rg) = (uint64_t)pack4<E5M2>(lo, inv) | ((uint64_t)pack4<E5M2>(hi, inv) << 32);
  }
  __syncthreads();
  store_transposed(tile, Qt + ex * K * ldqt, ldqt, k0, K, n0);
}

bool vec_ok(int es, const void* X, int64_t ldx, const void* gate, int64_t ldg) {
  return (uintptr_t)X % 16 == 0 && (ldx * es) % 16 == 0 && (uintptr_t)gate % 16 == 0 && (!gate || (ldg * es) % 16 == 0);
}

}  // namespace

hipError_t launch_fp8_quantize(int dt, const QuantArgs& a, hipStream_t s) {
  const int64_t nkb = (a.K + 127) / 128;
  const dim3 grid((unsigned)((a.R + 31) / 32), (unsigned)((nkb + 3) / 4));
  if (dt == DT_BF16) {
    const bool vec = vec_ok(2, a.X, a.ldx, a.gate, a.ldg);
    if (a.e5m2) hipLaunchKernelGGL((fp8_quantize_kernel<uint16_t, true>), grid, dim3(256), 0, s, a, vec);
    else hipLaunchKernelGGL((fp8_quantize_kernel<uint16_t, false>), grid, dim3(256), 0, s, a, vec);
  } else {
    const bool vec = vec_ok(4, a.X, a.ldx, a.gate, a.ldg);
    if (a.e5m2) hipLaunchKernelGGL((fp8_quantize_kernel<uint32_t, true>), grid, dim3(256), 0, s, a, vec);
    else hipLaunchKernelGGL((fp8_quantize_kernel<uint32_t, false>), grid, dim3(256), 0, s, a, vec);
  }
  return hipGetLastError();
}

hipError_t launch_fp8_quantize_t(int dt, const QuantArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.R + 127) / 128), (unsigned)((a.K + 127) / 128));
  if (dt == DT_BF16) {
    const bool vec = vec_ok(2, a.X, a.ldx, a.gate, a.ldg);
    if (a.e5m2) hipLaunchKernelGGL((fp8_quantize_t_kernel<uint16_t, true>), grid, dim3(256), 0, s, a, vec);
    else hipLaunchKernelGGL((fp8_quantize_t_kernel<uint16_t, false>), grid, dim3(256), 0, s, a, vec);
  } else {
    const bool vec = vec_ok(4, a.X, a.ldx, a.gate, a.ldg);
    if (a.e5m2) hipLaunchKernelGGL((fp8_quantize_t_kernel<uint32_t, true>), grid, dim3(256), 0, s, a, vec);
    else hipLaunchKernelGGL((fp8_quantize_t_kernel<uint32_t, false>), grid, dim3(256), 0, s, a, vec);
  }
  return hipGetLastError();
}

hipError_t launch_fp8_quantize_weight(int dt, const void* W, int64_t ldw, int64_t E, int64_t N, int64_t K, int e5m2,
                                      uint8_t* Q, int64_t ldq, float* S, uint8_t* Qt, int64_t ldqt, float* St,
                                      hipStream_t s) {
  const dim3 grid((unsigned)(((N + 127) / 128) * ((K + 127) / 128)), (unsigned)E);
  const int es = dt == DT_BF16 ? 2 : 4;
  const bool vec = vec_ok(es, W, ldw, nullptr, 0);
  auto go = [&](auto kern, auto* w) {
    hipLaunchKernelGGL(kern, grid, dim3(256), 0, s, w, ldw, N, K, Q, ldq, S, Qt, ldqt, St, vec);
    return hipGetLastError();
  };
  if (dt == DT_BF16)
    return e5m2 ? go(fp8_quantize_weight_kernel<uint16_t, true>, (const uint16_t*)W)
                : go(fp8_quantize_weight_kernel<uint16_t, false>, (const uint16_t*)W);
  return e5m2 ? go(fp8_quantize_weight_kernel<uint32_t, true>, (const uint32_t*)W)
              : go(fp8_quantize_weight_kernel<uint32_t, false>, (const uint32_t*)W);
}

}  // namespace nms
