// The weighted sum of each token's expert rows, and its gradients.
#include "common.hpp"
#include "launch.hpp"
#include "pieces.hpp"

namespace nms {
namespace {

// V consecutive elements of a row as fp32 and back: whole vectors, or one at a time in the tail and
// for rows that are not 16-byte aligned.  Stores are non-temporal: the rows still to be gathered keep
// their place in the caches (8192 tokens, forward and gradients, 198 -> 176 us).
template <typename T, int V>
__device__ inline void load_row(const T* p, int64_t c, int64_t D, bool vec, float (&x)[V]) {
  T b[V];
  if (vec) {
    __builtin_memcpy(b, __builtin_assume_aligned(p + c, V * sizeof(T)), sizeof(b));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = c + i < D ? p[c + i] : (T)0;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) x[i] = Elem<T>::to_f32(b[i]);
}
template <typename T, int V>
__device__ inline void store_row(T* p, int64_t c, int64_t D, bool vec, const float (&x)[V]) {
  T b[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (sizeof(T) == 2) b[i] = f32_to_bf16_rne(x[i]); else b[i] = __float_as_uint(x[i]);
  }
  if (vec) {
    u32x4 w;
    __builtin_memcpy(&w, b, sizeof(b));
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(p + c));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c + i < D) p[c + i] = b[i];
  }
}

// One workgroup per token and run of blockDim.x * V columns, eight of the k rows' loads in flight.  Bound
// by its bytes: 8192 tokens of 8 rows of 2048 bf16 (302 MB) in 52 us, 5.8 TB/s.
template <typename T>
__global__ __launch_bounds__(256) void moe_combine_kernel(const T* __restrict__ O, int64_t ldo, int64_t rows,
                                                          const int32_t* __restrict__ pos, const float* __restrict__ w,
                                                          int k, int64_t D, T* __restrict__ Y, int64_t ldy, bool vec) {
  constexpr int V = 16 / sizeof(T), J = 8;   // J rows in flight
  const int64_t t = blockIdx.x;
  for (int64_t c = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * V; c < D;
       c += (int64_t)gridDim.y * blockDim.x * V) {
    const bool whole = vec && c + V <= D;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < k; j0 += J) {
      float x[J][V], wj[J];
      bool on[J];
#pragma unroll
      for (int q = 0; q < J; ++q) {
        const int64_t p = j0 + q < k ? pos[t * k + j0 + q] : -1;
        on[q] = p >= 0 && p < rows;
        wj[q] = on[q] && w ? w[t * k + j0 + q] : 1.f;
        load_row<T, V>(O + (on[q] ? p : 0) * ldo, c, D, whole, x[q]);   // row 0 where there is none
      }
#pragma unroll
      for (int q = 0; q < J; ++q)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = on[q] ? acc[i] + wj[q] * x[q][i] : acc[i];
    }
    store_row<T, V>(Y + t * ldy, c, D, whole, acc);
  }
}

// Workgroups 0 .. T-1: one token each: dY's row is read once for its k rows of dO and k dot products
// (summed per thread, then over the wave and the four waves in a fixed order).  Workgroups from T
// on: 16 rows of dO each, those of no slot are cleared.  Bound by its bytes: the same tokens (588 MB with
// 4096 rows of padding) in 104 us, 5.7 TB/s.
constexpr int kPadRows = 16;
template <typename T>
__global__ __launch_bounds__(256) void moe_combine_bwd_kernel(const T* __restrict__ dY, int64_t lddy,
                                                              const T* __restrict__ O, int64_t ldo, int64_t rows,
                                                              const int32_t* __restrict__ src,
                                                              const int32_t* __restrict__ pos,
                                                              const float* __restrict__ w, int64_t Tn, int k, int64_t D,
                                                              T* __restrict__ dO, int64_t lddo, float* __restrict__ dw,
                                                              bool vec) {
  constexpr int V = 16 / sizeof(T);
  if ((int64_t)blockIdx.x >= Tn) {
    const int64_t r0 = ((int64_t)blockIdx.x - Tn) * kPadRows;
    const float zero[V] = {};
    for (int64_t r = r0; r < r0 + kPadRows && r < rows; ++r) {
      if (src[r] >= 0) continue;
      for (int64_t c = threadIdx.x * V; c < D; c += 256 * V) store_row<T, V>(dO + r * lddo, c, D, vec && c + V <= D, zero);
    }
    return;
  }
  __shared__ float part[64][4];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr int J = 4;   // rows in flight
  for (int j0 = 0; j0 < k; j0 += J) {
    int64_t p[J];
    float wj[J], dot[J];
#pragma unroll
    for (int q = 0; q < J; ++q) {
      p[q] = j0 + q < k ? pos[t * k + j0 + q] : -1;
      if (p[q] >= rows) p[q] = -1;
      wj[q] = p[q] >= 0 ? w[t * k + j0 + q] : 0.f;
      dot[q] = 0.f;
    }
    for (int64_t c = threadIdx.x * V; c < D; c += 256 * V) {
      const bool whole = vec && c + V <= D;
      float g[V], o[J][V];
      load_row<T, V>(dY + t * lddy, c, D, whole, g);
#pragma unroll
      for (int q = 0; q < J; ++q)
        if (p[q] >= 0) load_row<T, V>(O + p[q] * ldo, c, D, whole, o[q]);
#pragma unroll
      for (int q = 0; q < J; ++q) {
        if (p[q] < 0) continue;
        float d[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          dot[q] += g[i] * o[q][i];
          d[i] = wj[q] * g[i];
        }
        store_row<T, V>(dO + p[q] * lddo, c, D, whole, d);
      }
    }
#pragma unroll
    for (int q = 0; q < J; ++q) {
#pragma unroll
      for (int d = 32; d > 0; d /= 2) dot[q] += __shfl_xor(dot[q], d);
      if (lane == 0 && j0 + q < k) part[j0 + q][wave] = dot[q];
    }
  }
  __syncthreads();
  if ((int)threadIdx.x < k) {
    const float* s = part[threadIdx.x];
    dw[t * k + threadIdx.x] = (s[0] + s[1]) + (s[2] + s[3]);
  }
}

template <typename T>
bool vec_rows(const void* p, int64_t ld) {
  return (uintptr_t)p % 16 == 0 && (ld * (int64_t)sizeof(T)) % 16 == 0;
}

template <typename T>
hipError_t combine_t(const T* O, int64_t ldo, int64_t rows, const int32_t* pos, const float* w, int64_t Tn, int k,
                     int64_t D, T* Y, int64_t ldy, hipStream_t s) {
  constexpr int V = 16 / sizeof(T);
  const int64_t need = (D + V - 1) / V;
  const int nt = need <= 64 ? 64 : need <= 128 ? 128 : 256;
  const int64_t runs = (need + nt - 1) / nt;
  const bool vec = vec_rows<T>(O, ldo) && vec_rows<T>(Y, ldy);
  return in_pieces(Tn, kPieceRows256, [&](int64_t t0, int64_t n) {
    hipLaunchKernelGGL(moe_combine_kernel<T>, dim3((unsigned)n, (unsigned)(runs < 65535 ? runs : 65535)), dim3(nt), 0, s, O,
                       ldo, rows, pos + t0 * k, w ? w + t0 * k : nullptr, k, D, Y + t0 * ldy, ldy, vec);
    return hipGetLastError();
  });
}

template <typename T>
hipError_t combine_bwd_t(const T* dY, int64_t lddy, const T* O, int64_t ldo, int64_t rows, const int32_t* src,
                         const int32_t* pos, const float* w, int64_t Tn, int k, int64_t D, T* dO, int64_t lddo, float* dw,
                         hipStream_t s) {
  const int64_t pads = (rows + kPadRows - 1) / kPadRows;
  const bool vec = vec_rows<T>(dY, lddy) && vec_rows<T>(O, ldo) && vec_rows<T>(dO, lddo);
  // the rows to clear go with the last tokens, unless those and they are too many for one launch
  const bool together = pads <= kPieceRows256;
  const hipError_t e = in_pieces(Tn, kPieceRows256, [&](int64_t t0, int64_t n) {
    const int64_t clear = together && t0 + n == Tn ? pads : 0;
    hipLaunchKernelGGL(moe_combine_bwd_kernel<T>, dim3((unsigned)(n + clear)), dim3(256), 0, s, dY + t0 * lddy, lddy, O, ldo,
                       rows, src, pos + t0 * k, w + t0 * k, n, k, D, dO, lddo, dw + t0 * k, vec);
    return hipGetLastError();
  });
  if (e != hipSuccess || together) return e;
  return in_pieces(rows, kPieceRows256 * kPadRows, [&](int64_t r0, int64_t n) {
    hipLaunchKernelGGL(moe_combine_bwd_kernel<T>, dim3((unsigned)((n + kPadRows - 1) / kPadRows)), dim3(256), 0, s, dY, lddy, O,
                       ldo, n, src + r0, pos, w, (int64_t)0, k, D, dO + r0 * lddo, lddo, dw, vec);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_moe_combine(int dt, const void* O, int64_t ldo, int64_t rows, const int32_t* pos, const float* w,
                              int64_t T, int k, int64_t D, void* Y, int64_t ldy, hipStream_t s) {
  if (dt == DT_BF16)
    return combine_t<uint16_t>((const uint16_t*)O, ldo, rows, pos, w, T, k, D, (uint16_t*)Y, ldy, s);
  return combine_t<uint32_t>((const uint32_t*)O, ldo, rows, pos, w, T, k, D, (uint32_t*)Y, ldy, s);
}

hipError_t launch_moe_combine_bwd(int dt, const void* dY, int64_t lddy, const void* O, int64_t ldo, int64_t rows,
                                  const int32_t* src, const int32_t* pos, const float* w, int64_t T, int k, int64_t D,
                                  void* dO, int64_t lddo, float* dw, hipStream_t s) {
  if (dt == DT_BF16)
    return combine_bwd_t<uint16_t>((const uint16_t*)dY, lddy, (const uint16_t*)O, ldo, rows, src, pos, w, T, k, D,
                                   (uint16_t*)dO, lddo, dw, s);
  return combine_bwd_t<uint32_t>((const uint32_t*)dY, lddy, (const uint32_t*)O, ldo, rows, src, pos, w, T, k, D,
                                 (uint32_t*)dO, lddo, dw, s);
}

}  // namespace nms
