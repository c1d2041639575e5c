// Root-mean-square norm of rows, with the residual's addition in front and, where asked for, an 8-bit
// result behind; and its gradients.
#include "fp8.hpp"
#include "launch.hpp"
#include "pieces.hpp"
#include "rows8.hpp"

namespace nms {
namespace {

// Sum of v over the NT threads of a row, in every one of them: over the waves' lanes, then over the waves
// in their order.  `part` holds a float per wave.
template <int NT>
__device__ inline float row_sum(float v, float* part) {
  v = wave_sum(v);
  if constexpr (NT > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) part[wave] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) v += part[w];
  }
  return v;
}

template <int CTRL>
__device__ inline uint32_t dpp_umax(uint32_t m) {
  return umax2(m, (uint32_t)__builtin_amdgcn_update_dpp((int)m, (int)m, CTRL, 0xF, 0xF, false));
}
// Maximum over 16 consecutive lanes, in each of them.
__device__ inline uint32_t max16(uint32_t m) {
  return dpp_umax<0x121>(dpp_umax<0x122>(dpp_umax<0x124>(dpp_umax<0x128>(m))));
}

// A row of D columns by NT threads, each with V vectors of eight columns: vector t + NT i is thread t's
// i-th, so that neighbours read neighbouring bytes and a block of 128 columns lies in 16 neighbouring
// lanes.  The row stays in registers between its two uses.
//   h = x + residual, rstd = 1 / sqrt(mean h^2 + eps), y = h rstd w.
template <typename T, typename TW, int NT, int V, bool F8>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void rms_norm_kernel(NormArgs a) {
  constexpr int ROWS = NT < 256 ? 256 / NT : 1;
  __shared__ float part[16];
  const int t = threadIdx.x % NT;
  const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / NT;
  if (row >= a.T) return;   // NT == 64: no barrier follows; else ROWS is 1 and every row exists
  const T* X = (const T*)a.X + row * a.ldx;
  const T* R = a.R ? (const T*)a.R + row * a.ldr : nullptr;
  const TW* W = (const TW*)a.w;
  const int64_t D = a.D, Dq = F8 ? (D + 127) / 128 * 128 : D;
  float h[V][8];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t c = 8 * (int64_t)(t + NT * i);
    if (c < D) {
      load8f(X, c, D, h[i]);
      if (R) {
        float r[8];
        load8f(R, c, D, r);
#pragma unroll
        for (int q = 0; q < 8; ++q) h[i][q] += r[q];
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) sum = __builtin_fmaf(h[i][q], h[i][q], sum);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) h[i][q] = 0.f;
    }
  }
  sum = row_sum<NT>(sum, part);
  const float rstd = 1.f / sqrtf(sum / (float)D + a.eps);
  if (a.rstd && t == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t c = 8 * (int64_t)(t + NT * i);
    if (c >= Dq) continue;   // whole blocks: all of their 16 lanes go on
    if (c < D && a.H) store8f((T*)a.H + row * a.ldh, c, D, h[i]);
    float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (c < D) {
      float w[8];
      load8f(W, c, D, w);
#pragma unroll
      for (int q = 0; q < 8; ++q) y[q] = h[i][q] * rstd * w[q];
      if (a.Y) store8f((T*)a.Y + row * a.ldy, c, D, y);
    }
    if constexpr (F8) {
      Raw8<uint32_t> x;
#pragma unroll
      for (int q = 0; q < 8; ++q) x.w[q] = c + q < D ? __float_as_uint(y[q]) : 0u;
      uint32_t m = max16(x.row_max());
      if (m >= 0x7F800000u) {   // the same in a block's 16 lanes
        x.clean();
        Raw8<uint32_t> f = x;
#pragma unroll
        for (int q = 0; q < 8; ++q) f.w[q] = f.mag_finite(q);
        m = max16(f.row_max());
      }
      const float scale = power2(block_exponent(m, a.e5m2));
      const u32x2 q8 = a.e5m2 ? pack_row<true>(x, scale) : pack_row<false>(x, scale);
      __builtin_memcpy(a.Q + row * a.ldq + c, &q8, 8);
      if ((t & 15) == 0) a.S[c / 128 * a.lds + row] = scale;
    }
  }
}

// dx = dh + rstd (g - xh mean(g xh)) with g = dy w and xh = h rstd; a workgroup takes every gridDim-th
// row (NT 64: each wave its own) and sums dy xh of its rows for its columns.  The sums leave through
// `part` [gridDim][D] and are added in the order of the workgroups.
template <typename T, typename TW, int NT, int V>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void rms_norm_bwd_kernel(NormBwdArgs a, float* dw) {
  constexpr int ROWS = NT < 256 ? 256 / NT : 1;
  __shared__ float part[2][16];
  const int t = threadIdx.x % NT;
  const int64_t D = a.D;
  const TW* W = (const TW*)a.w;
  float acc[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[i][q] = 0.f;
  int buf = 0;
  for (int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / NT; row < a.T; row += (int64_t)gridDim.x * ROWS) {
    const T* dY = (const T*)a.dY + row * a.lddy;
    const T* H = (const T*)a.H + row * a.ldh;
    const float rstd = a.rstd[row];
    float g[V][8], xh[V][8];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int64_t c = 8 * (int64_t)(t + NT * i);
      if (c >= D) continue;
      float w[8];
      load8f(dY, c, D, g[i]);
      load8f(H, c, D, xh[i]);
      load8f(W, c, D, w);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        xh[i][q] *= rstd;
        acc[i][q] = __builtin_fmaf(g[i][q], xh[i][q], acc[i][q]);
        g[i][q] *= w[q];
        sum = __builtin_fmaf(g[i][q], xh[i][q], sum);
      }
    }
    sum = row_sum<NT>(sum, part[buf]);
    buf ^= 1;   // the next row's sums go to the other buffer: one barrier a row
    const float mean = sum / (float)D;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int64_t c = 8 * (int64_t)(t + NT * i);
      if (c >= D) continue;
      float d[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (a.dH) load8f((const T*)a.dH + row * a.lddh, c, D, d);
#pragma unroll
      for (int q = 0; q < 8; ++q) d[q] += rstd * (g[i][q] - xh[i][q] * mean);
      store8f((T*)a.dX + row * a.lddx, c, D, d);
    }
  }
  if constexpr (ROWS > 1) {
    // the waves' sums, added in their order
    __shared__ float sh[ROWS - 1][V * 512];
    const int wave = threadIdx.x / NT;
    if (wave > 0) {
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int q = 0; q < 8; ++q) sh[wave - 1][(i * 8 + q) * 64 + t] = acc[i][q];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int w = 0; w < ROWS - 1; ++w)
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[i][q] += sh[w][(i * 8 + q) * 64 + t];
  }
  float* out = dw + blockIdx.x * D;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t c = 8 * (int64_t)(t + NT * i);
    if (c < D) store8f((uint32_t*)out, c, D, acc[i]);
  }
}

template <typename T, typename TW, int NT, int V>
hipError_t run_fwd(const NormArgs& a, hipStream_t s) {
  constexpr int ROWS = NT < 256 ? 256 / NT : 1, TH = NT < 256 ? 256 : NT;
  return in_pieces(a.T, kPieceRows256, [&](int64_t r0, int64_t n) {
    NormArgs p = a;
    p.X = (const T*)a.X + r0 * a.ldx;
    if (a.R) p.R = (const T*)a.R + r0 * a.ldr;
    if (a.H) p.H = (T*)a.H + r0 * a.ldh;
    if (a.Y) p.Y = (T*)a.Y + r0 * a.ldy;
    if (a.Q) p.Q = a.Q + r0 * a.ldq;
    if (a.S) p.S = a.S + r0;
    if (a.rstd) p.rstd = a.rstd + r0;
    p.T = n;
    const dim3 grid((unsigned)((n + ROWS - 1) / ROWS));
    if (a.Q) hipLaunchKernelGGL((rms_norm_kernel<T, TW, NT, V, true>), grid, dim3(TH), 0, s, p);
    else hipLaunchKernelGGL((rms_norm_kernel<T, TW, NT, V, false>), grid, dim3(TH), 0, s, p);
    return hipGetLastError();
  });
}

template <typename T, typename TW, int NT, int V>
hipError_t run_bwd(const NormBwdArgs& a, hipStream_t s) {
  constexpr int TH = NT < 256 ? 256 : NT;
  const int64_t g = norm_bwd_groups(a.T, a.D);
  hipLaunchKernelGGL((rms_norm_bwd_kernel<T, TW, NT, V>), dim3((unsigned)g), dim3(TH), 0, s, a, g > 1 ? a.work : a.dw);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || g == 1 ? e : launch_sum_partials(a.work, g, a.D, a.dw, s);
}

// The threads of a row and their vectors, by its width.
template <typename T, typename TW, typename A, typename F>
hipError_t by_width(const A& a, F run) {
  const int64_t n = (a.D + 7) / 8;
  if (n <= 64) return run.template operator()<T, TW, 64, 1>(a);
  if (n <= 128) return run.template operator()<T, TW, 64, 2>(a);
  if (n <= 256) return run.template operator()<T, TW, 256, 1>(a);
  if (n <= 512) return run.template operator()<T, TW, 256, 2>(a);
  if (n <= 1024) return run.template operator()<T, TW, 256, 4>(a);
  if (n <= 2048) return run.template operator()<T, TW, 1024, 2>(a);
  return run.template operator()<T, TW, 1024, 4>(a);   // D <= 32768
}
struct Fwd {
  hipStream_t s;
  template <typename T, typename TW, int NT, int V>
  hipError_t operator()(const NormArgs& a) { return run_fwd<T, TW, NT, V>(a, s); }
};
struct Bwd {
  hipStream_t s;
  template <typename T, typename TW, int NT, int V>
  hipError_t operator()(const NormBwdArgs& a) { return run_bwd<T, TW, NT, V>(a, s); }
};
template <typename A, typename F>
hipError_t by_type(int dt, int wdt, const A& a, F run) {
  if (dt == DT_BF16)
    return wdt == DT_BF16 ? by_width<uint16_t, uint16_t>(a, run) : by_width<uint16_t, uint32_t>(a, run);
  return wdt == DT_BF16 ? by_width<uint32_t, uint16_t>(a, run) : by_width<uint32_t, uint32_t>(a, run);
}

}  // namespace

// Workgroups of the gradient, each with one row of sums: enough to fill the GPU, few enough that their
// sums stay small beside the rows.
int64_t norm_bwd_groups(int64_t T, int64_t D) {
  const int64_t rows = D <= 1024 ? 4 : 1, g = (T + rows - 1) / rows;
  return g < 512 ? g : 512;
}
hipError_t launch_rms_norm(int dt, int wdt, const NormArgs& a, hipStream_t s) { return by_type(dt, wdt, a, Fwd{s}); }
hipError_t launch_rms_norm_bwd(int dt, int wdt, const NormBwdArgs& a, hipStream_t s) {
  return by_type(dt, wdt, a, Bwd{s});
}

}  // namespace nms
