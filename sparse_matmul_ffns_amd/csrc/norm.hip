// Root-mean-square norm of rows, with the residual's addition in front and, where asked for, an 8-bit
// result behind; and its gradients.
#include <type_traits>

#include "fp8.hpp"
#include "launch.hpp"
#include "pieces.hpp"
#include "rows8.hpp"

namespace nms {
namespace {

// Sum of v over the NT threads of a row, in every one of them: over the waves' lanes, then over the waves
// in their order.  `part` holds a value per wave.
template <int NT, typename F>
__device__ inline F row_sum(F v, F* part) {
#pragma unroll
  for (int d = 32; d >= 1; d /= 2) v += __shfl_xor(v, d);
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

// The bits of an fp32 value that lies where y lies: y's first 20 bits behind the point and, where more follow, the last of them set
// (rounding to odd).  Rounding that to 8 bits, or comparing it with a border of 8 bits, comes out as for y
// itself, ties included; rounding y's nearest fp32 value would round twice.  (Below fp32's normal numbers it is rounded again.)
__device__ inline uint32_t odd_bits(double y) {
  const uint64_t b = __builtin_bit_cast(uint64_t, y);
  const uint32_t rest = (uint32_t)b, hi = (uint32_t)(b >> 32) | (rest < 1u ? rest : 1u);
  return __float_as_uint((float)__builtin_bit_cast(double, (uint64_t)hi << 32));
}

template <bool TAIL>
__device__ inline void load_w(const void* w, int bf16, int64_t c, int64_t D, float (&v)[8]) {
  if (bf16) load8f<uint16_t, TAIL>((const uint16_t*)w, c, D, v);
  else load8f<uint32_t, TAIL>((const uint32_t*)w, c, D, v);
}

// A row of D columns by NT threads, each with V vectors of eight columns: vector t + NT i is thread t's
// i-th, so that neighbours read neighbouring bytes and a block of 128 columns lies in 16 neighbouring
// lanes.  The row stays in registers between its two uses.
//   h = x + residual, rstd = 1 / sqrt(mean h^2 + eps), y = h rstd w.
// F8: y decides between 8-bit values and scales, so everything behind the loads is 64-bit (which the vector unit does at fp32's
// rate) and y is rounded once, to 8 bits.
template <typename T, int NT, int V, bool F8, bool TAIL>
__global__ __launch_bounds__(NT == 64 ? 256 : NT) void rms_norm_kernel(NormArgs a) {
  constexpr int ROWS = NT == 64 ? 4 : 1;
  typedef std::conditional_t<F8, double, float> Sum;
  __shared__ Sum part[16];
  const int t = threadIdx.x % NT;
  int64_t group = blockIdx.x;
  if constexpr (F8) {
    // Workgroups are dealt to the 8 XCDs in turn; an XCD takes a run of rows, so that their scales, which
    // lie together, meet in its L2
    const int64_t x = group % 8, per = gridDim.x / 8, rest = gridDim.x % 8;
    group = x * per + (x < rest ? x : rest) + group / 8;
  }
  const int64_t row = group * ROWS + threadIdx.x / NT;
  if (row >= a.T) return;   // NT 64: no barrier follows; else ROWS is 1 and every row exists
  const T* X = (const T*)a.X + row * a.ldx;
  const T* R = a.R ? (const T*)a.R + row * a.ldr : nullptr;
  const int64_t D = a.D, Dq = F8 ? (D + 127) / 128 * 128 : D;
  Row8<T> x[V], r[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t c = 8 * (int64_t)(t + NT * i);
    if (c < D) {
      x[i].template load<TAIL>(X, c, D);
      if (R) r[i].template load<TAIL>(R, c, D);
    }
  }
  Sum h[V][8], sum = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t c = 8 * (int64_t)(t + NT * i);
#pragma unroll
    for (int q = 0; q < 8; ++q) h[i][q] = 0;
    if (c >= D) continue;
    float f[8];
    x[i].get(f);
#pragma unroll
    for (int q = 0; q < 8; ++q) h[i][q] = (Sum)f[q];
    if (R) {
      float e[8];
      r[i].get(e);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        f[q] += e[q];
        if constexpr (F8) h[i][q] += (double)e[q];
        else h[i][q] = f[q];
      }
    }
    if (a.H) store8f<T, TAIL>((T*)a.H + row * a.ldh, c, D, f);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if constexpr (F8) sum = __builtin_fma(h[i][q], h[i][q], sum);
      else sum = __builtin_fmaf(h[i][q], h[i][q], sum);
    }
  }
  sum = row_sum<NT>(sum, part);
  Sum rho;
  if constexpr (F8) {
    // two Newton steps in 64 bits from the 32-bit result (the second for its last eight bits), of the mean scaled by a power of four: fp32 does
    // not hold the squares of all fp32 rows
    const double m = sum / (double)D + (double)a.eps;
    const int k = __builtin_amdgcn_frexp_exp(m) >> 1;
    const double n = __builtin_amdgcn_ldexp(m, -2 * k);
    rho = (double)(1.f / sqrtf((float)n));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const double e = rho * __builtin_fma(-0.5 * n * rho, rho, 1.5);
      rho = __builtin_isfinite(e) ? e : rho;   // an infinite sum's 0 stays
    }
    rho = __builtin_amdgcn_ldexp(rho, -k);
  } else {
    rho = 1.f / sqrtf(sum / (float)D + a.eps);
  }
  const float rstd = (float)rho;
  if (a.rstd && t == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t c = 8 * (int64_t)(t + NT * i);
    if (c >= Dq) continue;   // whole blocks: all of their 16 lanes go on
    float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    Raw8<uint32_t> v;
    if constexpr (F8) v.zero();
    if (c < D) {
      float w[8];
      load_w<TAIL>(a.w, a.w_bf16, c, D, w);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const Sum p = h[i][q] * rho * (Sum)w[q];
        y[q] = (float)p;
        if constexpr (F8) {
          v.w[q] = !TAIL || c + q < D ? odd_bits(p) : 0u;
          if constexpr (sizeof(T) == 2) y[q] = __uint_as_float(v.w[q]);   // for its one rounding to bf16
        }
      }
      if (a.Y) store8f<T, TAIL>((T*)a.Y + row * a.ldy, c, D, y);
    }
    if constexpr (F8) {
      uint32_t m = max16(v.row_max());
      if (m >= 0x7F800000u) {   // the same in a block's 16 lanes
        v.clean();
        Raw8<uint32_t> f = v;
#pragma unroll
        for (int q = 0; q < 8; ++q) f.w[q] = f.mag_finite(q);
        m = max16(f.row_max());
      }
      const float scale = power2(block_exponent(m, a.e5m2));
      const u32x2 q8 = a.e5m2 ? pack_row<true>(v, scale) : pack_row<false>(v, scale);
      __builtin_memcpy(a.Q + row * a.ldq + c, &q8, 8);
      if ((t & 15) == 0) a.S[c / 128 * a.lds + row] = scale;
    }
  }
}

// dx = dh + rstd (g - xh mean(g xh)) with g = dy w and xh = h rstd; a workgroup takes every gridDim-th
// row (NT 64: each wave its own) and sums dy xh of its rows for its columns.  The sums leave through
// `part` [gridDim][D] and are added in the order of the workgroups.  A row is kept as it lies in memory and widened twice.
// AHEAD: its loads are issued before the row in front of it is reduced (the widest rows leave no registers for that).
template <typename T, int NT, int V, bool DH, bool TAIL>
__global__ __launch_bounds__(NT == 64 ? 256 : NT) void rms_norm_bwd_kernel(NormBwdArgs a, float* dw) {
  constexpr int ROWS = NT == 64 ? 4 : 1;
  constexpr bool AHEAD = NT < 1024;
  __shared__ float part[2][16];
  const int t = threadIdx.x % NT;
  const int64_t D = a.D, step = (int64_t)gridDim.x * ROWS;
  float acc[V][8], wk[AHEAD ? V : 1][8];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t c = 8 * (int64_t)(t + NT * i);
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[i][q] = 0.f;
    if constexpr (AHEAD) {
#pragma unroll
      for (int q = 0; q < 8; ++q) wk[i][q] = 0.f;
      if (c < D) load_w<TAIL>(a.w, a.w_bf16, c, D, wk[i]);
    }
  }
  struct Row {
    Row8<T> dy[V], h[V], dh[DH && AHEAD ? V : 1];
    float rstd;
  };
  auto fetch = [&](int64_t row, Row& x) {
    if (row >= a.T) return;
    x.rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int64_t c = 8 * (int64_t)(t + NT * i);
      if (c >= D) continue;
      x.dy[i].template load<TAIL>((const T*)a.dY + row * a.lddy, c, D);
      x.h[i].template load<TAIL>((const T*)a.H + row * a.ldh, c, D);
      if constexpr (DH && AHEAD) x.dh[i].template load<TAIL>((const T*)a.dH + row * a.lddh, c, D);
    }
  };
  // dy, xh and w of a thread's vector i
  auto widen = [&](const Row& x, int i, int64_t c, float (&dy)[8], float (&xh)[8], float (&w)[8]) {
    x.dy[i].get(dy);
    x.h[i].get(xh);
    if constexpr (!AHEAD) load_w<TAIL>(a.w, a.w_bf16, c, D, w);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      xh[q] *= x.rstd;
      if constexpr (AHEAD) w[q] = wk[i][q];
    }
  };
  int buf = 0;
  auto work = [&](int64_t row, const Row& x) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int64_t c = 8 * (int64_t)(t + NT * i);
      if (c >= D) continue;
      float dy[8], xh[8], w[8];
      widen(x, i, c, dy, xh, w);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        acc[i][q] = __builtin_fmaf(dy[q], xh[q], acc[i][q]);
        sum = __builtin_fmaf(dy[q] * w[q], xh[q], sum);
      }
    }
    sum = row_sum<NT>(sum, part[buf]);
    buf ^= 1;   // the next row's sums go to the other buffer: one barrier a row
    const float mean = sum / (float)D;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int64_t c = 8 * (int64_t)(t + NT * i);
      if (c >= D) continue;
      float dy[8], xh[8], w[8], d[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if constexpr (DH && AHEAD) x.dh[i].get(d);
      if constexpr (DH && !AHEAD) load8f<T, TAIL>((const T*)a.dH + row * a.lddh, c, D, d);
      widen(x, i, c, dy, xh, w);
#pragma unroll
      for (int q = 0; q < 8; ++q) d[q] += x.rstd * (dy[q] * w[q] - xh[q] * mean);
      store8f<T, TAIL>((T*)a.dX + row * a.lddx, c, D, d);
    }
  };
  int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / NT;
  if constexpr (AHEAD) {
    Row x, y;
    fetch(row, x);
    while (row < a.T) {
      fetch(row + step, y);
      work(row, x);
      row += step;
      if (row >= a.T) break;
      fetch(row + step, x);
      work(row, y);
      row += step;
    }
  } else {
    for (; row < a.T; row += step) {
      Row x;
      fetch(row, x);
      work(row, x);
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
    for (int k = 0; k < ROWS - 1; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[i][q] += sh[k][(i * 8 + q) * 64 + t];
  }
  float* out = dw + blockIdx.x * D;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t c = 8 * (int64_t)(t + NT * i);
    if (c < D) store8f<uint32_t, TAIL>((uint32_t*)out, c, D, acc[i]);
  }
}

template <typename T, int NT, int V>
hipError_t run_fwd(const NormArgs& a, hipStream_t s) {
  constexpr int ROWS = NT == 64 ? 4 : 1, TH = NT * ROWS;
  constexpr int64_t PIECE = (int64_t(1) << 30) / NT;   // rows of a launch: 2^30 work-items
  return in_pieces(a.T, PIECE, [&](int64_t r0, int64_t n) {
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
    auto go = [&](auto f8, auto tail) {
      hipLaunchKernelGGL((rms_norm_kernel<T, NT, V, decltype(f8)::value, decltype(tail)::value>), grid, dim3(TH), 0, s, p);
    };
    const std::true_type yes;
    const std::false_type no;
    if (a.Q) a.D % 8 ? go(yes, yes) : go(yes, no);
    else a.D % 8 ? go(no, yes) : go(no, no);
    return hipGetLastError();
  });
}

template <typename T, int NT, int V>
hipError_t run_bwd(const NormBwdArgs& a, hipStream_t s) {
  constexpr int TH = NT == 64 ? 256 : NT;
  const int64_t g = norm_bwd_groups(a.T, a.D);
  float* out = g > 1 ? a.work : a.dw;
  auto go = [&](auto dh, auto tail) {
    hipLaunchKernelGGL((rms_norm_bwd_kernel<T, NT, V, decltype(dh)::value, decltype(tail)::value>), dim3((unsigned)g), dim3(TH),
                       0, s, a, out);
  };
  const std::true_type yes;
  const std::false_type no;
  if (a.dH) a.D % 8 ? go(yes, yes) : go(yes, no);
  else a.D % 8 ? go(no, yes) : go(no, no);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || g == 1 ? e : launch_sum_partials(a.work, g, a.D, a.dw, s);
}

// The threads of a row and their vectors, by its width (at most 16384).  Measured on bf16 rows that are not in
// a cache, us: 8192 x 4096 with a residual (268 MB) 44.5 with 256 threads, 43.4 with 128, 49 with 64, 51 with 1024 (its gradients, 268 MB,
// 48.7, 55.6, - and 75); 64 x 4096 3.6, 4.3, 5.5, 3.3; 4096 x 2048 13.0, 11.3, 11.6, 16.9; 4096 x 8192 45.5 with 256 and 44.0 with 512.  To 8
// bits 4096 x 2048 takes 15.3 (with 32-bit products 15.2, which with 64 threads a row were 0.7 slower, and 1.1 before an XCD's workgroups took
// neighbouring rows).
template <typename T>
hipError_t fwd_by_width(const NormArgs& a, hipStream_t s) {
  const int64_t n = (a.D + 7) / 8;
  if (n <= 64) return run_fwd<T, 64, 1>(a, s);
  if (n <= 128) return run_fwd<T, 64, 2>(a, s);
  if (n <= 256) return run_fwd<T, 128, 2>(a, s);
  if (n <= 512) return run_fwd<T, 256, 2>(a, s);
  if (n <= 1024) return run_fwd<T, 512, 2>(a, s);
  return run_fwd<T, 1024, 2>(a, s);
}
template <typename T>
hipError_t bwd_by_width(const NormBwdArgs& a, hipStream_t s) {
  const int64_t n = (a.D + 7) / 8;
  if (n <= 64) return run_bwd<T, 64, 1>(a, s);
  if (n <= 128) return run_bwd<T, 64, 2>(a, s);
  if (n <= 256) return run_bwd<T, 256, 1>(a, s);
  if (n <= 512) return run_bwd<T, 256, 2>(a, s);
  if (n <= 1024) return run_bwd<T, 512, 2>(a, s);
  return run_bwd<T, 1024, 2>(a, s);
}

}  // namespace

// Workgroups of the gradient, each with a row of sums: enough to fill the GPU, few enough that their
// sums stay small beside the rows.  8192 x 4096 takes 53.3, 48.7, 54.7, 62.0 us with 256, 512, 1024, 2048; 4096 x 8192 47.9 and
// 53.1, 2048 x 16384 61.1 and 67.1 with 256 and 512.
int64_t norm_bwd_groups(int64_t T, int64_t D) {
  const int64_t rows = D <= 1024 ? 4 : 1, g = (T + rows - 1) / rows, most = D <= 4096 ? 512 : 256;
  return g < most ? g : most;
}
hipError_t launch_rms_norm(int dt, const NormArgs& a, hipStream_t s) {
  return dt == DT_BF16 ? fwd_by_width<uint16_t>(a, s) : fwd_by_width<uint32_t>(a, s);
}
hipError_t launch_rms_norm_bwd(int dt, const NormBwdArgs& a, hipStream_t s) {
  return dt == DT_BF16 ? bwd_by_width<uint16_t>(a, s) : bwd_by_width<uint32_t>(a, s);
}

}  // namespace nms
