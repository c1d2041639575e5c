// Products of bf16 matrices with fp32 sums, for the dense FFN's forward (bias, activation and residual in
// the epilogue) and its gradients (the activation's derivative, or addition to the result, in the epilogue).
//
// Every kernel gives B the matrix instruction's row operand and A its column operand, so a lane holds four
// consecutive columns n of one row m of C.
#include "act.hpp"
#include "launch.hpp"
#include "pieces.hpp"

namespace nms {
namespace {

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

// Four consecutive elements from p[n] as fp32, 0 beyond N.
__device__ inline f32x4 load4(const uint16_t* p, int64_t n, int64_t N) {
  uint16_t b[4];
  if (n + 4 <= N) {
    __builtin_memcpy(b, p + n, sizeof(b));
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) b[q] = n + q < N ? p[n + q] : (uint16_t)0;
  }
  return f32x4{Elem<uint16_t>::to_f32(b[0]), Elem<uint16_t>::to_f32(b[1]), Elem<uint16_t>::to_f32(b[2]),
               Elem<uint16_t>::to_f32(b[3])};
}
__device__ inline f32x4 load4(const float* p, int64_t n, int64_t N) {
  f32x4 v;
  if (n + 4 <= N) {
    __builtin_memcpy(&v, p + n, sizeof(v));
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = n + q < N ? p[n + q] : 0.f;
  }
  return v;
}
// Four consecutive elements to p[n], bf16 rounded to nearest even; nothing beyond N.
__device__ inline void store4(uint16_t* p, int64_t n, int64_t N, const f32x4& v) {
  uint16_t b[4];
  const bf16x4 h = __builtin_convertvector(v, bf16x4);
  __builtin_memcpy(b, &h, sizeof(b));
  if (n + 4 <= N) {
    __builtin_memcpy(p + n, b, sizeof(b));
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (n + q < N) p[n + q] = b[q];
  }
}
__device__ inline void store4(float* p, int64_t n, int64_t N, const f32x4& v) {
  if (n + 4 <= N) {
    __builtin_memcpy(p + n, &v, sizeof(v));
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (n + q < N) p[n + q] = v[q];
  }
}

__device__ inline f32x4 bias4(const Linear& g, int64_t n) {
  if (!g.bias) return f32x4{0.f, 0.f, 0.f, 0.f};
  return g.bias_bf16 ? load4((const uint16_t*)g.bias, n, g.N) : load4((const float*)g.bias, n, g.N);
}
__device__ inline f32x4 act4(int act, f32x4 v) {
  with_act(act, [&](auto a) {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = act_fwd<decltype(a)::value>(v[q]);
  });
  return v;
}
__device__ inline f32x4 dact4(int act, f32x4 v) {
  with_act(act, [&](auto a) {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = act_bwd<decltype(a)::value>(v[q]);
  });
  return v;
}

// What C(m, n .. n + 3) becomes of the sums v, with n < N; everything is fp32 until the one rounding to C's type.
__device__ inline f32x4 epilogue4(const Linear& g, int64_t m, int64_t n, f32x4 v) {
  if (g.epi == EPI_FWD) {
    v += bias4(g, n);
    if (g.Z) store4(g.Z + m * g.ldz, n, g.N, v);
    v = act4(g.act, v);
    if (g.R) v += load4(g.R + m * g.ldr, n, g.N);
  } else if (g.epi == EPI_GATE) {
    v *= dact4(g.act, load4(g.P + m * g.ldp, n, g.N));
  } else if (g.accumulate) {
    v += load4((const float*)g.C + m * g.ldc, n, g.N);
  }
  return v;
}
__device__ inline void finish4(const Linear& g, int64_t m, int64_t n, const f32x4& v) {
  if (n >= g.N) return;
  const f32x4 c = epilogue4(g, m, n, v);
  if (g.bf16_out) store4((uint16_t*)g.C + m * g.ldc, n, g.N, c);
  else store4((float*)g.C + m * g.ldc, n, g.N, c);
}

// General kernel: any sizes, strides, alignments and operand orders.  64 x 64 tile, four waves of 32 x 32,
// 64 k a stage through LDS, with zeros beyond the rows and beyond K.
constexpr int GP = 72;   // LDS row pitch in elements: 64 and a shift of the banks per row
__global__ __launch_bounds__(256) void linear_general_kernel(Linear g) {
  __shared__ __align__(16) uint16_t sA[64 * GP], sB[64 * GP];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l16 = lane & 15, lq = lane >> 4;
  const int64_t m0 = (int64_t)blockIdx.x * 64, n0 = (int64_t)blockIdx.y * 64;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  f32x4 acc[2][2] = {};
  // 64 rows x 64 k in pieces of eight elements along the operand's contiguous dimension
  auto stage = [&](uint16_t* dst, const uint16_t* X, int64_t ld, bool t, int64_t r0, int64_t R, int64_t k0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int id = tid + 256 * i, line = id >> 3, c = (id & 7) * 8;
      const int64_t at = (t ? k0 : r0) + line, lines = t ? g.K : R;   // the piece's place along the stride
      const int64_t from = (t ? r0 : k0) + c, to = t ? R : g.K;       // and along the contiguous dimension
      uint16_t b[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      if (at < lines && from < to) {
        const uint16_t* p = X + at * ld + from;
        if (from + 8 <= to) {
          __builtin_memcpy(b, p, sizeof(b));
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) b[q] = from + q < to ? p[q] : (uint16_t)0;
        }
      }
      if (t) {
#pragma unroll
        for (int q = 0; q < 8; ++q) dst[(c + q) * GP + line] = b[q];
      } else {
        __builtin_memcpy(__builtin_assume_aligned(dst + line * GP + c, 16), b, sizeof(b));
      }
    }
  };
  for (int64_t k0 = 0; k0 < g.K; k0 += 64) {
    __syncthreads();
    stage(sA, g.A, g.lda, g.a_t, m0, g.M, k0);
    stage(sB, g.B, g.ldb, g.b_t, n0, g.N, k0);
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 64; kk += 32) {
      bf16x8 a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i] = *reinterpret_cast<const bf16x8*>(sA + (wm + 16 * i + l16) * GP + kk + 8 * lq);
        b[i] = *reinterpret_cast<const bf16x8*>(sB + (wn + 16 * i + l16) * GP + kk + 8 * lq);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b[j], a[i], acc[i][j], 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = m0 + wm + 16 * i + l16;
    if (m >= g.M) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j) finish4(g, m, n0 + wn + 16 * j + 4 * lq, acc[i][j]);
  }
}

hipError_t run_general(const Linear& g, hipStream_t s) {
  const int64_t ntm = (g.M + 63) / 64, ntn = (g.N + 63) / 64;
  if (ntn > 65535 || !grid_ok(ntm, 256)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(linear_general_kernel, dim3((unsigned)ntm, (unsigned)ntn), dim3(256), 0, s, g);
  return hipGetLastError();
}

hipError_t linear_piece(const Linear& g, hipStream_t s) { return run_general(g, s); }

}  // namespace

hipError_t launch_linear(const Linear& g, hipStream_t s) {
  return in_pieces(g.M, kPieceRows, [&](int64_t m0, int64_t n) {
    Linear p = g;
    p.A += g.a_t ? m0 : m0 * g.lda;
    p.M = n;
    p.C = (uint8_t*)g.C + m0 * g.ldc * (g.bf16_out ? 2 : 4);
    if (g.R) p.R += m0 * g.ldr;
    if (g.Z) p.Z += m0 * g.ldz;
    if (g.P) p.P += m0 * g.ldp;
    return linear_piece(p, s);
  });
}

}  // namespace nms
