// Products of 8-bit matrices with a scale for each block of 128 along the reduction: one product,
// one per group of A's rows, or one per run of the reduction.
//
// v_mfma_f32_16x16x128_f8f6f4 spans exactly one scale block: its result is the block's fp32 sum,
// which the vector unit scales and adds to the accumulator.  B takes the instruction's row operand
// and A its column operand, so a lane holds four consecutive columns n of one row m of C.
#include "common.hpp"
#include "launch.hpp"

namespace nms {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// D[i][j] = sum_k X[i][k] Y[j][k] over 128 k; fx, fy: 0 e4m3, 1 e5m2.
template <int FX, int FY>
__device__ inline f32x4 mfma128(i32x8 x, i32x8 y) {
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, zero, FX, FY, 0, 0, 0, 0);
}

// What a workgroup computes: rows m0 .. m_end - 1 (at most a tile of them) of A and C times B's rows
// from n0, over the 128-blocks kb0 .. kb1 - 1.
struct Tile {
  int64_t m0, m_end, n0, kb0, kb1;
  int e;       // group
  bool zero;   // rows of no group: C is cleared
};

__device__ inline int clamp_off(int v, int64_t rows) { return v < 0 ? 0 : (v > rows ? (int)rows : v); }

// Row tile t of the groups' rows, BM rows at a time per group, then of the rows behind the last
// group (and before the first).  Every wave finds it by itself: 64 groups at a time, an inclusive
// sum of their tile counts over the lanes, and the first lane whose sum exceeds t.
template <int BM>
__device__ inline bool find_rows(const Fp8Gemm& g, int64_t t, Tile& out) {
  const int lane = threadIdx.x & 63;
  int64_t before = 0;
  int end = 0, first = 0;   // rows covered so far
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    const int e = e0 + lane;
    int lo = 0, hi = 0;
    if (e < g.E) {
      lo = clamp_off(g.offsets[e], g.M);
      hi = clamp_off(g.offsets[e + 1], g.M);
      hi = hi < lo ? lo : hi;
    }
    if (e0 == 0) first = __shfl(lo, 0);
    int sum = (hi - lo + BM - 1) / BM;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int o = __shfl_up(sum, d);
      if (lane >= d) sum += o;
    }
    const uint64_t past = __ballot(before + sum > t);
    if (past) {
      const int w = __builtin_ctzll(past);
      const int64_t prev = before + (w ? __shfl(sum, w - 1) : 0);
      const int glo = __shfl(lo, w), ghi = __shfl(hi, w);
      out.e = e0 + w;
      out.m0 = glo + (t - prev) * BM;
      out.m_end = out.m0 + BM < ghi ? out.m0 + BM : ghi;
      out.zero = false;
      return true;
    }
    before += __shfl(sum, 63);
    const int last = __shfl(hi, g.E - 1 - e0 < 63 ? g.E - 1 - e0 : 63);
    end = last;
  }
  // the rows of no group: [0, first) and [end, M)
  t -= before;
  const int64_t head = (first + BM - 1) / BM;
  out.e = 0;
  out.zero = true;
  if (t < head) {
    out.m0 = t * BM;
    out.m_end = out.m0 + BM < first ? out.m0 + BM : first;
    return true;
  }
  out.m0 = end + (t - head) * BM;
  out.m_end = out.m0 + BM < g.M ? out.m0 + BM : g.M;
  return out.m0 < g.M;
}

__device__ inline void store4(const Fp8Gemm& g, int64_t crow, int64_t n, const float (&v)[4]) {
  if (g.bf16_out) {
    uint16_t* p = (uint16_t*)g.C + crow * g.ldc + n;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < g.N) p[i] = f32_to_bf16_rne(v[i]);
  } else {
    float* p = (float*)g.C + crow * g.ldc + n;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < g.N) p[i] = v[i];
  }
}

// General kernel: any sizes, strides and alignments.  64 x 64 tile, four waves of 32 x 32; each
// 128-block of both operands goes through LDS byte by byte where the rows are not 16-byte aligned,
// with zeros beyond the rows and beyond K.
constexpr int GP = 144;   // LDS row pitch: 128 bytes and a shift of the banks per row
template <int FA, int FB>
__global__ __launch_bounds__(256) void fp8_gemm_general_kernel(Fp8Gemm g, bool vec_a, bool vec_b) {
  __shared__ __align__(16) unsigned char sA[64 * GP], sB[64 * GP];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l16 = lane & 15, lq = lane >> 4;
  Tile t;
  t.n0 = (int64_t)blockIdx.y * 64;
  t.kb0 = 0;
  t.kb1 = (g.K + 127) / 128;
  t.zero = false;
  t.e = 0;
  if (g.mode == G_ROWS) {
    if (!find_rows<64>(g, blockIdx.x, t)) return;
  } else {
    t.m0 = (int64_t)blockIdx.x * 64;
    t.m_end = t.m0 + 64 < g.M ? t.m0 + 64 : g.M;
    if (g.mode == G_RED) {
      t.e = blockIdx.z;
      t.kb0 = clamp_off(g.offsets[t.e], g.K) / 128;
      t.kb1 = clamp_off(g.offsets[t.e + 1], g.K) / 128;
    }
  }
  const int64_t crow0 = g.mode == G_RED ? (int64_t)t.e * g.M : 0;
  const uint8_t* B = g.B;
  const float* sb = g.sb;
  if (g.mode == G_ROWS) {
    B += (int64_t)t.e * g.N * g.ldb;
    sb += (int64_t)t.e * ((g.N + 127) / 128) * g.ldsb;
  }
  if (t.zero) t.kb1 = t.kb0;

  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  float acc[2][2][4] = {};   // [m fragment][n fragment][n]
  auto stage = [&](unsigned char* dst, const uint8_t* X, int64_t ld, int64_t r0, int64_t r_end, int64_t k0, bool vec) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int id = tid + 256 * i, r = id >> 3, c = (id & 7) * 16;
      const int64_t row = r0 + r, k = k0 + c;
      u32x4 v = {0, 0, 0, 0};
      if (row < r_end && k < g.K) {
        const uint8_t* p = X + row * ld + k;
        if (vec && k + 16 <= g.K) {
          v = *reinterpret_cast<const u32x4*>(p);
        } else {
          unsigned char b[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) b[q] = k + q < g.K ? p[q] : 0;
          __builtin_memcpy(&v, b, 16);
        }
      }
      *reinterpret_cast<u32x4*>(dst + r * GP + c) = v;
    }
  };
  auto frag = [&](const unsigned char* s, int row) {
    i32x8 v;
    u32x4* h = reinterpret_cast<u32x4*>(&v);
    h[0] = *reinterpret_cast<const u32x4*>(s + row * GP + lq * 32);
    h[1] = *reinterpret_cast<const u32x4*>(s + row * GP + lq * 32 + 16);
    return v;
  };
  for (int64_t kb = t.kb0; kb < t.kb1; ++kb) {
    __syncthreads();
    stage(sA, g.A, g.lda, t.m0, t.m_end, kb * 128, vec_a);
    stage(sB, B, g.ldb, t.n0, g.N, kb * 128, vec_b);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t m = t.m0 + wm + i * 16 + l16;
      const float sam = m < t.m_end ? g.sa[kb * g.ldsa + m] : 0.f;
      const i32x8 fa = frag(sA, wm + i * 16 + l16);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t n = t.n0 + wn + j * 16 + lq * 4;
        const f32x4 p = mfma128<FB, FA>(frag(sB, wn + j * 16 + l16), fa);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float sbn = 0.f;
          if (n + q < g.N) sbn = g.b_block == 1 ? sb[kb * g.ldsb + n + q] : sb[(n + q) / 128 * g.ldsb + kb];
          if (m < t.m_end && n + q < g.N) acc[i][j][q] += p[q] * (sam * sbn);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = t.m0 + wm + i * 16 + l16;
    if (m >= t.m_end) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j) store4(g, crow0 + m, t.n0 + wn + j * 16 + lq * 4, acc[i][j]);
  }
}

template <int FA, int FB>
hipError_t run_general(const Fp8Gemm& g, hipStream_t s) {
  const bool va = (uintptr_t)g.A % 16 == 0 && g.lda % 16 == 0, vb = (uintptr_t)g.B % 16 == 0 && g.ldb % 16 == 0;
  const int64_t ntn = (g.N + 63) / 64;
  const int64_t ntm = g.mode == G_ROWS ? g.M / 64 + g.E + 2 : (g.M + 63) / 64;
  hipLaunchKernelGGL((fp8_gemm_general_kernel<FA, FB>), dim3((unsigned)ntm, (unsigned)ntn, g.mode == G_RED ? g.E : 1),
                     dim3(256), 0, s, g, va, vb);
  return hipGetLastError();
}

template <int FA, int FB>
hipError_t run(const Fp8Gemm& g, hipStream_t s) {
  return run_general<FA, FB>(g, s);
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8Gemm& g, hipStream_t s) {
  if (g.a_e5m2) return g.b_e5m2 ? run<1, 1>(g, s) : run<1, 0>(g, s);
  return g.b_e5m2 ? run<0, 1>(g, s) : run<0, 0>(g, s);
}

}  // namespace nms
