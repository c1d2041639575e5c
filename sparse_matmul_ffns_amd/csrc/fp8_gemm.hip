// Products of 8-bit matrices with a scale for each block of 128 along the reduction: one product,
// one per group of A's rows, or one per run of the reduction.
//
// v_mfma_f32_16x16x128_f8f6f4 spans exactly one scale block: its result is the block's sum, which the
// vector unit scales and adds to the fp32 accumulator.  B takes the instruction's row operand
// and A its column operand, so a lane holds four consecutive columns n of one row m of C.
#include "common.hpp"
#include "dma.hpp"
#include "launch.hpp"
#include "pieces.hpp"

namespace nms {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

// Eight 8-bit values (F: 0 e4m3, 1 e5m2) as bf16, exactly.
template <int F>
__device__ inline bf16x8 widen8(uint32_t lo, uint32_t hi) {
  u32x4 w;
  if constexpr (F) {
    w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.f, false));
    w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(lo, 1.f, true));
    w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.f, false));
    w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(hi, 1.f, true));
  } else {
    w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false));
    w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true));
    w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false));
    w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true));
  }
  return __builtin_bit_cast(bf16x8, w);
}

// D[i][j] = sum_k X[i][k] Y[j][k] over 128 k, a lane holding 32 k of row l % 16 of each (the same ones);
// FX, FY: 0 e4m3, 1 e5m2.  The 8-bit matrix instruction aligns the products of eight consecutive bytes of
// a lane (k = 8 i .. 8 i + 7 in every kernel here) to the largest 2^(ea + eb) = u of them and cuts each
// to a multiple of 2^-13 u, towards zero; across the eights it adds like fp32.  Less than 7 * 2^-13 u for
// each eight, 1.5e-5 of the result of normal operands (root mean square).  A bf16 result's own rounding
// is up to 2^-8 of it, so bf16 results take this; where an eight's large products cancel, the loss shows.
// EXACT (fp32 results): the bytes widened to bf16 and four bf16 instructions, whose products and sums
// are fp32, at half the rate.
template <int FX, int FY, bool EXACT>
__device__ inline f32x4 mfma128(i32x8 x, i32x8 y) {
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  if constexpr (!EXACT) return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, zero, FX, FY, 0, 0, 0, 0);
  f32x4 d = zero;
#pragma unroll
  for (int s = 0; s < 4; ++s)
    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<FX>(x[2 * s], x[2 * s + 1]), widen8<FY>(y[2 * s], y[2 * s + 1]), d,
                                               0, 0, 0);
  return d;
}

// What a workgroup computes: rows m0 .. m_end - 1 (at most a tile of them) of A and C times B's rows
// from n0, over the 128-blocks kb0 .. kb1 - 1.
struct Tile {
  int64_t m0, m_end, n0, kb0, kb1;
  int e;       // group
  bool zero;   // rows of no group: C is cleared
};

__device__ inline int clamp_off(int v, int64_t rows) { return v < 0 ? 0 : (v > rows ? (int)rows : v); }

// The row tiles of a grouped product: every group's rows BM at a time, in order, then the rows before
// the first group and those behind the last (which are cleared).  Every wave counts them by itself, 64
// groups at a time: a sum of the tile counts over the lanes.
struct RowTiles {
  int64_t grouped;    // tiles of the groups
  int64_t total;
  int first, end;     // rows [0, first) and [end, M) belong to no group
};
__device__ inline void group_rows(const Fp8Gemm& g, int e, int& lo, int& hi) {
  lo = hi = 0;
  if (e < g.E) {
    lo = clamp_off(g.offsets[e], g.M);
    hi = clamp_off(g.offsets[e + 1], g.M);
    hi = hi < lo ? lo : hi;
  }
}
__device__ inline int wave_scan(int v, int lane) {   // sum of the lanes up to and including this one
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}
template <int BM>
__device__ inline RowTiles count_rows(const Fp8Gemm& g) {
  const int lane = threadIdx.x & 63;
  RowTiles r;
  int sum = 0;
  for (int e = lane; e < g.E; e += 64) {
    int lo, hi;
    group_rows(g, e, lo, hi);
    sum += (hi - lo + BM - 1) / BM;
  }
  r.grouped = __builtin_amdgcn_readlane(wave_scan(sum, lane), 63);
  r.first = clamp_off(g.offsets[0], g.M);
  const int last = clamp_off(g.offsets[g.E], g.M);
  r.end = last < r.first ? r.first : last;
  r.total = r.grouped + (r.first + BM - 1) / BM + (g.M - r.end + BM - 1) / BM;
  return r;
}
// Row tile t < r.total.
template <int BM>
__device__ inline void find_rows(const Fp8Gemm& g, const RowTiles& r, int64_t t, Tile& out) {
  const int lane = threadIdx.x & 63;
  if (t >= r.grouped) {
    t -= r.grouped;
    const int64_t head = (r.first + BM - 1) / BM;
    const bool front = t < head;
    const int64_t stop = front ? r.first : g.M;
    out.e = 0;
    out.zero = true;
    out.m0 = front ? t * BM : r.end + (t - head) * BM;
    out.m_end = out.m0 + BM < stop ? out.m0 + BM : stop;
    return;
  }
  int64_t before = 0;
  out.zero = false;
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    int lo, hi;
    group_rows(g, e0 + lane, lo, hi);
    const int sum = wave_scan((hi - lo + BM - 1) / BM, lane);
    const uint64_t past = __ballot(before + sum > t);
    if (past) {
      const int w = __builtin_ctzll(past);   // the first lane whose sum exceeds t
      const int64_t prev = before + (w ? __builtin_amdgcn_readlane(sum, w - 1) : 0);
      const int glo = __builtin_amdgcn_readlane(lo, w), ghi = __builtin_amdgcn_readlane(hi, w);
      out.e = e0 + w;
      out.m0 = glo + (t - prev) * BM;
      out.m_end = out.m0 + BM < ghi ? out.m0 + BM : ghi;
      return;
    }
    before += __builtin_amdgcn_readlane(sum, 63);
  }
}

// Four consecutive elements of row crow of C from column n: one store when the row allows it (vec),
// else one at a time.
template <typename T>
__device__ inline void store4(T* p, int64_t n, int64_t N, bool vec, const f32x4& v) {
  T b[4];
  if constexpr (sizeof(T) == 2) {
    const bf16x4 h = __builtin_convertvector(v, bf16x4);   // nearest even
    __builtin_memcpy(b, &h, sizeof(b));
  } else {
    __builtin_memcpy(b, &v, sizeof(b));
  }
  if (vec && n + 4 <= N) {
    __builtin_memcpy(__builtin_assume_aligned(p + n, 4 * sizeof(T)), b, sizeof(b));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) p[n + i] = b[i];
  }
}
__device__ inline void store4(const Fp8Gemm& g, int64_t crow, int64_t n, const f32x4& v) {
  const bool vec = g.ldc % 4 == 0 && (uintptr_t)g.C % (g.bf16_out ? 8 : 16) == 0;
  if (g.bf16_out) store4((uint16_t*)g.C + crow * g.ldc, n, g.N, vec, v);
  else store4((float*)g.C + crow * g.ldc, n, g.N, vec, v);
}

// A wave's FM x FN fragments to rows 0 .. rows - 1 and columns n .. of C.  A fragment's row is 16
// columns in four lanes (64 bytes of fp32).  Stored as they lie, a wave's store touches 16 half lines;
// two exchanges make it eight whole 128-byte lines, which (stored non-temporally: half lines and ordinary
// stores gain nothing alone) took the experts' fp32 weight gradients, then of the
// 8-bit instruction, from 255 to 173 us:
//   - bf16: the 16-lane rows of two neighbouring fragments are swapped so that a lane holds eight
//     consecutive columns (16 bytes) of one of them;
//   - lanes 0-7 and 8-15 of each 16 trade, so that one store holds rows 0-7 of two such 64-byte runs
//     and the next rows 8-15.
template <int FM, int FN, typename T>
__device__ inline void store_tile(const f32x4 (&acc)[FM][FN], T* C, int64_t ldc, int rows, int64_t n, int64_t N, int lane) {
  constexpr bool BF = sizeof(T) == 2;
  constexpr int STEP = BF ? 4 : 2;   // fragments in a 128-byte run
  static_assert(FN % STEP == 0, "");
  const int l16 = lane & 15, lq = lane >> 4;
  if ((uintptr_t)C % 16 == 0 && (ldc * (int64_t)sizeof(T)) % 16 == 0) {
    const bool low = l16 < 8;
    constexpr int PER = 16 / (int)sizeof(T);   // elements a store
    // this lane's place in a run: its half, and its 16 bytes of that half
    const int64_t col = n + (low ? 0 : 64 / (int)sizeof(T)) + (BF ? (lq & 1) * 2 + (lq >> 1) : lq) * PER;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
      for (int j = 0; j < FN; j += STEP) {
        u32x4 u, v;
        if constexpr (BF) {
          auto pair = [&](const f32x4& x, const f32x4& y) {
            const u32x2 a = __builtin_bit_cast(u32x2, __builtin_convertvector(x, bf16x4));   // nearest even
            const u32x2 b = __builtin_bit_cast(u32x2, __builtin_convertvector(y, bf16x4));
            const auto r0 = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
            const auto r1 = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
            return u32x4{r0[0], r1[0], r0[1], r1[1]};
          };
          u = pair(acc[i][j], acc[i][j + 1]);
          v = pair(acc[i][j + STEP - 2], acc[i][j + STEP - 1]);
        } else {
          u = __builtin_bit_cast(u32x4, acc[i][j]);
          v = __builtin_bit_cast(u32x4, acc[i][j + 1]);
        }
        u32x4 first, second;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t t = low ? v[q] : u[q];
          const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)t, (int)t, 0x128, 0xF, 0xF, false);   // lane ^ 8
          first[q] = low ? u[q] : o;
          second[q] = low ? o : v[q];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 16 * i + 8 * h + (l16 & 7);
          const int64_t c = col + 16 * j;
          if (r >= rows) continue;
          const u32x4 w = h ? second : first;
          T* p = C + r * ldc + c;
          if (c + PER <= N) {
            __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(p));
          } else {
            T e[PER];
            __builtin_memcpy(e, &w, 16);
#pragma unroll
            for (int q = 0; q < PER; ++q)
              if (c + q < N) p[q] = e[q];
          }
        }
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    if (16 * i + l16 >= rows) continue;
#pragma unroll
    for (int j = 0; j < FN; ++j) store4(C + (16 * i + l16) * ldc, n + 16 * j + 4 * lq, N, false, acc[i][j]);
  }
}

// General kernel: any sizes, strides and alignments.  64 x 64 tile, four waves of 32 x 32; each
// 128-block of both operands goes through LDS byte by byte where the rows are not 16-byte aligned,
// with zeros beyond the rows and beyond K.
constexpr int GP = 144;   // LDS row pitch: 128 bytes and a shift of the banks per row
template <int FA, int FB, bool EXACT>
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
    const RowTiles r = count_rows<64>(g);
    if (blockIdx.x >= r.total) return;
    find_rows<64>(g, r, blockIdx.x, t);
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
  f32x4 acc[2][2] = {};   // [m fragment][n fragment], four n a lane
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
        const f32x4 p = mfma128<FB, FA, EXACT>(frag(sB, wn + j * 16 + l16), fa);
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

// The most row tiles that M rows in E groups can make: a partial one per group and at both ends, and
// never more than one per row.
int64_t most_row_tiles(const Fp8Gemm& g, int bm) {
  const int64_t n = g.M / bm + g.E + 2;
  return n < g.M ? n : g.M;
}

template <int FA, int FB>
hipError_t run_general(const Fp8Gemm& g, hipStream_t s) {
  const bool va = (uintptr_t)g.A % 16 == 0 && g.lda % 16 == 0, vb = (uintptr_t)g.B % 16 == 0 && g.ldb % 16 == 0;
  const int64_t ntn = (g.N + 63) / 64;
  const int64_t ntm = g.mode == G_ROWS ? most_row_tiles(g, 64) : (g.M + 63) / 64;
  if (!grid_ok(ntm, 256)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)ntm, (unsigned)ntn, g.mode == G_RED ? g.E : 1);
  if (g.bf16_out) hipLaunchKernelGGL((fp8_gemm_general_kernel<FA, FB, false>), grid, dim3(256), 0, s, g, va, vb);
  else hipLaunchKernelGGL((fp8_gemm_general_kernel<FA, FB, true>), grid, dim3(256), 0, s, g, va, vb);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Tiled kernel: BM x BN tiles of C, 128-k stages of both operands in two LDS buffers filled by
// direct-to-LDS loads, which for stage kt + 1 are in flight while stage kt is computed.
//
// An LDS row is 128 bytes of one row, its 16-byte chunk c at slot c ^ (row / 2 % 8): sixteen rows' reads
// of the same chunk cover all 64 banks once.  A wave computes TM rows of A by TN rows of B as fragments of 16 x 16:
// it keeps the TM / 16 fragments of A for the stage and walks over B's, so that per B fragment TM / 16
// matrix instructions run while the vector unit scales the previous fragment's results.  Two waves per
// SIMD (their accumulators stay in vector registers: the scaling cannot read accumulation registers).
// 8192 x 16384 x 4096 with bf16 results 471 to 500 us (2.2 to 2.3 PFLOP/s): the matrix cores are busy 54% of the
// cycles, vector instructions 44%; 8192 x 2048 x 4096 with fp32 results 139 to 145 us, 41% and 57%.
// The scales of a stage are a row of floats behind the operands, loaded the same way.
// ---------------------------------------------------------------------------
template <int BM_, int BN_, int WM_, int WN_, int D_>
struct TileCfg {
  static constexpr int D = D_;   // how many slots ahead B's fragments are read
  static constexpr int BM = BM_, BN = BN_, WAVES_M = WM_, WAVES_N = WN_, WAVES = WM_ * WN_, NT = 64 * WAVES;
  static constexpr int TM = BM / WAVES_M, TN = BN / WAVES_N, FM = TM / 16, FN = TN / 16;
  static constexpr int OPER = (BM + BN) * 128, STAGE = OPER + (BM + BN) * 4, LDS = 2 * STAGE;
  static constexpr int LOADS = OPER / 1024 / WAVES;   // 16-byte loads a lane and stage
  static_assert((BM + BN) / 64 == WAVES, "one load of 64 scales a wave");
};

template <int FA, int FB, bool ROWB, bool EXACT, typename Cfg>
__global__ __launch_bounds__(Cfg::NT, 2) void fp8_gemm_tile_kernel(Fp8Gemm g) {
  constexpr int BM = Cfg::BM, BN = Cfg::BN, FM = Cfg::FM, FN = Cfg::FN;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  const int ntn = (int)((g.N + BN - 1) / BN);

  Tile t;
  t.e = 0;
  t.zero = false;
  t.kb0 = 0;
  t.kb1 = (g.K + 127) / 128;
  if (g.mode == G_ROWS) {
    // XCD x takes a run of the row tiles that there are, all column tiles of one after the other
    const RowTiles r = count_rows<BM>(g);
    const int x = blockIdx.x % 8, local = blockIdx.x / 8;
    const int64_t per = (r.total + 7) / 8, rt = x * per + local / ntn;
    if (local / ntn >= per || rt >= r.total) return;
    find_rows<BM>(g, r, rt, t);
    t.n0 = (int64_t)(local % ntn) * BN;
    if (t.zero) t.kb1 = 0;
  } else {
    const int ntm = (int)((g.M + BM - 1) / BM);
    int tm, tn;
    if (g.mode == G_RED) {
      const int wg = xcd_remap(blockIdx.x, gridDim.x);
      t.e = wg / (ntm * ntn);
      const int within = wg % (ntm * ntn);
      tm = within / ntn;
      tn = within % ntn;
      t.kb0 = clamp_off(g.offsets[t.e], g.K) / 128;
      t.kb1 = clamp_off(g.offsets[t.e + 1], g.K) / 128;
    } else {
      panel_major_tile(blockIdx.x, ntm, ntn, 4, tm, tn);
    }
    t.m0 = (int64_t)tm * BM;
    t.m_end = t.m0 + BM < g.M ? t.m0 + BM : g.M;
    t.n0 = (int64_t)tn * BN;
  }
  // the same in every lane, in scalar registers (rows and columns are below 2^31)
  t.m0 = (int)uniform((uint32_t)t.m0);
  t.m_end = (int)uniform((uint32_t)t.m_end);
  t.n0 = (int)uniform((uint32_t)t.n0);
  t.e = (int)uniform((uint32_t)t.e);
  t.kb0 = (int)uniform((uint32_t)t.kb0);
  t.kb1 = (int)uniform((uint32_t)t.kb1);
  const uint8_t* B = g.B;
  const float* sb = g.sb;
  if (g.mode == G_ROWS) {
    B += (int64_t)t.e * g.N * g.ldb;
    sb += (int64_t)t.e * ((g.N + 127) / 128) * g.ldsb;
  }
  const int wm = (wave / Cfg::WAVES_N) * Cfg::TM, wn = (wave % Cfg::WAVES_N) * Cfg::TN;
  const int KT = (int)(t.kb1 - t.kb0);

  // A wave fills 8 LOADS consecutive LDS rows, all of A's or all of B's: load q rows 8 q .. 8 q + 7 of
  // them, lane -> row lane / 8, slot lane % 8 (LOADS is even, so the slot's source chunk depends on the
  // parity of q).  The descriptor ends behind the wave's last row: lanes beyond it get zeros.
  constexpr int ROWS = 8 * Cfg::LOADS;
  static_assert(Cfg::LOADS % 2 == 0 && BM % ROWS == 0 && BN % ROWS == 0, "a wave's rows are of one operand");
  const bool of_a = wave < BM / ROWS;
  const int64_t ldx = of_a ? g.lda : g.ldb;
  const int64_t row0 = of_a ? t.m0 + wave * ROWS : t.n0 + wave * ROWS - BM;
  const int64_t left = (of_a ? t.m_end : g.N) - row0;
  const int rows = left < 0 ? 0 : left < ROWS ? (int)left : ROWS;
  const int rem = (int)(g.K - (t.kb1 - 1) * 128 < 128 ? g.K - (t.kb1 - 1) * 128 : 128);   // of the last block
  const uint32_t span = uniform(rows > 0 && KT > 0 ? (uint32_t)((rows - 1) * ldx + (KT - 1) * 128 + (rem + 15) / 16 * 16) : 0u);
  const u32x4 desc = buffer_desc((of_a ? g.A : B) + row0 * ldx + t.kb0 * 128, span);
  const uint32_t voff0 = (uint32_t)((lane >> 3) * ldx) + ((lane & 7) ^ (lane >> 4)) * 16;
  const uint32_t voff1 = (uint32_t)((lane >> 3) * ldx) + ((lane & 7) ^ (lane >> 4) ^ 4) * 16;
  // and the 64 scales of 64 of the tile's rows (clamped to the last)
  const float* sc;
  int64_t sc_step;
  uint32_t sc_off;
  if (wave < BM / 64) {
    const int64_t m = t.m0 + wave * 64 + lane;
    sc = g.sa + t.kb0 * g.ldsa + t.m0;
    sc_off = (uint32_t)((m < g.M ? m : g.M - 1) - t.m0) * 4;
    sc_step = g.ldsa;
  } else {
    int64_t n = t.n0 + wave * 64 - BM + lane;
    n = n < g.N ? n : g.N - 1;
    sc = ROWB ? sb + t.kb0 * g.ldsb + t.n0 : sb + t.n0 / 128 * g.ldsb + t.kb0;
    sc_off = (uint32_t)(ROWB ? n - t.n0 : (n / 128 - t.n0 / 128) * g.ldsb) * 4;
    sc_step = ROWB ? g.ldsb : 1;
  }
  const uint32_t lds0 = lds_addr(smem);
  // load q < LOADS of stage kt, or (q == LOADS) its scales; past the last stage nothing is read: the
  // descriptor is empty (the scales are the last stage's again)
  auto dma = [&](int kt, int q) {
    const uint32_t dst = lds0 + (kt & 1) * Cfg::STAGE;
    if (q == Cfg::LOADS) {
      dma4s(sc_off, sc + (kt < KT ? kt : KT - 1) * sc_step, uniform(dst + Cfg::OPER + wave * 256));
    } else {
      u32x4 d = desc;
      d[2] = kt < KT ? span : 0u;
      dma16b((q & 1 ? voff1 : voff0) + uniform((uint32_t)(q * 8 * ldx) + kt * 128), d,
             uniform(dst + (Cfg::LOADS * wave + q) * 1024));
    }
  };
  // this wave's loads of stage kt have landed and its reads of the stage before are done; then every wave's
  auto land = [&](int kt) {
    wait_vmcnt<0>();
    lds_barrier();
    if (kt == KT - 1 && rem < 128) {
      // K ends inside the block: clear the bytes behind it in every row of both operands
      for (int r = tid; r < BM + BN; r += Cfg::NT) {
        unsigned char* row = smem + (kt & 1) * Cfg::STAGE + r * 128;
        for (int c = rem / 16; c < 8; ++c) {
          u32x4* p = reinterpret_cast<u32x4*>(row + ((c ^ (r >> 1 & 7)) * 16));
          u32x4 v = *p;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int keep = rem - 16 * c - 4 * w;   // bytes of this word before K
            v[w] = keep >= 4 ? v[w] : keep <= 0 ? 0u : v[w] & ((1u << (8 * keep)) - 1);
          }
          *p = v;
        }
      }
      lds_barrier();
    }
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // a lane's 32 bytes of a fragment row: chunks 2 lq and 2 lq + 1
  const int sl0 = ((2 * lq) ^ (l16 >> 1)) * 16, sl1 = ((2 * lq + 1) ^ (l16 >> 1)) * 16;
  const int a_row = (wm + l16) * 128, b_row = (BM + wn + l16) * 128;
  auto frag = [&](int kt, int row) {
    const unsigned char* st = smem + (kt & 1) * Cfg::STAGE + row;
    i32x8 v;
    u32x4* h = reinterpret_cast<u32x4*>(&v);
    h[0] = *reinterpret_cast<const u32x4*>(st + sl0);
    h[1] = *reinterpret_cast<const u32x4*>(st + sl1);
    return v;
  };
  auto scales = [&](int kt) { return reinterpret_cast<const float*>(smem + (kt & 1) * Cfg::STAGE + Cfg::OPER); };

  constexpr int D = Cfg::D;
  i32x8 a[FM], b[D + 1];
  bf16x8 aw[EXACT ? FM : 1][4];   // EXACT: the stage's A fragments widened
  f32x4 p[2][FM], sn = {0.f, 0.f, 0.f, 0.f}, late[D];   // late: the row scales of the last D slots
  float s[FM], sprev[FM];
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    p[1][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    s[i] = 0.f;
  }
#pragma unroll
  for (int d = 0; d < D; ++d) late[d] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto row_scales = [&](int kt, int j) {
    return *reinterpret_cast<const f32x4*>(scales(kt) + BM + wn + 16 * j + 4 * lq);
  };
  auto load_scales = [&](int kt) {
    const float sbw = scales(kt)[BM + wn];
#pragma unroll
    for (int i = 0; i < FM; ++i) s[i] = scales(kt)[wm + 16 * i + l16] * (ROWB ? 1.f : sbw);
  };
  auto scale = [&](int i, int j, const float (&sc_)[FM]) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      // the block's scale is formed first, as in the other kernels: a sum times one scale alone can pass
      // fp32's range where the result does not
      const float f = ROWB ? sc_[i] * (j < FN - D ? sn[q] : late[j < FN - D ? 0 : j - (FN - D)][q]) : sc_[i];
      acc[i][j][q] = __builtin_fmaf(p[j & 1][i][q], f, acc[i][j][q]);
    }
    asm volatile("" : "+v"(acc[i][j]));   // here, not sunk to the end of the loop
  };
  // Stage kt.  Slot j: fragment j's FM matrix instructions, and between them the scaling of the slot
  // before (a result is read FM matrix instructions after its own was issued; slot 0 finishes the stage
  // before).  B's fragments are read D slots ahead, and the last D slots' row scales before slot FN - D,
  // so from there on nothing of this stage is read: there the waves meet, and the last D slots read the
  // next stage's first fragments and issue the loads of the stage after it into the buffer just left.
  auto stage = [&](int kt) {
#pragma unroll
    for (int i = 0; i < FM; ++i) sprev[i] = s[i];
    if constexpr (EXACT) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int h = 0; h < 4; ++h) aw[i][h] = widen8<FA>(a[i][2 * h], a[i][2 * h + 1]);
    }
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      if (j == FN - D) land(kt + 1);
      if (j + D < FN) b[(j + D) % (D + 1)] = frag(kt, b_row + (j + D) * 2048);
      else b[(j + D) % (D + 1)] = frag(kt + 1, b_row + (j + D - FN) * 2048);
      if (j == 0) load_scales(kt);
#pragma unroll
      for (int h = 0; h < (EXACT ? 4 : 1); ++h) {
        bf16x8 bw;
        if constexpr (EXACT) bw = widen8<FB>(b[j % (D + 1)][2 * h], b[j % (D + 1)][2 * h + 1]);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (EXACT)
            p[j & 1][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                bw, aw[i][h], h == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : p[j & 1][i], 0, 0, 0);
          else
            p[j & 1][i] = mfma128<FB, FA, false>(b[j % (D + 1)], a[i]);
          __builtin_amdgcn_sched_barrier(0);
          if (h > 0) continue;
          if (j == 0) scale(i, FN - 1, sprev); else scale(i, j - 1, s);
          if (j == FN - 1) a[i] = frag(kt + 1, a_row + i * 2048);
          if (j >= FN - D) {
            constexpr int PER = Cfg::LOADS / (D * FM);
#pragma unroll
            for (int u = 0; u < PER; ++u) dma(kt + 2, ((j - (FN - D)) * FM + i) * PER + u);
          }
        }
      }
      if (ROWB) {
        if (j < FN - D) sn = row_scales(kt, j);
        if (j == FN - D - 1) {
#pragma unroll
          for (int d = 0; d < D; ++d) late[d] = row_scales(kt, FN - D + d);
        }
      }
    }
    dma(kt + 2, Cfg::LOADS);
    if constexpr (FN % (D + 1) != 0) {
      i32x8 r[D];
#pragma unroll
      for (int d = 0; d < D; ++d) r[d] = b[(FN + d) % (D + 1)];
#pragma unroll
      for (int d = 0; d < D; ++d) b[d] = r[d];
    }
  };
  static_assert(Cfg::LOADS % (D * FM) == 0, "the last slots issue all loads");
  if (KT > 0) {
#pragma unroll
    for (int q = 0; q <= Cfg::LOADS; ++q) dma(0, q);
    land(0);
#pragma unroll
    for (int q = 0; q <= Cfg::LOADS; ++q) dma(1, q);
#pragma unroll
    for (int i = 0; i < FM; ++i) a[i] = frag(0, a_row + i * 2048);
#pragma unroll
    for (int d = 0; d < D; ++d) b[d] = frag(0, b_row + d * 2048);
    if (t.m0 + wm < t.m_end) {
      for (int kt = 0; kt < KT; ++kt) stage(kt);
#pragma unroll
      for (int i = 0; i < FM; ++i) scale(i, FN - 1, s);
    } else {
      // a wave whose rows lie behind the group's last (a group's partial tile) only loads
      for (int kt = 0; kt < KT; ++kt) {
        land(kt + 1);
#pragma unroll
        for (int q = 0; q <= Cfg::LOADS; ++q) dma(kt + 2, q);
      }
    }
    wait_vmcnt<0>();   // no load may land in LDS after the workgroup ends
  }

  const int64_t crow = (g.mode == G_RED ? (int64_t)t.e * g.M : 0) + t.m0 + wm;
  const int rows_left = (int)(t.m_end - t.m0) - wm;
  const int64_t n = t.n0 + wn;
  if (g.bf16_out) store_tile<FM, FN>(acc, (uint16_t*)g.C + crow * g.ldc, g.ldc, rows_left, n, g.N, lane);
  else store_tile<FM, FN>(acc, (float*)g.C + crow * g.ldc, g.ldc, rows_left, n, g.N, lane);
}

template <int FA, int FB, bool ROWB, bool EXACT, typename Cfg>
hipError_t run_tile(const Fp8Gemm& g, hipStream_t s) {
  auto kern = fp8_gemm_tile_kernel<FA, FB, ROWB, EXACT, Cfg>;
  (void)hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, Cfg::LDS);
  const int64_t ntn = (g.N + Cfg::BN - 1) / Cfg::BN, ntm = (g.M + Cfg::BM - 1) / Cfg::BM;
  int64_t wgs = ntm * ntn;
  if (g.mode == G_ROWS) wgs = (most_row_tiles(g, Cfg::BM) + 7) / 8 * 8 * ntn;
  if (g.mode == G_RED) wgs *= g.E;
  if (!grid_ok(wgs, Cfg::NT)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(kern, dim3((unsigned)wgs), dim3(Cfg::NT), Cfg::LDS, s, g);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Few rows per group (or few rows at all): B is read once and that bounds the call, so its bytes go
// straight from memory to the registers of the matrix instruction, with no LDS and no barrier on the
// way.  A workgroup computes 16 FM rows of A by 32 rows of B; its KS waves take every KS-th chunk of
// two 128-blocks, each with the next chunk's loads in flight, and add their sums through LDS in the
// order of the waves.  The lanes of a row that does not exist load nothing.
// ---------------------------------------------------------------------------
template <int FA, int FB, bool ROWB, bool EXACT, int FM, int KS>
__global__ __launch_bounds__(64 * KS) void fp8_gemm_rows_kernel(Fp8Gemm g) {
  constexpr int BM = 16 * FM, BN = 32, FN = 2, CH = 2;   // CH: 128-blocks a chunk
  __shared__ f32x4 part[KS][FM * FN][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  const int ntn = (int)((g.N + BN - 1) / BN);
  Tile t;
  t.e = 0;
  t.zero = false;
  t.kb0 = 0;
  t.kb1 = (g.K + 127) / 128;
  const int64_t rt = blockIdx.x / ntn;
  t.n0 = (int64_t)(blockIdx.x % ntn) * BN;
  if (g.mode == G_ROWS) {
    const RowTiles r = count_rows<BM>(g);
    if (rt >= r.total) return;
    find_rows<BM>(g, r, rt, t);
    if (t.zero) t.kb1 = 0;
  } else {
    t.m0 = rt * BM;
    t.m_end = t.m0 + BM < g.M ? t.m0 + BM : g.M;
  }
  t.m0 = (int)uniform((uint32_t)t.m0);
  t.m_end = (int)uniform((uint32_t)t.m_end);
  t.e = (int)uniform((uint32_t)t.e);
  t.kb1 = (int)uniform((uint32_t)t.kb1);
  const uint8_t* B = g.B;
  const float* sb = g.sb;
  if (g.mode == G_ROWS) {
    B += (int64_t)t.e * g.N * g.ldb;
    sb += (int64_t)t.e * ((g.N + 127) / 128) * g.ldsb;
  }
  const int kbs = (int)t.kb1, nchunks = (kbs + CH - 1) / CH;

  // a lane's 32 bytes of a block: 16 at 16 lq and 16 at 64 + 16 lq (the same for both operands, so the
  // order inside a block does not matter), which makes 64 contiguous bytes of each row per load
  const uint8_t* arow[FM];
  bool aon[FM], bon[FN];
  const uint8_t* brow[FN];
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t m = t.m0 + 16 * i + l16;
    aon[i] = m < t.m_end;
    arow[i] = g.A + (aon[i] ? m : t.m0) * g.lda;
  }
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int64_t n = t.n0 + 16 * j + l16;
    bon[j] = n < g.N;
    brow[j] = B + (bon[j] ? n : t.n0) * g.ldb;
  }
  auto load16 = [&](const uint8_t* row, bool on, int64_t k) {
    u32x4 v = {0, 0, 0, 0};
    if (on && k < g.K) v = *reinterpret_cast<const u32x4*>(row + k);
    return v;
  };
  auto trim = [&](u32x4 v, int64_t k) {   // clear the bytes from K on
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const int64_t keep = g.K - k - 4 * w;
      v[w] = keep >= 4 ? v[w] : keep <= 0 ? 0u : v[w] & ((1u << (8 * keep)) - 1);
    }
    return v;
  };
  struct Chunk {
    u32x4 a[CH][FM][2], b[CH][FN][2];
    float sa[CH][FM], sb[CH][ROWB ? 4 * FN : 1];
  };
  auto load = [&](int c, Chunk& x) {
#pragma unroll
    for (int u = 0; u < CH; ++u) {
      const int kb = c * CH + u;
      const int64_t k = (int64_t)kb * 128 + 16 * lq;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        x.b[u][j][0] = load16(brow[j], bon[j], k);
        x.b[u][j][1] = load16(brow[j], bon[j], k + 64);
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        x.a[u][i][0] = load16(arow[i], aon[i], k);
        x.a[u][i][1] = load16(arow[i], aon[i], k + 64);
        x.sa[u][i] = aon[i] && kb < kbs ? g.sa[kb * g.ldsa + t.m0 + 16 * i + l16] : 0.f;
      }
      if constexpr (ROWB) {
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int64_t n = t.n0 + 16 * j + 4 * lq + q;
            x.sb[u][4 * j + q] = n < g.N && kb < kbs ? sb[kb * g.ldsb + n] : 0.f;
          }
      } else {
        x.sb[u][0] = kb < kbs ? sb[t.n0 / 128 * g.ldsb + kb] : 0.f;   // a tile's 32 rows lie in one block
      }
    }
  };
  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](int c, Chunk& x) {
#pragma unroll
    for (int u = 0; u < CH; ++u) {
      const int64_t k = (int64_t)(c * CH + u) * 128 + 16 * lq;
      if ((int64_t)(c * CH + u + 1) * 128 > g.K) {   // K ends in this block
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int j = 0; j < FN; ++j) x.b[u][j][h] = trim(x.b[u][j][h], k + 64 * h);
#pragma unroll
          for (int i = 0; i < FM; ++i) x.a[u][i][h] = trim(x.a[u][i][h], k + 64 * h);
        }
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const i32x8 fb = __builtin_bit_cast(i32x8, x.b[u][j]);
#pragma unroll
        for (int i = 0; i < FM; ++i) {
          const f32x4 p = mfma128<FB, FA, EXACT>(fb, __builtin_bit_cast(i32x8, x.a[u][i]));
#pragma unroll
          for (int q = 0; q < 4; ++q)
            acc[i][j][q] += p[q] * (x.sa[u][i] * (ROWB ? x.sb[u][4 * j + q] : x.sb[u][0]));
        }
      }
    }
  };
  Chunk x, y;
  int c = wave;
  if (c < nchunks) load(c, x);
  while (c < nchunks) {
    if (c + KS < nchunks) load(c + KS, y);
    compute(c, x);
    c += KS;
    if (c >= nchunks) break;
    if (c + KS < nchunks) load(c + KS, x);
    compute(c, y);
    c += KS;
  }
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) part[wave][i * FN + j][lane] = acc[i][j];
  __syncthreads();
  for (int f = wave; f < FM * FN; f += KS) {
    f32x4 sum = part[0][f][lane];
#pragma unroll
    for (int w = 1; w < KS; ++w) sum += part[w][f][lane];
    const int64_t m = t.m0 + 16 * (f / FN) + l16;
    if (m < t.m_end) store4(g, m, t.n0 + 16 * (f % FN) + 4 * lq, sum);
  }
}

template <int FA, int FB, bool ROWB, int FM, int KS>
hipError_t run_rows(const Fp8Gemm& g, hipStream_t s) {
  const int64_t ntn = (g.N + 31) / 32;
  const int64_t ntm = g.mode == G_ROWS ? most_row_tiles(g, 16 * FM) : (g.M + 16 * FM - 1) / (16 * FM);
  if (!grid_ok(ntm * ntn, 64 * KS)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)(ntm * ntn)), wg(64 * KS);
  if (g.bf16_out) hipLaunchKernelGGL((fp8_gemm_rows_kernel<FA, FB, ROWB, false, FM, KS>), grid, wg, 0, s, g);
  else hipLaunchKernelGGL((fp8_gemm_rows_kernel<FA, FB, ROWB, true, FM, KS>), grid, wg, 0, s, g);
  return hipGetLastError();
}

// The tiled kernel's conditions: 16-byte loads of both operands, 32-bit offsets inside a tile.
bool tile_ok(const Fp8Gemm& g) {
  return (uintptr_t)g.A % 16 == 0 && (uintptr_t)g.B % 16 == 0 && g.lda % 16 == 0 && g.ldb % 16 == 0 &&
         g.lda < (1 << 23) && g.ldb < (1 << 23) && g.ldsb < (1 << 28);
}

using Tile256 = TileCfg<256, 256, 4, 2, 1>;
using Tile128 = TileCfg<128, 128, 2, 2, 2>;

template <int FA, int FB>
hipError_t run(const Fp8Gemm& g, hipStream_t s) {
  if (force_generic() || !tile_ok(g)) return run_general<FA, FB>(g, s);
  auto tiles = [&](int64_t b) { return (g.M + b - 1) / b * ((g.N + b - 1) / b) * (g.mode == G_RED ? g.E : 1); };
  // Few rows a group, and at most one 128 x 128 tile a CU: the kernel without LDS.  It and the tiled
  // kernel, in us: 1 x 8192 x 2048 5.3 and 12; 64 x 8192 x 2048 11.0 and 12.5; 128 x 8192 x 2048 18.6 and
  // 12.7; 1 x 16384 x 4096 14 and 24; experts of 1024 x 2048, 8 rows of 8 of them 6.2 and 13, 128 rows of 64
  // of them 23.5 and 21.6.
  const int64_t groups = g.mode == G_ROWS ? (g.E < g.M ? g.E : g.M) : 1, per_group = (g.M + groups - 1) / groups;
  if (g.mode != G_RED && per_group <= 64 && groups * ((g.N + 127) / 128) <= 256) {
    const bool two = per_group > 16;
    if (g.b_block == 1)
      return two ? run_rows<FA, FB, true, 2, 4>(g, s) : run_rows<FA, FB, true, 1, 4>(g, s);
    return two ? run_rows<FA, FB, false, 2, 4>(g, s) : run_rows<FA, FB, false, 1, 4>(g, s);
  }
  // fp32 results: the widened fragments fit beside the small tile's accumulators only
  if (!g.bf16_out)
    return g.b_block == 1 ? run_tile<FA, FB, true, true, Tile128>(g, s) : run_tile<FA, FB, false, true, Tile128>(g, s);
  // Time of a round of 256 large tiles : of 512 small ones (two a CU) = 5 : 3 (65 and 39 us at K 4096), as
  // measured on dense products.  The groups' partial tiles are not counted, so with uneven groups the
  // rule is right at many rows and can be a fifth off at few (large, small, in us: 4096 tokens, 8 of 128
  // experts 1024 x 2048, 112 and 128; 8 of 64 experts 2048 x 1024, 98 and 113; but 8 of 64 experts 1024 x 2048,
  // 4096 tokens 96 and 94, 2048 tokens 60 and 54; 1024 tokens, 2048 x 1024, 49 and 40).
  const bool large = (tiles(256) + 255) / 256 * 5 <= (tiles(128) + 511) / 512 * 3;
  if (g.b_block == 1)
    return large ? run_tile<FA, FB, true, false, Tile256>(g, s) : run_tile<FA, FB, true, false, Tile128>(g, s);
  return large ? run_tile<FA, FB, false, false, Tile256>(g, s) : run_tile<FA, FB, false, false, Tile128>(g, s);
}

}  // namespace

static hipError_t gemm_piece(const Fp8Gemm& g, hipStream_t s) {
  if (g.a_e5m2) return g.b_e5m2 ? run<1, 1>(g, s) : run<1, 0>(g, s);
  return g.b_e5m2 ? run<0, 1>(g, s) : run<0, 0>(g, s);
}

hipError_t launch_fp8_gemm(const Fp8Gemm& g, hipStream_t s) {
  if (g.mode != G_DENSE) return gemm_piece(g, s);
  return in_pieces(g.M, kPieceRows, [&](int64_t m0, int64_t n) {
    Fp8Gemm p = g;
    p.A += m0 * g.lda;
    p.sa += m0;
    p.M = n;
    p.C = (uint8_t*)g.C + m0 * g.ldc * (g.bf16_out ? 2 : 4);
    return gemm_piece(p, s);
  });
}

}  // namespace nms
