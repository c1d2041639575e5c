// Products of bf16 matrices with fp32 sums, for the dense FFN's forward (bias, activation and residual in
// the epilogue) and its gradients (the activation's derivative, or addition to the result, in the epilogue).
//
// Every kernel gives B the matrix instruction's row operand and A its column operand, so a lane holds four
// consecutive columns n of one row m of C.
#include "act.hpp"
#include "dma.hpp"
#include "launch.hpp"
#include "pieces.hpp"
#include "rows8.hpp"

#include <utility>

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
__device__ inline f32x4 gate4(int act, f32x4 v, const f32x4& z) {
  with_act(act, [&](auto a) {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = act_gate<decltype(a)::value>(v[q], z[q]);
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
    v = gate4(g.act, v, load4(g.P + m * g.ldp, n, g.N));
  } else if (g.epi == EPI_ADD) {
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
  if (!grid_ok(ntm, 256)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(linear_general_kernel, dim3((unsigned)ntm, (unsigned)ntn), dim3(256), 0, s, g);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Tiled kernel: BM x BN tiles of C by four waves (2 x 2) of 16 FM x 16 FN, one workgroup a CU.  The operands pass through LDS
// in buffers of 64 k, NA of A's and NA + 1 of B's, filled by direct-to-LDS loads.
//
// An operand lies in LDS as it does in memory:
//   reduction contiguous   a row of C per 128-byte LDS row, its 16-byte chunk c at slot c ^ (row / 2 % 8): sixteen
//                          rows' reads of one chunk cover all 64 banks once; a fragment is one 16-byte read.  (A row's
//                          128 bytes are a cache line: with buffers of 32 k and 64-byte pieces the L2s give half);
//   reduction strided      a k per LDS row of 2 BM bytes, its 32-byte segment s (16 columns: a fragment's) at
//                          s ^ (k % 4 + 4 (k / 8 % 2)).  The transposing read gives a lane four k of one column from
//                          four rows; a read's half wave touches eight rows (k % 4 and k / 8 % 2 all different), so
//                          eight segments in different banks; a fragment is two reads.
// Unit u (64 k) runs 2 FM x FN matrix instructions a wave, the first half on fragments that were read during unit
// u - 1.  Between those it reads the second half's fragments and issues B's loads of unit u + NA, into the buffer of
// unit u - 1; then the waves meet, once a unit: all have read unit u.  Between the second half's instructions it reads
// unit u + 1's first fragments and issues A's loads of unit u + NA into the buffer that unit u was read from.  So a load has
// NA - 1 units or more to arrive, and a unit's matrix instructions take about 1, 0.5 and 0.25 us with the three tiles: NA is what LDS holds.
// With operands that are not in a cache that counts: 256 x 128 with NA 2 takes 139 us for 4096 x 2048 x 8192 and with 3 127
// (bias and residual); 128 x 128 tiles with a ring of five buffers of 32 k, two workgroups a CU, 93 us for 2048 x 2048 x 8192, and
// with NA 4 71.  8192 x 16384 x 4096 takes 812 us (1350 TFLOP/s, a large library product's rate), 4096^3 97 us.
// Rows and columns beyond the operands, and k beyond K, are zeros: a lane's
// 16 bytes lie inside the operand or outside (the contiguous sizes are multiples of eight), and outside its offset
// is moved beyond the descriptor's size, where nothing is read.
// ---------------------------------------------------------------------------
constexpr uint32_t kOutside = 0x80000000u;   // added to an offset: beyond every descriptor's size

// f(0) .. f(N - 1) with the index as a constant
template <typename F, int... I>
__device__ __forceinline__ void each_of(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each_of(F f) {
  each_of(std::make_integer_sequence<int, N>(), f);
}

constexpr int KU = 64;   // the k of an LDS buffer

// NA: A's buffers; B has one more
template <int FM_, int FN_, int NA_>
struct LinCfg {
  static constexpr int FM = FM_, FN = FN_, BM = 32 * FM, BN = 32 * FN, NA = NA_, NB = NA + 1;
  static constexpr int A_BYTES = BM * 2 * KU, B_BYTES = BN * 2 * KU, LDS = NA * A_BYTES + NB * B_BYTES;
  static constexpr int LA = A_BYTES / 4096, LB = B_BYTES / 4096, LOADS = LA + LB;   // 1 KB loads a wave and buffer
  static_assert(LDS <= 163840, "a CU's LDS");
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Where a wave's loads of one operand come from, and where a lane's fragments lie in LDS.
template <bool T, int BR, int LN>
struct Operand {
  static constexpr int ROW = T ? 2 * BR : 2 * KU;     // bytes of an LDS row
  static constexpr int CH = KU / 8;                   // not T: chunks of a row
  static_assert(LN % 2 == 0, "the swizzle of a wave's loads alternates");
  const uint16_t* base;
  int64_t step;          // elements from a buffer's k to the next one's
  int64_t K;
  uint32_t width;        // T: bytes of the tile's columns that exist
  uint32_t ldb;          // bytes of a row
  uint32_t off[LN];      // of this wave's loads, this lane
  int c[2];              // not T: the lane's chunk in the even and the odd loads
  __device__ void init(const uint16_t* X, int64_t ld, int64_t r0, int64_t R, int64_t K_, int wave, int lane) {
    K = K_;
    ldb = (uint32_t)(2 * ld);
    if constexpr (T) {
      base = X + r0;
      step = KU * ld;
      width = (uint32_t)(2 * (R - r0 < BR ? R - r0 : BR));
#pragma unroll
      for (int t = 0; t < LN; ++t) {
        const int at = (wave * LN + t) * 1024 + lane * 16, k = at / ROW, chunk = at % ROW / 16;
        const uint32_t col = 32 * ((chunk >> 1) ^ ((k & 3) | (k >> 3 & 1) << 2)) + 16 * (chunk & 1);
        off[t] = k * ldb + col + (col < width ? 0u : kOutside);
      }
    } else {
      base = X + r0 * ld;
      step = KU;
      constexpr int RL = 64 / CH;   // rows of a load
      c[0] = (lane % CH) ^ ((lane / CH) >> 1 & (CH - 1));
      c[1] = c[0] ^ 4;
#pragma unroll
      for (int t = 0; t < LN; ++t) {
        const int r = RL * (wave * LN + t) + lane / CH;
        off[t] = r * ldb + 16 * c[t & 1] + (r0 + r < R ? 0u : kOutside);
      }
    }
  }
  // the descriptor of buffer u's k; nothing is read behind the last
  __device__ u32x4 desc(int u) const {
    const int64_t left = K - (int64_t)u * KU;
    uint32_t bytes = left > 0 ? kOutside : 0u;
    if constexpr (T) bytes = left > 0 ? (uint32_t)((left < KU ? left : KU) - 1) * ldb + width : 0u;
    return buffer_desc(base + u * step, bytes);
  }
  // what the offsets of buffer u's even and odd loads carry besides
  __device__ uint32_t tail(int u, int odd) const {
    if constexpr (T) return 0u;
    else return 8 * c[odd] < K - (int64_t)u * KU ? 0u : kOutside;
  }
  // a lane's address in LDS of its part of fragment 0 of k 0 .. 31, `first` the wave's first row or column
  __device__ static uint32_t lds0(uint32_t part, int first, int lane) {
    const int l16 = lane & 15, lq = lane >> 4;
    if constexpr (T) {
      const int k = 8 * lq + (l16 >> 2);
      return part + k * ROW + 32 * ((first >> 4) ^ ((k & 3) | (k >> 3 & 1) << 2)) + 8 * (l16 & 3);
    }
    return part + (first + l16) * ROW + ((lq ^ (l16 >> 1 & (CH - 1))) << 4);
  }
  // fragment i of k 32 kk ..
  __device__ static bf16x8 frag(uint32_t at, int kk, int i) {
    if constexpr (T) {
      // segment first / 16 + i: first is a multiple of the wave's fragments, so its low bits are i's alone
      const uint32_t a = (at ^ (uint32_t)(32 * i)) + kk * (32 * ROW);
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)a);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a + 4 * ROW));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    typedef __attribute__((address_space(3))) const bf16x8 lds_bf16x8;
    return *(lds_bf16x8*)((at ^ (uint32_t)(64 * kk)) + i * (16 * ROW));
  }
};

// A wave's FM x FN fragments to C, by way of LDS (`region`: the wave's part of the ring): a lane then holds four
// consecutive columns of rows lane / 16, and 16 lanes 64 columns, so every load and store of C and of what lies
// like C takes whole 128-byte lines of bf16.  Row r's 16-byte chunk c lies at c ^ (r % 16): a fragment's rows are written to
// different banks, and read in order.
template <int FM, int FN>
struct Out {
  static constexpr int COLS = 16 * FN, H = COLS / 64;                 // H: runs of 64 columns
  static constexpr int ROWS = 64, PF = ROWS / 16, PASSES = FM / PF;   // ROWS: of a pass
  static constexpr int REGION = ROWS * COLS * 4;                      // a wave's bytes of LDS
  static_assert(FM % PF == 0, "a pass is whole fragments");
  template <int P>
  __device__ static void put(const f32x4 (&acc)[FM][FN], unsigned char* region, int lane) {
    const int l16 = lane & 15, lq = lane >> 4;
#pragma unroll
    for (int i = 0; i < PF; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
        *reinterpret_cast<f32x4*>(region + (16 * i + l16) * (COLS * 4) + ((4 * j + lq) ^ l16) * 16) = acc[P * PF + i][j];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // other lanes of this wave read it
  }
  __device__ static f32x4 get(const unsigned char* region, int r, int h, int lane) {
    return *reinterpret_cast<const f32x4*>(region + r * (COLS * 4) + ((16 * h + (lane & 15)) ^ (r & 15)) * 16);
  }
};

// Any tile, element by element where it ends.
template <int FM, int FN>
__device__ __forceinline__ void epilogue_edge(const Linear& g, const f32x4 (&acc)[FM][FN], unsigned char* region, int64_t m0,
                                              int64_t n0, int lane) {
  typedef Out<FM, FN> O;
  each_of<O::PASSES>([&](auto p) {
    O::template put<decltype(p)::value>(acc, region, lane);
    const int64_t mp = m0 + decltype(p)::value * O::ROWS;
    const int rows = g.M - mp < O::ROWS ? (int)(g.M - mp) : O::ROWS;
#pragma unroll 1
    for (int r = lane >> 4; r < rows; r += 4) {
#pragma unroll
      for (int h = 0; h < O::H; ++h) finish4(g, mp + r, n0 + 64 * h + 4 * (lane & 15), O::get(region, r, h, lane));
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // before the next pass's values
  });
}

typedef __amdgpu_buffer_rsrc_t Rsrc;
// 2 GiB from p (wave-uniform), or nothing: loads give 0 and stores are dropped
__device__ inline Rsrc rsrc(const void* p, bool on) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, on ? (int)0x7FFFFFFF : 0, 0x00020000);
}

// A tile that lies whole inside C.  Addresses are a lane's 32-bit offset, so a row costs its arithmetic, its loads and
// stores and one addition a matrix.  Stores take no scalar offset: behind a 16-byte store that has one the compiler lets the
// next instruction overwrite the data's registers, and on this GPU the last lanes' data then is what that wrote
// (tests/test_dense_codegen.py).  OTHER: something is read beside the sums (the residual, the gate, C itself)
// or the pre-activations are stored; all of a pass's reads are in flight together, since with one or two waves a SIMD
// nothing else hides their latency.
template <int EPI, int ACT, bool OTHER, typename T, int FM, int FN>
__device__ __forceinline__ void epilogue_whole(const Linear& g, const f32x4 (&acc)[FM][FN], unsigned char* region, int64_t m0,
                                      int64_t n0, int lane) {
  typedef Out<FM, FN> O;
  typedef std::conditional_t<EPI == EPI_ADD, u32x4, u32x2> Raw;
  constexpr int G = O::ROWS / 4, H = O::H;
  const int l16 = lane & 15, lq = lane >> 4;
  f32x4 bias[H];
#pragma unroll
  for (int h = 0; h < H; ++h)
    bias[h] = EPI == EPI_FWD ? bias4(g, n0 + 4 * l16 + 64 * h) : f32x4{0.f, 0.f, 0.f, 0.f};
  // what is read: one row stride and element size
  const void* x = EPI == EPI_FWD ? (const void*)g.R : EPI == EPI_GATE ? (const void*)g.P : g.C;
  const int64_t ldx = EPI == EPI_FWD ? g.ldr : EPI == EPI_GATE ? g.ldp : g.ldc;
  constexpr int XS = EPI == EPI_ADD ? 4 : 2;
  each_of<O::PASSES>([&](auto p) {
    const int64_t mp = m0 + decltype(p)::value * O::ROWS;
    const Rsrc rc = rsrc((T*)g.C + mp * g.ldc + n0, true);
    const uint32_t vc = (uint32_t)((lq * g.ldc + 4 * l16) * sizeof(T)), sc = (uint32_t)(4 * g.ldc * sizeof(T));
    const Rsrc rx = rsrc((const char*)x + (mp * ldx + n0) * XS, x != nullptr);
    const uint32_t vx = (uint32_t)((lq * ldx + 4 * l16) * XS), sx = (uint32_t)(4 * ldx * XS);
    const Rsrc rz = rsrc(g.Z + mp * g.ldz + n0, EPI == EPI_FWD && g.Z);
    const uint32_t vz = (uint32_t)((lq * g.ldz + 4 * l16) * 2), sz = (uint32_t)(8 * g.ldz);
    Raw r[G][H];
    if constexpr (OTHER) {
#pragma unroll
      for (int u = 0; u < G; ++u)
#pragma unroll
        for (int h = 0; h < H; ++h) {
          if constexpr (EPI == EPI_ADD) r[u][h] = __builtin_amdgcn_raw_buffer_load_b128(rx, vx + 64 * h * XS, u * sx, 0);
          else r[u][h] = __builtin_amdgcn_raw_buffer_load_b64(rx, vx + 64 * h * XS, u * sx, 0);
        }
    }
    O::template put<decltype(p)::value>(acc, region, lane);
#pragma unroll
    for (int u = 0; u < G; ++u)
#pragma unroll
      for (int h = 0; h < H; ++h) {
        f32x4 v = O::get(region, 4 * u + lq, h, lane), w = {0.f, 0.f, 0.f, 0.f};
        if constexpr (OTHER && EPI == EPI_ADD) w = __builtin_bit_cast(f32x4, r[u][h]);
        if constexpr (OTHER && EPI != EPI_ADD)
          w = f32x4{__uint_as_float(r[u][h][0] << 16), __uint_as_float(r[u][h][0] & 0xFFFF0000u),
                    __uint_as_float(r[u][h][1] << 16), __uint_as_float(r[u][h][1] & 0xFFFF0000u)};
        if constexpr (EPI == EPI_FWD) {
          v += bias[h];
          if constexpr (OTHER)
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, __builtin_convertvector(v, bf16x4)), rz,
                                                  vz + u * sz + 128 * h, 0, 0);
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = act_fwd<ACT>(v[q]) + w[q];
        }
        if constexpr (EPI == EPI_GATE) {
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = act_gate<ACT>(v[q], w[q]);
        }
        if constexpr (EPI == EPI_ADD) v += w;
        if constexpr (sizeof(T) == 2)
          __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, __builtin_convertvector(v, bf16x4)), rc,
                                                vc + u * sc + 128 * h, 0, 0);
        else
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), rc, vc + u * sc + 256 * h, 0, 0);
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // before the next pass's values
  });
}

// A matrix whose rows four consecutive elements at a multiple of four columns can be read from at once, with 31-bit
// offsets inside a pass.
__device__ inline bool fours(const void* p, int64_t ld, int size) {
  return !p || ((uintptr_t)p % (4 * size) == 0 && ld % 4 == 0 && ld < (1 << 22));
}

template <int EPI, int ACT, int FM, int FN>
__device__ __forceinline__ void tile_epilogue(const Linear& g, const f32x4 (&acc)[FM][FN], unsigned char* region,
                                              int64_t m0, int64_t n0, int lane) {
  if (m0 >= g.M || n0 >= g.N) return;
  const bool whole = m0 + 16 * FM <= g.M && n0 + 16 * FN <= g.N && fours(g.C, g.ldc, g.bf16_out ? 2 : 4) &&
                     fours(g.R, g.ldr, 2) && fours(g.Z, g.ldz, 2) && fours(g.P, g.ldp, 2);
  if (!whole) {
    epilogue_edge(g, acc, region, m0, n0, lane);
  } else if constexpr (EPI == EPI_FWD) {
    const bool other = g.R || g.Z;
    if (g.bf16_out) {
      if (other) epilogue_whole<EPI, ACT, true, uint16_t>(g, acc, region, m0, n0, lane);
      else epilogue_whole<EPI, ACT, false, uint16_t>(g, acc, region, m0, n0, lane);
    } else {
      if (other) epilogue_whole<EPI, ACT, true, float>(g, acc, region, m0, n0, lane);
      else epilogue_whole<EPI, ACT, false, float>(g, acc, region, m0, n0, lane);
    }
  } else if constexpr (EPI == EPI_ADD) {
    epilogue_whole<EPI, ACT, true, float>(g, acc, region, m0, n0, lane);
  } else {
    if (g.bf16_out) epilogue_whole<EPI, ACT, EPI == EPI_GATE, uint16_t>(g, acc, region, m0, n0, lane);
    else epilogue_whole<EPI, ACT, EPI == EPI_GATE, float>(g, acc, region, m0, n0, lane);
  }
}

// The tile of a workgroup.  Workgroups are dealt to the 8 XCDs in turn; an XCD takes a run of the tiles in the order of
// groups of kGroupRows row tiles, column after column, so the 32 tiles that it computes together are about square and
// share their operands' rows in its L2.
constexpr int kGroupRows = 4;
__device__ inline void xcd_tile(int id, int ntm, int ntn, int& tm, int& tn) {
  const int tiles = ntm * ntn, x = id % 8, per = tiles / 8, rest = tiles % 8;
  const int t = x * per + (x < rest ? x : rest) + id / 8;
  const int group = t / (kGroupRows * ntn), first = group * kGroupRows;
  const int rows = ntm - first < kGroupRows ? ntm - first : kGroupRows, within = t - first * ntn;
  tm = first + within % rows;
  tn = within / rows;
}

template <bool AT, bool BT, int EPI, int ACT, typename Cfg>
__global__ __launch_bounds__(256) void linear_tile_kernel(Linear g) {
  if (gridDim.y > 1) {
    // a part of the reduction, whose sums go to a matrix of their own
    const int64_t k0 = (int64_t)blockIdx.y * g.part_k;
    auto rest = [&](int64_t k) { return k - k0 < g.part_k ? k - k0 : g.part_k; };
    g.A += AT ? k0 * g.lda : k0;
    g.B += BT ? k0 * g.ldb : k0;
    g.K = rest(g.K);
    g.ka = rest(g.ka);
    g.kb = rest(g.kb);
    g.C = (float*)g.C + blockIdx.y * g.M * g.ldc;
  }
  constexpr int FM = Cfg::FM, FN = Cfg::FN, LA = Cfg::LA, LB = Cfg::LB, LOADS = Cfg::LOADS;
  extern __shared__ __align__(1024) unsigned char smem[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = (wave >> 1) * 16 * FM, wn = (wave & 1) * 16 * FN;
  const int ntm = (int)((g.M + Cfg::BM - 1) / Cfg::BM), ntn = (int)((g.N + Cfg::BN - 1) / Cfg::BN);
  int tm, tn;
  xcd_tile(blockIdx.x, ntm, ntn, tm, tn);
  const int64_t m0 = (int64_t)(int)uniform((uint32_t)(tm * Cfg::BM)), n0 = (int64_t)(int)uniform((uint32_t)(tn * Cfg::BN));
  const int units = (int)((g.K + KU - 1) / KU);

  Operand<AT, Cfg::BM, LA> A;
  Operand<BT, Cfg::BN, LB> B;
  A.init(g.A, g.lda, m0, g.ra, g.ka, wave, lane);
  B.init(g.B, g.ldb, n0, g.rb, g.kb, wave, lane);
  const uint32_t lds_base = uniform(lds_addr(smem));
  const uint32_t a_first = A.lds0(lds_base, wm, lane), b_first = B.lds0(lds_base + Cfg::NA * Cfg::A_BYTES, wn, lane);

  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // load t of this wave's of an operand, into the buffer at byte `at` of the operand's
  const uint32_t lds_a = uniform(lds_base + wave * (LA * 1024)), lds_b = uniform(lds_base + Cfg::NA * Cfg::A_BYTES + wave * (LB * 1024));
  auto load_a = [&](auto t, uint32_t at, const u32x4& d, uint32_t t0, uint32_t t1) {
    constexpr int T = decltype(t)::value;
    dma16b_at<T * 1024>(A.off[T] | (T & 1 ? t1 : t0), d, lds_a + at);
  };
  auto load_b = [&](auto t, uint32_t at, const u32x4& d, uint32_t t0, uint32_t t1) {
    constexpr int T = decltype(t)::value;
    dma16b_at<T * 1024>(B.off[T] | (T & 1 ? t1 : t0), d, lds_b + at);
  };
  auto fill_a = [&](int u) {   // the loads of a whole buffer
    const u32x4 d = A.desc(u);
    each_of<LA>([&](auto t) { load_a(t, u % Cfg::NA * Cfg::A_BYTES, d, A.tail(u, 0), A.tail(u, 1)); });
  };
  auto fill_b = [&](int u) {
    const u32x4 d = B.desc(u);
    each_of<LB>([&](auto t) { load_b(t, u % Cfg::NB * Cfg::B_BYTES, d, B.tail(u, 0), B.tail(u, 1)); });
  };
  auto forward = [](u32x4& d, uint64_t by) {
    const uint64_t at = ((uint64_t)d[1] << 32 | d[0]) + by;
    d[0] = (uint32_t)at;
    d[1] = (uint32_t)(at >> 32);
  };
  const uint64_t adv_a = 2 * A.step, adv_b = 2 * B.step;
  // the matrix instructions of 32 k on (a, b); f(m) behind instruction m
  auto multiply = [&](const bf16x8 (&a)[FM], const bf16x8 (&b)[FN], auto f) {
    each_of<FM * FN>([&](auto m_) {
      constexpr int m = decltype(m_)::value, j = m / FM, i = m % FM;
      // tied in and out of the instruction in the accumulation registers (as a builtin, the compiler moves the
      // small accumulators between registers every step)
      asm("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc[i][j]) : "v"(b[j]), "v"(a[i]));
      __builtin_amdgcn_sched_barrier(0);
      f(m_);
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  constexpr int N = FM * FN;
  // operand fragment q (A's first) of k 32 kk .. of the buffers at pa and pb, behind instruction READ q: the reads end well
  // before the next meeting of the waves, which waits for them
  constexpr int READ = N / (FM + FN) > 3 ? 3 : N / (FM + FN);
  auto read = [&](auto m_, int kk, uint32_t pa, uint32_t pb, bf16x8 (&an)[FM], bf16x8 (&bn)[FN]) {
    constexpr int m = decltype(m_)::value, q = m / READ;
    if constexpr (m % READ == 0) {
      if constexpr (q < FM) an[q] = A.frag(pa, kk, q);
      else if constexpr (q < FM + FN) bn[q - FM] = B.frag(pb, kk, q - FM);
    }
  };
  bf16x8 a0[FM], b0[FN], a1[FM], b1[FN];
  auto first = [&] {
#pragma unroll
    for (int i = 0; i < FM; ++i) a0[i] = A.frag(a_first, 0, i);
#pragma unroll
    for (int j = 0; j < FN; ++j) b0[j] = B.frag(b_first, 0, j);
  };
  // WHOLE below: the k that are loaded lie whole inside K, so the descriptor is the last one moved on
  constexpr int NA = Cfg::NA;
  fill_a(0);
  fill_b(0);
#pragma unroll
  for (int u = 1; u < NA; ++u) {
    fill_b(u);
    fill_a(u);
  }
  wait_vmcnt<(NA - 1) * LOADS>();   // unit 0
  lds_barrier();
  first();
  uint32_t ca = 0, cb = 0;   // unit u's buffers, in bytes
  u32x4 na = A.desc(NA), nb = B.desc(NA);
  auto next = [](uint32_t at, uint32_t bytes, int n) { return at == (n - 1) * bytes ? 0 : at + bytes; };
  auto unit = [&](auto whole, int u) {
    constexpr bool WHOLE = decltype(whole)::value;
    constexpr int LOAD_B = N / LB, LOAD_A = N / 2 / LA;
    uint32_t t[4] = {0, 0, 0, 0};
    if constexpr (!WHOLE) {
      na = A.desc(u + NA);
      nb = B.desc(u + NA);
      t[0] = A.tail(u + NA, 0), t[1] = A.tail(u + NA, 1), t[2] = B.tail(u + NA, 0), t[3] = B.tail(u + NA, 1);
    }
    const uint32_t xa = next(ca, Cfg::A_BYTES, NA), xb = next(cb, Cfg::B_BYTES, NA + 1);   // of unit u + 1
    const uint32_t free = cb == 0 ? NA * Cfg::B_BYTES : cb - Cfg::B_BYTES;                 // B's of unit u - 1
    // unit u's second half is read; B's unit u + NA goes where unit u - 1 was
    multiply(a0, b0, [&](auto m_) {
      constexpr int m = decltype(m_)::value;
      read(m_, 1, a_first + ca, b_first + cb, a1, b1);
      if constexpr (m % LOAD_B == LOAD_B / 2) {
        load_b(std::integral_constant<int, m / LOAD_B>(), free, nb, t[2], t[3]);
        if constexpr (WHOLE && m / LOAD_B == LB - 1) forward(nb, adv_b);
      }
    });
    wait_vmcnt<(NA - 2) * LOADS + LB>();   // this wave's loads of unit u + 1
    lds_barrier();                         // every wave's; and every wave has read unit u
    multiply(a1, b1, [&](auto m_) {
      constexpr int m = decltype(m_)::value;
      read(m_, 0, a_first + xa, b_first + xb, a0, b0);
      if constexpr (m % LOAD_A == LOAD_A / 2 && m / LOAD_A < LA) {
        load_a(std::integral_constant<int, m / LOAD_A>(), ca, na, t[0], t[1]);
        if constexpr (WHOLE && m / LOAD_A == LA - 1) forward(na, adv_a);
      }
    });
    ca = xa;
    cb = xb;
  };
  int u = 0;
  for (const int whole = (int)(g.K / 64) - NA; u < whole; ++u) unit(std::true_type(), u);
  for (; u < units; ++u) unit(std::false_type(), u);
  wait_vmcnt<0>();   // no load may land in LDS any more
  // the last instructions' results before any other instruction reads them (the compiler does not see
  // the instructions inside the assembly statements)
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
  lds_barrier();   // every wave has read its last operands: the buffers are free
  tile_epilogue<EPI, ACT>(g, acc, smem + wave * Out<FM, FN>::REGION, m0 + wm, n0 + wn, lane);
}

// What C becomes of the parts' sums, added in their order.
__global__ __launch_bounds__(256) void linear_join_kernel(Linear g, const float* part, int64_t ld, int parts) {
  const int64_t per = (g.N + 3) / 4, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = id / per, n = id % per * 4;
  if (m >= g.M) return;
  const float* p = part + m * ld + n;
  f32x4 v = *reinterpret_cast<const f32x4*>(p);
  for (int s = 1; s < parts; ++s) v += *reinterpret_cast<const f32x4*>(p + s * g.M * ld);
  finish4(g, m, n, v);
}

template <bool AT, bool BT, int EPI, int ACT, typename Cfg>
hipError_t run_tile(const Linear& g, int parts, hipStream_t s) {
  auto kern = linear_tile_kernel<AT, BT, EPI, ACT, Cfg>;
  (void)hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, Cfg::LDS);
  const int64_t wgs = (g.M + Cfg::BM - 1) / Cfg::BM * ((g.N + Cfg::BN - 1) / Cfg::BN);
  if (!grid_ok(wgs, 256)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(kern, dim3((unsigned)wgs, (unsigned)parts), dim3(256), Cfg::LDS, s, g);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Few rows of A (serving): B is read once and that bounds the call, so its bytes go straight from memory to
// the registers of the matrix instruction, with no LDS and no barrier on the way.  A workgroup computes 16 FM rows of A by
// 16 FN rows of B; its KS waves take every KS-th chunk of 32 CH k, each with the next chunk's loads in flight, and
// add their sums through LDS in the order of the waves.  The lanes of a row that does not exist load nothing.
// Weights that are not in a cache, replayed from a graph: 16 x 8192 x 2048 11.8 us, 16 x 2048 x 8192 18.8 (one workgroup a 16 columns leaves half
// of the CUs without work there; 16 waves gain nothing), 32 x 8192 x 2048 13.4, 16 x 4096 x 16384 42.
// ---------------------------------------------------------------------------
template <int FM, int FN, int KS, int CH, bool TAIL>
__global__ __launch_bounds__(64 * KS) void linear_rows_kernel(Linear g) {
  __shared__ f32x4 part[KS][FM * FN][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, lq = lane >> 4;
  const int ntn = (int)((g.N + 16 * FN - 1) / (16 * FN));
  const int64_t m0 = (int64_t)(blockIdx.x / ntn) * (16 * FM), n0 = (int64_t)(blockIdx.x % ntn) * (16 * FN);
  const uint16_t *arow[FM], *brow[FN];
  bool aon[FM], bon[FN];
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int64_t m = m0 + 16 * i + l16;
    aon[i] = m < g.M;
    arow[i] = g.A + (aon[i] ? m : m0) * g.lda + 8 * lq;
  }
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int64_t n = n0 + 16 * j + l16;
    bon[j] = n < g.N;
    brow[j] = g.B + (bon[j] ? n : n0) * g.ldb + 8 * lq;
  }
  struct Chunk {
    u32x4 a[CH][FM], b[CH][FN];
  };
  const int64_t kl = g.K - 8 * lq;
  // any alignment: memory takes 16-byte loads at every element; TAIL: a lane's last eight k may not all exist
  auto load16 = [&](const uint16_t* p, bool on, int64_t k) {
    u32x4 v = {0, 0, 0, 0};
    if (!on || k >= kl) return v;
    if (!TAIL || k + 8 <= kl) {
      __builtin_memcpy(&v, p + k, 16);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (k + q < kl) v[q / 2] |= (uint32_t)p[k + q] << (16 * (q & 1));
    }
    return v;
  };
  auto load = [&](int64_t c, Chunk& x) {
#pragma unroll
    for (int u = 0; u < CH; ++u) {
      const int64_t k = (c * CH + u) * 32;
#pragma unroll
      for (int j = 0; j < FN; ++j) x.b[u][j] = load16(brow[j], bon[j], k);
#pragma unroll
      for (int i = 0; i < FM; ++i) x.a[u][i] = load16(arow[i], aon[i], k);
    }
  };
  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto compute = [&](const Chunk& x) {
#pragma unroll
    for (int u = 0; u < CH; ++u)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int i = 0; i < FM; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x.b[u][j]),
                                                             __builtin_bit_cast(bf16x8, x.a[u][i]), acc[i][j], 0, 0, 0);
  };
  const int64_t chunks = (g.K + 32 * CH - 1) / (32 * CH);
  Chunk x, y;
  int64_t c = wave;
  if (c < chunks) load(c, x);
  while (c < chunks) {
    if (c + KS < chunks) load(c + KS, y);
    compute(x);
    c += KS;
    if (c >= chunks) break;
    if (c + KS < chunks) load(c + KS, x);
    compute(y);
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
    const int64_t m = m0 + 16 * (f / FN) + l16;
    if (m < g.M) finish4(g, m, n0 + 16 * (f % FN) + 4 * lq, sum);
  }
}

template <int FM, int FN, int KS, int CH>
hipError_t run_rows(const Linear& g, hipStream_t s) {
  const int64_t wgs = (g.M + 16 * FM - 1) / (16 * FM) * ((g.N + 16 * FN - 1) / (16 * FN));
  if (!grid_ok(wgs, 64 * KS)) return hipErrorInvalidConfiguration;
  if (g.K % 8) hipLaunchKernelGGL((linear_rows_kernel<FM, FN, KS, CH, true>), dim3((unsigned)wgs), dim3(64 * KS), 0, s, g);
  else hipLaunchKernelGGL((linear_rows_kernel<FM, FN, KS, CH, false>), dim3((unsigned)wgs), dim3(64 * KS), 0, s, g);
  return hipGetLastError();
}
// ---------------------------------------------------------------------------
// One row of A (a token): products on the vector unit, so that a wave's load of B is a kilobyte of one row (the matrix
// instruction's operand is 64 bytes of each of 16 rows, which costs where rows lie far apart).  A workgroup takes four rows
// of B, its waves every blockDim / 64-th chunk of 512 k, two chunks in flight; sums over the lanes, then over the waves in their order.
// Weights that are not in a cache, replayed from a graph, us (in brackets the kernel for few rows): 2048 x 8192 10.0 (12.4),
// 4096 x 16384 29.2 (35.3; 4.6 TB/s), 16384 x 4096 28.7 (29.7), 8192 x 2048 9.5 (9.5), 8192 x 2049 11.1 (17.4), 1000 x 1000 3.8 (3.1).
// Two rows in this manner take 12.0 and 10.4 for the first and the fourth (13.4 and 10.0), four 14.3 and 13.0 (14.6 and 10.6).
// ---------------------------------------------------------------------------
template <bool TAIL>
__global__ __launch_bounds__(512) void linear_token_kernel(Linear g) {
  constexpr int NR = 4, U = 2;
  __shared__ float part[8][NR];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int64_t n0 = (int64_t)blockIdx.x * NR;
  const uint16_t* brow[NR];
#pragma unroll
  for (int j = 0; j < NR; ++j) brow[j] = g.B + (n0 + j < g.N ? n0 + j : n0) * g.ldb;
  float acc[NR] = {};
  const int64_t step = (int64_t)waves * 512;
  for (int64_t k0 = wave * 512 + lane * 8; k0 < g.K; k0 += U * step) {
    Row8<uint16_t> a[U], b[U][NR];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = k0 + u * step;
      if (k >= g.K) break;
#pragma unroll
      for (int j = 0; j < NR; ++j) b[u][j].template load<TAIL>(brow[j], k, g.K);
      a[u].template load<TAIL>(g.A, k, g.K);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k0 + u * step >= g.K) break;
      float x[8];
      a[u].get(x);
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        float w[8];
        b[u][j].get(w);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[j] = __builtin_fmaf(x[q], w[q], acc[j]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NR; ++j) {
#pragma unroll
    for (int d = 32; d >= 1; d /= 2) acc[j] += __shfl_xor(acc[j], d);
    if (lane == 0) part[wave][j] = acc[j];
  }
  __syncthreads();
  if (threadIdx.x > 0) return;
  f32x4 v;
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    v[j] = part[0][j];
    for (int w = 1; w < waves; ++w) v[j] += part[w][j];
  }
  finish4(g, 0, n0, v);
}

hipError_t run_token(const Linear& g, hipStream_t s) {
  const int threads = g.K > 7168 ? 512 : (int)((g.K + 1023) / 1024) * 64;   // two chunks a wave, up to eight waves
  const int64_t wgs = (g.N + 3) / 4;
  if (!grid_ok(wgs, threads)) return hipErrorInvalidConfiguration;
  if (g.K % 8) hipLaunchKernelGGL(linear_token_kernel<true>, dim3((unsigned)wgs), dim3(threads), 0, s, g);
  else hipLaunchKernelGGL(linear_token_kernel<false>, dim3((unsigned)wgs), dim3(threads), 0, s, g);
  return hipGetLastError();
}

// What the tiled kernel asks of an operand: 16-byte loads that lie inside it or outside, and 31-bit offsets
// inside a tile.  `line` is its contiguous size.
bool line_ok(const uint16_t* X, int64_t ld, int64_t line) {
  return (uintptr_t)X % 16 == 0 && ld % 8 == 0 && ld < (1 << 22) && line % 8 == 0;
}

using Lin256 = LinCfg<8, 8, 2>;
using Lin256x128 = LinCfg<8, 4, 3>;
using Lin128 = LinCfg<4, 4, 4>;

template <bool AT, bool BT, int EPI, int ACT>
hipError_t run_sized(const Linear& g, const LinearPlan& p, hipStream_t s) {
  switch (p.tile) {
    case LinearPlan::T256: return run_tile<AT, BT, EPI, ACT, Lin256>(g, p.parts, s);
    case LinearPlan::T256x128: return run_tile<AT, BT, EPI, ACT, Lin256x128>(g, p.parts, s);
  }
  return run_tile<AT, BT, EPI, ACT, Lin128>(g, p.parts, s);
}
template <bool BT, int EPI>
hipError_t run_act(const Linear& g, const LinearPlan& p, hipStream_t s) {
  switch (g.act) {
    case ACT_RELU: return run_sized<false, BT, EPI, ACT_RELU>(g, p, s);
    case ACT_GELU_TANH: return run_sized<false, BT, EPI, ACT_GELU_TANH>(g, p, s);
    case ACT_SILU: return run_sized<false, BT, EPI, ACT_SILU>(g, p, s);
  }
  if constexpr (EPI == EPI_FWD) return run_sized<false, BT, EPI, ACT_NONE>(g, p, s);
  return hipErrorInvalidValue;   // a gate has an activation
}

hipError_t run_tiles(const Linear& g, const LinearPlan& p, hipStream_t s) {
  if (!g.a_t && !g.b_t) {
    return g.epi == EPI_FWD ? run_act<false, EPI_FWD>(g, p, s) : run_sized<false, false, EPI_PLAIN, ACT_NONE>(g, p, s);
  }
  if (g.a_t) {
    return g.epi == EPI_ADD ? run_sized<true, true, EPI_ADD, ACT_NONE>(g, p, s)
                            : run_sized<true, true, EPI_PLAIN, ACT_NONE>(g, p, s);
  }
  return g.epi == EPI_GATE ? run_act<true, EPI_GATE>(g, p, s) : run_sized<false, true, EPI_PLAIN, ACT_NONE>(g, p, s);
}

int64_t part_bytes(const LinearPlan& p, int64_t M, int64_t N) {
  return p.parts > 1 ? p.parts * M * ((N + 3) / 4 * 4) * 4 : 0;
}

// Copies of operands that the tiled kernel cannot load: X [rows][line] to P [rows][up to a multiple of eight], zeros behind
// the line.  The first `na` workgroups copy A, the others B; the launch's are those from `first` on.
struct Pack {
  const uint16_t* X;
  int64_t ld, rows, line;
  uint16_t* P;             // null: nothing to copy
};
__global__ __launch_bounds__(256) void linear_pack_kernel(Pack a, Pack b, int64_t na, int64_t first) {
  const int64_t wg = first + blockIdx.x;
  const bool second = wg >= na;
  const Pack& p = second ? b : a;
  const int64_t per = (p.line + 7) / 8, id = (wg - (second ? na : 0)) * 256 + threadIdx.x;
  const int64_t r = id / per, c = id % per * 8;
  if (r >= p.rows) return;
  const uint16_t* x = p.X + r * p.ld;
  u32x4 v = {0, 0, 0, 0};
  if (c + 8 <= p.line) {
    __builtin_memcpy(&v, x + c, 16);
  } else {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (c + q < p.line) v[q / 2] |= (uint32_t)x[c + q] << (16 * (q & 1));
  }
  *reinterpret_cast<u32x4*>(p.P + (r * per + c / 8) * 8) = v;
}
int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }
int64_t pack_bytes(int t, int64_t R, int64_t K) { return t ? K * up8(R) * 2 : R * up8(K) * 2; }

hipError_t run_pack(const Pack& a, const Pack& b, hipStream_t s) {
  auto wgs = [](const Pack& p) { return p.P ? (p.rows * ((p.line + 7) / 8) + 255) / 256 : 0; };
  const int64_t na = wgs(a), nb = wgs(b);
  constexpr int64_t PIECE = int64_t(1) << 23;   // workgroups of a launch: 2^31 work-items
  return in_pieces(na + nb, PIECE, [&](int64_t first, int64_t n) {
    hipLaunchKernelGGL(linear_pack_kernel, dim3((unsigned)n), dim3(256), 0, s, a, b, na, first);
    return hipGetLastError();
  });
}

hipError_t linear_piece(const Linear& g, LinearPlan p, void* work, int64_t work_bytes, hipStream_t s) {
  if (force_generic()) return run_general(g, s);
  if (p.tile == LinearPlan::ROWS && g.M == 1) return run_token(g, s);
  if (p.tile == LinearPlan::ROWS) return g.M > 16 ? run_rows<2, 2, 8, 4>(g, s) : run_rows<1, 1, 8, 4>(g, s);
  Linear q = g;
  q.ra = g.M, q.rb = g.N, q.ka = q.kb = g.K;
  const bool ca = !line_ok(g.A, g.lda, g.a_t ? g.M : g.K), cb = !line_ok(g.B, g.ldb, g.b_t ? g.N : g.K);
  if (ca || cb) {
    const int64_t ba = ca ? pack_bytes(g.a_t, g.M, g.K) : 0, bb = cb ? pack_bytes(g.b_t, g.N, g.K) : 0;
    if (!p.pack || work_bytes < ba + bb || up8(g.a_t ? g.M : g.K) >= (1 << 22) || up8(g.b_t ? g.N : g.K) >= (1 << 22))
      return run_general(g, s);
    Pack a{}, b{};
    if (ca) {
      a = Pack{g.A, g.lda, g.a_t ? g.K : g.M, g.a_t ? g.M : g.K, (uint16_t*)work};
      q.A = a.P;
      q.lda = up8(a.line);
      (g.a_t ? q.ra : q.ka) = q.lda;
    }
    if (cb) {
      b = Pack{g.B, g.ldb, g.b_t ? g.K : g.N, g.b_t ? g.N : g.K, (uint16_t*)((char*)work + ba)};
      q.B = b.P;
      q.ldb = up8(b.line);
      (g.b_t ? q.rb : q.kb) = q.ldb;
    }
    const hipError_t e = run_pack(a, b, s);
    if (e != hipSuccess) return e;
    work = (char*)work + ba + bb;
    work_bytes -= ba + bb;
  }
  if (work_bytes < part_bytes(p, g.M, g.N)) p.parts = 1;
  if (p.parts == 1) return run_tiles(q, p, s);
  q.epi = EPI_PLAIN;
  q.C = work;
  q.ldc = (g.N + 3) / 4 * 4;
  q.bf16_out = 0;
  q.act = ACT_NONE;
  q.bias = nullptr;
  q.R = nullptr;
  q.Z = nullptr;
  q.P = nullptr;
  q.part_k = p.part_k;
  const hipError_t e = run_tiles(q, p, s);
  if (e != hipSuccess) return e;
  const int64_t wgs = (g.M * ((g.N + 3) / 4) + 255) / 256;
  if (!grid_ok(wgs, 256)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL(linear_join_kernel, dim3((unsigned)wgs), dim3(256), 0, s, g, (const float*)work, q.ldc, p.parts);
  return hipGetLastError();
}

// The kernel for a product, by what each is expected to take: rounds of one workgroup a CU, each a fixed time and one
// per 1024 k that grows with the part x of the GPU that is at work (its power and the memory behind the L2s are shared),
// and where the reduction is cut a launch, the parts' bytes and a step per part.  The constants are fits of measured
// times of operands that are not in a cache, in us, of 54 products in three operand orders; the choice by them is
// at most 11 % behind the best one there, 0.5 % on average.  With 256 x 256, 256 x 128 and 128 x 128 tiles, each with its best number of
// parts: 4096 x 4096 x 4096 97, 118, 151; 4096 x 2048 x 8192 123, 113, 134; 1024 x 8192 x 2048 48, 35, 45; 2048 x 2048 x 8192 72, 71, 71 (4, 2 and 1
// parts); 1000^3 26, 22, 16; 512 x 2048 x 8192 37, 33, 33 (12, 8 and 4).
struct TileCost {
  int tile, bm, bn;
  double fixed, alone, shared;     // a round: fixed + (alone + shared x^2) per 1024 k
};
constexpr TileCost kTiles[] = {{LinearPlan::T128, 128, 128, 5.2, 8.6, 0.4},
                               {LinearPlan::T256x128, 256, 128, 7.4, 11.8, 1.8},
                               {LinearPlan::T256, 256, 256, 10.6, 16.6, 5.6}};
constexpr int kRound = 256;        // workgroups that the GPU computes at once

double round_us(const TileCost& t, double k, int64_t workgroups) {
  const double x = (double)workgroups / kRound;
  return t.fixed + (t.alone + t.shared * x * x) * k;
}

LinearPlan linear_plan(int a_t, int b_t, int64_t M, int64_t N, int64_t K, bool aligned) {
  // Few rows: the kernel without LDS, against the best of the tiles in us: 1 x 2048 x 8192 12 and 16 (10 by the kernel for one
  // row), 16 x 8192 x 2048 12 and 15, 16 x 2048 x 8192 19 and 18; 32 x 8192 x 2048 13 and 15, but 32 x 2048 x 8192 26 and 18
  if (!a_t && !b_t && (M <= 16 || (M <= 32 && K <= 2048))) return LinearPlan{LinearPlan::ROWS, 1, K, false};
  LinearPlan best{LinearPlan::T256, 1, K, false};
  double least = 1e30;
  for (const TileCost& t : kTiles) {
    const int64_t tiles = (M + t.bm - 1) / t.bm * ((N + t.bn - 1) / t.bn);
    for (int p = 1; p <= 16 && (p == 1 || (K >= 256 * p && tiles * p <= 4 * kRound)); ++p) {
      const int64_t part_k = p == 1 ? K : ((K + p - 1) / p + 63) / 64 * 64, parts = (K + part_k - 1) / part_k, wgs = tiles * parts;
      const double k = part_k / 1024.0;
      double us = (double)(wgs / kRound) * round_us(t, k, kRound);
      if (wgs % kRound) us += round_us(t, k, wgs % kRound);
      if (parts > 1) us += 3.6 + 0.3 * (double)parts + 1e-6 * (double)(parts * M) * (double)N;
      if (us < least) {
        least = us;
        best = LinearPlan{t.tile, (int)parts, part_k, false};
      }
    }
  }
  // Operands that the tiles cannot load are copied first, unless the general kernel is done sooner: 1.7 us per 64 k
  // and 1536 of its 64 x 64 tiles.  With a copy and without, us: 1000 x 1111 x 777 22 and 27, 4096 x 5001 x 3333
  // 200 and 649, its gradients 137 and 795, 189 and 1139; 200 x 500 x 300 14 and 11.
  if (!aligned) {
    const double general = 4 + 1.7 / 64 * (double)K * (double)(((M + 63) / 64 * ((N + 63) / 64) + 1535) / 1536);
    const double elements = ((double)M + (double)N) * (double)K;   // the copies: 2 bytes each, in one launch
    best.pack = elements < 1LL << 35 && least + 4 + 4e-6 / 5 * elements < general;
  }
  return best;
}

}  // namespace

// Columns of a launch, at most: below every kernel's limit of workgroups.
constexpr int64_t kPieceCols = int64_t(1) << 21;

int64_t linear_work_bytes(int a_t, int b_t, int64_t M, int64_t N, int64_t K, bool aligned) {
  const int64_t m = M < kPieceRows ? M : kPieceRows;
  N = N < kPieceCols ? N : kPieceCols;
  aligned = aligned && (a_t ? M : K) % 8 == 0 && (b_t ? N : K) % 8 == 0;
  const LinearPlan p = linear_plan(a_t, b_t, m, N, K, aligned);
  if (p.tile == LinearPlan::ROWS || (!aligned && !p.pack)) return 0;
  return part_bytes(p, m, N) + (aligned ? 0 : pack_bytes(a_t, m, K) + pack_bytes(b_t, N, K));
}

hipError_t launch_linear(const Linear& g, void* work, int64_t work_bytes, hipStream_t s) {
  auto piece = [&](int64_t m0, int64_t m, int64_t n0, int64_t n) {
    Linear p = g;
    p.A += g.a_t ? m0 : m0 * g.lda;
    p.B += g.b_t ? n0 : n0 * g.ldb;
    p.M = m;
    p.N = n;
    p.C = (uint8_t*)g.C + (m0 * g.ldc + n0) * (g.bf16_out ? 2 : 4);
    if (g.bias) p.bias = (const uint8_t*)g.bias + n0 * (g.bias_bf16 ? 2 : 4);
    if (g.R) p.R += m0 * g.ldr + n0;
    if (g.Z) p.Z += m0 * g.ldz + n0;
    if (g.P) p.P += m0 * g.ldp + n0;
    const bool aligned = line_ok(p.A, p.lda, p.a_t ? m : p.K) && line_ok(p.B, p.ldb, p.b_t ? n : p.K);
    return linear_piece(p, linear_plan(g.a_t, g.b_t, m, n, g.K, aligned), work, work_bytes, s);
  };
  return in_pieces(g.M, kPieceRows, [&](int64_t m0, int64_t m) {
    return in_pieces(g.N, kPieceCols, [&](int64_t n0, int64_t n) { return piece(m0, m, n0, n); });
  });
}

}  // namespace nms
