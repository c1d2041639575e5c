// Quantisation to 8-bit floating point in blocks of 128 with a power-of-two scale.
#include "fp8.hpp"
#include "launch.hpp"
#include "pieces.hpp"

namespace nms {
namespace {

// Eight consecutive elements of a row from column c: 16-byte loads (VEC: the row is aligned, and the
// columns exist), or one at a time with 0 beyond K.
template <bool VEC, typename T>
__device__ inline void load8(const T* p, int64_t c, int64_t K, Raw8<T>& x) {
  if constexpr (VEC) {
    __builtin_memcpy(x.w, __builtin_assume_aligned(p + c, 16), sizeof(x.w));
  } else {
    T b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = c + i < K ? p[c + i] : (T)0;
    __builtin_memcpy(x.w, b, sizeof(x.w));
  }
}

// Source row of row r of the quantisers' input, -1 for a row of zeros.
__device__ inline int source_row(const QuantArgs& a, int r) {
  if (!a.src) return r;
  const int sl = a.src[r];
  const uint32_t t = __umulhi(a.div.mul, (uint32_t)sl);
  const int row = (int)((t + (((uint32_t)sl - t) >> a.div.s1)) >> a.div.s2);
  return sl >= 0 && row < a.RX ? row : -1;
}
// Eight elements of N rows of the input from column c (rows[i] their sources, -1: zeros; r[i] their own
// numbers, for the gate).  All loads are issued before any is used; what is zero reads a place that
// exists.  VEC: K % 8 == 0 and aligned rows, so a lane's eight columns exist or do not, together.
template <bool VEC, typename T, int N>
__device__ inline void input_rows(const QuantArgs& a, const int (&rows)[N], const int (&r)[N], int64_t c,
                                  Raw8<T> (&x)[N]) {
  const T* X = (const T*)a.X;
  const T* G = (const T*)a.gate;
  const bool own = G && (const void*)G == a.X && !a.src && a.ldg == a.ldx;   // the gate is the row itself
  const bool in = c < a.K;
  const int64_t at = in ? c : 0;
#pragma unroll
  for (int i = 0; i < N; ++i) load8<VEC>(X + (rows[i] < 0 ? 0 : rows[i]) * a.ldx, at, a.K, x[i]);
  if (G && !own) {
    Raw8<T> g[N];
#pragma unroll
    for (int i = 0; i < N; ++i) load8<VEC>(G + r[i] * a.ldg, at, a.K, g[i]);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i].gate(g[i]);
  } else if (own) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i].gate(Raw8<T>(x[i]));
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (rows[i] < 0 || !in) x[i].zero();
}

template <int CTRL>
__device__ inline uint32_t dpp_max(uint32_t m) {
  return umax2(m, (uint32_t)__builtin_amdgcn_update_dpp((int)m, (int)m, CTRL, 0xF, 0xF, false));
}
// Maximum over 16 consecutive lanes, in each of them (rotations by 8, 4, 2, 1).
__device__ inline uint32_t row16_max(uint32_t m) { return dpp_max<0x121>(dpp_max<0x122>(dpp_max<0x124>(dpp_max<0x128>(m)))); }

// Rows: 16 lanes hold a block (8 elements a lane), a wave four consecutive blocks of N rows, a
// workgroup 4 N rows x 4 blocks; the scales leave through LDS so that a block's are written together.
// One pass over the data; bound by its bytes (36864 x 2048 bf16, 226 MB: 41 us, 5.5 TB/s; the same rows
// gathered from 4096 tokens: 28 us).  N = 4 keeps four rows' loads in flight (eight, with fewer waves:
// 32 us); N = 1 spreads few rows over more CUs (128 rows of 1024: 3.0 us, eight rows a wave 8.9).
template <typename T, bool E5M2, int N, bool VEC>
__global__ __launch_bounds__(256) void fp8_quantize_kernel(QuantArgs a) {
  __shared__ float sc[4][4 * N];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t r0 = (int64_t)blockIdx.x * (4 * N);
  const int64_t kb0 = (int64_t)blockIdx.y * 4, nkb = (a.K + 127) / 128;
  const int64_t kb = kb0 + (lane >> 4);
  const int64_t c = kb * 128 + (lane & 15) * 8;
  int r[N], rows[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t row = r0 + wave * N + i;
    r[i] = (int)(row < a.R ? row : a.R - 1);   // repeats that are not stored
    rows[i] = source_row(a, r[i]);
  }
  Raw8<T> x[N];
  input_rows<VEC, T, N>(a, rows, r, c, x);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int rl = wave * N + i;
    uint32_t m = row16_max(x[i].row_max());
    if (__any(m >= 0x7F800000u)) {
      x[i].clean();
      Raw8<T> f = x[i];
#pragma unroll
      for (int q = 0; q < Raw8<T>::NMAX; ++q) {
        const auto v = f.mag_finite(q);
        __builtin_memcpy(&f.w[q], &v, 4);
      }
      m = row16_max(f.row_max());
    }
    const float scale = power2(block_exponent(m, E5M2));
    const u32x2 q = pack_row<E5M2>(x[i], scale);
    if (r0 + rl < a.R && kb < nkb) {
      uint8_t* dst = a.Q + (r0 + rl) * a.ldq + c;
      if (((uintptr_t)dst & 7) == 0) {
        *reinterpret_cast<u32x2*>(dst) = q;
      } else {
#pragma unroll
        for (int b = 0; b < 8; ++b) dst[b] = (uint8_t)(q[b >> 2] >> (8 * (b & 3)));
      }
    }
    if ((lane & 15) == 0) sc[lane >> 4][rl] = scale;
  }
  __syncthreads();
  if (threadIdx.x < 16 * N) {
    const int kq = threadIdx.x / (4 * N), rl = threadIdx.x % (4 * N);
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

// Transposed: 256 rows (two blocks) x 64 columns a workgroup, so that a column of the result leaves as
// 256 contiguous bytes (36864 gathered rows of 2048: 34 us, of their own: 40 us, 5.7 TB/s).  Thread -> columns
// 8 (tid % 8) .. +7, rows 8 (tid / 8) .. +7, in registers; the column maxima are reduced over a block's
// two waves; the bytes pass through LDS, where column j is 32 slots of 8 rows, slot s at s ^ 4 (j / 8):
// a wave's writes cover all banks twice, and 16-byte reads keep their order.
template <typename T, bool E5M2, bool VEC>
__global__ __launch_bounds__(256) void fp8_quantize_t_kernel(QuantArgs a) {
  constexpr int NM = Raw8<T>::NMAX;
  __shared__ __align__(16) unsigned char tile[64][256];
  __shared__ typename Raw8<T>::Max cmax[4][8][NM];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t r0 = (int64_t)blockIdx.x * 256, k0 = (int64_t)blockIdx.y * 64;
  const int cg = tid & 7, rg = tid >> 3;
  const int64_t c = k0 + cg * 8;
  Raw8<T> x[8];
  int r[8], rows[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = r0 + rg * 8 + i;
    const bool in = row < a.R;
    r[i] = (int)(in ? row : a.R - 1);
    rows[i] = source_row(a, r[i]);
    if (!in) rows[i] = -1;   // the padding columns of the result are 0
  }
  input_rows<VEC, T, 8>(a, rows, r, c, x);
  typename Raw8<T>::Max m[NM];
  auto maxima = [&](auto mag) {
#pragma unroll
    for (int q = 0; q < NM; ++q) {
      m[q] = mag(x[0], q);
#pragma unroll
      for (int i = 1; i < 8; ++i) m[q] = vmax(m[q], mag(x[i], q));
#pragma unroll
      for (int d = 8; d <= 32; d *= 2) {
        uint32_t o;
        __builtin_memcpy(&o, &m[q], 4);
        o = __shfl_xor(o, d);
        typename Raw8<T>::Max om;
        __builtin_memcpy(&om, &o, 4);
        m[q] = vmax(m[q], om);
      }
      if (lane < 8) cmax[wave][cg][q] = m[q];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < NM; ++q) m[q] = vmax(cmax[wave & 2][cg][q], cmax[(wave & 2) + 1][cg][q]);
  };
  maxima([](const Raw8<T>& v, int q) { return v.mag(q); });
  bool odd = false;   // a column with an infinity or NaN
#pragma unroll
  for (int q = 0; q < 8; ++q) odd |= Raw8<T>::column(m, q) >= 0x7F800000u;
  if (__syncthreads_or(odd)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i].clean();
    maxima([](const Raw8<T>& v, int q) { return v.mag_finite(q); });
  }
  const int64_t rp = (a.R + 127) / 128 * 128;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float scale = power2(block_exponent(Raw8<T>::column(m, q), E5M2));
    const u32x2 b = pack_column<E5M2>(x, q, scale);
    *reinterpret_cast<u32x2*>(&tile[cg * 8 + q][(rg ^ (cg * 4)) * 8]) = b;
    if ((rg & 15) == 0 && c + q < a.K && r0 + rg * 8 < rp) a.S[(r0 / 128 + (rg >> 4)) * a.lds + c + q] = scale;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int id = tid + 256 * i, col = id >> 4, piece = id & 15;   // 16 rows a piece
    if (k0 + col >= a.K || r0 + 16 * piece >= rp) continue;
    const u32x4 v = *reinterpret_cast<const u32x4*>(&tile[col][((2 * piece) ^ ((col >> 3) * 4)) * 8]);
    uint8_t* dst = a.Q + (k0 + col) * a.ldq + r0 + 16 * piece;
    if (((uintptr_t)dst & 15) == 0) {
      *reinterpret_cast<u32x4*>(dst) = v;
    } else {
      for (int b = 0; b < 16; ++b) dst[b] = (uint8_t)(v[b >> 2] >> (8 * (b & 3)));
    }
  }
}

// One 128 x 128 block of a weight: its bytes row by row, and the same bytes transposed.  Bound by its
// bytes: 64 weights of 1024 x 2048 bf16 in 77 us (403 MB, 5.3 TB/s), with the transposed bytes 102 us (537 MB).
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
  Raw8<T> x[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = n0 + rg * 8 + i;
    x[i].zero();
    if (r < N && c < K) {
      if (vec && c + 8 <= K) load8<true>(W + r * ldw, c, K, x[i]);
      else load8<false>(W + r * ldw, c, K, x[i]);
    }
    m = umax2(m, x[i].row_max());
  }
  auto block_max = [&](uint32_t v) {
#pragma unroll
    for (int d = 32; d > 0; d /= 2) v = umax2(v, __shfl_xor(v, d));
    if (lane == 0) bmax[wave] = v;
    __syncthreads();
    return umax2(umax2(bmax[0], bmax[1]), umax2(bmax[2], bmax[3]));
  };
  m = block_max(m);
  if (m >= 0x7F800000u) {   // the same for the whole workgroup
    __syncthreads();        // bmax has been read
    m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i].clean();
      Raw8<T> f = x[i];
#pragma unroll
      for (int q = 0; q < Raw8<T>::NMAX; ++q) {
        const auto v = f.mag_finite(q);
        __builtin_memcpy(&f.w[q], &v, 4);
      }
      m = umax2(m, f.row_max());
    }
    m = block_max(m);
  }
  const float scale = power2(block_exponent(m, E5M2));
  if (tid == 0) {
    S[(ex * nb + ib) * kbn + jb] = scale;
    if (St) St[(ex * kbn + jb) * nb + ib] = scale;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = n0 + rg * 8 + i;
    if (r >= N) continue;
    const u32x2 q = pack_row<E5M2>(x[i], scale);
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
    const u32x2 b = pack_column<E5M2>(x, q, scale);
    *tile_slot(tile, cg * 8 + q, rg) = (uint64_t)b[0] | ((uint64_t)b[1] << 32);
  }
  __syncthreads();
  store_transposed(tile, Qt + ex * K * ldqt, ldqt, k0, K, n0);
}

bool vec_ok(int es, const void* X, int64_t ldx, const void* gate, int64_t ldg) {
  return (uintptr_t)X % 16 == 0 && (ldx * es) % 16 == 0 && (uintptr_t)gate % 16 == 0 && (!gate || (ldg * es) % 16 == 0);
}

}  // namespace

template <typename T, bool E5M2, bool VEC>
static hipError_t quantize_rows(const QuantArgs& a, hipStream_t s) {
  const unsigned gy = (unsigned)((a.K + 511) / 512);
  // four rows a wave once that fills the chip's 256 CUs twice
  if ((a.R + 15) / 16 * gy >= 512)
    hipLaunchKernelGGL((fp8_quantize_kernel<T, E5M2, 4, VEC>), dim3((unsigned)((a.R + 15) / 16), gy), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((fp8_quantize_kernel<T, E5M2, 1, VEC>), dim3((unsigned)((a.R + 3) / 4), gy), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <typename T, bool E5M2, bool VEC>
static hipError_t quantize_columns(const QuantArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((fp8_quantize_t_kernel<T, E5M2, VEC>), dim3((unsigned)((a.R + 255) / 256), (unsigned)((a.K + 63) / 64)),
                     dim3(256), 0, s, a);
  return hipGetLastError();
}

// Rows r0 .. r0 + n - 1 of a.
static QuantArgs rows_of(const QuantArgs& a, int es, int64_t r0, int64_t n) {
  QuantArgs p = a;
  if (a.src) p.src += r0;
  else p.X = (const uint8_t*)a.X + r0 * a.ldx * es;
  if (a.gate) p.gate = (const uint8_t*)a.gate + r0 * a.ldg * es;
  p.R = n;
  p.Q += r0 * a.ldq;
  p.S += r0;
  return p;
}

static hipError_t quantize_piece(int dt, const QuantArgs& a, hipStream_t s) {
  const bool vec = a.K % 8 == 0 && vec_ok(dt == DT_BF16 ? 2 : 4, a.X, a.ldx, a.gate, a.ldg);
  if (dt == DT_BF16) {
    if (a.e5m2) return vec ? quantize_rows<uint16_t, true, true>(a, s) : quantize_rows<uint16_t, true, false>(a, s);
    return vec ? quantize_rows<uint16_t, false, true>(a, s) : quantize_rows<uint16_t, false, false>(a, s);
  }
  if (a.e5m2) return vec ? quantize_rows<uint32_t, true, true>(a, s) : quantize_rows<uint32_t, true, false>(a, s);
  return vec ? quantize_rows<uint32_t, false, true>(a, s) : quantize_rows<uint32_t, false, false>(a, s);
}

hipError_t launch_fp8_quantize(int dt, const QuantArgs& a, hipStream_t s) {
  return in_pieces(a.R, kPieceRows, [&](int64_t r0, int64_t n) {
    return quantize_piece(dt, rows_of(a, dt == DT_BF16 ? 2 : 4, r0, n), s);
  });
}

hipError_t launch_fp8_quantize_t(int dt, const QuantArgs& a, hipStream_t s) {
  const bool vec = a.K % 8 == 0 && vec_ok(dt == DT_BF16 ? 2 : 4, a.X, a.ldx, a.gate, a.ldg);
  if (dt == DT_BF16) {
    if (a.e5m2) return vec ? quantize_columns<uint16_t, true, true>(a, s) : quantize_columns<uint16_t, true, false>(a, s);
    return vec ? quantize_columns<uint16_t, false, true>(a, s) : quantize_columns<uint16_t, false, false>(a, s);
  }
  if (a.e5m2) return vec ? quantize_columns<uint32_t, true, true>(a, s) : quantize_columns<uint32_t, true, false>(a, s);
  return vec ? quantize_columns<uint32_t, false, true>(a, s) : quantize_columns<uint32_t, false, false>(a, s);
}

hipError_t launch_fp8_quantize_weight(int dt, const void* W, int64_t ldw, int64_t E, int64_t N, int64_t K, int e5m2,
                                      uint8_t* Q, int64_t ldq, float* S, uint8_t* Qt, int64_t ldqt, float* St,
                                      hipStream_t s) {
  const int64_t blocks = ((N + 127) / 128) * ((K + 127) / 128);
  if (!grid_ok(blocks, 256)) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks, (unsigned)E);
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
