// C ABI of libnmsparse: argument validation and dispatch to the gfx950 kernels.
// Every check runs on the host before anything is launched; a call that
// returns an error has touched no device memory.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <new>
#include <utility>

#include "../../include/nmsparse.h"
#include "launch.hpp"

namespace {

thread_local char g_last_hip_error[256] = "";

nm_status hip_status(hipError_t e) {
  if (e == hipSuccess) return NM_OK;
  const char* s = hipGetErrorString(e);
  strncpy(g_last_hip_error, s ? s : "unknown HIP error", sizeof(g_last_hip_error) - 1);
  g_last_hip_error[sizeof(g_last_hip_error) - 1] = '\0';
  return NM_ERR_HIP;
}

bool dtype_ok(nm_dtype dt) { return dt == NM_F32 || dt == NM_BF16; }
int esize(nm_dtype dt) { return dt == NM_BF16 ? 2 : 4; }
bool aligned(const void* p, int a) { return ((uintptr_t)p % (uintptr_t)a) == 0; }
bool m_ok(int M) { return M == 4 || M == 8 || M == 16; }
bool nm_ok(int N, int M) { return m_ok(M) && N >= 1 && N < M; }
bool v_ok(int V) { return V >= 1 && V <= 256; }
hipStream_t hs(nm_stream s) { return reinterpret_cast<hipStream_t>(s); }

bool score_ok(nm_score s) { return s == NM_SOFTMAX || s == NM_SIGMOID; }
bool scale_ok(float s) { return s != 0.f && s - s == 0.f; }   // not 0, infinite or NaN
bool fp8_ok(nm_fp8 f) { return f == NM_E4M3 || f == NM_E5M2; }
int64_t up128(int64_t n) { return (n + 127) / 128 * 128; }

// the checks fp8_quantize and fp8_quantize_t share
nm_status quantize_check(nm_dtype dt, const void* X, int64_t ldx, int64_t RX, const int32_t* src, int div,
                         const void* gate, int64_t ldg, int64_t R, int64_t K, nm_fp8 fmt, const void* Q, const void* S) {
  if (!X || !Q || !S) return NM_ERR_NULL;
  if (!dtype_ok(dt) || !fp8_ok(fmt)) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || RX <= 0 || R > INT32_MAX || K > INT32_MAX || ldx < K || (src ? div < 1 : R > RX) ||
      (gate && ldg < K))
    return NM_ERR_SHAPE;
  if (!aligned(X, esize(dt)) || !aligned(gate, esize(dt)) || !aligned(src, 4) || !aligned(S, 4)) return NM_ERR_ALIGN;
  return NM_OK;
}

// the checks the 8-bit products share
nm_status fp8_gemm_check(nm_fp8 fa, const void* A, int64_t lda, const void* sa, int64_t ldsa, nm_fp8 fb, const void* B,
                         int64_t ldb, const void* sb, int64_t M, int64_t N, int64_t K, nm_dtype out, const void* C,
                         int64_t ldc) {
  if (!A || !sa || !B || !sb || !C) return NM_ERR_NULL;
  if (!fp8_ok(fa) || !fp8_ok(fb) || !dtype_ok(out)) return NM_ERR_UNSUPPORTED;
  if (M <= 0 || N <= 0 || K <= 0 || M > INT32_MAX || N > INT32_MAX || K > INT32_MAX || lda < K || ldb < K || ldsa < M ||
      ldc < N)
    return NM_ERR_SHAPE;
  if (!aligned(sa, 4) || !aligned(sb, 4) || !aligned(C, esize(out))) return NM_ERR_ALIGN;
  return NM_OK;
}

bool act_ok(nm_act a) { return a >= NM_ACT_NONE && a <= NM_ACT_SILU; }
// A number of rows and a width that an int holds.
bool rows_ok(int64_t R, int64_t C) { return R > 0 && C > 0 && R <= INT32_MAX && C <= INT32_MAX; }

// The bytes of a matrix: rows of `width` bytes, `stride` apart; an empty one where p is null.
struct Area {
  uintptr_t lo, hi;   // hi: behind the last byte
  int64_t rows;
  uintptr_t width, stride;
};
Area area(const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t es) {
  if (!p || rows <= 0 || cols <= 0) return Area{0, 0, 0, 0, 0};
  const uintptr_t lo = (uintptr_t)p, width = (uintptr_t)(cols * es);
  if (rows == 1 || ld == cols) {   // one run of bytes
    const uintptr_t all = (uintptr_t)rows * width, hi = lo + all < lo ? UINTPTR_MAX : lo + all;
    return Area{lo, hi, 1, hi - lo, hi - lo};
  }
  const unsigned __int128 end = (unsigned __int128)(rows - 1) * ((uintptr_t)ld * (uintptr_t)es) + width + lo;
  return Area{lo, end > UINTPTR_MAX ? UINTPTR_MAX : (uintptr_t)end, rows, width, (uintptr_t)ld * (uintptr_t)es};
}
bool same(const Area& a, const Area& b) {
  return a.lo == b.lo && a.rows == b.rows && a.width == b.width && a.stride == b.stride;
}
// Whether two matrices share a byte: exactly, since columns of one buffer interleave without meeting.
bool meet(Area a, Area b) {
  if (a.lo >= b.hi || b.lo >= a.hi) return false;
  if (a.stride == b.stride && a.rows > 1 && b.rows > 1) {
    if (a.lo > b.lo) std::swap(a, b);
    const uintptr_t r = (b.lo - a.lo) / a.stride, off = (b.lo - a.lo) % a.stride;   // b's first row begins behind a's row r
    return (r < (uintptr_t)a.rows && off < a.width) || (r + 1 < (uintptr_t)a.rows && off + b.width > a.stride);
  }
  if (a.rows > b.rows) std::swap(a, b);
  // every row of the one that has fewer (one, unless both have gaps and other strides) against the first of b's rows that ends behind its start
  for (int64_t i = 0; i < a.rows; ++i) {
    const uintptr_t lo = a.lo + (uintptr_t)i * a.stride;
    if (lo >= b.hi) return false;
    const uintptr_t k = lo < b.lo + b.width ? 0 : (lo - b.lo - b.width) / b.stride + 1;
    if (k < (uintptr_t)b.rows && b.lo + k * b.stride < lo + a.width) return true;
  }
  return false;
}
// Whether an output meets another output or an input.  in_place: bit j of entry i where output i may be input j itself.
template <size_t NO, size_t NI>
bool overlap(const Area (&out)[NO], const Area (&in)[NI], const unsigned (&in_place)[NO]) {
  for (size_t i = 0; i < NO; ++i) {
    for (size_t j = 0; j < i; ++j)
      if (meet(out[i], out[j])) return true;
    for (size_t j = 0; j < NI; ++j)
      if (meet(out[i], in[j]) && !(in_place[i] >> j & 1 && same(out[i], in[j]))) return true;
  }
  return false;
}
constexpr int64_t kNormWidth = 16384;   // a row stays in the registers of a workgroup

// the checks rms_norm and rms_norm_fp8 share
nm_status norm_check(nm_dtype dt, const void* X, int64_t ldx, const void* residual, int64_t ldr, nm_dtype wdt,
                     const void* w, float eps, int64_t T, int64_t D, const void* H, int64_t ldh, const void* Y,
                     int64_t ldy, const float* rstd, const void* Q = nullptr, int64_t ldq = 0, const float* S = nullptr,
                     int64_t lds = 0) {
  if (!X || !w) return NM_ERR_NULL;
  if (!dtype_ok(dt) || !dtype_ok(wdt) || !(eps > 0.f) || eps - eps != 0.f) return NM_ERR_UNSUPPORTED;
  if (!rows_ok(T, D) || ldx < D || (residual && ldr < D) || (H && ldh < D) || (Y && ldy < D)) return NM_ERR_SHAPE;
  if (D > kNormWidth) return NM_ERR_UNSUPPORTED;
  if (Q && (ldq < up128(D) || lds < T)) return NM_ERR_SHAPE;
  if (!aligned(X, esize(dt)) || !aligned(residual, esize(dt)) || !aligned(w, esize(wdt)) || !aligned(H, esize(dt)) ||
      !aligned(Y, esize(dt)) || !aligned(rstd, 4) || !aligned(S, 4))
    return NM_ERR_ALIGN;
  const int64_t e = esize(dt), Dp = up128(D);
  const Area out[] = {area(H, T, D, ldh, e), area(Y, T, D, ldy, e), area(rstd, 1, T, T, 4), area(Q, T, Dp, ldq, 1),
                      area(S, Dp / 128, T, lds, 4)};
  const Area in[] = {area(X, T, D, ldx, e), area(residual, T, D, ldr, e)};
  return overlap(out, in, {3, 3, 0, 0, 0}) ? NM_ERR_SHAPE : NM_OK;
}

// A contiguous range of device memory that a call over many tensors reads, or writes (out).
struct Range {
  uintptr_t lo, hi;
  bool out;
};

// Whether an output meets another range (in place, an output is its own gradient).
bool outputs_overlap(const Range* r, int64_t n) {
  // sorted by address: the ranges that started before and reach furthest, among the outputs and among all
  uintptr_t hi_out = 0, hi_any = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (r[i].lo < hi_out || (r[i].out && r[i].lo < hi_any)) return true;
    if (r[i].out && r[i].hi > hi_out) hi_out = r[i].hi;
    if (r[i].hi > hi_any) hi_any = r[i].hi;
  }
  return false;
}

// the checks grad_norm and grad_clip share
nm_status grads_check(int64_t n, const nm_dtype* dt, const void* const* grads, const int64_t* counts,
                      const float* norm, const void* work, int64_t work_bytes, bool need_work) {
  if (n <= 0 || n > 65536) return NM_ERR_SHAPE;
  if (!dt || !grads || !counts || !norm) return NM_ERR_NULL;
  for (int64_t i = 0; i < n; ++i) {
    if (!dtype_ok(dt[i])) return NM_ERR_UNSUPPORTED;
    if (counts[i] < 0 || counts[i] > INT64_MAX / 8 / n) return NM_ERR_SHAPE;
    if (counts[i] == 0) continue;
    if (!grads[i]) return NM_ERR_NULL;
    if (!aligned(grads[i], esize(dt[i]))) return NM_ERR_ALIGN;
  }
  if (!aligned(norm, 4)) return NM_ERR_ALIGN;
  if (need_work) {
    const int64_t need = nms::grad_partials(counts, n) * 8;
    if (need > 0 && !work) return NM_ERR_NULL;
    if (work_bytes < need) return NM_ERR_SHAPE;
    if (!aligned(work, 8)) return NM_ERR_ALIGN;
  }
  return NM_OK;
}

}  // namespace

extern "C" {

nm_status nm_prune(nm_dtype dt, const void* A, int64_t lda, int64_t R, int64_t K, int N, int M, uint8_t* mask,
                   int64_t ldmask, nm_stream stream) {
  if (!A || !mask) return NM_ERR_NULL;
  if (!dtype_ok(dt) || !nm_ok(N, M)) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || K % M != 0 || lda < K || ldmask < K) return NM_ERR_SHAPE;
  if (!aligned(A, esize(dt))) return NM_ERR_ALIGN;
  return hip_status(nms::launch_nm_prune(dt, A, lda, R, K, N, M, mask, ldmask, hs(stream)));
}

nm_status nm_compress(nm_dtype dt, const void* A, int64_t lda, const uint8_t* mask, int64_t ldmask, int64_t R,
                      int64_t K, int N, int M, void* values, uint8_t* meta, int32_t* bad_groups,
                      nm_stream stream) {
  if (!A || !mask || !values || !meta) return NM_ERR_NULL;
  if (!dtype_ok(dt) || !nm_ok(N, M)) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || K % M != 0 || lda < K || ldmask < K) return NM_ERR_SHAPE;
  if (!aligned(A, esize(dt)) || !aligned(values, esize(dt)) || !aligned(bad_groups, 4)) return NM_ERR_ALIGN;
  return hip_status(
      nms::launch_nm_compress(dt, A, lda, mask, ldmask, R, K, N, M, values, meta, bad_groups, hs(stream)));
}

nm_status nm_prune_compress(nm_dtype dt, const void* A, int64_t lda, int64_t R, int64_t K, int N, int M,
                            uint8_t* mask, int64_t ldmask, void* values, uint8_t* meta, nm_stream stream) {
  if (!A || !mask || !values || !meta) return NM_ERR_NULL;
  if (!dtype_ok(dt) || !nm_ok(N, M)) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || K % M != 0 || lda < K || ldmask < K) return NM_ERR_SHAPE;
  if (!aligned(A, esize(dt)) || !aligned(values, esize(dt))) return NM_ERR_ALIGN;
  return hip_status(nms::launch_nm_prune_compress(dt, A, lda, R, K, N, M, mask, ldmask, values, meta, hs(stream)));
}

nm_status nm_prune_compress_transpose(nm_dtype dt, const void* A, int64_t lda, int64_t R, int64_t K, int N, int M,
                                      uint8_t* mask, int64_t ldmask, void* values, uint8_t* meta, const void* B,
                                      int64_t ldb, int64_t KB, int64_t Nc, void* Bt, int64_t ldbt, nm_stream stream) {
  if (!A || !mask || !values || !meta || !B || !Bt) return NM_ERR_NULL;
  if (dt != NM_BF16 || !nm_ok(N, M)) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || K % M != 0 || lda < K || ldmask < K) return NM_ERR_SHAPE;
  if (KB <= 0 || Nc <= 0 || ldb < Nc || ldbt < KB) return NM_ERR_SHAPE;
  if (!aligned(A, esize(dt)) || !aligned(values, esize(dt)) || !aligned(B, esize(dt)) || !aligned(Bt, esize(dt)))
    return NM_ERR_ALIGN;
  return hip_status(nms::launch_nm_prune_compress_transpose(dt, A, lda, R, K, N, M, mask, ldmask, values, meta, B,
                                                            ldb, KB, Nc, Bt, ldbt, hs(stream)));
}

nm_status nm_decompress(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R, int64_t K, int N, int M,
                        void* A_out, int64_t lda, nm_stream stream) {
  if (!values || !meta || !A_out) return NM_ERR_NULL;
  if (!dtype_ok(dt) || !nm_ok(N, M)) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || K % M != 0 || lda < K) return NM_ERR_SHAPE;
  if (!aligned(values, esize(dt)) || !aligned(A_out, esize(dt))) return NM_ERR_ALIGN;
  return hip_status(nms::launch_nm_decompress(dt, values, meta, R, K, N, M, A_out, lda, hs(stream)));
}

nm_status spmm_nm(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R, int64_t K, const void* B,
                  int64_t ldb, int64_t Nc, float* C, int64_t ldc, nm_stream stream) {
  if (!values || !meta || !B || !C) return NM_ERR_NULL;
  if (!dtype_ok(dt)) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || Nc <= 0 || K % 4 != 0 || ldb < Nc || ldc < Nc) return NM_ERR_SHAPE;
  if (!aligned(values, esize(dt)) || !aligned(B, esize(dt)) || !aligned(C, 4)) return NM_ERR_ALIGN;
  return hip_status(nms::launch_spmm_nm(dt, values, meta, R, K, B, ldb, Nc, C, ldc, hs(stream)));
}

nm_status spmm_nm_t(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R, int64_t K, const void* Bt,
                    int64_t ldbt, int64_t Nc, float* C, int64_t ldc, nm_stream stream) {
  if (!values || !meta || !Bt || !C) return NM_ERR_NULL;
  if (!dtype_ok(dt)) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || Nc <= 0 || K % 4 != 0 || ldbt < K || ldc < Nc) return NM_ERR_SHAPE;
  if (!aligned(values, esize(dt)) || !aligned(Bt, esize(dt)) || !aligned(C, 4)) return NM_ERR_ALIGN;
  return hip_status(nms::launch_spmm_nm_t(dt, values, meta, R, K, Bt, ldbt, Nc, C, ldc, hs(stream)));
}

nm_status spmm_nm_t_out_bf16(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R, int64_t K,
                             const void* Bt, int64_t ldbt, int64_t Nc, void* C, int64_t ldc, nm_stream stream) {
  if (!values || !meta || !Bt || !C) return NM_ERR_NULL;
  if (!dtype_ok(dt)) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || Nc <= 0 || K % 4 != 0 || ldbt < K || ldc < Nc) return NM_ERR_SHAPE;
  if (!aligned(values, esize(dt)) || !aligned(Bt, esize(dt)) || !aligned(C, 2)) return NM_ERR_ALIGN;
  return hip_status(nms::launch_spmm_nm_t_bf16out(dt, values, meta, R, K, Bt, ldbt, Nc, (uint16_t*)C, ldc,
                                                  hs(stream)));
}

nm_status spmm_nm_t_lowrank(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R, int64_t K,
                            const void* Bt, int64_t ldbt, int64_t Nc, const void* U, int64_t ldu, const void* Vt,
                            int64_t ldvt, int64_t rank, float* Tt, float* C, int64_t ldc, nm_stream stream) {
  if (!values || !meta || !Bt || !U || !Vt || !Tt || !C) return NM_ERR_NULL;
  if (!dtype_ok(dt)) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || Nc <= 0 || rank <= 0 || rank > (1 << 20) || K % 4 != 0 || ldbt < K || ldc < Nc ||
      ldu < rank || ldvt < K)
    return NM_ERR_SHAPE;
  if (!aligned(values, esize(dt)) || !aligned(Bt, esize(dt)) || !aligned(U, esize(dt)) || !aligned(Vt, esize(dt)) ||
      !aligned(Tt, 4) || !aligned(C, 4))
    return NM_ERR_ALIGN;
  return hip_status(nms::launch_spmm_nm_t_lowrank(dt, values, meta, R, K, Bt, ldbt, Nc, U, ldu, Vt, ldvt, rank, Tt, C,
                                                  ldc, hs(stream)));
}

nm_status spmm_nm_general(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R, int64_t K, int N, int M,
                          const void* Bt, int64_t ldbt, int64_t Nc, float* C, int64_t ldc, void* work,
                          int64_t work_bytes, nm_stream stream) {
  if (!values || !meta || !Bt || !C) return NM_ERR_NULL;
  if (!dtype_ok(dt) || !nm_ok(N, M)) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || Nc <= 0 || K % M != 0 || ldbt < K || ldc < Nc || work_bytes < 0) return NM_ERR_SHAPE;
  if (!aligned(values, esize(dt)) || !aligned(Bt, esize(dt)) || !aligned(C, 4)) return NM_ERR_ALIGN;
  return hip_status(nms::launch_spmm_nm_general(dt, values, meta, R, K, N, M, Bt, ldbt, Nc, C, ldc, work, work_bytes,
                                                hs(stream)));
}

nm_status spmm_nm_general_noalloc(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R, int64_t K, int N,
                                  int M, const void* Bt, int64_t ldbt, int64_t Nc, float* C, int64_t ldc,
                                  nm_stream stream) {
  if (!values || !meta || !Bt || !C) return NM_ERR_NULL;
  if (!dtype_ok(dt) || !nm_ok(N, M)) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || Nc <= 0 || K % M != 0 || ldbt < K || ldc < Nc) return NM_ERR_SHAPE;
  if (!aligned(values, esize(dt)) || !aligned(Bt, esize(dt)) || !aligned(C, 4)) return NM_ERR_ALIGN;
  if (nms::general_work_bytes(esize(dt), R, K, N, M) > nms::GENERAL_SCRATCH_BYTES) return NM_ERR_TOO_LARGE;
  return hip_status(nms::launch_spmm_nm_general_noalloc(dt, values, meta, R, K, N, M, Bt, ldbt, Nc, C, ldc,
                                                        hs(stream)));
}

nm_status sddmm_venom(nm_dtype dt, const void* dY, int64_t lddy, const void* W_down, int64_t ldw, int64_t T,
                      int64_t F, int64_t Nc, int V, int M, const void* h_values, const uint8_t* h_meta,
                      const uint8_t* h_colsel, int apply_relu, float* dz, void* dYt, int64_t lddyt,
                      nm_stream stream) {
  if (!dY || !W_down || !h_values || !h_meta || !h_colsel || !dz) return NM_ERR_NULL;
  if (!dtype_ok(dt) || !m_ok(M) || !v_ok(V) || (dYt && dt != NM_BF16)) return NM_ERR_UNSUPPORTED;
  if (T <= 0 || F <= 0 || Nc <= 0 || F % M != 0 || T % V != 0 || lddy < Nc || ldw < Nc || (dYt && lddyt < T))
    return NM_ERR_SHAPE;
  if (!aligned(dY, esize(dt)) || !aligned(W_down, esize(dt)) || !aligned(h_values, 2 * esize(dt)) ||
      !aligned(h_colsel, 4) || !aligned(dz, 8) || !aligned(dYt, esize(dt)))
    return NM_ERR_ALIGN;
  return hip_status(nms::launch_sddmm_venom(dt, dY, lddy, W_down, ldw, T, F, Nc, V, M, h_values, h_meta, h_colsel,
                                            apply_relu ? 1 : 0, dz, dYt, lddyt, hs(stream)));
}

nm_status spmm_venom_tn(nm_dtype dt, const void* h_values, const uint8_t* h_meta, const uint8_t* h_colsel, int64_t T,
                        int64_t F, int V, int M, const void* dYt, int64_t lddyt, int64_t Nc, float* dW, int64_t lddw,
                        void* work, int64_t work_bytes, nm_stream stream) {
  if (!h_values || !h_meta || !h_colsel || !dYt || !dW) return NM_ERR_NULL;
  if (!dtype_ok(dt) || !m_ok(M) || !v_ok(V)) return NM_ERR_UNSUPPORTED;
  if (T <= 0 || F <= 0 || Nc <= 0 || F % M != 0 || T % V != 0 || lddyt < T || lddw < Nc || work_bytes < 0)
    return NM_ERR_SHAPE;
  if (!aligned(h_values, 2 * esize(dt)) || !aligned(h_colsel, 4) || !aligned(dYt, esize(dt)) || !aligned(dW, 4))
    return NM_ERR_ALIGN;
  return hip_status(nms::launch_spmm_venom_tn(dt, h_values, h_meta, h_colsel, T, F, V, M, dYt, lddyt, Nc, dW, lddw,
                                              work, work_bytes, hs(stream)));
}

int64_t nm_venom_tn_work_bytes(nm_dtype dt, int64_t T, int64_t F) {
  if (!dtype_ok(dt) || T <= 0 || F <= 0) return 0;
  return nms::venom_tn_work_bytes(esize(dt), T, F);
}

int nm_gmp_n_at(int M, int n_final, int64_t t_begin, int64_t t_end, int64_t interval, int64_t t_dense, int64_t step,
                int* prune_now) {
  if (prune_now) *prune_now = 0;
  if (!m_ok(M) || n_final < 1 || n_final >= M || t_begin < 0 || t_end < t_begin || interval < 1) return -1;
  if (step < t_begin || (t_dense >= 0 && step >= t_dense)) return M;   // dense before the ramp and after the switch
  const int64_t events = (t_end - t_begin) / interval + 1;           // at t_begin + e * interval
  int64_t e = (step - t_begin) / interval;                             // the last event at or before step
  if (e > events - 1) e = events - 1;
  if (prune_now && (step - t_begin) % interval == 0 && (step - t_begin) / interval < events) *prune_now = 1;
  const int64_t removed = ((int64_t)(M - n_final) * (e + 1) + events - 1) / events;   // ceil
  return M - (int)removed;
}

int64_t nm_general_scratch_bytes(void) { return nms::GENERAL_SCRATCH_BYTES; }

int64_t nm_general_work_bytes(nm_dtype dt, int64_t R, int64_t K, int N, int M) {
  if (!dtype_ok(dt) || !nm_ok(N, M) || R <= 0 || K <= 0 || K % M != 0) return 0;
  return nms::general_work_bytes(esize(dt), R, K, N, M);
}

nm_status spmm_nm_t_relu_venom(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R, int64_t K,
                               const void* Bt, int64_t ldbt, int64_t Nc, int V, int M, void* h_values,
                               uint8_t* h_meta, uint8_t* h_colsel, nm_stream stream) {
  if (!values || !meta || !Bt || !h_values || !h_meta || !h_colsel) return NM_ERR_NULL;
  if (dt != NM_BF16 || (V != 64 && V != 128 && V != 256) || (M != 4 && M != 8 && M != 16)) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || Nc <= 0 || K % 4 != 0 || ldbt < K || R % M != 0 || Nc % V != 0) return NM_ERR_SHAPE;
  if (!aligned(values, 2) || !aligned(Bt, 2) || !aligned(h_values, 2)) return NM_ERR_ALIGN;
  const hipError_t e = nms::launch_spmm_nm_t_relu_venom(values, meta, R, K, Bt, ldbt, Nc, V, M, h_values, h_meta,
                                                        h_colsel, hs(stream));
  if (e == hipErrorNotSupported) return NM_ERR_UNSUPPORTED;
  return hip_status(e);
}

nm_status nm_transpose(nm_dtype dt, const void* src, int64_t lds, int64_t R, int64_t Cn, void* dst, int64_t ldd,
                       nm_stream stream) {
  if (!src || !dst) return NM_ERR_NULL;
  if (dt != NM_BF16) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || Cn <= 0 || lds < Cn || ldd < R) return NM_ERR_SHAPE;
  if (!aligned(src, esize(dt)) || !aligned(dst, esize(dt))) return NM_ERR_ALIGN;
  return hip_status(nms::launch_nm_transpose(dt, src, lds, R, Cn, dst, ldd, hs(stream)));
}

nm_status prune_act_venom(nm_dtype dt, const void* Z, int64_t ldz, int64_t R, int64_t K, int V, int M,
                          int apply_relu, void* values, uint8_t* meta, uint8_t* colsel, uint8_t* mask,
                          int64_t ldmask, nm_stream stream) {
  if (!Z || !values || !meta || !colsel) return NM_ERR_NULL;
  if (!dtype_ok(dt) || !m_ok(M) || !v_ok(V)) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || R % V != 0 || K % M != 0 || ldz < K || (mask && ldmask < K)) return NM_ERR_SHAPE;
  if (!aligned(Z, esize(dt)) || !aligned(values, esize(dt))) return NM_ERR_ALIGN;
  return hip_status(nms::launch_prune_act_venom(dt, Z, ldz, R, K, V, M, apply_relu != 0, values, meta, colsel,
                                                mask, ldmask, hs(stream)));
}

nm_status spmm_venom(nm_dtype dt, const void* values, const uint8_t* meta, const uint8_t* colsel, int64_t R,
                     int64_t K, int V, int M, const void* B, int64_t ldb, int64_t Nc, float* C, int64_t ldc,
                     nm_stream stream) {
  if (!values || !meta || !colsel || !B || !C) return NM_ERR_NULL;
  if (!dtype_ok(dt) || !m_ok(M) || !v_ok(V)) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || Nc <= 0 || R % V != 0 || K % M != 0 || ldb < Nc || ldc < Nc) return NM_ERR_SHAPE;
  if (!aligned(values, esize(dt)) || !aligned(B, esize(dt)) || !aligned(C, 4)) return NM_ERR_ALIGN;
  return hip_status(
      nms::launch_spmm_venom(dt, values, meta, colsel, R, K, V, M, B, ldb, Nc, C, ldc, hs(stream)));
}

nm_status nm_reprune_t(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R, int64_t K, void* values_t,
                       uint8_t* meta_t, nm_stream stream) {
  if (!values || !meta || !values_t || !meta_t) return NM_ERR_NULL;
  if (!dtype_ok(dt)) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || R % 4 != 0 || K % 4 != 0) return NM_ERR_SHAPE;
  if (!aligned(values, esize(dt)) || !aligned(values_t, esize(dt))) return NM_ERR_ALIGN;
  return hip_status(nms::launch_nm_reprune_t(dt, values, meta, R, K, values_t, meta_t, hs(stream)));
}

nm_status nm_reprune_t_transpose(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R, int64_t K,
                                 void* values_t, uint8_t* meta_t, const void* X, int64_t ldx, int64_t RX, int64_t CX,
                                 void* Xt, int64_t ldxt, nm_stream stream) {
  if (!values || !meta || !values_t || !meta_t || !X || !Xt) return NM_ERR_NULL;
  if (dt != NM_BF16) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || R % 4 != 0 || K % 4 != 0) return NM_ERR_SHAPE;
  if (RX <= 0 || CX <= 0 || ldx < CX || ldxt < RX) return NM_ERR_SHAPE;
  if (!aligned(values, esize(dt)) || !aligned(values_t, esize(dt)) || !aligned(X, esize(dt)) || !aligned(Xt, esize(dt)))
    return NM_ERR_ALIGN;
  return hip_status(nms::launch_nm_reprune_t_transpose(dt, values, meta, R, K, values_t, meta_t, X, ldx, RX, CX, Xt,
                                                       ldxt, hs(stream)));
}

nm_status nm_mfma_rate_probe(int kind, int64_t iters, float* sink, int64_t* flops, nm_stream stream) {
  if (!sink || !flops) return NM_ERR_NULL;
  if (kind != 0 && kind != 1) return NM_ERR_UNSUPPORTED;
  if (iters <= 0 || iters > (int64_t(1) << 24)) return NM_ERR_SHAPE;
  if (!aligned(sink, 4)) return NM_ERR_ALIGN;
  *flops = nms::mfma_probe_flops(kind, iters);
  return hip_status(nms::launch_mfma_rate_probe(kind, iters, sink, hs(stream)));
}

nm_status nm_to_panels(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R, int64_t K, void* values_p,
                       uint8_t* meta_p, nm_stream stream) {
  if (!values || !meta || !values_p || !meta_p) return NM_ERR_NULL;
  if (dt != NM_BF16) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || R % 4 != 0 || K % 256 != 0) return NM_ERR_SHAPE;
  if (!aligned(values, 16) || !aligned(meta, 16) || !aligned(values_p, 16) || !aligned(meta_p, 16)) return NM_ERR_ALIGN;
  return hip_status(nms::launch_nm_to_panels(values, meta, R, K, values_p, meta_p, hs(stream)));
}

nm_status nm_reprune_t_transpose_panels(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R, int64_t K,
                                        void* values_t, uint8_t* meta_t, const void* X, int64_t ldx, int64_t RX,
                                        int64_t CX, void* Xt, int64_t ldxt, nm_stream stream) {
  if (!values || !meta || !values_t || !meta_t || !X || !Xt) return NM_ERR_NULL;
  if (dt != NM_BF16) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || R % 256 != 0 || K % 128 != 0) return NM_ERR_SHAPE;
  if (RX <= 0 || CX <= 0 || ldx < CX || ldxt < RX) return NM_ERR_SHAPE;
  if (!aligned(values, 16) || !aligned(meta, 2) || !aligned(values_t, 16) || !aligned(meta_t, 2) ||
      !aligned(X, esize(dt)) || !aligned(Xt, esize(dt)))
    return NM_ERR_ALIGN;
  return hip_status(nms::launch_nm_reprune_t_transpose_panels(values, meta, R, K, values_t, meta_t, X, ldx, RX, CX, Xt,
                                                              ldxt, hs(stream)));
}

nm_status spmm_nm_t_panels(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R, int64_t K, const void* Bt,
                           int64_t ldbt, int64_t Nc, float* C, int64_t ldc, nm_stream stream) {
  if (!values || !meta || !Bt || !C) return NM_ERR_NULL;
  if (dt != NM_BF16) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || K <= 0 || Nc <= 0 || R % 256 != 0 || K % 256 != 0 || ldbt < K || ldbt % 8 != 0 || ldc < Nc)
    return NM_ERR_SHAPE;
  if (!aligned(values, 16) || !aligned(meta, 16) || !aligned(Bt, 16) || !aligned(C, 4)) return NM_ERR_ALIGN;
  if (R * K >= (int64_t(1) << 32) || Nc * ldbt * 2 >= (int64_t(1) << 32)) return NM_ERR_TOO_LARGE;
  const hipError_t e = nms::launch_spmm_nm_t_panels(values, meta, R, K, Bt, ldbt, Nc, C, ldc, hs(stream));
  if (e == hipErrorNotSupported) return NM_ERR_UNSUPPORTED;
  return hip_status(e);
}

nm_status sddmm_nm(nm_dtype dt, const void* D, int64_t ldd, const void* X, int64_t ldx, int64_t R, int64_t Kc,
                   int64_t T, const uint8_t* meta, float* values_out, nm_stream stream) {
  if (!D || !X || !meta || !values_out) return NM_ERR_NULL;
  if (!dtype_ok(dt)) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || Kc <= 0 || T <= 0 || Kc % 4 != 0 || ldd < T || ldx < T) return NM_ERR_SHAPE;
  if (!aligned(D, esize(dt)) || !aligned(X, esize(dt)) || !aligned(values_out, 4)) return NM_ERR_ALIGN;
  return hip_status(nms::launch_sddmm_nm(dt, D, ldd, X, ldx, R, Kc, T, meta, values_out, hs(stream)));
}

nm_status sddmm_nm_dt(nm_dtype dt, const void* D, int64_t ldd, const void* X, int64_t ldx, int64_t R, int64_t Kc,
                      int64_t T, const uint8_t* meta, float* values_out, void* Dt, int64_t lddt, nm_stream stream) {
  if (!D || !X || !meta || !values_out || !Dt) return NM_ERR_NULL;
  if (dt != NM_BF16) return NM_ERR_UNSUPPORTED;
  if (R <= 0 || Kc <= 0 || T <= 0 || Kc % 4 != 0 || ldd < T || ldx < T || lddt < R) return NM_ERR_SHAPE;
  if (!aligned(D, esize(dt)) || !aligned(X, esize(dt)) || !aligned(values_out, 4) || !aligned(Dt, esize(dt)))
    return NM_ERR_ALIGN;
  return hip_status(nms::launch_sddmm_nm_dt(dt, D, ldd, X, ldx, R, Kc, T, meta, values_out, Dt, lddt, hs(stream)));
}

nm_status moe_route(nm_dtype dt, const void* logits, int64_t ldl, int64_t T, int64_t E, nm_score score,
                    const float* bias, int groups, int topk_groups, int group_top, int k, int renorm, float scale,
                    int32_t* ids, float* weights, nm_stream stream) {
  if (!logits || !ids || !weights) return NM_ERR_NULL;
  if (!dtype_ok(dt) || !score_ok(score) || E > 1024 || k > 64 || groups > 64 || group_top < 1 || group_top > 2 ||
      !scale_ok(scale))
    return NM_ERR_UNSUPPORTED;
  if (T <= 0 || E <= 0 || k <= 0 || groups <= 0 || topk_groups <= 0 || topk_groups > groups || E % groups != 0 ||
      k > E / groups * topk_groups || ldl < E || T > INT32_MAX / k)
    return NM_ERR_SHAPE;
  if (!aligned(logits, esize(dt)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4)) return NM_ERR_ALIGN;
  const nms::RouteArgs a{logits, ldl, T, (int)E, score == NM_SIGMOID, bias, groups, topk_groups, group_top, k,
                         renorm != 0, scale, ids, weights};
  return hip_status(nms::launch_moe_route(dt, a, hs(stream)));
}

nm_status moe_route_bwd(nm_dtype dt, const void* logits, int64_t ldl, int64_t T, int64_t E, nm_score score, int k,
                        int renorm, float scale, const int32_t* ids, const float* weights, const float* dweights,
                        void* dlogits, int64_t lddl, nm_stream stream) {
  if (!logits || !ids || !weights || !dweights || !dlogits) return NM_ERR_NULL;
  if (!dtype_ok(dt) || !score_ok(score) || E > 1024 || k > 64 || !scale_ok(scale)) return NM_ERR_UNSUPPORTED;
  if (T <= 0 || E <= 0 || k <= 0 || k > E || ldl < E || lddl < E || T > INT32_MAX / k) return NM_ERR_SHAPE;
  if (!aligned(logits, esize(dt)) || !aligned(dlogits, esize(dt)) || !aligned(ids, 4) || !aligned(weights, 4) ||
      !aligned(dweights, 4))
    return NM_ERR_ALIGN;
  return hip_status(nms::launch_moe_route_bwd(dt, logits, ldl, T, (int)E, score == NM_SIGMOID, k, renorm != 0, scale,
                                              ids, weights, dweights, dlogits, lddl, hs(stream)));
}

nm_status moe_plan_work_bytes(int64_t T, int k, int64_t E, int64_t* bytes) {
  if (!bytes) return NM_ERR_NULL;
  *bytes = 0;
  if (E > 1024 || k > 64) return NM_ERR_UNSUPPORTED;
  if (T <= 0 || k <= 0 || E <= 0 || T > (int64_t(1) << 30) / k) return NM_ERR_SHAPE;
  *bytes = nms::moe_plan_work_bytes(T * k, E);
  return NM_OK;
}

nm_status moe_plan(const int32_t* ids, int64_t T, int k, int64_t E, int align, int32_t* offsets, int32_t* counts,
                   int32_t* src, int64_t rows, int32_t* pos, void* work, int64_t work_bytes, nm_stream stream) {
  if (!ids || !offsets || !counts || !src || !pos) return NM_ERR_NULL;
  if (E > 1024 || k > 64 || align < 1 || align > 256 || (align & (align - 1)) != 0) return NM_ERR_UNSUPPORTED;
  if (T <= 0 || k <= 0 || E <= 0 || T > (int64_t(1) << 30) / k || rows > INT32_MAX) return NM_ERR_SHAPE;
  const int64_t n = T * k;
  const int64_t need = (n + (n < E ? n : E) * (align - 1) + align - 1) / align * align;
  if (rows < need) return NM_ERR_SHAPE;
  const int64_t wb = nms::moe_plan_work_bytes(n, E);
  if (wb > 0 && !work) return NM_ERR_NULL;
  if (work_bytes < wb) return NM_ERR_SHAPE;
  if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(counts, 4) || !aligned(src, 4) || !aligned(pos, 4) ||
      !aligned(work, 4))
    return NM_ERR_ALIGN;
  return hip_status(nms::launch_moe_plan(ids, n, (int)E, align, offsets, counts, src, rows, pos, (int32_t*)work,
                                         hs(stream)));
}

nm_status fp8_quantize(nm_dtype dt, const void* X, int64_t ldx, int64_t RX, const int32_t* src, int div,
                       const void* gate, int64_t ldg, int64_t R, int64_t K, nm_fp8 fmt, uint8_t* Q, int64_t ldq,
                       float* S, int64_t lds, nm_stream stream) {
  const nm_status st = quantize_check(dt, X, ldx, RX, src, div, gate, ldg, R, K, fmt, Q, S);
  if (st != NM_OK) return st;
  if (ldq < up128(K) || lds < R) return NM_ERR_SHAPE;
  const nms::QuantArgs a{X, ldx, RX, src, nms::fast_div(src ? div : 1), gate, ldg, R, K, fmt == NM_E5M2, Q, ldq, S, lds};
  return hip_status(nms::launch_fp8_quantize(dt, a, hs(stream)));
}

nm_status fp8_quantize_t(nm_dtype dt, const void* X, int64_t ldx, int64_t RX, const int32_t* src, int div,
                         const void* gate, int64_t ldg, int64_t R, int64_t K, nm_fp8 fmt, uint8_t* Qt, int64_t ldqt,
                         float* St, int64_t ldst, nm_stream stream) {
  const nm_status st = quantize_check(dt, X, ldx, RX, src, div, gate, ldg, R, K, fmt, Qt, St);
  if (st != NM_OK) return st;
  if (ldqt < up128(R) || ldst < K) return NM_ERR_SHAPE;
  const nms::QuantArgs a{X, ldx, RX, src, nms::fast_div(src ? div : 1), gate, ldg, R, K, fmt == NM_E5M2, Qt, ldqt, St, ldst};
  return hip_status(nms::launch_fp8_quantize_t(dt, a, hs(stream)));
}

nm_status fp8_quantize_weight(nm_dtype dt, const void* W, int64_t ldw, int64_t E, int64_t N, int64_t K, nm_fp8 fmt,
                              uint8_t* Q, int64_t ldq, float* S, uint8_t* Qt, int64_t ldqt, float* St,
                              nm_stream stream) {
  if (!W || !Q || !S || (!Qt != !St)) return NM_ERR_NULL;
  if (!dtype_ok(dt) || !fp8_ok(fmt)) return NM_ERR_UNSUPPORTED;
  if (E <= 0 || E > 65535 || N <= 0 || K <= 0 || N > INT32_MAX || K > INT32_MAX || ldw < K || ldq < up128(K) ||
      (Qt && ldqt < up128(N)))
    return NM_ERR_SHAPE;
  if (!aligned(W, esize(dt)) || !aligned(S, 4) || !aligned(St, 4)) return NM_ERR_ALIGN;
  return hip_status(nms::launch_fp8_quantize_weight(dt, W, ldw, E, N, K, fmt == NM_E5M2, Q, ldq, S, Qt, ldqt, St,
                                                    hs(stream)));
}

nm_status fp8_gemm_nt(nm_fp8 fa, const uint8_t* A, int64_t lda, const float* sa, int64_t ldsa, nm_fp8 fb,
                      const uint8_t* B, int64_t ldb, const float* sb, int64_t ldsb, int b_block, int64_t M, int64_t N,
                      int64_t K, nm_dtype out, void* C, int64_t ldc, nm_stream stream) {
  const nm_status st = fp8_gemm_check(fa, A, lda, sa, ldsa, fb, B, ldb, sb, M, N, K, out, C, ldc);
  if (st != NM_OK) return st;
  if (b_block != 1 && b_block != 128) return NM_ERR_UNSUPPORTED;
  if (ldsb < (b_block == 1 ? N : up128(K) / 128)) return NM_ERR_SHAPE;
  const nms::Fp8Gemm g{nms::G_DENSE, fa == NM_E5M2, fb == NM_E5M2, b_block, out == NM_BF16, A, lda, sa, ldsa, B, ldb,
                       sb, ldsb, nullptr, 1, M, N, K, C, ldc};
  return hip_status(nms::launch_fp8_gemm(g, hs(stream)));
}

nm_status fp8_gemm_nt_grouped(nm_fp8 fa, const uint8_t* A, int64_t lda, const float* sa, int64_t ldsa, nm_fp8 fb,
                              const uint8_t* B, int64_t ldb, const float* sb, int64_t ldsb, const int32_t* offsets,
                              int64_t E, int64_t rows, int64_t N, int64_t K, nm_dtype out, void* C, int64_t ldc,
                              nm_stream stream) {
  if (!offsets) return NM_ERR_NULL;
  const nm_status st = fp8_gemm_check(fa, A, lda, sa, ldsa, fb, B, ldb, sb, rows, N, K, out, C, ldc);
  if (st != NM_OK) return st;
  if (E > 1024) return NM_ERR_UNSUPPORTED;
  if (E <= 0 || rows > INT32_MAX || ldsb < up128(K) / 128) return NM_ERR_SHAPE;
  if (!aligned(offsets, 4)) return NM_ERR_ALIGN;
  const nms::Fp8Gemm g{nms::G_ROWS, fa == NM_E5M2, fb == NM_E5M2, 128, out == NM_BF16, A, lda, sa, ldsa, B, ldb, sb,
                       ldsb, offsets, (int)E, rows, N, K, C, ldc};
  return hip_status(nms::launch_fp8_gemm(g, hs(stream)));
}

nm_status fp8_gemm_nt_grouped_k(nm_fp8 fa, const uint8_t* A, int64_t lda, const float* sa, int64_t ldsa, nm_fp8 fb,
                                const uint8_t* B, int64_t ldb, const float* sb, int64_t ldsb, const int32_t* offsets,
                                int64_t E, int64_t M, int64_t N, int64_t rows, nm_dtype out, void* C, int64_t ldc,
                                nm_stream stream) {
  if (!offsets) return NM_ERR_NULL;
  const nm_status st = fp8_gemm_check(fa, A, lda, sa, ldsa, fb, B, ldb, sb, M, N, rows, out, C, ldc);
  if (st != NM_OK) return st;
  if (E > 1024) return NM_ERR_UNSUPPORTED;
  if (E <= 0 || rows > INT32_MAX || rows % 128 != 0 || ldsb < N) return NM_ERR_SHAPE;
  if (!aligned(offsets, 4)) return NM_ERR_ALIGN;
  const nms::Fp8Gemm g{nms::G_RED, fa == NM_E5M2, fb == NM_E5M2, 1, out == NM_BF16, A, lda, sa, ldsa, B, ldb, sb, ldsb,
                       offsets, (int)E, M, N, rows, C, ldc};
  return hip_status(nms::launch_fp8_gemm(g, hs(stream)));
}

nm_status moe_combine(nm_dtype dt, const void* O, int64_t ldo, int64_t rows, const int32_t* pos, const float* weights,
                      int64_t T, int k, int64_t D, void* Y, int64_t ldy, nm_stream stream) {
  if (!O || !pos || !Y) return NM_ERR_NULL;
  if (!dtype_ok(dt) || k > 64) return NM_ERR_UNSUPPORTED;
  if (T <= 0 || k <= 0 || D <= 0 || rows <= 0 || rows > INT32_MAX || T > INT32_MAX / k || ldo < D || ldy < D)
    return NM_ERR_SHAPE;
  if (!aligned(O, esize(dt)) || !aligned(Y, esize(dt)) || !aligned(pos, 4) || !aligned(weights, 4)) return NM_ERR_ALIGN;
  return hip_status(nms::launch_moe_combine(dt, O, ldo, rows, pos, weights, T, k, D, Y, ldy, hs(stream)));
}

nm_status moe_combine_bwd(nm_dtype dt, const void* dY, int64_t lddy, const void* O, int64_t ldo, int64_t rows,
                          const int32_t* src, const int32_t* pos, const float* weights, int64_t T, int k, int64_t D,
                          void* dO, int64_t lddo, float* dweights, nm_stream stream) {
  if (!dY || !O || !src || !pos || !weights || !dO || !dweights) return NM_ERR_NULL;
  if (!dtype_ok(dt) || k > 64) return NM_ERR_UNSUPPORTED;
  if (T <= 0 || k <= 0 || D <= 0 || rows <= 0 || rows > INT32_MAX || T > INT32_MAX / k || lddy < D || ldo < D || lddo < D)
    return NM_ERR_SHAPE;
  if (!aligned(dY, esize(dt)) || !aligned(O, esize(dt)) || !aligned(dO, esize(dt)) || !aligned(src, 4) ||
      !aligned(pos, 4) || !aligned(weights, 4) || !aligned(dweights, 4))
    return NM_ERR_ALIGN;
  return hip_status(nms::launch_moe_combine_bwd(dt, dY, lddy, O, ldo, rows, src, pos, weights, T, k, D, dO, lddo,
                                                dweights, hs(stream)));
}

nm_status rms_norm(nm_dtype dt, const void* X, int64_t ldx, const void* residual, int64_t ldr, nm_dtype wdt,
                   const void* w, float eps, int64_t T, int64_t D, void* H, int64_t ldh, void* Y, int64_t ldy,
                   float* rstd, nm_stream stream) {
  if (!Y) return NM_ERR_NULL;
  const nm_status st = norm_check(dt, X, ldx, residual, ldr, wdt, w, eps, T, D, H, ldh, Y, ldy, rstd);
  if (st != NM_OK) return st;
  const nms::NormArgs a{X, ldx, residual, ldr, w, wdt == NM_BF16, eps, T, D, H, ldh, Y, ldy, rstd, nullptr, 0, nullptr, 0, 0};
  return hip_status(nms::launch_rms_norm(dt, a, hs(stream)));
}

nm_status rms_norm_fp8(nm_dtype dt, const void* X, int64_t ldx, const void* residual, int64_t ldr, nm_dtype wdt,
                       const void* w, float eps, int64_t T, int64_t D, nm_fp8 fmt, uint8_t* Q, int64_t ldq, float* S,
                       int64_t lds, void* H, int64_t ldh, void* Y, int64_t ldy, float* rstd, nm_stream stream) {
  if (!Q || !S) return NM_ERR_NULL;
  if (!fp8_ok(fmt)) return NM_ERR_UNSUPPORTED;
  const nm_status st = norm_check(dt, X, ldx, residual, ldr, wdt, w, eps, T, D, H, ldh, Y, ldy, rstd, Q, ldq, S, lds);
  if (st != NM_OK) return st;
  const nms::NormArgs a{X, ldx, residual, ldr, w, wdt == NM_BF16, eps, T, D, H, ldh, Y, ldy, rstd, Q, ldq, S, lds, fmt == NM_E5M2};
  return hip_status(nms::launch_rms_norm(dt, a, hs(stream)));
}

nm_status rms_norm_bwd_work_bytes(int64_t T, int64_t D, int64_t* bytes) {
  if (!bytes) return NM_ERR_NULL;
  if (!rows_ok(T, D)) return NM_ERR_SHAPE;
  if (D > kNormWidth) return NM_ERR_UNSUPPORTED;
  const int64_t g = nms::norm_bwd_groups(T, D);
  *bytes = g > 1 ? g * D * 4 : 0;
  return NM_OK;
}

nm_status rms_norm_bwd(nm_dtype dt, const void* dY, int64_t lddy, const void* H, int64_t ldh, nm_dtype wdt,
                       const void* w, const float* rstd, const void* dH, int64_t lddh, int64_t T, int64_t D, void* dX,
                       int64_t lddx, float* dw, void* work, int64_t work_bytes, nm_stream stream) {
  if (!dY || !H || !w || !rstd || !dX || !dw) return NM_ERR_NULL;
  if (!dtype_ok(dt) || !dtype_ok(wdt)) return NM_ERR_UNSUPPORTED;
  if (!rows_ok(T, D) || lddy < D || ldh < D || (dH && lddh < D) || lddx < D) return NM_ERR_SHAPE;
  int64_t need;
  const nm_status st = rms_norm_bwd_work_bytes(T, D, &need);
  if (st != NM_OK) return st;
  if (need > 0 && !work) return NM_ERR_NULL;
  if (work_bytes < need) return NM_ERR_SHAPE;
  if (!aligned(dY, esize(dt)) || !aligned(H, esize(dt)) || !aligned(w, esize(wdt)) || !aligned(rstd, 4) ||
      !aligned(dH, esize(dt)) || !aligned(dX, esize(dt)) || !aligned(dw, 4) || !aligned(work, 4))
    return NM_ERR_ALIGN;
  const int64_t e = esize(dt);
  const Area out[] = {area(dX, T, D, lddx, e), area(dw, 1, D, D, 4), area(work, 1, need, need, 1)};
  const Area in[] = {area(dY, T, D, lddy, e), area(H, T, D, ldh, e), area(dH, T, D, lddh, e)};
  if (overlap(out, in, {7, 0, 0})) return NM_ERR_SHAPE;
  const nms::NormBwdArgs a{dY, lddy, H, ldh, w, wdt == NM_BF16, rstd, dH, lddh, T, D, dX, lddx, dw, (float*)work};
  return hip_status(nms::launch_rms_norm_bwd(dt, a, hs(stream)));
}

nm_status linear_fwd(nm_dtype dt, const void* X, int64_t ldx, const void* W, int64_t ldw, nm_dtype bdt,
                     const void* bias, nm_act act, const void* residual, int64_t ldr, int64_t M, int64_t N, int64_t K,
                     nm_dtype out, void* Y, int64_t ldy, void* pre, int64_t ldp, void* work, int64_t work_bytes,
                     nm_stream stream) {
  if (!X || !W || !Y) return NM_ERR_NULL;
  if (dt != NM_BF16 || !dtype_ok(out) || (bias && !dtype_ok(bdt)) || !act_ok(act)) return NM_ERR_UNSUPPORTED;
  if (!rows_ok(M, N) || !rows_ok(K, 1) || ldx < K || ldw < K || (residual && ldr < N) || ldy < N || (pre && ldp < N))
    return NM_ERR_SHAPE;
  if (!aligned(X, 2) || !aligned(W, 2) || (bias && !aligned(bias, esize(bdt))) || !aligned(residual, 2) ||
      !aligned(Y, esize(out)) || !aligned(pre, 2) || !aligned(work, 16))
    return NM_ERR_ALIGN;
  const Area written[] = {area(Y, M, N, ldy, esize(out)), area(pre, M, N, ldp, 2), area(work, 1, work_bytes, work_bytes, 1)};
  const Area read[] = {area(X, M, K, ldx, 2), area(W, N, K, ldw, 2), area(residual, M, N, ldr, 2)};
  if (overlap(written, read, {out == NM_BF16 ? 4u : 0u, 0, 0})) return NM_ERR_SHAPE;
  const nms::Linear g{(const uint16_t*)X, ldx, (const uint16_t*)W, ldw, 0, 0, M, N, K, Y, ldy, out == NM_BF16,
                      nms::EPI_FWD, bias, bdt == NM_BF16, act, (const uint16_t*)residual, ldr, (uint16_t*)pre, ldp,
                      nullptr, 0, 0, 0, 0, 0, 0};
  return hip_status(nms::launch_linear(g, work, work ? work_bytes : 0, hs(stream)));
}

nm_status linear_bwd_act_work_bytes(int64_t M, int64_t N, int64_t* bytes) {
  if (!bytes) return NM_ERR_NULL;
  if (!rows_ok(M, N)) return NM_ERR_SHAPE;
  const int64_t g = nms::act_bwd_groups(M, N);
  *bytes = g > 1 ? g * N * 4 : 0;
  return NM_OK;
}

nm_status linear_bwd_act(nm_dtype dt, const void* dY, int64_t lddy, const void* pre, int64_t ldp, nm_act act, int64_t M,
                         int64_t N, void* dZ, int64_t lddz, float* db, void* work, int64_t work_bytes,
                         nm_stream stream) {
  if (!dY || (!pre && act != NM_ACT_NONE) || (!dZ && !db)) return NM_ERR_NULL;
  if (dt != NM_BF16 || !act_ok(act)) return NM_ERR_UNSUPPORTED;
  if (!rows_ok(M, N) || lddy < N || (act != NM_ACT_NONE && ldp < N) || (dZ && lddz < N)) return NM_ERR_SHAPE;
  int64_t need = 0;
  if (db) (void)linear_bwd_act_work_bytes(M, N, &need);
  if (need > 0 && !work) return NM_ERR_NULL;
  if (work_bytes < need) return NM_ERR_SHAPE;
  if (!aligned(dY, 2) || !aligned(pre, 2) || !aligned(dZ, 2) || !aligned(db, 4) || !aligned(work, 4)) return NM_ERR_ALIGN;
  const Area out[] = {area(dZ, M, N, lddz, 2), area(db, 1, N, N, 4), area(work, 1, need, need, 1)};
  const Area in[] = {area(dY, M, N, lddy, 2), area(act == NM_ACT_NONE ? nullptr : pre, M, N, ldp, 2)};
  if (overlap(out, in, {3, 0, 0})) return NM_ERR_SHAPE;
  const nms::ActBwdArgs a{dY, lddy, pre, ldp, act, M, N, dZ, lddz, db, (float*)work};
  return hip_status(nms::launch_linear_bwd_act(a, hs(stream)));
}

nm_status linear_bwd_x(nm_dtype dt, const void* dZ, int64_t lddz, const void* W, int64_t ldw, const void* pre,
                       int64_t ldp, nm_act act, int64_t M, int64_t N, int64_t K, nm_dtype out, void* dX, int64_t lddx,
                       void* work, int64_t work_bytes, nm_stream stream) {
  if (!dZ || !W || !dX || (!pre && act != NM_ACT_NONE)) return NM_ERR_NULL;
  if (dt != NM_BF16 || !dtype_ok(out) || !act_ok(act)) return NM_ERR_UNSUPPORTED;
  if (!rows_ok(M, N) || !rows_ok(K, 1) || lddz < N || ldw < K || (act != NM_ACT_NONE && ldp < K) || lddx < K)
    return NM_ERR_SHAPE;
  if (!aligned(dZ, 2) || !aligned(W, 2) || !aligned(pre, 2) || !aligned(dX, esize(out)) || !aligned(work, 16))
    return NM_ERR_ALIGN;
  const Area written[] = {area(dX, M, K, lddx, esize(out)), area(work, 1, work_bytes, work_bytes, 1)};
  const Area read[] = {area(dZ, M, N, lddz, 2), area(W, N, K, ldw, 2), area(act == NM_ACT_NONE ? nullptr : pre, M, K, ldp, 2)};
  if (overlap(written, read, {out == NM_BF16 ? 4u : 0u, 0})) return NM_ERR_SHAPE;
  // rows of dZ times columns of W: the product's columns are W's, its reduction runs over W's rows
  const nms::Linear g{(const uint16_t*)dZ, lddz, (const uint16_t*)W, ldw, 0, 1, M, K, N, dX, lddx, out == NM_BF16,
                      act == NM_ACT_NONE ? nms::EPI_PLAIN : nms::EPI_GATE, nullptr, 0, act, nullptr, 0, nullptr, 0,
                      (const uint16_t*)pre, ldp, 0, 0, 0, 0, 0};
  return hip_status(nms::launch_linear(g, work, work ? work_bytes : 0, hs(stream)));
}

nm_status linear_bwd_w(nm_dtype dt, const void* dZ, int64_t lddz, const void* X, int64_t ldx, int64_t M, int64_t N,
                       int64_t K, int accumulate, nm_dtype out, void* dW, int64_t lddw, void* work, int64_t work_bytes,
                       nm_stream stream) {
  if (!dZ || !X || !dW) return NM_ERR_NULL;
  if (dt != NM_BF16 || !dtype_ok(out) || (accumulate && out != NM_F32)) return NM_ERR_UNSUPPORTED;
  if (!rows_ok(M, N) || !rows_ok(K, 1) || lddz < N || ldx < K || lddw < K) return NM_ERR_SHAPE;
  if (!aligned(dZ, 2) || !aligned(X, 2) || !aligned(dW, esize(out)) || !aligned(work, 16)) return NM_ERR_ALIGN;
  const Area written[] = {area(dW, N, K, lddw, esize(out)), area(work, 1, work_bytes, work_bytes, 1)};
  const Area read[] = {area(dZ, M, N, lddz, 2), area(X, M, K, ldx, 2)};
  if (overlap(written, read, {0, 0})) return NM_ERR_SHAPE;
  const nms::Linear g{(const uint16_t*)dZ, lddz, (const uint16_t*)X, ldx, 1, 1, N, K, M, dW, lddw, out == NM_BF16,
                      accumulate ? nms::EPI_ADD : nms::EPI_PLAIN, nullptr, 0, NM_ACT_NONE, nullptr, 0, nullptr, 0, nullptr, 0, 0, 0, 0, 0, 0};
  return hip_status(nms::launch_linear(g, work, work ? work_bytes : 0, hs(stream)));
}

nm_status linear_work_bytes(nm_linear call, int64_t M, int64_t N, int64_t K, int aligned, int64_t* bytes) {
  if (!bytes) return NM_ERR_NULL;
  if (!rows_ok(M, N) || !rows_ok(K, 1)) return NM_ERR_SHAPE;
  switch (call) {
    case NM_LINEAR_FWD: *bytes = nms::linear_work_bytes(0, 0, M, N, K, aligned != 0); return NM_OK;
    case NM_LINEAR_BWD_X: *bytes = nms::linear_work_bytes(0, 1, M, K, N, aligned != 0); return NM_OK;
    case NM_LINEAR_BWD_W: *bytes = nms::linear_work_bytes(1, 1, N, K, M, aligned != 0); return NM_OK;
  }
  return NM_ERR_UNSUPPORTED;
}

nm_status grad_work_bytes(int64_t n, const int64_t* counts, int64_t* bytes) {
  if (!bytes || !counts) return NM_ERR_NULL;
  if (n <= 0 || n > 65536) return NM_ERR_SHAPE;
  for (int64_t i = 0; i < n; ++i)
    if (counts[i] < 0 || counts[i] > INT64_MAX / 8 / n) return NM_ERR_SHAPE;
  *bytes = nms::grad_partials(counts, n) * 8;
  return NM_OK;
}

nm_status grad_norm(int64_t n, const nm_dtype* dt, const void* const* grads, const int64_t* counts, float* norm,
                    void* work, int64_t work_bytes, nm_stream stream) {
  const nm_status st = grads_check(n, dt, grads, counts, norm, work, work_bytes, true);
  if (st != NM_OK) return st;
  const int64_t need = nms::grad_partials(counts, n) * 8;
  const Area out[] = {area(norm, 1, 1, 1, 4), area(work, 1, need, need, 1)};
  if (meet(out[0], out[1])) return NM_ERR_SHAPE;
  for (int64_t i = 0; i < n; ++i) {
    const Area g = area(grads[i], 1, counts[i], counts[i], esize(dt[i]));
    if (meet(out[0], g) || meet(out[1], g)) return NM_ERR_SHAPE;
  }
  const nms::Grads g{n, (const int*)dt, grads, counts, nullptr, nullptr};
  return hip_status(nms::launch_grads(g, false, norm, 0.f, (double*)work, hs(stream)));
}

nm_status grad_clip(int64_t n, const nm_dtype* dt, const void* const* grads, const int64_t* counts, float max_norm,
                    int have_norm, float* norm, const nm_dtype* odt, void* const* out, void* work, int64_t work_bytes,
                    nm_stream stream) {
  if (!odt || !out) return NM_ERR_NULL;
  const nm_status st = grads_check(n, dt, grads, counts, norm, work, work_bytes, !have_norm);
  if (st != NM_OK) return st;
  if (!(max_norm >= 0.f)) return NM_ERR_UNSUPPORTED;
  for (int64_t i = 0; i < n; ++i) {
    if (!dtype_ok(odt[i])) return NM_ERR_UNSUPPORTED;
    if (counts[i] == 0) continue;
    if (!out[i]) return NM_ERR_NULL;
    if (!aligned(out[i], esize(odt[i]))) return NM_ERR_ALIGN;
  }
  Range* r = new (std::nothrow) Range[2 * n + 2];
  if (!r) return hip_status(hipErrorOutOfMemory);
  int64_t k = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (counts[i] == 0) continue;
    const uintptr_t o = (uintptr_t)out[i], p = (uintptr_t)grads[i];
    r[k++] = Range{o, o + (uintptr_t)(counts[i] * esize(odt[i])), true};
    if (o != p || odt[i] != dt[i]) r[k++] = Range{p, p + (uintptr_t)(counts[i] * esize(dt[i])), false};
  }
  // the norm and the work memory are written too
  r[k++] = Range{(uintptr_t)norm, (uintptr_t)norm + 4, true};
  if (!have_norm && work)
    r[k++] = Range{(uintptr_t)work, (uintptr_t)work + (uintptr_t)(nms::grad_partials(counts, n) * 8), true};
  std::sort(r, r + k, [](const Range& a, const Range& b) { return a.lo < b.lo; });
  const bool bad = outputs_overlap(r, k);
  delete[] r;
  if (bad) return NM_ERR_SHAPE;
  const nms::Grads g{n, (const int*)dt, grads, counts, (const int*)odt, out};
  return hip_status(nms::launch_grads(g, have_norm != 0, norm, max_norm, (double*)work, hs(stream)));
}

void nm_sizes(int64_t R, int64_t K, int N, int M, int V, int64_t* n_values, int64_t* meta_bytes,
              int64_t* colsel_bytes) {
  if (M <= 0) M = 4;
  const int64_t G = K / M;
  if (V > 0) {
    if (n_values) *n_values = R * G * 2;
    if (meta_bytes) *meta_bytes = R * ((G + 1) / 2);
    if (colsel_bytes) *colsel_bytes = (R / V) * G * 4;
  } else {
    if (n_values) *n_values = R * G * N;
    if (meta_bytes) *meta_bytes = R * nms::meta_row_bytes(K, N, M);
    if (colsel_bytes) *colsel_bytes = 0;
  }
}

const char* nm_status_str(nm_status status) {
  switch (status) {
    case NM_OK: return "ok";
    case NM_ERR_NULL: return "a required pointer is NULL";
    case NM_ERR_SHAPE: return "invalid shape or leading dimension";
    case NM_ERR_UNSUPPORTED: return "unsupported dtype, N:M pattern, block size or option";
    case NM_ERR_ALIGN: return "pointer not aligned to its element size";
    case NM_ERR_HIP: return "HIP launch failed";
    case NM_ERR_TOO_LARGE: return "the operand needs more scratch memory than the library's fixed buffer holds";
  }
  return "unknown status";
}

const char* nm_last_hip_error(void) { return g_last_hip_error; }

int nm_version(void) { return 100; }

}  // extern "C"
