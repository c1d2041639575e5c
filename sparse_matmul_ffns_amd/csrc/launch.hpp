// Host-side launchers of the gfx950 kernels (internal to libnmsparse).
// Arguments are validated by api.cpp before any of these is called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nms {

enum { DT_F32 = 0, DT_BF16 = 1 };

inline int64_t meta_row_bytes(int64_t K, int N, int M) {
  int b = 1;
  while ((1 << b) < M) ++b;
  return ((K / M) * N * b + 7) / 8;
}

hipError_t launch_nm_prune(int dt, const void* A, int64_t lda, int64_t R, int64_t K, int N, int M,
                           uint8_t* mask, int64_t ldmask, hipStream_t s);
hipError_t launch_nm_compress(int dt, const void* A, int64_t lda, const uint8_t* mask, int64_t ldmask,
                              int64_t R, int64_t K, int N, int M, void* values, uint8_t* meta, int32_t* bad,
                              hipStream_t s);
hipError_t launch_nm_prune_compress(int dt, const void* A, int64_t lda, int64_t R, int64_t K, int N, int M,
                                    uint8_t* mask, int64_t ldmask, void* values, uint8_t* meta, hipStream_t s);
hipError_t launch_nm_prune_compress_transpose(int dt, const void* A, int64_t lda, int64_t R, int64_t K, int N, int M,
                                              uint8_t* mask, int64_t ldmask, void* values, uint8_t* meta,
                                              const void* B, int64_t ldb, int64_t KB, int64_t Nc, void* Bt,
                                              int64_t ldbt, hipStream_t s);
hipError_t launch_nm_decompress(int dt, const void* values, const uint8_t* meta, int64_t R, int64_t K, int N,
                                int M, void* out, int64_t lda, hipStream_t s);
hipError_t launch_prune_act_venom(int dt, const void* Z, int64_t ldz, int64_t R, int64_t K, int V, int M,
                                  int relu, void* values, uint8_t* meta, uint8_t* colsel, uint8_t* mask,
                                  int64_t ldmask, hipStream_t s);
hipError_t launch_nm_reprune_t(int dt, const void* values, const uint8_t* meta, int64_t R, int64_t K,
                               void* values_t, uint8_t* meta_t, hipStream_t s);
hipError_t launch_nm_reprune_t_transpose(int dt, const void* values, const uint8_t* meta, int64_t R, int64_t K,
                                         void* values_t, uint8_t* meta_t, const void* X, int64_t ldx, int64_t RX,
                                         int64_t CX, void* Xt, int64_t ldxt, hipStream_t s);
hipError_t launch_spmm_nm(int dt, const void* values, const uint8_t* meta, int64_t R, int64_t K, const void* B,
                          int64_t ldb, int64_t Nc, float* C, int64_t ldc, hipStream_t s);
hipError_t launch_spmm_venom(int dt, const void* values, const uint8_t* meta, const uint8_t* colsel, int64_t R,
                             int64_t K, int V, int M, const void* B, int64_t ldb, int64_t Nc, float* C,
                             int64_t ldc, hipStream_t s);
bool spmm_dma_ok(const void* values, const uint8_t* meta, const void* B, int64_t ldb, int64_t Nc, int64_t Kd);
hipError_t launch_spmm_nm_dma(const void* values, const uint8_t* meta, int64_t R, int64_t K, const void* B,
                              int64_t ldb, int64_t Nc, float* C, int64_t ldc, hipStream_t s);
hipError_t launch_spmm_venom_dma(const void* values, const uint8_t* meta, const uint8_t* colsel, int64_t R,
                                 int64_t Kd, int V, int M, int64_t G, const void* B, int64_t ldb, int64_t Nc,
                                 float* C, int64_t ldc, hipStream_t s);
bool spmm_vnm_reg_ok(const uint8_t* colsel, int V, int M, int64_t G, int64_t Kd, int64_t ldb, int64_t Nc, const float* C,
                     int64_t ldc);
hipError_t launch_spmm_vnm_reg(const void* values, const uint8_t* meta, const uint8_t* colsel, int64_t R, int64_t Kd,
                               int V, int M, int64_t G, const void* B, int64_t ldb, int64_t Nc, float* C, int64_t ldc,
                               hipStream_t s);
bool spmm_nt_ok(const void* values, const uint8_t* meta, const void* Bt, int64_t ldbt, int64_t R, int64_t Nc,
                int64_t Kd);
hipError_t launch_spmm_nm_t(int dt, const void* values, const uint8_t* meta, int64_t R, int64_t K, const void* Bt,
                            int64_t ldbt, int64_t Nc, float* C, int64_t ldc, hipStream_t s);
hipError_t launch_spmm_nm_nt_dma(const void* values, const uint8_t* meta, int64_t R, int64_t K, const void* Bt,
                                 int64_t ldbt, int64_t Nc, float* C, int64_t ldc, hipStream_t s);
hipError_t launch_spmm_nm_nt_dma_bf16out(const void* values, const uint8_t* meta, int64_t R, int64_t K, const void* Bt,
                                         int64_t ldbt, int64_t Nc, uint16_t* C, int64_t ldc, hipStream_t s);
hipError_t launch_spmm_nm_t_bf16out(int dt, const void* values, const uint8_t* meta, int64_t R, int64_t K,
                                   const void* Bt, int64_t ldbt, int64_t Nc, uint16_t* C, int64_t ldc, hipStream_t s);
hipError_t launch_spmm_nm_nt_dma_lowrank(const void* values, const uint8_t* meta, int64_t R, int64_t K, const void* Bt,
                                         int64_t ldbt, int64_t Nc, const void* U, int64_t ldu, const float* Tt,
                                         int rank, float* C, int64_t ldc, hipStream_t s);
hipError_t launch_spmm_nm_t_lowrank(int dt, const void* values, const uint8_t* meta, int64_t R, int64_t K,
                                    const void* Bt, int64_t ldbt, int64_t Nc, const void* U, int64_t ldu,
                                    const void* Vt, int64_t ldvt, int64_t rank, float* Tt, float* C, int64_t ldc,
                                    hipStream_t s);
hipError_t launch_spmm_nm_t_relu_venom(const void* values, const uint8_t* meta, int64_t R, int64_t K, const void* Bt,
                                      int64_t ldbt, int64_t Nc, int V, int M, void* hv, uint8_t* hm, uint8_t* hc,
                                      hipStream_t s);
int64_t general_work_bytes(int esz, int64_t R, int64_t K, int N, int M);
// Size of the fixed scratch memory of spmm_nm_general_noalloc (64 MiB per GPU).
constexpr int64_t GENERAL_SCRATCH_BYTES = int64_t(64) << 20;
hipError_t launch_spmm_nm_general_noalloc(int dt, const void* values, const uint8_t* meta, int64_t R, int64_t K,
                                          int N, int M, const void* Bt, int64_t ldbt, int64_t Nc, float* C,
                                          int64_t ldc, hipStream_t s);
hipError_t launch_spmm_nm_general(int dt, const void* values, const uint8_t* meta, int64_t R, int64_t K, int N, int M,
                                  const void* Bt, int64_t ldbt, int64_t Nc, float* C, int64_t ldc, void* work,
                                  int64_t work_bytes, hipStream_t s);
hipError_t launch_nm_transpose(int dt, const void* src, int64_t lds, int64_t R, int64_t Cn, void* dst, int64_t ldd,
                               hipStream_t s);
bool spmm_panels_ok(const void* values, const uint8_t* meta, const void* Bt, int64_t ldbt, int64_t R, int64_t K,
                    int64_t Nc);
hipError_t launch_spmm_nm_t_panels(const void* values, const uint8_t* meta, int64_t R, int64_t K, const void* Bt,
                                   int64_t ldbt, int64_t Nc, float* C, int64_t ldc, hipStream_t s);
hipError_t launch_nm_reprune_t_transpose_panels(const void* values, const uint8_t* meta, int64_t R, int64_t K,
                                                void* values_t, uint8_t* meta_t, const void* X, int64_t ldx,
                                                int64_t RX, int64_t CX, void* Xt, int64_t ldxt, hipStream_t s);
hipError_t launch_nm_to_panels(const void* values, const uint8_t* meta, int64_t R, int64_t K, void* values_p,
                               uint8_t* meta_p, hipStream_t s);
int64_t mfma_probe_flops(int kind, int64_t iters);
hipError_t launch_mfma_rate_probe(int kind, int64_t iters, float* sink, hipStream_t s);
hipError_t launch_sddmm_nm_dt(int dt, const void* D, int64_t ldd, const void* X, int64_t ldx, int64_t R, int64_t Kc,
                              int64_t Tn, const uint8_t* meta, float* out, void* Dt, int64_t lddt, hipStream_t s);
bool sddmm_venom_fast_ok(const void* dY, int64_t lddy, const void* Wd, int64_t ldw, int64_t Tn, int64_t F, int64_t Nc,
                         int V, int M, const void* hv, const float* dz, const void* dYt, int64_t lddyt);
hipError_t launch_sddmm_venom_dma(const void* dY, int64_t lddy, const void* Wd, int64_t ldw, int64_t Tn, int64_t F,
                                  int64_t Nc, int V, int M, const void* hv, const uint8_t* hm, const uint8_t* hc,
                                  int relu, float* dz, void* dYt, int64_t lddyt, hipStream_t s);
bool dense_nt_fast_ok(const void* A, int64_t lda, const void* B, int64_t ldb, const float* out, int64_t ldo,
                      int64_t Tn);
hipError_t launch_dense_nt(const void* A, int64_t lda, const void* B, int64_t ldb, int64_t R, int64_t Kc, int64_t Tn,
                           float* out, int64_t ldo, hipStream_t s);
int64_t venom_tn_work_bytes(int esz, int64_t Tn, int64_t F);
hipError_t launch_sddmm_venom(int dt, const void* dY, int64_t lddy, const void* Wd, int64_t ldw, int64_t Tn,
                              int64_t F, int64_t Nc, int V, int M, const void* hv, const uint8_t* hm,
                              const uint8_t* hc, int relu, float* dz, void* dYt, int64_t lddyt, hipStream_t s);
hipError_t launch_spmm_venom_tn(int dt, const void* hv, const uint8_t* hm, const uint8_t* hc, int64_t Tn, int64_t F,
                                int V, int M, const void* dYt, int64_t lddyt, int64_t Nc, float* dW, int64_t lddw,
                                void* work, int64_t work_bytes, hipStream_t s);
hipError_t launch_sddmm_nm(int dt, const void* D, int64_t ldd, const void* X, int64_t ldx, int64_t R,
                           int64_t Kc, int64_t T, const uint8_t* meta, float* out, hipStream_t s);

// The mixture-of-experts FFN in 8 bits.
struct RouteArgs {
  const void* logits;
  int64_t ldl, T;
  int E, sigmoid;
  const float* bias;
  int groups, topk_groups, group_top, k, renorm;
  float scale;
  int32_t* ids;
  float* weights;
};
hipError_t launch_moe_route(int dt, const RouteArgs& a, hipStream_t s);
hipError_t launch_moe_route_bwd(int dt, const void* logits, int64_t ldl, int64_t T, int E, int sigmoid, int k, int renorm,
                                float scale, const int32_t* ids, const float* weights, const float* dweights,
                                void* dlogits, int64_t lddl, hipStream_t s);
int64_t moe_plan_work_bytes(int64_t n, int64_t E);
hipError_t launch_moe_plan(const int32_t* ids, int64_t n, int E, int align, int32_t* offsets, int32_t* counts,
                           int32_t* src, int64_t rows, int32_t* pos, int32_t* work, hipStream_t s);
hipError_t launch_moe_combine(int dt, const void* O, int64_t ldo, int64_t rows, const int32_t* pos, const float* w,
                              int64_t T, int k, int64_t D, void* Y, int64_t ldy, hipStream_t s);
hipError_t launch_moe_combine_bwd(int dt, const void* dY, int64_t lddy, const void* O, int64_t ldo, int64_t rows,
                                  const int32_t* src, const int32_t* pos, const float* w, int64_t T, int k, int64_t D,
                                  void* dO, int64_t lddo, float* dw, hipStream_t s);
// n / d for 0 <= n < 2^31 as a product and shifts (d fixed by the host): q = (t + ((n - t) >> s1)) >> s2
// with t the high half of mul * n, mul = floor(2^32 (2^l - d) / d) + 1, l = ceil(log2 d).
struct FastDiv {
  uint32_t mul;
  int s1, s2;
};
inline FastDiv fast_div(int d) {
  int l = 0;
  while ((int64_t(1) << l) < d) ++l;
  const uint64_t mul = ((uint64_t)((int64_t(1) << l) - d) << 32) / (uint64_t)d + 1;
  return FastDiv{(uint32_t)mul, l < 1 ? l : 1, l < 1 ? 0 : l - 1};
}
struct QuantArgs {
  const void* X;
  int64_t ldx, RX;
  const int32_t* src;
  FastDiv div;
  const void* gate;
  int64_t ldg, R, K;
  int e5m2;
  uint8_t* Q;
  int64_t ldq;
  float* S;
  int64_t lds;
};
hipError_t launch_fp8_quantize(int dt, const QuantArgs& a, hipStream_t s);
hipError_t launch_fp8_quantize_t(int dt, const QuantArgs& a, hipStream_t s);
hipError_t launch_fp8_quantize_weight(int dt, const void* W, int64_t ldw, int64_t E, int64_t N, int64_t K, int e5m2,
                                      uint8_t* Q, int64_t ldq, float* S, uint8_t* Qt, int64_t ldqt, float* St,
                                      hipStream_t s);
// One product (mode 0), or one for every group of A's rows (1) or of the reduction (2).
enum { G_DENSE = 0, G_ROWS = 1, G_RED = 2 };
struct Fp8Gemm {
  int mode, a_e5m2, b_e5m2, b_block, bf16_out;
  const uint8_t* A;
  int64_t lda;
  const float* sa;
  int64_t ldsa;
  const uint8_t* B;
  int64_t ldb;
  const float* sb;
  int64_t ldsb;
  const int32_t* offsets;   // G_ROWS, G_RED
  int E;
  int64_t M, N, K;          // G_ROWS: M = rows; G_RED: K = rows
  void* C;
  int64_t ldc;
};
hipError_t launch_fp8_gemm(const Fp8Gemm& g, hipStream_t s);

// The dense FFN block: norms, products with their epilogue and gradients, the gradients' norm.
struct NormArgs {
  const void* X;
  int64_t ldx;
  const void* R;            // null: nothing is added
  int64_t ldr;
  const void* w;
  int w_bf16;
  float eps;
  int64_t T, D;
  void* H;                  // null: the sum is not stored
  int64_t ldh;
  void* Y;                  // null with Q only
  int64_t ldy;
  float* rstd;              // null: not stored
  uint8_t* Q;               // null: no 8-bit result
  int64_t ldq;
  float* S;
  int64_t lds;
  int e5m2;
};
hipError_t launch_rms_norm(int dt, const NormArgs& a, hipStream_t s);
struct NormBwdArgs {
  const void* dY;
  int64_t lddy;
  const void* H;
  int64_t ldh;
  const void* w;
  int w_bf16;
  const float* rstd;
  const void* dH;           // null: nothing comes through the residual
  int64_t lddh, T, D;
  void* dX;
  int64_t lddx;
  float* dw;
  float* work;
};
int64_t norm_bwd_groups(int64_t T, int64_t D);
hipError_t launch_rms_norm_bwd(int dt, const NormBwdArgs& a, hipStream_t s);
// out[c] = sum of part[0 .. G - 1][c], in fp32 in a fixed order.
hipError_t launch_sum_partials(const float* part, int64_t G, int64_t N, float* out, hipStream_t s);
struct ActBwdArgs {
  const void* dY;
  int64_t lddy;
  const void* pre;
  int64_t ldp;
  int act;
  int64_t M, N;
  void* dZ;                 // null: only the sums
  int64_t lddz;
  float* db;                // null: no sums
  float* work;
};
int64_t act_bwd_groups(int64_t M, int64_t N);
hipError_t launch_linear_bwd_act(const ActBwdArgs& a, hipStream_t s);
// C[m][n] = sum over k of A(m, k) B(n, k), bf16 operands: A(m, k) at A[m * lda + k], or with a_t at
// A[k * lda + m]; B alike.
// EPI_ADD: added to C, which is fp32 then.
enum { EPI_FWD = 0, EPI_GATE = 1, EPI_PLAIN = 2, EPI_ADD = 3 };
struct Linear {
  const uint16_t* A;
  int64_t lda;
  const uint16_t* B;
  int64_t ldb;
  int a_t, b_t;
  int64_t M, N, K;
  void* C;
  int64_t ldc;
  int bf16_out, epi;
  const void* bias;         // EPI_FWD; null: none
  int bias_bf16, act;
  const uint16_t* R;        // EPI_FWD: added behind the activation; null: none
  int64_t ldr;
  uint16_t* Z;              // EPI_FWD: the sum before the activation; null: not stored
  int64_t ldz;
  const uint16_t* P;        // EPI_GATE: the activation's derivative at P
  int64_t ldp;
  int64_t part_k;           // the reduction's length of a part, where it is cut
  // what may be read of the operands: A's rows (or columns) and k, and B's; more than M, N and K where a copy is padded
  int64_t ra, ka, rb, kb;
};
// How a product is computed: its kernel and tile, and in how many parts of part_k the reduction is cut.
struct LinearPlan {
  enum { ROWS = 0, T128 = 1, T256x128 = 2, T256 = 3 };
  int tile, parts;
  int64_t part_k;
  bool pack;        // copy operands whose rows are not aligned
};
// aligned: both operands have 16-byte aligned rows.
int64_t linear_work_bytes(int a_t, int b_t, int64_t M, int64_t N, int64_t K, bool aligned);
// work: 16-byte aligned; with fewer than linear_work_bytes the general kernel, or an uncut reduction, does without
hipError_t launch_linear(const Linear& g, void* work, int64_t work_bytes, hipStream_t s);
struct Grads {
  int64_t n;
  const int* dt;
  const void* const* in;
  const int64_t* count;
  const int* odt;           // with out
  void* const* out;         // null for the norm alone
};
int64_t grad_partials(const int64_t* count, int64_t n);
// The norm, and with g.out the scaling (have_norm: *norm is given, and work is not used).
hipError_t launch_grads(const Grads& g, bool have_norm, float* norm, float max_norm, double* work, hipStream_t s);

}  // namespace nms
