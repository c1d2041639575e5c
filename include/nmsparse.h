/*
 * nmsparse.h -- C ABI of the MI355X (gfx950) library for semi-structured
 * sparse feed-forward matmuls: magnitude N:M and V:N:M pruning, compression
 * to values plus packed position metadata, and the sparse x dense products of
 * the FFN forward pass and of the double-pruned backward pass.  The last part
 * is the mixture-of-experts FFN in 8-bit floating point: routing, the rows'
 * order by expert, quantisation to blocks of 128, products with a scale per
 * block, and the weighted combine.
 *
 * Sources (page title, section):
 *   "Success story: ESPLAG" (inno4scale) -- Highlights, Research Topic,
 *       Solution: semi-structured N:M magnitude pruning, a compressed storage
 *       format (VENOM) and an SpMM kernel library; figures 1-3 (the formats)
 *       are missing from the page.
 *   "To 2:4 Sparsity and Beyond: Neuron-level Activation Function to
 *       Accelerate LLM Pre-Training" -- abstract: 2:4 weights and v:n:m
 *       (Venom) activations in every FFN matmul.
 *   NSF PAR award 2340011 listing -- SLOPE abstract: the backward pass uses
 *       the transposed weight re-pruned with N:M ("double pruned"); lazy
 *       low-rank adapters join the sparse weight late in pre-training.
 *   "Sparser, Faster, Lighter Transformer Language Models" -- Methodologie:
 *       ReLU activations, the FFN as the dominant cost.
 *
 * Conventions shared by every call
 *   - Matrices are row-major.  Leading dimensions (lda, ldb, ...) count
 *     elements, not bytes, and must be >= the row width.
 *   - Groups are M consecutive elements along the reduction dimension K of the
 *     left (sparse) operand, starting at column 0.  K must be a multiple of M.
 *   - Selection keeps the N largest magnitudes of a group; on equal magnitude
 *     the lower position wins.  A group always keeps exactly N elements, zeros
 *     included.  +0.0 and -0.0 have equal magnitude.
 *   - Compressed form of an R x K matrix, N:M:
 *       values [R][(K/M)*N]  kept elements in ascending position, raw bits of
 *                            the input dtype (signed zeros preserved);
 *       meta   [R][ceil((K/M)*N*b/8)] bytes, b = ceil(log2 M): per row one
 *                            LSB-first bit stream of b-bit positions, survivor
 *                            s of group g at bit (g*N + s)*b.  For 2:4 this is
 *                            one nibble p0 | p1 << 2 per group, even groups in
 *                            the low nibble (ceil(K/8) bytes per row).
 *   - V:N:M form (N = 2): per V-row block and M-column group the 4 columns with
 *     the largest block L1 norm (fp64, rows summed top to bottom) are kept,
 *     then 2 of those 4 per row by magnitude:
 *       colsel [R/V][K/M][4] u8  the 4 kept columns of each group, ascending;
 *       values [R][(K/M)*2]       kept elements;
 *       meta   [R][ceil(K/M/2)]   2:4 nibbles j0 | j1 << 2 over j = 0..3,
 *                                 j indexing the group's colsel entries.
 *   - Device pointers: every array argument is device memory owned by the
 *     caller, naturally aligned for its element type.  Outputs are fully
 *     overwritten and must not overlap inputs.  The library allocates nothing
 *     and keeps no state: calls are reentrant and thread-safe -- except
 *     spmm_nm_general_noalloc, whose calls share a fixed scratch buffer per
 *     GPU (see there).
 *   - Streams: `stream` is a hipStream_t (NULL = the null stream).  Every call
 *     is asynchronous on that stream; argument errors are returned before
 *     anything is launched.  No call allocates, clears memory with a memset or
 *     synchronises, so a sequence of calls on one stream can be captured into a
 *     HIP graph and replayed.
 *   - Floating point: products accumulate in fp32 and are written as fp32,
 *     except where a call states a bf16 result (rounded to nearest even).
 *   - Errors: NM_ERR_NULL for a NULL required pointer, NM_ERR_SHAPE for
 *     non-positive sizes, sizes that are not multiples of the group/block, or
 *     a leading dimension below the row width, NM_ERR_UNSUPPORTED for a dtype
 *     or (N, M, V) the call does not implement, NM_ERR_ALIGN for a pointer
 *     that is not aligned to its element size, NM_ERR_HIP when the launch
 *     fails (nm_last_hip_error() names the HIP error), NM_ERR_TOO_LARGE when
 *     an operand does not fit a fixed scratch buffer (spmm_nm_general_noalloc).
 */
#ifndef NMSPARSE_H
#define NMSPARSE_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  NM_OK = 0,
  NM_ERR_NULL = 1,
  NM_ERR_SHAPE = 2,
  NM_ERR_UNSUPPORTED = 3,
  NM_ERR_ALIGN = 4,
  NM_ERR_HIP = 5,
  NM_ERR_TOO_LARGE = 6
} nm_status;

typedef enum { NM_F32 = 0, NM_BF16 = 1 } nm_dtype;

/* A hipStream_t, passed as an opaque pointer (NULL = the null stream). */
typedef void* nm_stream;

/*
 * nm_prune -- magnitude N:M pruning along K ("Success story: ESPLAG",
 * Highlights and Solution; "To 2:4 Sparsity and Beyond", abstract).
 *   A     [R][lda]    fp32 or bf16 input (dt)
 *   mask  [R][ldmask] u8 output: 1 where kept, 0 elsewhere (columns 0..K-1)
 * N:M: M in {4, 8, 16}, 1 <= N < M.
 */
nm_status nm_prune(nm_dtype dt, const void* A, int64_t lda, int64_t R, int64_t K, int N, int M,
                   uint8_t* mask, int64_t ldmask, nm_stream stream);

/*
 * nm_compress -- gather the kept elements of each group in ascending position
 * and pack their positions ("Success story: ESPLAG", Solution: compressed
 * storage format).
 *   A          [R][lda] input; mask [R][ldmask] u8 (nonzero = kept)
 *   values     [R][(K/M)*N] output, dtype dt
 *   meta       [R][ceil((K/M)*N*b/8)] u8 output
 *   bad_groups nullable device int32: incremented (never reset) by the number
 *              of groups whose mask keeps a count other than N.  Such a group
 *              is stored as +0.0 values at positions 0..N-1.
 */
nm_status nm_compress(nm_dtype dt, const void* A, int64_t lda, const uint8_t* mask, int64_t ldmask,
                      int64_t R, int64_t K, int N, int M, void* values, uint8_t* meta,
                      int32_t* bad_groups, nm_stream stream);

/*
 * nm_prune_compress -- nm_prune and nm_compress in one call: the N:M magnitude
 * selection of A ("Success story: ESPLAG", Highlights and Solution: pruning to
 * N:M and its compressed storage) written both as the mask and as values +
 * metadata.  Outputs are byte-identical to nm_prune followed by nm_compress.
 *   A [R][lda], mask [R][ldmask] u8 output, values [R][(K/M)*N] and
 *   meta [R][ceil((K/M)*N*ceil(log2 M)/8)] outputs, dtype dt.
 * 2:4 with 16-byte aligned rows (A, mask, values) and K % 16 == 0 runs as one
 * pass over A; other calls run the two passes.  Errors as for nm_compress.
 */
nm_status nm_prune_compress(nm_dtype dt, const void* A, int64_t lda, int64_t R, int64_t K, int N,
                            int M, uint8_t* mask, int64_t ldmask, void* values, uint8_t* meta,
                            nm_stream stream);

/*
 * nm_prune_compress_transpose -- nm_prune_compress of A and nm_transpose of B
 * in one launch: the two passes that prepare the 2:4 product of an FFN layer
 * ("Success story: ESPLAG", Solution: the weight pruned to 2:4 and stored
 * compressed; the activations then feed spmm_nm_t K-contiguous).
 *   A, mask, values, meta as for nm_prune_compress;
 *   B [KB][ldb] dense input, Bt [Nc][ldbt] output (ldbt >= KB): Bt[c][k] = B[k][c].
 * Outputs are byte-identical to nm_prune_compress followed by nm_transpose.
 * bf16 only (NM_ERR_UNSUPPORTED otherwise).  2:4 with the single-pass layout of
 * nm_prune_compress runs as one kernel; other calls run the two kernels.
 * Bt must not overlap B; no output may overlap an input.  Errors as for the
 * two calls.
 */
nm_status nm_prune_compress_transpose(nm_dtype dt, const void* A, int64_t lda, int64_t R,
                                      int64_t K, int N, int M, uint8_t* mask, int64_t ldmask,
                                      void* values, uint8_t* meta, const void* B, int64_t ldb,
                                      int64_t KB, int64_t Nc, void* Bt, int64_t ldbt,
                                      nm_stream stream);

/*
 * nm_decompress -- inverse of nm_compress: dense A_out [R][lda] with +0.0 at
 * every position that is not kept.
 */
nm_status nm_decompress(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R, int64_t K,
                        int N, int M, void* A_out, int64_t lda, nm_stream stream);

/*
 * spmm_nm -- C = decompress(values, meta) * B for a 2:4 left operand
 * ("Success story: ESPLAG", Research Topic: the SpMM; "To 2:4 Sparsity and
 * Beyond", abstract: 2:4 weights in every FFN matmul).
 *   values [R][K/2], meta [R][ceil(K/8)] (2:4 form of an R x K matrix), dtype dt
 *   B      [K][ldb] dense, dtype dt
 *   C      [R][ldc] fp32 output, C[r][n] for n < Nc
 * K must be a multiple of 4.
 */
nm_status spmm_nm(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R, int64_t K,
                  const void* B, int64_t ldb, int64_t Nc, float* C, int64_t ldc, nm_stream stream);

/*
 * spmm_nm_t -- spmm_nm with the dense operand given K-contiguous:
 * C[r][n] = sum_k decompress(values, meta)[r][k] * Bt[n][k]
 * ("Success story: ESPLAG", Research Topic: the SpMM of a 2:4 layer).
 *   values [R][K/2], meta [R][ceil(K/8)] (2:4 form of an R x K matrix), dtype dt
 *   Bt     [Nc][ldbt] dense, dtype dt: row n holds column n of B (the token-major
 *          activation layout of an FFN, [tokens][d_model])
 *   C      [R][ldc] fp32 output, C[r][n] for n < Nc
 * K must be a multiple of 4.  Errors as for spmm_nm.  The pipelined bf16 kernel
 * runs when K % 256 == 0, ldbt % 8 == 0 and values, meta and Bt are 16-byte
 * aligned; other calls take a slower general kernel.
 */
nm_status spmm_nm_t(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R, int64_t K,
                    const void* Bt, int64_t ldbt, int64_t Nc, float* C, int64_t ldc, nm_stream stream);

/*
 * spmm_nm_t_out_bf16 -- spmm_nm_t with a bf16 result: each fp32 sum is rounded
 * to the nearest bf16, ties to even, as it is stored.  The output an FFN's
 * up-projection hands to the next step in bf16 (the activations that
 * prune_act_venom selects from; "To 2:4 Sparsity and Beyond", abstract).
 *   values, meta, Bt as for spmm_nm_t (dtype dt, bf16 or fp32 products);
 *   C [R][ldc] bf16 output (uint16 bit patterns), C[r][n] for n < Nc.
 * Errors as for spmm_nm_t (C aligned to 2 bytes).
 */
nm_status spmm_nm_t_out_bf16(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R,
                             int64_t K, const void* Bt, int64_t ldbt, int64_t Nc, void* C,
                             int64_t ldc, nm_stream stream);

/*
 * spmm_nm_t_lowrank -- spmm_nm_t of a 2:4 weight plus a low-rank adapter,
 * applied lazily (SLOPE abstract, NSF PAR award 2340011: low-rank adapters
 * joined to the sparse weight late in pre-training).  The adapted weight
 * W_s + U Vt is never formed:
 *   Tt[n][j] = sum_k Bt[n][k] * Vt[j][k]                   (adapter's inner activations)
 *   C[r][n]  = sum_k decompress(values, meta)[r][k] * Bt[n][k] + sum_j U[r][j] * Tt[n][j]
 *   values, meta, Bt as for spmm_nm_t (dtype dt)
 *   U      [R][ldu] dense, dtype dt, ldu >= rank
 *   Vt     [rank][ldvt] dense, dtype dt, ldvt >= K
 *   Tt     [Nc][rank] fp32 output, contiguous (row n holds the rank inner
 *          activations of column n of B; caller-allocated, kept for the
 *          adapter's backward)
 *   C      [R][ldc] fp32 output, C[r][n] for n < Nc
 * Two launches on the stream.  K must be a multiple of 4 and 0 < rank <= 2^20;
 * no output may overlap an input or the other output.  Errors as for
 * spmm_nm_t (U and Vt aligned to their element size, Tt and C to 4 bytes).
 * With bf16, rank % 16 == 0, K % 16 == 0, ldbt, ldvt and ldu multiples of 8
 * and Bt, Vt, U and Tt 16-byte aligned, Tt comes from matrix instructions and
 * the adapter term is added inside the pipelined SpMM (when that kernel's own
 * conditions hold) as extra steps after the sparse ones; each Tt value then
 * enters that term as two bf16 parts (about 16 significant bits).  Other calls
 * take plain fp32 kernels after the SpMM.
 */
nm_status spmm_nm_t_lowrank(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R,
                            int64_t K, const void* Bt, int64_t ldbt, int64_t Nc, const void* U,
                            int64_t ldu, const void* Vt, int64_t ldvt, int64_t rank, float* Tt,
                            float* C, int64_t ldc, nm_stream stream);

/*
 * spmm_nm_t_relu_venom -- an FFN up-projection whose activations leave the
 * kernel already pruned ("To 2:4 Sparsity and Beyond", abstract: 2:4 weights
 * and v:n:m activations in the FFN; "Sparser, Faster, Lighter Transformer
 * Language Models", Methodologie: ReLU).  With C = decompress(values, meta) Bt^T
 * as in spmm_nm_t ([R][Nc]: R the FFN width, Nc the tokens), the activations
 * h = ReLU(bf16(C))^T [Nc][R] (each fp32 sum rounded to nearest even, then
 * every value <= 0 made +0.0) are pruned to V:N:M along R with V-blocks of
 * tokens, exactly as prune_act_venom(h, V, M, apply_relu) would, and only the
 * compressed form is written: h is never stored.
 *   values, meta, Bt as for spmm_nm_t, bf16 only
 *   h_values [Nc][(R/M)*2] bf16, h_meta [Nc][ceil((R/M)/2)], h_colsel
 *            [Nc/V][R/M][4]: the outputs of prune_act_venom for h
 * V in {64, 128, 256} and M in {4, 8, 16} (NM_ERR_UNSUPPORTED otherwise, and
 * for dtypes other than bf16); R % 256 == 0, Nc % 256 == 0, K % 256 == 0, ldbt % 8 == 0,
 * values, meta and Bt 16-byte aligned, values and Bt each below 4 GiB,
 * h_values 16-byte and h_meta, h_colsel 4-byte aligned (NM_ERR_UNSUPPORTED
 * otherwise: compose spmm_nm_t_out_bf16,
 * nm_transpose and prune_act_venom instead).  NM_ERR_SHAPE for non-positive
 * sizes, K % 4 != 0, ldbt < K, R % M != 0 or Nc % V != 0.
 */
nm_status spmm_nm_t_relu_venom(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R,
                               int64_t K, const void* Bt, int64_t ldbt, int64_t Nc, int V, int M,
                               void* h_values, uint8_t* h_meta, uint8_t* h_colsel,
                               nm_stream stream);

/*
 * spmm_nm_general -- spmm_nm_t for any N:M form nm_compress writes ("Success
 * story: ESPLAG", Solution: N:M patterns beyond 2:4):
 * C[r][n] = sum_k decompress(values, meta, N, M)[r][k] * Bt[n][k]
 *   values [R][(K/M)*N], meta [R][ceil((K/M)*N*ceil(log2 M)/8)] (the layout of
 *          nm_compress), dtype dt
 *   Bt     [Nc][ldbt] dense, dtype dt (K-contiguous, as for spmm_nm_t)
 *   C      [R][ldc] fp32 output
 *   work   optional device memory of work_bytes bytes, 16-byte aligned, that
 *          must not overlap any other argument (NULL allowed)
 * M in {4, 8, 16}, 1 <= N < M, K % M == 0.  When N <= 2 every aligned run of
 * 4 columns holds at most two survivors: with work of at least
 * nm_general_work_bytes(dt, R, K, N, M) bytes the matrix is rewritten there
 * in 2:4 form (runs padded with +0.0) and spmm_nm_t computes the product; 2:4
 * itself goes to spmm_nm_t directly.  With N > 2 (bf16, K % 64 == 0, ldbt % 8
 * == 0, ldc % 4 == 0, 16-byte aligned Bt and C) the work memory receives the
 * matrix as dense bf16 rows [R][K] and a dense matrix-core GEMM computes the
 * product.  Other calls, and any without enough work memory, take a plain SIMT
 * kernel.  Errors as for spmm_nm_t, plus
 * NM_ERR_UNSUPPORTED for an N:M outside the set above and NM_ERR_SHAPE for
 * K % M != 0 or work_bytes < 0.
 */
nm_status spmm_nm_general(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R,
                          int64_t K, int N, int M, const void* Bt, int64_t ldbt, int64_t Nc,
                          float* C, int64_t ldc, void* work, int64_t work_bytes,
                          nm_stream stream);

/*
 * sddmm_venom -- gradient reaching V:N:M activations through a down-projection
 * ("To 2:4 Sparsity and Beyond", abstract: v:n:m activations in every FFN
 * matmul).  For Y = h_s . W_down with h_s the V:N:M form (prune_act_venom,
 * apply_relu) of h = ReLU(z) [T][F]:
 *   dz[t][2g+s] = sum_c dY[t][c] * W_down[g*M + colsel[t/V][g][j_s]][c]
 *                 (times [h_values[t][2g+s] > 0] when apply_relu)
 * i.e. dY . W_down^T at the entries h_s keeps -- the only ones through which
 * the gradient flows -- gated by ReLU's derivative.
 *   dY       [T][lddy] dtype dt         W_down [F][ldw] dtype dt (Nc columns)
 *   h_values [T][(F/M)*2], h_meta [T][ceil(F/M/2)], h_colsel [T/V][F/M][4]:
 *            h_s as prune_act_venom writes it (N = 2, 4 kept columns per group)
 *   dz       [T][(F/M)*2] fp32 output, aligned with h_values
 *   dYt      optional (NULL allowed, bf16 only): dYt [Nc][lddyt] receives
 *            dY^T, the operand spmm_venom_tn takes
 * M in {4, 8, 16}, 1 <= V <= 256, F % M == 0, T % V == 0.  bf16 with
 * V % 128 == 0, Nc % 64 == 0 and 16-byte aligned rows runs the pipelined
 * matrix-core kernel (B rows gathered per V-block); other calls a SIMT kernel
 * (then dYt by nm_transpose).  Errors as for sddmm_nm.
 */
nm_status sddmm_venom(nm_dtype dt, const void* dY, int64_t lddy, const void* W_down, int64_t ldw,
                      int64_t T, int64_t F, int64_t Nc, int V, int M, const void* h_values,
                      const uint8_t* h_meta, const uint8_t* h_colsel, int apply_relu, float* dz,
                      void* dYt, int64_t lddyt, nm_stream stream);

/*
 * spmm_venom_tn -- weight gradient of the same down-projection:
 *   dW[k][c] = sum_t h_s[t][k] * dY[t][c]      (h_s^T . dY)
 *   h_values, h_meta, h_colsel: h_s [T][F] in V:N:M form (as for sddmm_venom)
 *   dYt  [Nc][lddyt] dY^T, dtype dt (token index contiguous)
 *   dW   [F][lddw] fp32 output
 *   work optional device memory of work_bytes bytes, 16-byte aligned, not
 *        overlapping any argument (NULL allowed)
 * The reduction runs over tokens and every V-block of tokens keeps a different
 * half of each group's rows, so the product has no empty blocks for the matrix
 * instructions to skip.  bf16 with work of at least
 * nm_venom_tn_work_bytes(dt, T, F) bytes, T % 64 == 0, lddyt % 8 == 0,
 * lddw % 4 == 0 and 16-byte aligned operands writes h_s^T densely into work
 * and runs a matrix-core NT GEMM; other calls a SIMT kernel on the compressed
 * form.  Errors as for spmm_venom, plus NM_ERR_SHAPE for work_bytes < 0.
 */
nm_status spmm_venom_tn(nm_dtype dt, const void* h_values, const uint8_t* h_meta,
                        const uint8_t* h_colsel, int64_t T, int64_t F, int V, int M,
                        const void* dYt, int64_t lddyt, int64_t Nc, float* dW, int64_t lddw,
                        void* work, int64_t work_bytes, nm_stream stream);

/* Work bytes spmm_venom_tn uses for T tokens and F columns of h (host only; 0 = none). */
int64_t nm_venom_tn_work_bytes(nm_dtype dt, int64_t T, int64_t F);

/*
 * spmm_nm_general_noalloc -- spmm_nm_general for callers that cannot allocate
 * device memory (code under stream capture, tight serving loops, harnesses that
 * forbid allocation): the same product and kernels, with the work memory (the
 * 2:4 rewrite or the dense rows) held in a fixed 64 MiB scratch buffer that the library keeps in each GPU's memory
 * for the life of the process (nm_general_scratch_bytes() gives the size).
 * The call allocates nothing and takes no work argument; the caller still
 * passes inputs and outputs as for spmm_nm_general.  Every call on one GPU
 * shares that buffer: calls that overlap on one GPU (two streams, or two host
 * threads) race and must be serialised by the caller.  Nothing in the buffer
 * needs clearing between calls.  Errors as for spmm_nm_general, plus
 * NM_ERR_TOO_LARGE, returned before any launch, when the rewrite needs more
 * than the buffer holds (nm_general_work_bytes(dt, R, K, N, M) >
 * nm_general_scratch_bytes()).
 */
nm_status spmm_nm_general_noalloc(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R,
                                  int64_t K, int N, int M, const void* Bt, int64_t ldbt, int64_t Nc,
                                  float* C, int64_t ldc, nm_stream stream);

/*
 * nm_gmp_n_at -- host only: the N:M pattern a gradual magnitude pruning
 * schedule has in effect at a training step ("Success story: ESPLAG",
 * Highlights and Research Topic: semi-structured gradual magnitude pruning;
 * "To 2:4 Sparsity and Beyond", abstract: sparse steps, then regular dense
 * steps towards the end).  The pages give no schedule; the one implemented:
 *   - dense (returns M) before t_begin and, when t_dense >= 0, from t_dense on;
 *   - pruning events at t_begin + e*interval for e = 0 .. E-1,
 *     E = (t_end - t_begin) / interval + 1;
 *   - after event e the pattern is N_e : M with
 *     N_e = M - ceil((M - n_final) * (e + 1) / E), falling linearly to n_final
 *     at the last event and held until the dense switch.
 * *prune_now (nullable) is set to 1 when `step` is a pruning event: the caller
 * then magnitude-prunes its current weight to N_e:M (nm_prune_compress) and
 * keeps the pruned entries at zero.  Returns -1 for invalid parameters
 * (M not in {4, 8, 16}, n_final outside 1 .. M-1, t_begin < 0,
 * t_end < t_begin, interval < 1).
 */
int nm_gmp_n_at(int M, int n_final, int64_t t_begin, int64_t t_end, int64_t interval,
                int64_t t_dense, int64_t step, int* prune_now);

/* Bytes of the fixed scratch buffer of spmm_nm_general_noalloc (host only). */
int64_t nm_general_scratch_bytes(void);

/*
 * nm_general_work_bytes -- host only: the work bytes spmm_nm_general uses for
 * an R x K matrix in N:M form (0 when it uses none, or for invalid arguments).
 */
int64_t nm_general_work_bytes(nm_dtype dt, int64_t R, int64_t K, int N, int M);

/*
 * nm_transpose -- dst[c][r] = src[r][c] for an R x Cn matrix: turns a row-major
 * dense operand B [K][Nc] into the K-contiguous form spmm_nm_t takes.
 *   src [R][lds], dst [Cn][ldd] (ldd >= R), dtype dt; dst must not overlap src.
 * bf16 only (NM_ERR_UNSUPPORTED for other dtypes).
 */
nm_status nm_transpose(nm_dtype dt, const void* src, int64_t lds, int64_t R, int64_t Cn, void* dst,
                       int64_t ldd, nm_stream stream);

/*
 * prune_act_venom -- V:N:M prune (N = 2) and compress in one pass, optionally
 * after ReLU ("To 2:4 Sparsity and Beyond", abstract: v:n:m activations;
 * "Sparser, Faster, Lighter Transformer Language Models", Methodologie: ReLU;
 * "Success story: ESPLAG", Solution: VENOM format).
 *   Z       [R][ldz] input, dtype dt
 *   apply_relu  nonzero: select on h = ReLU(Z) (every z <= 0, and -0.0,
 *               becomes +0.0) and store h's values
 *   values  [R][(K/M)*2], meta [R][ceil(K/M/2)], colsel [R/V][K/M][4] outputs
 *   mask    nullable [R][ldmask] u8 output: 1 at the 2 kept columns per group
 * M in {4, 8, 16}; 1 <= V <= 256; R % V == 0; K % M == 0.
 */
nm_status prune_act_venom(nm_dtype dt, const void* Z, int64_t ldz, int64_t R, int64_t K, int V,
                          int M, int apply_relu, void* values, uint8_t* meta, uint8_t* colsel,
                          uint8_t* mask, int64_t ldmask, nm_stream stream);

/*
 * spmm_venom -- C = decompress_venom(values, meta, colsel) * B:
 * C[r][n] = sum_g sum_s values[r][2g+s] * B[g*M + colsel[r/V][g][j_s]][n]
 * ("To 2:4 Sparsity and Beyond", abstract; "Success story: ESPLAG",
 * Solution: VENOM format and its SpMM).
 *   B [K][ldb] dense, dtype dt; C [R][ldc] fp32 output.
 * M in {4, 8, 16}; 1 <= V <= 256; R % V == 0; K % M == 0.
 */
nm_status spmm_venom(nm_dtype dt, const void* values, const uint8_t* meta, const uint8_t* colsel,
                     int64_t R, int64_t K, int V, int M, const void* B, int64_t ldb, int64_t Nc,
                     float* C, int64_t ldc, nm_stream stream);

/*
 * nm_reprune_t -- double pruning (NSF PAR award 2340011, SLOPE abstract): the
 * 2:4-compressed W_s [R x K] is decompressed with +0.0 fill, transposed to
 * [K x R], pruned 2:4 by magnitude along R and compressed.
 *   values [R][K/2], meta [R][ceil(K/8)]      input (2:4 along K)
 *   values_t [K][R/2], meta_t [K][ceil(R/8)]  output (2:4 along R)
 * R and K must be multiples of 4.
 */
nm_status nm_reprune_t(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R, int64_t K,
                       void* values_t, uint8_t* meta_t, nm_stream stream);

/*
 * nm_reprune_t_transpose -- nm_reprune_t of W_s and nm_transpose of X in one
 * launch: the two passes of a double-pruned training step (NSF PAR award
 * 2340011, SLOPE abstract: the transposed weight re-pruned for the backward
 * pass; the layer input then feeds spmm_nm_t K-contiguous) that touch
 * disjoint data.
 *   values, meta, R, K, values_t, meta_t as for nm_reprune_t;
 *   X [RX][ldx] dense input, Xt [CX][ldxt] output (ldxt >= RX): Xt[c][r] = X[r][c].
 * Outputs are byte-identical to nm_reprune_t followed by nm_transpose.  bf16
 * only (NM_ERR_UNSUPPORTED otherwise).  With R and K multiples of 128 and the
 * re-prune's aligned layout the two run as one kernel; otherwise as the two
 * kernels.  No output may overlap an input.  Errors as for the two calls.
 */
nm_status nm_reprune_t_transpose(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R,
                                 int64_t K, void* values_t, uint8_t* meta_t, const void* X,
                                 int64_t ldx, int64_t RX, int64_t CX, void* Xt, int64_t ldxt,
                                 nm_stream stream);

/*
 * nm_mfma_rate_probe -- a measurement aid, not a step of the sparse path: a
 * chip-wide loop of independent bf16 matrix instructions on register operands
 * (kind 0: v_mfma_f32_32x32x16_bf16; kind 1: v_smfmac_f32_32x32x32_bf16, 2:4),
 * eight accumulators per wave, two waves per SIMD on 256 CUs, no memory traffic.
 * Timed by the caller (events around it on `stream`), it gives the matrix rate
 * the chip sustains under its power limit, the reference the benchmark reports
 * next to the nominal peak.
 *   iters  loop count per wave (1 .. 2^24)
 *   sink   device fp32 [512 * 256]: one value per thread, written so that
 *          nothing is optimised away (its contents mean nothing)
 *   flops  host output: the dense-equivalent flops one launch performs
 * NM_ERR_UNSUPPORTED for another kind, NM_ERR_SHAPE for iters out of range.
 */
nm_status nm_mfma_rate_probe(int kind, int64_t iters, float* sink, int64_t* flops, nm_stream stream);

/*
 * The panel layout of a bf16 2:4 form (R rows, K dense columns, R % 4 == 0,
 * K % 256 == 0): the same values and nibbles as the row-major form
 * (values [R][K/2], meta [R][K/8]), in another order, with the same total sizes:
 *   values: the 64 bytes of row r for the 64-column step s (its 32 kept values,
 *           in column order) at byte ((r / 2) * (K / 64) + s) * 128 + (r % 2) * 64;
 *   meta:   the 32 bytes of row r for the 256-column chunk c (its 64 nibbles,
 *           group 0 in bits 0..3) at byte ((r / 4) * (K / 256) + c) * 128 + (r % 4) * 32.
 * Every 64-column step of a 256-row tile is then whole 128-byte lines of each
 * operand, which the four-wave SpMM below needs to load two steps ahead.
 */

/*
 * nm_to_panels -- the panel layout of a bf16 2:4 form given row-major.
 *   values [R][K/2], meta [R][K/8] in; values_p, meta_p (same sizes) out.
 * R % 4 == 0 and K % 256 == 0 (NM_ERR_SHAPE), all four pointers 16-byte aligned
 * (NM_ERR_ALIGN), bf16 only (NM_ERR_UNSUPPORTED).  No output may overlap an input.
 */
nm_status nm_to_panels(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R, int64_t K,
                       void* values_p, uint8_t* meta_p, nm_stream stream);

/*
 * nm_reprune_t_transpose_panels -- nm_reprune_t_transpose with the re-pruned
 * transposed weight written in the panel layout (a K x R form compressed along
 * R): the double-pruned backward's operand (NSF PAR award 2340011, SLOPE
 * abstract) for spmm_nm_t_panels.  Xt as for nm_reprune_t_transpose.
 * bf16 only; R % 256 == 0 and K % 128 == 0 (NM_ERR_SHAPE); values and values_t
 * 16-byte, meta and meta_t 2-byte aligned (NM_ERR_ALIGN).  Outputs equal
 * nm_to_panels of nm_reprune_t's, byte for byte.
 */
nm_status nm_reprune_t_transpose_panels(nm_dtype dt, const void* values, const uint8_t* meta,
                                        int64_t R, int64_t K, void* values_t, uint8_t* meta_t,
                                        const void* X, int64_t ldx, int64_t RX, int64_t CX,
                                        void* Xt, int64_t ldxt, nm_stream stream);

/*
 * spmm_nm_t_panels -- spmm_nm_t of a weight given in the panel layout
 * ("Success story: ESPLAG", Research Topic: the SpMM of a 2:4 layer; the
 * backward's product with the re-pruned transposed weight, SLOPE abstract):
 * C[r][n] = sum_k decompress(values, meta)[r][k] * Bt[n][k].
 *   values, meta: panel layout of the R x K form; Bt [Nc][ldbt]; C [R][ldc] fp32.
 * bf16 only; R % 256 == 0, K % 256 == 0, ldbt >= K, ldbt % 8 == 0, ldc >= Nc
 * (NM_ERR_SHAPE); values, meta and Bt 16-byte, C 4-byte aligned (NM_ERR_ALIGN);
 * NM_ERR_TOO_LARGE when values or Bt reach 4 GiB.  The products are added in the
 * order of spmm_nm_t's pipelined kernel, so C equals spmm_nm_t's bit for bit.
 */
nm_status spmm_nm_t_panels(nm_dtype dt, const void* values, const uint8_t* meta, int64_t R,
                           int64_t K, const void* Bt, int64_t ldbt, int64_t Nc, float* C,
                           int64_t ldc, nm_stream stream);

/*
 * sddmm_nm -- the weight gradient of a 2:4 layer, sampled at the weight's
 * survivors ("Success story: ESPLAG", Research Topic: kernels for the full
 * sparse training step):
 *   values_out[r][2g+s] = sum_t D[r][t] * X[4g + p_s(r, g)][t]
 * with p_s from meta (the 2:4 metadata of the R x Kc weight).
 *   D [R][ldd] (the output gradient), X [Kc][ldx] (the layer input, one row
 *   per input feature), dtype dt; values_out [R][Kc/2] fp32.
 * Kc must be a multiple of 4.
 */
nm_status sddmm_nm(nm_dtype dt, const void* D, int64_t ldd, const void* X, int64_t ldx, int64_t R,
                   int64_t Kc, int64_t T, const uint8_t* meta, float* values_out, nm_stream stream);

/*
 * sddmm_nm_dt -- sddmm_nm that also writes the transpose of the output
 * gradient, Dt[t][r] = D[r][t], which the input gradient's product then reads
 * K-contiguous (spmm_nm_t of the re-pruned transposed weight; "Success story:
 * ESPLAG", Research Topic: the kernels of the sparse training step).  The
 * SDDMM stages every tile of D through LDS, so the transpose costs no extra
 * read of D.
 *   D, X, meta, values_out as for sddmm_nm; Dt [T][lddt] bf16 output
 *   (lddt >= R), not overlapping any input.
 * bf16 only (NM_ERR_UNSUPPORTED otherwise).  Outputs are those of sddmm_nm and
 * nm_transpose(D); without the pipelined SDDMM's conditions the call runs the
 * two.  Errors as for the two calls.
 */
nm_status sddmm_nm_dt(nm_dtype dt, const void* D, int64_t ldd, const void* X, int64_t ldx, int64_t R,
                      int64_t Kc, int64_t T, const uint8_t* meta, float* values_out, void* Dt,
                      int64_t lddt, nm_stream stream);

/*
 * ---------------------------------------------------------------------------
 * The mixture-of-experts FFN in 8-bit floating point ("To 2:4 Sparsity and
 * Beyond", abstract: the method is orthogonal to quantisation and applies to
 * mixture-of-experts FFNs).  A layer's forward is
 *   moe_route -> moe_plan -> fp8_quantize (rows gathered by expert)
 *   -> fp8_gemm_nt_grouped (up) -> fp8_quantize (ReLU) -> fp8_gemm_nt_grouped (down) -> moe_combine
 * and its backward moe_combine_bwd, the same products on transposed weights
 * (input gradient), fp8_quantize_t and fp8_gemm_nt_grouped_k (weight
 * gradients), moe_combine with no weights, and moe_route_bwd.
 *
 * 8-bit matrices are OCP e4m3 (largest value 448, no infinities) or e5m2
 * (57344) bytes with an fp32 scale for each block of 128 elements along the
 * reduction dimension: value = byte's value * scale.  Scales lie block-major:
 *   by rows   s[kb][lds], kb = k / 128: one per row and 128-block, contiguous
 *             along the rows (a tile's scales of one block are one load);
 *   by blocks s[r / 128][lds], lds >= ceil(K / 128): one per 128 x 128 block.
 * ---------------------------------------------------------------------------
 */

typedef enum { NM_E4M3 = 0, NM_E5M2 = 1 } nm_fp8;
typedef enum { NM_SOFTMAX = 0, NM_SIGMOID = 1 } nm_score;

/*
 * moe_route -- the experts of every token and their weights.
 *   s[t][e] = softmax over e of logits[t], or sigmoid(logits[t][e])
 *   c[t][e] = s[t][e] + bias[e]                (bias NULL: c = s)
 *   With groups > 1, the E experts are `groups` equal runs; a run's score is the
 *   sum of its group_top (1 or 2) largest c; only experts of the topk_groups best
 *   runs stay.  ids[t][0..k-1] are the k experts of largest c, in descending
 *   order; on equal c (and equal run scores) the lower index wins.
 *   weights[t][j] = scale * s[t][ids[t][j]], divided by the sum of the chosen s
 *   when renorm.
 *   logits [T][ldl] dtype dt; bias fp32 [E]; ids int32 [T][k], weights fp32 [T][k]
 * An expert whose logit is -infinity or NaN (or whose bias is NaN) is never
 * chosen; +infinity counts as the largest finite value.  Where fewer than k
 * experts can be chosen, the remaining ids are -1 and their weights 0.  Scores
 * are computed in fp32; with no bias the order is that of the logits themselves.
 * 1 <= E <= 1024, 1 <= k <= 64, groups <= 64 (NM_ERR_UNSUPPORTED, also for a
 * scale that is 0 or not finite); E % groups == 0, topk_groups <= groups,
 * k <= E / groups * topk_groups, T * k < 2^31 (NM_ERR_SHAPE).
 */
nm_status moe_route(nm_dtype dt, const void* logits, int64_t ldl, int64_t T, int64_t E, nm_score score,
                    const float* bias, int groups, int topk_groups, int group_top, int k, int renorm,
                    float scale, int32_t* ids, float* weights, nm_stream stream);

/*
 * moe_route_bwd -- the gradient of moe_route's weights with respect to the logits.
 * The choice itself has no gradient.  With g = sum_j dweights_j weights_j / scale:
 *   softmax, renorm   dl_j = weights_j (dweights_j - g) at the chosen, 0 elsewhere
 *   sigmoid, renorm   the same times 1 - s_j
 *   softmax           dl_e = weights_e dweights_e (chosen e) - s_e g scale
 *   sigmoid           dl_j = weights_j dweights_j (1 - s_j) at the chosen, 0 elsewhere
 *   logits, ids, weights as moe_route takes and writes them (the ids of a token
 *   are distinct; an id outside 0 .. E-1 has no part in it); dweights fp32
 *   [T][k]; dlogits [T][lddl] dtype dt output.  Limits and errors as for moe_route.
 */
nm_status moe_route_bwd(nm_dtype dt, const void* logits, int64_t ldl, int64_t T, int64_t E, nm_score score, int k,
                        int renorm, float scale, const int32_t* ids, const float* weights, const float* dweights,
                        void* dlogits, int64_t lddl, nm_stream stream);

/*
 * moe_plan -- the order of the T * k (token, choice) slots by expert, slots of one
 * expert in ascending order; each expert's run of rows starts at a multiple of
 * `align` (1, or a power of two up to 256).
 *   ids [T][k]; a slot whose id lies outside 0 .. E-1 belongs to no expert
 *   offsets int32 [E + 1]: expert e's rows are offsets[e] .. offsets[e + 1] - 1, the
 *           last of them padding; counts int32 [E]: how many are not padding
 *   src int32 [rows]: the slot t * k + j of each row, -1 for padding and for every
 *           row from offsets[E] on
 *   pos int32 [T][k]: the row of each slot, -1 for a slot of no expert
 *   rows >= T * k + min(T * k, E) * (align - 1) rounded up to align (NM_ERR_SHAPE)
 *   work device memory, 4-byte aligned, of moe_plan_work_bytes bytes (NULL when that is 0;
 *           NM_ERR_SHAPE when work_bytes is less)
 * rows < 2^31, 1 <= E <= 1024 and T * k <= 2^30.  The result does not depend on the
 * order in which threads run.
 */
nm_status moe_plan(const int32_t* ids, int64_t T, int k, int64_t E, int align, int32_t* offsets, int32_t* counts,
                   int32_t* src, int64_t rows, int32_t* pos, void* work, int64_t work_bytes, nm_stream stream);

/* Host only: the work bytes moe_plan uses (*bytes; 0 for small T * k). */
nm_status moe_plan_work_bytes(int64_t T, int k, int64_t E, int64_t* bytes);

/*
 * fp8_quantize -- rows to 8 bits in blocks of 128 along K, with a power-of-two scale:
 *   x[r][c] = X[src[r] / div][c] (src NULL: X[r][c]); 0 where src[r] / div is not a row of X;
 *             0 where gate is given and gate[r][c] is not > 0 (gate = X: ReLU; gate = the
 *             forward's pre-activations: the gradient of ReLU); a NaN gate is not > 0, so ReLU
 *             takes a NaN to 0, and keeps +infinity
 *   S[kb][r] = the smallest power of two (at least 2^-126) that is >= amax / 448 (e4m3) or
 *             amax / 57344 (e5m2), amax the largest finite |x| of the block; 1 when that is 0
 *   Q[r][c] = x[r][c] / S[kb][r] rounded to nearest even (the division is exact)
 * so no finite value saturates, and a NaN or infinite x becomes NaN.
 *   X [RX][ldx] dtype dt, src int32 [R], gate [R][ldg] dtype dt
 *   Q [R][ldq] bytes, ldq >= Kp = K rounded up to 128: columns K .. Kp-1 are written 0
 *   S fp32 [Kp / 128][lds], lds >= R
 * src == NULL needs R <= RX.  16-byte aligned rows run with vector loads.
 */
nm_status fp8_quantize(nm_dtype dt, const void* X, int64_t ldx, int64_t RX, const int32_t* src, int div,
                       const void* gate, int64_t ldg, int64_t R, int64_t K, nm_fp8 fmt, uint8_t* Q, int64_t ldq,
                       float* S, int64_t lds, nm_stream stream);

/*
 * fp8_quantize_t -- the same x transposed, in blocks of 128 along its rows: the operands of a
 * weight gradient, whose reduction runs over the rows.
 *   Qt [K][ldqt] bytes, ldqt >= Rp = R rounded up to 128: columns R .. Rp-1 are written 0
 *   St fp32 [Rp / 128][ldst], ldst >= K
 */
nm_status fp8_quantize_t(nm_dtype dt, const void* X, int64_t ldx, int64_t RX, const int32_t* src, int div,
                         const void* gate, int64_t ldg, int64_t R, int64_t K, nm_fp8 fmt, uint8_t* Qt, int64_t ldqt,
                         float* St, int64_t ldst, nm_stream stream);

/*
 * fp8_quantize_weight -- E weights [N][K] (W[e] = W + e * N * ldw) to 8 bits in 128 x 128 blocks
 * (scales as fp8_quantize's), and optionally the same bytes transposed, for the input gradient.
 *   Q [E][N][ldq], ldq >= Kp, columns K .. Kp-1 written 0; S fp32 [E][ceil(N / 128)][Kp / 128]
 *   Qt [E][K][ldqt], ldqt >= Np = N rounded up to 128, columns N .. Np-1 written 0, and
 *   St fp32 [E][Kp / 128][Np / 128]: both given or both NULL
 */
nm_status fp8_quantize_weight(nm_dtype dt, const void* W, int64_t ldw, int64_t E, int64_t N, int64_t K, nm_fp8 fmt,
                              uint8_t* Q, int64_t ldq, float* S, uint8_t* Qt, int64_t ldqt, float* St,
                              nm_stream stream);

/*
 * fp8_gemm_nt -- the product of two 8-bit matrices, both K-contiguous:
 *   C[m][n] = sum_kb sa[kb][m] sb(n, kb) sum_{k in kb} A[m][k] B[n][k]
 *   A [M][lda] format fa, sa fp32 [ceil(K / 128)][ldsa], ldsa >= M
 *   B [N][ldb] format fb; sb by blocks (b_block 128): [ceil(N / 128)][ldsb], ldsb >= ceil(K / 128),
 *     or by rows (b_block 1): [ceil(K / 128)][ldsb], ldsb >= N
 *   C [M][ldc] fp32 or bf16 (out)
 * Each 128-block's sum is scaled and added in fp32; the result is rounded once.  The product of a block's
 * two scales is formed first, in fp32, and has to be finite (scales of magnitude below 2^64 always
 * do; an infinite product gives NaN where the sum is 0).  The sum itself:
 *   out NM_F32   products and sums are fp32.
 *   out NM_BF16  the 8-bit matrix instruction.  Of every eight products k = 8 i .. 8 i + 7 each is cut
 *     towards zero to a multiple of 2^-13 u, u the largest 2^(ea + eb) among the eight that are not 0
 *     (ea, eb the operands' exponents, at least -6 in e4m3 and -14 in e5m2, so u is no more than the
 *     largest product unless it has a subnormal operand); the cut products are added in fp32.  That is
 *     off by less than 7 * 2^-13 u for every eight products and 1.5e-5 of a result of normal operands
 *     (root mean square).  Where large products of one group of eight cancel it can be more than the
 *     rounding to bf16: a caller who needs fp32 sums there asks for an fp32 result.
 * The tiled kernels run when lda and ldb are multiples of 16, A and B are 16-byte
 * aligned (the rows are then read whole, up to K rounded up to 16); other calls take a slower
 * general kernel.
 */
nm_status fp8_gemm_nt(nm_fp8 fa, const uint8_t* A, int64_t lda, const float* sa, int64_t ldsa, nm_fp8 fb,
                      const uint8_t* B, int64_t ldb, const float* sb, int64_t ldsb, int b_block, int64_t M,
                      int64_t N, int64_t K, nm_dtype out, void* C, int64_t ldc, nm_stream stream);

/*
 * fp8_gemm_nt_grouped -- fp8_gemm_nt with a B for every group of A's rows (a mixture-of-experts
 * layer's forward, and its input gradient with the transposed weights):
 *   C[m][n] = the product of A's row m with B[e], offsets[e] <= m < offsets[e + 1]
 *   A [rows][lda], sa [ceil(K / 128)][ldsa], ldsa >= rows
 *   B [E][N][ldb], sb [E][ceil(N / 128)][ldsb] by blocks
 *   offsets device int32 [E + 1], not decreasing (values are taken as at least 0 and at most rows)
 *   C [rows][ldc]; rows outside every group are written 0.  1 <= E <= 1024, rows < 2^31.
 */
nm_status fp8_gemm_nt_grouped(nm_fp8 fa, const uint8_t* A, int64_t lda, const float* sa, int64_t ldsa, nm_fp8 fb,
                              const uint8_t* B, int64_t ldb, const float* sb, int64_t ldsb, const int32_t* offsets,
                              int64_t E, int64_t rows, int64_t N, int64_t K, nm_dtype out, void* C, int64_t ldc,
                              nm_stream stream);

/*
 * fp8_gemm_nt_grouped_k -- a product for every run of the reduction dimension (the experts' weight
 * gradients):
 *   C[e][m][n] = sum over offsets[e] <= k < offsets[e + 1] of A[m][k] B[n][k], scaled as above
 *   A [M][lda], sa [rows / 128][ldsa], ldsa >= M; B [N][ldb], sb [rows / 128][ldsb], ldsb >= N
 *   offsets device int32 [E + 1] multiples of 128, as moe_plan writes them with align 128 or 256
 *           (any other value counts as the next lower multiple of 128)
 *   C [E][M][ldc]; a group with no columns is written 0.  rows % 128 == 0 (NM_ERR_SHAPE).
 */
nm_status fp8_gemm_nt_grouped_k(nm_fp8 fa, const uint8_t* A, int64_t lda, const float* sa, int64_t ldsa, nm_fp8 fb,
                                const uint8_t* B, int64_t ldb, const float* sb, int64_t ldsb,
                                const int32_t* offsets, int64_t E, int64_t M, int64_t N, int64_t rows, nm_dtype out,
                                void* C, int64_t ldc, nm_stream stream);

/*
 * moe_combine -- Y[t][c] = sum_j weights[t][j] O[pos[t][j]][c], summed in fp32 in ascending j
 * (weights NULL: all 1, the gradient of gathering the tokens' rows); a pos outside 0 .. rows-1 adds
 * nothing, whatever its weight.
 *   O [rows][ldo] dtype dt, pos int32 [T][k], weights fp32 [T][k], Y [T][ldy] dtype dt.  1 <= k <= 64.
 */
nm_status moe_combine(nm_dtype dt, const void* O, int64_t ldo, int64_t rows, const int32_t* pos,
                      const float* weights, int64_t T, int k, int64_t D, void* Y, int64_t ldy, nm_stream stream);

/*
 * moe_combine_bwd -- the gradients of moe_combine:
 *   dO[pos[t][j]][c] = weights[t][j] dY[t][c], and 0 in the rows whose src is negative
 *   dweights[t][j] = sum_c dY[t][c] O[pos[t][j]][c], 0 where pos is outside 0 .. rows-1
 *   src [rows] and pos [T][k] as moe_plan writes them; dO [rows][lddo] dtype dt, dweights fp32 [T][k]
 */
nm_status moe_combine_bwd(nm_dtype dt, const void* dY, int64_t lddy, const void* O, int64_t ldo, int64_t rows,
                          const int32_t* src, const int32_t* pos, const float* weights, int64_t T, int k, int64_t D,
                          void* dO, int64_t lddo, float* dweights, nm_stream stream);

/*
 * nm_sizes -- host-only helper: element count of values, bytes of meta and of
 * colsel for an R x K matrix in N:M form (V > 0: V:N:M form with N = 2, where
 * N is ignored).  NULL outputs are skipped.
 */
void nm_sizes(int64_t R, int64_t K, int N, int M, int V, int64_t* n_values, int64_t* meta_bytes,
              int64_t* colsel_bytes);

/* Static description of a status code. */
const char* nm_status_str(nm_status status);

/* The HIP error string behind the last NM_ERR_HIP on this thread ("" if none). */
const char* nm_last_hip_error(void);

/* Library version, major * 10000 + minor * 100 + patch. */
int nm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* NMSPARSE_H */
