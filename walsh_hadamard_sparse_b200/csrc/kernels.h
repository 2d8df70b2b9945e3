// Internal launchers of libqwha (not part of the C ABI). Each enqueues its
// kernels on `s` and returns the launch status; argument checks live in api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "qwha.h"

namespace qwha {

// W_eff rows for Hadamard blocks of 2^logn, 7 <= logn <= 12 (fwht.cu).
bool weff_rows_supported(int logn);
cudaError_t launch_weff_rows(const int32_t *row_ptr, const int32_t *col_idx, const float *coef, int64_t p, int d_in,
                             int64_t n_rows, int logn, float scale, int bits, int group, const uint8_t *qw,
                             const float *scales, const uint8_t *zeros, void *out, cudaStream_t s);

// Transform `blocks` consecutive blocks of 2^logn elements; out = H_unnorm(in) * scale.
cudaError_t launch_fwht(qwha_dtype din, qwha_dtype dout, const void *x, void *z, int64_t blocks,
                        int logn, float scale, cudaStream_t s);

}  // namespace qwha

namespace qwha {

// Upper bound on the token chunks of the coefficient-gradient kernel (its
// partial sums take kSddmmMaxChunks * p floats of workspace at most).
constexpr int kSddmmMaxChunks = 16;

// out[t, i] = alpha * sum_{j in [seg_ptr[i], seg_ptr[i+1])} v_j * in[t, idx[j]], with
// v_j = val[perm[j]] when perm is given (the CSC view), else val[j]. scratch
// (256-byte aligned) holds the entries in the order the kernel reads them;
// spmm_scratch_bytes(nnz, n_seg, W_in) bytes always suffice. *launched (if
// given) receives the number of kernels enqueued.
size_t spmm_scratch_bytes(int64_t p, int n_seg, int W_in);
cudaError_t launch_seg_spmm(qwha_dtype din, qwha_dtype dout, const void *in, int64_t T, int W_in,
                            const int32_t *seg_ptr, const int32_t *idx, const float *val, const int32_t *perm,
                            int64_t nnz, int n_seg, float alpha, void *scratch, size_t scratch_bytes, void *out,
                            cudaStream_t s, int *launched = nullptr);

int sddmm_chunks(int64_t T, int32_t d_out, int32_t d_in);

// Bytes of the transposed copies of dY and Z that launch_sddmm can use (bf16).
size_t sddmm_transposed_bytes(int64_t T, int32_t d_out, int32_t d_in);

// dc[j] = alpha * sum_t dY[t, r_j] Z[t, k_j] through the tile view; partial is
// workspace of sddmm_chunks(...) * p floats. tscratch (16-byte aligned, at
// least sddmm_transposed_bytes(...)) lets bf16 inputs take the path that
// transposes dY and Z once and feeds the kernel by tensor copies; nullptr, or
// shapes that path does not take (fp32, d_out or d_in not a multiple of 8),
// keep the kernel that stages and transposes its own tiles. Both give
// bitwise the same dc. *launched (if given) receives the number of kernels
// enqueued.
cudaError_t launch_sddmm(qwha_dtype dt, const void *dY, const void *Z, int64_t T, int32_t d_out, int32_t d_in,
                         const int32_t *tile_ptr, const int32_t *tile_pos, const int32_t *tile_rk, int64_t p,
                         float alpha, float *partial, float *dc, cudaStream_t s, void *tscratch = nullptr,
                         int *launched = nullptr);

// A tensor map over a bf16 matrix of rows x cols with a row stride of ld
// elements (ld * 2 a multiple of 16, ptr 16-byte aligned), box box_cols x
// box_rows, no swizzle (gemm.cu).
bool make_map_rows(CUtensorMap *m, const void *ptr, int64_t rows, int64_t cols, int64_t ld, uint32_t box_cols,
                   uint32_t box_rows);

size_t plan_workspace(int32_t d_out, int32_t d_in);
int plan_max_row_blocks();
cudaError_t launch_plan_build(int32_t d_out, int32_t d_in, int64_t p, const int32_t *row_ptr,
                              const int32_t *col_idx, int32_t *col_ptr, int32_t *row_idx, int32_t *perm,
                              int32_t *tile_ptr, int32_t *tile_pos, int32_t *tile_rk, void *ws,
                              cudaStream_t s);

}  // namespace qwha

namespace qwha {

// AdaAlloc (init.cu)
size_t init_workspace(int32_t d_out, int32_t d_in);
int init_max_din();
// Value Refinement (refine.cu)
int refine_cap(int32_t d_in);
size_t refine_workspace(int32_t d_out, int32_t d_in);
cudaError_t launch_calib_hessian(const void *X, int64_t T, int32_t d_in, float *S, cudaStream_t s);
cudaError_t launch_refine(const float *dWq, int32_t d_out, int32_t d_in, int32_t had_block, const float *S,
                          float damp, const int32_t *row_ptr, const int32_t *col_idx, int64_t p, float *coef,
                          void *ws, cudaStream_t s);
size_t select_global_workspace(int32_t d_out, int32_t d_in);
cudaError_t launch_select_global(const float *dW, int32_t d_out, int32_t d_in, int32_t had_block, int64_t p, int sel,
                                 uint64_t seed, int32_t *budgets, int32_t *row_ptr, int32_t *col_idx, float *coef,
                                 void *ws, cudaStream_t s);
// Selection diagnostics (init.cu, diag.cu).
size_t energy_stats_workspace(int32_t d_out, int32_t d_in);
cudaError_t launch_energy_stats(const float *dW, int32_t d_out, int32_t d_in, int32_t had_block, int64_t k,
                                double *out, void *ws, cudaStream_t s);
size_t pattern_stats_workspace(int32_t d_in);
cudaError_t launch_pattern_stats(int32_t d_out, int32_t d_in, int64_t p, const int32_t *row_ptr,
                                 const int32_t *col_idx, int32_t *col_counts, int64_t *stats, void *ws,
                                 cudaStream_t s);
cudaError_t launch_init_norms(const float *dW, int32_t rows, int32_t d_in, double *e, cudaStream_t s);
cudaError_t launch_init_budgets(const double *e, int32_t d_out, int32_t d_in, int64_t p, int32_t min_per_row, int mode,
                                int32_t *budgets, int32_t *row_ptr, void *ws, cudaStream_t s);
cudaError_t launch_init_select(const float *dW, int32_t rows, int32_t d_in, int32_t had_block, const int32_t *budgets,
                               const int32_t *row_ptr, int64_t p, int32_t *col_idx, float *coef, cudaStream_t s);
cudaError_t launch_init_alloc(const float *dW, int32_t d_out, int32_t d_in, int32_t had_block, int64_t p,
                              int32_t min_per_row, int mode, int32_t *budgets, int32_t *row_ptr, int32_t *col_idx,
                              float *coef, void *ws, cudaStream_t s);

// Base weight (dequant.cu): bf16 W_Q [d_out, d_in].
size_t wdeq_bytes(int32_t d_out, int32_t d_in);
cudaError_t launch_dequant(int bits, int group, int32_t d_out, int32_t d_in, const uint8_t *qw, const float *scales,
                           const uint8_t *zeros, void *out, cudaStream_t s);

// Base GEMM with fp32 addend in the epilogue (gemm.cu).
cudaError_t launch_gemm_fwd(const void *X, const void *wdeq, const float *y_ad, void *Y, int64_t T, int32_t d_out,
                            int32_t d_in, cudaStream_t s);
// out[M, N] = A[M, K] B[N, K]^T (+ addend), A and B bf16 K-major, out fp32 or bf16.
cudaError_t launch_gemm_nt(const void *A, const void *B, const float *addend, void *out, bool f32_out, int64_t M,
                           int64_t N, int64_t K, cudaStream_t s);
// dc[j] = alpha * (A B^T)[r_j, col_idx[j]] for the CSR entries of E, written
// by the GEMM epilogue (no dense output).
// Forward GEMM Y = X W^T (bf16, K-major) whose launch also writes Z = X H
// (bf16, Hadamard blocks of 2^logn, times scale) from extra warps.
bool gemm_fused_fwht_supported(int64_t M, int logn);
cudaError_t launch_gemm_fwd_fused(const void *X, const void *W, void *Y, int64_t T, int32_t d_out, int32_t d_in,
                                  void *Z, int logn, float scale, cudaStream_t s);
cudaError_t launch_gemm_sampled(const void *A, bool a_mn, const void *B, bool b_mn, int64_t M, int64_t N, int64_t K,
                                const int32_t *row_ptr, const int32_t *col_idx, int64_t p, float alpha, float *dc,
                                cudaStream_t s);
// Same with either operand MN-major: A [K, M] when a_mn, B [K, N] when b_mn.
cudaError_t launch_gemm_any(const void *A, bool a_mn, const void *B, bool b_mn, const float *addend, void *out,
                            bool f32_out, int64_t M, int64_t N, int64_t K, cudaStream_t s);

// Device error word and plan validation (misc.cu).
cudaError_t read_and_clear_error_word(unsigned int *word, cudaStream_t s);
const char *validate_message(unsigned int code);
cudaError_t launch_validate(const qwha_adapter *a, cudaStream_t s, uint32_t *code, int64_t *where);

}  // namespace qwha

namespace qwha {

// Dense formulation (dense.cu).
size_t weff_smem(int32_t d_in);
// out = bf16(dequant(W_Q) + alpha * (F H)) [d_out, d_in]; wq may be NULL (adapter alone).
cudaError_t launch_weff(const qwha_adapter *a, const qwha_qweight *wq, float alpha, void *out, cudaStream_t s);

}  // namespace qwha

namespace qwha {

// Products with the packed weight for a few tokens (gemv.cu). A call is up to
// three launches on one stream, each overlapping the one before: the tokens'
// operands and transform (launch_decode_prepare), the entries of E
// (launch_decode_entries), the product (launch_gemv). qw NULL: no base term;
// row_ptr NULL: no adapter term.
constexpr unsigned int kErrEntries = 0x8000u;  // a wait of the decode call gave up
struct GemvArgs {
  const uint8_t *qw;
  const float *scales;
  const uint8_t *zeros;
  int bits, group, d_out, d_in;
  const void *x;
  int T, f32;  // tokens, and whether x and y are fp32 (else bf16)
  void *y;
  const int32_t *row_ptr, *col_idx;
  const float *coef;
  int64_t p;
  float alpha;
  // Z = X H in fp32 by groups of tg tokens: zt [tp / tg][z_cols(d_in)][tg]; the entries' sums y_ad [d_out][tp].
  float *zt, *y_ad;
  int tg, tp;
  unsigned int *ready;  // 1 once the preparing launch is complete (beside zt)
  unsigned int *err;    // the device's error word
  // The values as operands, `pieces` columns a token, TPN = 8 / G columns to an n-tile (G groups in a chunk of 128
  // columns): xpieces [chunk][n-tile][4][TPN][4 runs] of 16 bytes, xfac [chunk][n-tile][8] factors.
  int pieces;
  uint4 *xpieces;  // NULL: the product makes them itself
  float *xfac;
  // Many columns instead (npad > 0): passes of tpp tokens, padded to npad columns; xpieces [pass][chunk][2][npad][128]
  // bytes, fac [T] the factors of fp32 tokens.
  int tpp, npad;
  float *fac;
  int prepared;  // another launch of the call precedes the product
};
// Columns of zt: those of the layer, and zeros for entries that count nothing (four keep copies to whole 16 bytes).
__host__ __device__ constexpr int z_cols(int d_in) { return d_in + 4; }
__host__ __device__ constexpr int x_tiles(int cols, int G) { return (cols * G + 7) / 8; }
bool gemv_on_tensor_cores(const uint8_t *qw, int group);
bool gemv_own_x(int32_t d_in, int64_t T, bool f32);  // whether a product by itself needs no prepared values
// Workspaces, and where in them the arrays lie.
size_t gemv_x_bytes(int32_t d_in, int64_t T, bool f32);
void gemv_place_x(GemvArgs *a, void *ws);
size_t gemv_z_bytes(int32_t d_out, int32_t d_in, int64_t T);
void gemv_place_z(GemvArgs *a, void *ws);
// Fills a.zt (if set), a.xpieces and its factors (if set) and z_out (if not NULL) from a.x.
cudaError_t launch_decode_prepare(const GemvArgs &a, int logn, void *z_out, cudaStream_t s);
cudaError_t launch_decode_entries(const GemvArgs &a, cudaStream_t s);
cudaError_t launch_gemv(const GemvArgs &a, cudaStream_t s);
// Its tensor-core kernels (gemv_mma.cuh).
cudaError_t launch_gemv_b2(const GemvArgs &a, cudaStream_t s);
cudaError_t launch_gemv_b3(const GemvArgs &a, cudaStream_t s);
cudaError_t launch_gemv_b4(const GemvArgs &a, cudaStream_t s);

// The quantized cache (cache.cu): up to two caches (keys and values) whose rows
// move in one launch. unit = 1/sqrt(had_block).
struct CachePair {
  qwha_cache cache[2];
  const void *rows[2];
  double unit[2];
};
// Bits of the device error word.
constexpr unsigned int kErrSlot = 0x1000u, kErrPage = 0x2000u;
int cache_max_head_dim();
// Launches of a call: a pair whose caches need different kernels takes two.
int cache_write_launches(qwha_dtype dt, const CachePair &c, int n_caches);
int cache_read_launches(const CachePair &c, int n_caches);
cudaError_t launch_cache_write(qwha_dtype dt, const CachePair &c, int n_caches, const int64_t *slots, int64_t n,
                               cudaStream_t s);
// Where the rows of a read come from (qwha_cache_read).
struct ReadArgs {
  const int32_t *pages;
  int max_pages, n_seqs;
  const int64_t *row_start, *first;
};
cudaError_t launch_cache_read(qwha_dtype dt, const CachePair &c, int n_caches, const ReadArgs &r, int64_t n,
                              cudaStream_t s);
size_t check_slots_bytes(int64_t n_slots);
cudaError_t launch_check_slots(const int64_t *slots, int64_t n, int64_t n_slots, void *ws, unsigned long long *bad,
                               cudaStream_t s);

// Rotary positions (rotary.cu).
struct RotaryArgs {
  const void *x[2];
  void *y[2];
  int64_t x_stride[2], y_stride[2];
  int heads[2];  // heads[1] 0: one tensor
  int head_dim, rot;
  int64_t n;
  const int64_t *positions;
  const double *freq;
  float factor;
  bool pairs, inverse;
};
cudaError_t launch_rotary(qwha_dtype dt, const RotaryArgs &r, cudaStream_t s);

// Page table and moves of cached rows (pages.cu).
constexpr unsigned int kErrTable = 0x4000u;  // rows of a table or of a move that were refused
size_t pages_workspace(int64_t n_seqs, int64_t n_pages, int64_t m);
// from, to: NULL, or where the pages to copy are named (the table is guarded then).
cudaError_t launch_pages_resize(const qwha_page_table &t, const int64_t *want, int32_t *from, int32_t *to, void *ws,
                                cudaStream_t s);
cudaError_t launch_pages_fork(const qwha_page_table &t, const int64_t *src, const int64_t *dst, int32_t m,
                              int32_t *from, int32_t *to, void *ws, cudaStream_t s);
cudaError_t launch_copy_pages(const CachePair &c, int n_caches, const int32_t *from, const int32_t *to, int32_t m,
                              cudaStream_t s);
cudaError_t launch_compact(const CachePair &c, int n_caches, const int32_t *pages, int32_t max_pages,
                           const int64_t *first, const int32_t *keep, int32_t width, int32_t n_seqs, cudaStream_t s);

// Attention over the quantized cache (attention.cu, attention.cuh).
struct AttnArgs {
  qwha_cache k, v;
  float unit_k, unit_v;  // 1 / sqrt(had_block)
  const void *q;
  int64_t q_stride, n;
  int q_heads, grp;  // query heads, and of one cached head
  const int32_t *pages;
  int max_pages;
  int cap;  // tokens the page table has room for
  int longest;  // of a sequence, as far as the host knows: chooses the kernel
  unsigned int page_mul;  // t / page_size = t page_mul >> page_shift for t below 2^31
  int page_shift;
  const int64_t *q_start, *past;
  int n_seqs;
  const int64_t *tree;
  float scale2;  // scale log2(e)
  void *out;
  float *lse;
  int f32;
  unsigned int *err;
  // How the work is cut (launch_attention).
  int tq, gh, parts;  // new tokens and query heads (of a cached head) of a tile; parts of the group
  int hb, blocks;     // cached heads of a CTA; blocks of heads times parts
  int kt_log2;        // cached tokens of a unit: a power of two
  int ctas;
  // Pieces of tiles that are cut between CTAs.
  int part_rows;
  float *part, *part_stats;
  int4 *part_desc;  // of CTA c: [2 c] and [2 c + 1]
};
size_t attention_workspace(int32_t q_heads, int32_t head_dim, int32_t heads, int64_t n, bool f32);
int attention_launches(const AttnArgs &a);
cudaError_t launch_attention(AttnArgs a, void *ws, cudaStream_t s);
// The tensor-core kernels (attention_mma.cuh): heads padded to 64, 128 or 256
// channels, tiles of 8 nt rows. grid, warps and the cut are the caller's.
struct MmaLaunch {
  int nt, warps, per_head, ctas;
  size_t smem;
};
cudaError_t launch_attention_d64(const AttnArgs &a, const MmaLaunch &l, cudaStream_t s);
cudaError_t launch_attention_d128(const AttnArgs &a, const MmaLaunch &l, cudaStream_t s);
cudaError_t launch_attention_d256(const AttnArgs &a, const MmaLaunch &l, cudaStream_t s);
// The tcgen05 kernel (attention_tc.cu): tiles of up to 256 rows, runs of 128 cached tokens.
constexpr int kTcRows = 256, kTcKeysLog2 = 7;
bool attention_tc_takes(const AttnArgs &a);
cudaError_t launch_attention_tc(const AttnArgs &a, cudaStream_t s);

}  // namespace qwha
