/*
 * Ragged-M grouped GEMM for AMD Instinct MI355X (gfx950) -- C ABI.
 *
 * One call computes E independent bf16 products with fp32 accumulation,
 *     C[off[e]:off[e+1], :] = A[off[e]:off[e+1], :] x B[e]      for e < E,
 * where the row count m_e = off[e+1] - off[e] of every group is read on the
 * device at run time and may be zero or heavily skewed. This is the
 * expert-FFN projection of a Mixture-of-Experts layer after routing, as
 * defined by "Grouped GEMM for Imbalanced Experts on Blackwell: A WIP
 * Worklog" (section "What I am measuring" and section 2, "The Grouped
 * Problem and the flat tile list") and by the InferenceX glossary entry
 * "Grouped GEMM" ("Technical definition"): rows arrive grouped by expert,
 * K and N are fixed, the group sizes are only known at run time, and every
 * expert's product runs in a single launch.
 *
 * Conventions shared by every entry point below:
 *  - All array pointers are DEVICE pointers owned by the caller; the library
 *    keeps no reference to them after the call returns and allocates no
 *    device memory.
 *  - `stream` is a hipStream_t passed as void* (NULL = the null stream). The
 *    call only enqueues work on it: no host synchronisation, no device to
 *    host copy. Results are ready when the stream reaches that point.
 *  - Errors the host can see (bad sizes, null or misaligned pointers,
 *    unsupported shapes) return a status and enqueue nothing.
 *  - Malformed offsets (off[0] != 0, decreasing entries, entries outside
 *    [0, M_cap]) are the caller's bug; they never make the kernel read or
 *    write outside A[0:M_cap], B[0:E] and C[0:M_cap]: every offset is clamped
 *    into [0, M_cap] and a group whose clamped end precedes its clamped start
 *    is treated as empty. Decreasing offsets can make clamped groups
 *    overlap; if the tiles of all groups then outnumber what M_cap rows can
 *    produce with nondecreasing offsets, ((M_cap / h) + E) * ceil(N / 256)
 *    for the smallest height h in use, the call computes nothing at all.
 *  - An output may not share memory with another array of the call (all
 *    but the forward products return GG_ERR_INVALID_VALUE; the two exceptions are
 *    named there).
 *  - Calls on different streams may run concurrently; the library holds no
 *    mutable state besides a per-device cache of launch limits.
 */
#ifndef MOE_RAGGED_GROUPED_AMD_GROUPED_GEMM_H
#define MOE_RAGGED_GROUPED_AMD_GROUPED_GEMM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GG_OK = 0,
  GG_ERR_INVALID_VALUE = 1, /* null pointer, non-positive size, bad bm, output over an array */
  GG_ERR_MISALIGNED = 2,    /* pointer not 16-byte aligned, K or N not 8k     */
  GG_ERR_UNSUPPORTED = 3,   /* E, K or N above its limit, or index range beyond int32 */
  GG_ERR_LAUNCH = 4         /* the HIP runtime refused the launch             */
} gg_status_t;

/* Largest number of groups one call accepts (the per-group tables live in LDS). */
#define GG_MAX_EXPERTS 1024
/* Largest K and N gg_grouped_gemm_bf16 accepts. */
#define GG_MAX_K (1 << 22)
#define GG_MAX_N (1 << 24)
/* Largest N of the data gradients, which sum over it. */
#define GG_MAX_DGRAD_N (1 << 21)

/*
 * gg_grouped_gemm_bf16 -- the grouped product (worklog section 2; glossary
 * "Technical definition").
 *
 *   A   bf16 [M_cap][K], row-major (K fastest). Rows are grouped by expert:
 *       rows off[e] .. off[e+1]-1 belong to expert e. Rows at or beyond
 *       off[E] are never read.
 *   B   bf16 [E][K][N], row-major (N fastest): B[e] is expert e's weight.
 *       The slice of an expert with no rows is never read.
 *   group_offsets  int32 [E+1] on the device: 0 = off[0] <= off[1] <= ...
 *       <= off[E] = M_tot <= M_cap.
 *   C   fp32 [M_cap][N], row-major. Rows [0, M_tot) are overwritten with the
 *       product (not accumulated into); rows [M_tot, M_cap) are not touched.
 *   E in [1, GG_MAX_EXPERTS]; K >= 8 and N >= 8, both multiples of 8;
 *   K <= GG_MAX_K and N <= GG_MAX_N (the kernels address a tile's A rows and
 *   a K slice of B with 32-bit byte offsets);
 *   M_cap >= 0 (0: nothing is enqueued).
 *   bm  tile height: 16, 32, 64, 128 or 256 for every expert, or 0 to let
 *       the device choose per expert from its row count (the trade between
 *       padding in the last tile and per-tile work that the worklog
 *       describes in sections 2.1, 6 and 7).
 *   A, B and C must be 16-byte aligned; group_offsets 4-byte aligned.
 *
 * Accumulation is fp32 inside the matrix cores; a result differs from the
 * exact sum by at most a few units of K * 2^-24 relative to sum_k |a*b|.
 */
gg_status_t gg_grouped_gemm_bf16(const void *A, const void *B, const int32_t *group_offsets,
                                 float *C, int32_t E, int32_t K, int32_t N, int32_t M_cap,
                                 int32_t bm, void *stream);

/*
 * gg_grouped_gemm_bf16_bf16out -- the same product with bf16 output C.
 *
 * The worklog's compulsory-traffic model (section 2.1, about 474 MB at 16k)
 * counts C as 2-byte values. Every argument and rule is that of
 * gg_grouped_gemm_bf16 except C:
 *   C   bf16 [M_cap][N], row-major, 16-byte aligned. Each element is the fp32
 *       matrix-core result rounded once to the nearest bf16 (ties to even),
 *       so it is within half a bf16 unit (2^-8 relative) of the fp32 result
 *       gg_grouped_gemm_bf16 returns for the same inputs, and equal to that
 *       result rounded to bf16.
 */
gg_status_t gg_grouped_gemm_bf16_bf16out(const void *A, const void *B,
                                         const int32_t *group_offsets, void *C, int32_t E,
                                         int32_t K, int32_t N, int32_t M_cap, int32_t bm,
                                         void *stream);

/*
 * gg_grouped_gemm_bf16_swiglu -- the gate and up projections with the SwiGLU
 * activation applied in the epilogue.
 *
 * The Pearl Pulse page "Pearl's grouped GEMM kernel for MoE models,
 * explained" (section "What the 15% measures") benchmarks the kernel on
 * the gate and up projections of MoE models; the activation between them
 * and the next projection is silu(gate) * up. Here B holds both projections
 * with their columns interleaved, so the product's two columns of one output
 * are computed by the same lane and need no exchange:
 *   B   bf16 [E][K][N], N = 2 * I: column 2j is gate column j and column
 *       2j+1 is up column j (a caller holding [W_gate | W_up] interleaves
 *       the columns once, when the weights are loaded).
 *   H   bf16 [M_cap][N/2], row-major, 16-byte aligned:
 *       H[r][j] = silu(C[r][2j]) * C[r][2j+1], silu(x) = x / (1 + e^-x),
 *       where C is the fp32 product gg_grouped_gemm_bf16 computes for the
 *       same inputs. The activation is evaluated in fp32 as
 *       x * rcp(1 + 2^(-x log2 e)) with the hardware exp2 and reciprocal,
 *       within (|gate| + 3.5) * 2^-23 of the exact value relative to first
 *       order (-0 for gate below about -87.3, where the reciprocal would be
 *       subnormal: less than 1.1e-36 * |up| is lost), and rounded once to the
 *       nearest bf16 (ties to even). Rows at or past off[E] are not written.
 * A, group_offsets, E, K, N, M_cap, bm, the stream, the status codes and
 * the conditions for them are those of gg_grouped_gemm_bf16 (N a multiple
 * of 8, so I is a multiple of 4).
 */
gg_status_t gg_grouped_gemm_bf16_swiglu(const void *A, const void *B,
                                        const int32_t *group_offsets, void *H, int32_t E,
                                        int32_t K, int32_t N, int32_t M_cap, int32_t bm,
                                        void *stream);

/*
 * gg_grouped_gemm_bf16_gather -- the product with the expert grouping done by
 * index instead of by copying rows (the worklog's "What I am measuring" puts
 * the token permutation on either side of the grouped GEMM; here it is folded
 * into the A loads and the C stores).
 *
 *   X         bf16 [n_src][K], row-major, 16-byte aligned: the unpermuted
 *             rows (e.g. token activations).
 *   src_rows  int32 [M_cap] on the device, 4-byte aligned: grouped row r
 *             (expert e owns grouped rows off[e] .. off[e+1]-1, exactly as
 *             in gg_grouped_gemm_bf16) reads its A row from X[src_rows[r]].
 *             An index outside [0, n_src) reads a row of zeros. Entries at
 *             or past off[E] are never read.
 *   dst_rows  int32 [M_cap] on the device, 4-byte aligned, or NULL: grouped
 *             row r is written to C row dst_rows[r]; an index outside
 *             [0, M_cap) is not written. With NULL, grouped row r is written
 *             to C row r, as in gg_grouped_gemm_bf16. Two grouped rows that
 *             name the same C row race (either result may land).
 *   C         fp32 [M_cap][N], row-major; rows no grouped row names are not
 *             touched.
 *   n_src >= 0 and n_src * K * 2 <= 2^31 (GG_ERR_UNSUPPORTED otherwise).
 * The other arguments, rules and the accuracy are those of
 * gg_grouped_gemm_bf16. The result equals gg_grouped_gemm_bf16 applied to
 * A = X[src_rows] followed by C[dst_rows[r]] = C_grouped[r].
 */
gg_status_t gg_grouped_gemm_bf16_gather(const void *X, int32_t n_src, const int32_t *src_rows,
                                        const void *B, const int32_t *group_offsets, float *C,
                                        const int32_t *dst_rows, int32_t E, int32_t K, int32_t N,
                                        int32_t M_cap, int32_t bm, void *stream);

/*
 * gg_grouped_gemm_bf16_gather_combine -- the gathered product with the
 * weighted combine folded into the epilogue.
 *
 * After the expert products, each token's routed rows are weighted and
 * summed back into the token's row (the worklog's "What I am measuring"
 * places the permutation on either side of the grouped GEMM; the InferenceX
 * glossary's "Engineering details" name the weighted combine). Here:
 *   Y[dst_rows[r]][n] += row_weights[r] * C[r][n]
 * for every grouped row r < off[E] whose destination lies in [0, n_dst),
 * where C[r] is the product gg_grouped_gemm_bf16_gather computes for that
 * row (A row X[src_rows[r]], weights B[e] of its expert).
 *   X, n_src, src_rows, B, group_offsets, E, K, N, M_cap, bm, stream: as in
 *             gg_grouped_gemm_bf16_gather.
 *   dst_rows     int32 [M_cap] on the device, 4-byte aligned, required.
 *                Several grouped rows may name the same Y row (top-k).
 *   row_weights  fp32 [M_cap] on the device, 4-byte aligned, required.
 *   Y            fp32 [n_dst][N], row-major, 16-byte aligned, in device
 *                memory (hipMalloc; the adds are the GPU's fp32 atomics):
 *                accumulated into, not overwritten -- clear it first for a
 *                plain combine. Rows no grouped row names keep their values.
 *   n_dst >= 0.
 * Each term is the fp32 product row times its weight, rounded once; the
 * terms meeting in one element are added with fp32 atomic adds in an
 * unspecified order, so the result may differ between runs by the rounding
 * of that order (the product itself is as accurate as gg_grouped_gemm_bf16).
 * Status codes as for gg_grouped_gemm_bf16_gather; a null dst_rows or
 * row_weights, or n_dst < 0, is GG_ERR_INVALID_VALUE.
 */
gg_status_t gg_grouped_gemm_bf16_gather_combine(const void *X, int32_t n_src,
                                                const int32_t *src_rows, const void *B,
                                                const int32_t *group_offsets,
                                                const int32_t *dst_rows,
                                                const float *row_weights, float *Y, int32_t n_dst,
                                                int32_t E, int32_t K, int32_t N, int32_t M_cap,
                                                int32_t bm, void *stream);

/*
 * gg_grouped_gemm_fp8w -- the product with fp8 weights and per-column scales
 * (the Pearl Pulse page, "What the 15% measures", notes that its kernel
 * ships with an FP8 scheme; the scheme below is this library's reading).
 *
 *   C[r][n] = scale[e][n] * sum_k A[r][k] * dec(Bq[e][k][n])   for r in group e
 *
 *   A        bf16 [M_cap][K], as in gg_grouped_gemm_bf16.
 *   Bq       uint8 [E][K][N], row-major, 16-byte aligned: OCP fp8 E4M3 codes
 *            (1 sign, 4 exponent bits with bias 7, 3 mantissa bits; 0x7F and
 *            0xFF are NaN; largest finite magnitude 448).
 *   b_scale  fp32 [E][N] on the device, 16-byte aligned: one scale per expert
 *            and output column.
 *   C        fp32 [M_cap][N].
 * The weights stay fp8 in LDS and each is widened exactly to bf16 as the
 * matrix cores' operand is read from there; the products accumulate in fp32
 * in the bf16 matrix cores, and the epilogue multiplies by the column scale
 * (one more fp32 rounding). Weight bytes in HBM are halved;
 * this is a separate precision from gg_grouped_gemm_bf16, not a replacement.
 * Other arguments and rules are those of gg_grouped_gemm_bf16; b_scale NULL
 * is GG_ERR_INVALID_VALUE, misaligned b_scale GG_ERR_MISALIGNED.
 */
gg_status_t gg_grouped_gemm_fp8w(const void *A, const void *Bq, const float *b_scale,
                                 const int32_t *group_offsets, float *C, int32_t E, int32_t K,
                                 int32_t N, int32_t M_cap, int32_t bm, void *stream);

/*
 * gg_grouped_gemm_fp8 -- fp8 activations and fp8 weights on the fp8 matrix
 * cores (the article's FP8 scheme, read as one scale per activation row and
 * one per weight column).
 *
 *   C[r][n] = a_scale[r] * b_scale[e][n] * sum_k dec(Aq[r][k]) * dec(Bq[e][k][n])
 *
 *   Aq       uint8 [M_cap][K], row-major, 16-byte aligned: E4M3 codes, rows
 *            grouped by expert as A in gg_grouped_gemm_bf16.
 *   a_scale  fp32 [M_cap] on the device, 4-byte aligned: one scale per row.
 *   Bq       uint8 [E][K][N], 16-byte aligned: E4M3 codes, as for
 *            gg_grouped_gemm_fp8w.
 *   b_scale  fp32 [E][N], 16-byte aligned: one scale per expert and column.
 *   C        fp32 [M_cap][N].
 *   K and N must be multiples of 16 (GG_ERR_MISALIGNED otherwise).
 * The products of two E4M3 values are exact; they accumulate in fp32 in the
 * matrix cores (v_mfma_scale_f32_16x16x128_f8f6f4 with unit block scales),
 * and the epilogue multiplies by the row and the column scale (two fp32
 * roundings). Other arguments and rules are those of gg_grouped_gemm_bf16;
 * a NULL scale pointer is GG_ERR_INVALID_VALUE.
 */
gg_status_t gg_grouped_gemm_fp8(const void *Aq, const float *a_scale, const void *Bq,
                                const float *b_scale, const int32_t *group_offsets, float *C,
                                int32_t E, int32_t K, int32_t N, int32_t M_cap, int32_t bm,
                                void *stream);

/*
 * gg_grouped_gemm_fp8_bf16out -- gg_grouped_gemm_fp8 with bf16 output: C is
 * bf16 [M_cap][N], 16-byte aligned, each element the fp32 result of
 * gg_grouped_gemm_fp8 (scales applied) rounded once to the nearest bf16
 * (ties to even). Every other argument and rule is that of
 * gg_grouped_gemm_fp8.
 */
gg_status_t gg_grouped_gemm_fp8_bf16out(const void *Aq, const float *a_scale, const void *Bq,
                                        const float *b_scale, const int32_t *group_offsets,
                                        void *C, int32_t E, int32_t K, int32_t N, int32_t M_cap,
                                        int32_t bm, void *stream);

/*
 * gg_grouped_gemm_fp8_swiglu -- gg_grouped_gemm_fp8 for the gate and up
 * projections with the SwiGLU of gg_grouped_gemm_bf16_swiglu in the
 * epilogue: Bq's columns interleave gate (even) and up (odd), and
 *   H[r][j] = silu(C[r][2j]) * C[r][2j+1]   (bf16 [M_cap][N/2], 16-byte aligned)
 * where C is the scaled fp32 result gg_grouped_gemm_fp8 computes. The
 * activation and its rounding are those of gg_grouped_gemm_bf16_swiglu;
 * every other argument and rule is that of gg_grouped_gemm_fp8.
 */
gg_status_t gg_grouped_gemm_fp8_swiglu(const void *Aq, const float *a_scale, const void *Bq,
                                       const float *b_scale, const int32_t *group_offsets,
                                       void *H, int32_t E, int32_t K, int32_t N, int32_t M_cap,
                                       int32_t bm, void *stream);

/*
 * gg_grouped_gemm_bf16_dgrad -- the data gradient of the grouped product: with
 * dC the gradient of C = gg_grouped_gemm_bf16(A, B),
 *
 *   dA[r][k] = sum_n dC[r][n] * B[e][k][n]          for the rows r of expert e
 *
 *   dC  bf16 [M_cap][N], row-major, 16-byte aligned, rows grouped by expert as
 *       A's in the product. Rows at or beyond off[E] are never read.
 *   B   bf16 [E][K][N], the weights exactly as the product takes them (nothing
 *       is transposed beforehand). The slice of an expert with no rows is
 *       never read.
 *   dA  fp32 [M_cap][K], 16-byte aligned. Rows [0, off[E]) are overwritten;
 *       rows past them are not touched.
 * group_offsets, E, M_cap, bm, the stream, the status codes and the conditions
 * for them are those of gg_grouped_gemm_bf16 with K in the place of its N
 * (arrays of no rows, M_cap = 0, may be NULL here and below); K and N are
 * multiples of 8, N <= GG_MAX_DGRAD_N and K <= GG_MAX_N (the sum runs over N
 * here). Malformed offsets whose groups overlap compute nothing where their
 * row tiles outnumber M_cap / h + E (h = bm, or 16 for bm = 0).
 * Accumulation is fp32 in the matrix cores, as accurate as the product's with
 * N in the place of K.
 */
gg_status_t gg_grouped_gemm_bf16_dgrad(const void *dC, const void *B,
                                       const int32_t *group_offsets, float *dA, int32_t E,
                                       int32_t K, int32_t N, int32_t M_cap, int32_t bm,
                                       void *stream);

/*
 * gg_grouped_gemm_bf16_dgrad_bf16out -- the same with dA bf16 [M_cap][K], each
 * element the fp32 result rounded once to the nearest bf16 (ties to even).
 */
gg_status_t gg_grouped_gemm_bf16_dgrad_bf16out(const void *dC, const void *B,
                                               const int32_t *group_offsets, void *dA, int32_t E,
                                               int32_t K, int32_t N, int32_t M_cap, int32_t bm,
                                               void *stream);

/*
 * gg_grouped_gemm_bf16_dgrad_swiglu -- the data gradient of the down projection
 * taken through the SwiGLU before it, in one launch. An expert's layer is
 *   C = X B1 (gate in column 2j, up in column 2j+1),  H = silu(gate) * up,
 *   Y = H B2;
 * given dY, this entry point computes dH = dY B2^T (in fp32, never stored) and
 *   dC[r][2j]   = dH[r][j] * up * s * (1 + gate * (1 - s)),  s = 1 / (1 + e^-gate)
 *   dC[r][2j+1] = dH[r][j] * gate * s
 *   H[r][j]     = gate * s * up                    (where H is not NULL)
 *
 *   dY  bf16 [M_cap][N];  B  bf16 [E][K][N], the down projection (K = the width
 *       of H);  C  bf16 [M_cap][2K], the gate and up columns interleaved, as
 *       gg_grouped_gemm_bf16_bf16out gives them;
 *   dC  bf16 [M_cap][2K], and H bf16 [M_cap][K] or NULL: the operand of the down
 *       projection's weight gradient, which a forward pass that kept only C has
 *       not stored. dC may be C itself, from its start. Rows at or beyond off[E]
 *       of C are not read, of dC and H not written. All are 16-byte aligned.
 * Everything is evaluated in fp32 (hardware exp2 and reciprocal, each within one
 * ulp) and rounded once to bf16 on its way out. s is 0 where it would be subnormal
 * (gate below about -87.3); dC and H then are 0, off by less than 1.1e-36 *
 * |dH * up|, 1.1e-36 * |dH| and 1.1e-36 * |up|. An infinite gate gives NaN.
 * Sizes, offsets, bm, the stream and the status codes are those of
 * gg_grouped_gemm_bf16_dgrad.
 */
gg_status_t gg_grouped_gemm_bf16_dgrad_swiglu(const void *dY, const void *B,
                                              const int32_t *group_offsets, const void *C, void *dC,
                                              void *H, int32_t E, int32_t K, int32_t N,
                                              int32_t M_cap, int32_t bm, void *stream);

/*
 * gg_grouped_gemm_bf16_wgrad -- the weight gradient of the grouped product:
 *
 *   dB[e][k][n] = sum over the rows r of expert e of A[r][k] * dC[r][n]
 *
 *   A   bf16 [M_cap][K] and dC bf16 [M_cap][N], row-major, 16-byte aligned, rows
 *       grouped by expert. Rows at or beyond off[E] are never read. Both may be
 *       NULL where M_cap is 0.
 *   dB  fp32 [E][K][N], 16-byte aligned. Every element is written: an expert
 *       with no rows gets zeros. With accumulate != 0 the sums are added to what
 *       dB holds (each element by one fp32 addition), and experts with no rows
 *       are left as they are.
 *   group_offsets  int32 [E+1] on the device. Malformed offsets never make the
 *       kernel read or write outside its arrays (they are clamped as in
 *       gg_grouped_gemm_bf16).
 *   K and N are multiples of 8, at most GG_MAX_K; E in [1, GG_MAX_EXPERTS];
 *   M_cap in [0, 2^31 - 257]; E * 8 * ceil(ceil(K/128) * ceil(N/256) / 8) < 2^24
 *   (GG_ERR_UNSUPPORTED beyond; a launch counts its threads in 32 bits).
 * The sum over an expert's rows is taken in fp32 in the matrix cores, with no
 * atomics, in an order that E, K, N, M_cap and the expert's row count fix: equal
 * arguments give equal bits. M_cap takes part (its mean per expert chooses
 * between two tiles), so the same groups in a longer buffer may differ in the
 * last places.
 */
gg_status_t gg_grouped_gemm_bf16_wgrad(const void *A, const void *dC,
                                       const int32_t *group_offsets, float *dB,
                                       int32_t accumulate, int32_t E, int32_t K, int32_t N,
                                       int32_t M_cap, void *stream);

/*
 * gg_grouped_gemm_bf16_wgrad_bf16out -- the same with dB bf16 [E][K][N], each
 * element the fp32 sum rounded once to the nearest bf16 (ties to even). There
 * is no accumulating form: sums held in bf16 would lose what is added to them.
 */
gg_status_t gg_grouped_gemm_bf16_wgrad_bf16out(const void *A, const void *dC,
                                               const int32_t *group_offsets, void *dB, int32_t E,
                                               int32_t K, int32_t N, int32_t M_cap, void *stream);

/*
 * 4-bit microscaled operands ("mx4", the OCP Microscaling format MXFP4). Blocks
 * of 32 values along K share a scale 2^(s - 127), s a byte (E8M0; 255 is NaN).
 * A value is a 4-bit E2M1 code: bit 3 the sign, codes 0..7 the magnitudes
 * 0, 0.5, 1, 1.5, 2, 3, 4, 6.
 *   codes   uint8 [rows][K/2]: byte j of a row holds k = 2j in its low half and
 *           k = 2j + 1 in its high half.
 *   scales  uint8 [ceil(K/256)][rows][8]: the block of k = 32 b .. 32 b + 31 of
 *           row r has its scale at [b / 8][r][b % 8]. (A tile's scales of one
 *           slice of 256 k are then one run of memory.) Bytes past the last
 *           block are ignored by every entry point and written as 0.
 * Weights are kept per expert with the output columns as rows: codes
 * [E][N][K/2], scales [E][ceil(K/256)][N][8]. K is a multiple of 32.
 *
 * gg_mx4_quantize -- X bf16 [rows][K] to codes and scales. A block's scale is
 * 2^(floor(log2 max|x|) - 2), at least 2^-127; x over the scale goes to the
 * nearest value, ties to the even code, and magnitudes over 6 become 6 (the
 * format's own rule: the largest values of a block may be up to 8 scales). A
 * block of zeros gets scale byte 0. A block that holds an infinity or a NaN
 * gets scale byte 255 and codes 0, and so stands for NaN throughout.
 * X, q and scales are 16-byte aligned; rows in [0, 2^31 - 1], K <= GG_MAX_K,
 * rows * K <= 2^37 - 2^13 (GG_ERR_UNSUPPORTED beyond; a launch counts its
 * threads in 32 bits).
 */
gg_status_t gg_mx4_quantize(const void *X, void *q, void *scales, int64_t rows, int32_t K,
                            void *stream);

/*
 * gg_mx4_quantize_weights -- B bf16 [E][K][N] (the layout of the bf16 product)
 * to codes [E][N][K/2] and scales [E][ceil(K/256)][N][8], blocks along K, by the
 * rule of gg_mx4_quantize. N is a multiple of 8, at most GG_MAX_N, and E *
 * ceil(K/256) * ceil(N/256) < 2^23.
 */
gg_status_t gg_mx4_quantize_weights(const void *B, void *q, void *scales, int32_t E, int32_t K,
                                    int32_t N, void *stream);

/*
 * gg_mx4_dequantize -- the values that codes and scales stand for:
 * Y bf16 [batch][rows][K] from codes [batch][rows][K/2] and scales
 * [batch][ceil(K/256)][rows][8] (batch = E and rows = N for weights, batch = 1
 * for activations). Every such value is a bf16 value except 4 and 6 times
 * 2^127 (scale byte 254), which become infinite; scale byte 255 gives NaN.
 * batch in [0, 65535]; rows in [0, 2^31 - 1]; rows * K <= 2^37 - 2^13.
 */
gg_status_t gg_mx4_dequantize(const void *q, const void *scales, void *Y, int32_t batch,
                              int64_t rows, int32_t K, void *stream);

/*
 * gg_grouped_gemm_mx4 -- the grouped product of 4-bit microscaled activations
 * and weights on the matrix cores' own 4-bit format:
 *
 *   C[r][n] = sum_k val(Aq, a_scale)[r][k] * val(Bq, b_scale)[e][n][k]
 *
 *   Aq, a_scale  codes uint8 [M_cap][K/2] and scales uint8 [ceil(K/256)][M_cap][8].
 *                Codes of rows at or beyond off[E] are never used.
 *   Bq, b_scale  codes uint8 [E][N][K/2] and scales uint8 [E][ceil(K/256)][N][8].
 *   C            fp32 [M_cap][N]. Rows at or beyond off[E] are not touched.
 * K is a multiple of 32 and at most GG_MAX_K, N a multiple of 8 and at most
 * GG_MAX_N; all pointers but group_offsets (4) are 16-byte aligned. Offsets, E,
 * M_cap, bm, the stream and the status codes are those of gg_grouped_gemm_bf16.
 * Products of two values are exact and accumulate in fp32; a NaN scale makes the
 * row's or the column's results NaN.
 */
gg_status_t gg_grouped_gemm_mx4(const void *Aq, const void *a_scale, const void *Bq,
                                const void *b_scale, const int32_t *group_offsets, float *C,
                                int32_t E, int32_t K, int32_t N, int32_t M_cap, int32_t bm,
                                void *stream);

/*
 * gg_grouped_gemm_mx4_bf16out -- the same with C bf16 [M_cap][N], each element
 * the fp32 result rounded once to the nearest bf16 (ties to even).
 */
gg_status_t gg_grouped_gemm_mx4_bf16out(const void *Aq, const void *a_scale, const void *Bq,
                                        const void *b_scale, const int32_t *group_offsets, void *C,
                                        int32_t E, int32_t K, int32_t N, int32_t M_cap, int32_t bm,
                                        void *stream);

/*
 * gg_grouped_gemm_mx4_swiglu -- gg_grouped_gemm_mx4 for the gate and up
 * projections, N = 2 I interleaved columns, with the SwiGLU of
 * gg_grouped_gemm_bf16_swiglu in the epilogue: H bf16 [M_cap][N/2].
 */
gg_status_t gg_grouped_gemm_mx4_swiglu(const void *Aq, const void *a_scale, const void *Bq,
                                       const void *b_scale, const int32_t *group_offsets, void *H,
                                       int32_t E, int32_t K, int32_t N, int32_t M_cap, int32_t bm,
                                       void *stream);

/*
 * 8-bit operands with a scale for each block of 128 ("fp8_block"). A value is an
 * OCP E4M3 code (1 sign, 4 exponent and 3 mantissa bits, 448 at most) times its
 * block's fp32 scale.
 *   rows     codes uint8 [rows][K], scales fp32 [ceil(K/128)][rows]: one scale for
 *            128 values along K, those of a slice of 128 k side by side.
 *   weights  codes uint8 [E][N][K] (output columns as rows), scales fp32
 *            [E][ceil(N/128)][ceil(K/128)]: one scale for 128 x 128 values.
 *
 * gg_fp8_quantize -- X bf16 [rows][K] to codes and scales. With top the largest
 * magnitude of a block, counted as 2^-100 at least, and m = 448 / top cut to 16
 * significant bits, a value's code is the one nearest to x * m (which is exact in
 * fp32), ties to even, and the block's scale is 1 / m. A block that holds an
 * infinity or a NaN gets scale NaN and codes 0, and so stands for NaN throughout.
 * K is a multiple of 16, at most GG_MAX_K; rows in [0, 2^31 - 1]; ceil(rows/32) *
 * ceil(K/512) < 2^23 (GG_ERR_UNSUPPORTED beyond; a launch counts its threads in 32
 * bits). X, q and scales are 16-byte aligned.
 */
gg_status_t gg_fp8_quantize(const void *X, void *q, float *scales, int64_t rows, int32_t K,
                            void *stream);

/*
 * gg_fp8_quantize_weights -- B bf16 [E][K][N] (the layout of the bf16 product) to
 * codes and scales by the rule of gg_fp8_quantize, a block being 128 x 128 values.
 *   for_grad == 0: codes [E][N][K], scales [E][ceil(N/128)][ceil(K/128)], what
 *     gg_grouped_gemm_fp8_block takes; K a multiple of 16, N of 8.
 *   for_grad != 0: codes [E][K][N], scales [E][ceil(K/128)][ceil(N/128)], the same
 *     values with K and N exchanged: what the same entry point takes for the data
 *     gradient dA = dC B^T (its K is then this N); N a multiple of 16, K of 8.
 * The summed dimension is at most GG_MAX_K, the other at most GG_MAX_N, and
 * E * ceil(K/128) * ceil(N/128) < 2^24.
 */
gg_status_t gg_fp8_quantize_weights(const void *B, void *q, float *scales, int32_t for_grad,
                                    int32_t E, int32_t K, int32_t N, void *stream);

/*
 * gg_grouped_gemm_fp8_block -- the grouped product of 8-bit rows and weights with
 * a scale for each block of 128:
 *
 *   C[r][n] = sum_b a_scale[b][r] * b_scale[e][n / 128][b] *
 *             sum_{k in block b} dec(Aq[r][k]) * dec(Bq[e][n][k])
 *
 *   Aq, a_scale  codes uint8 [M_cap][K] and scales fp32 [ceil(K/128)][M_cap].
 *                Rows at or beyond off[E] are never used.
 *   Bq, b_scale  codes uint8 [E][N][K] and scales fp32 [E][ceil(N/128)][ceil(K/128)].
 *                The scales are any fp32 numbers, not only what the quantiser makes, and
 *                the product of a row's and the columns' may lie beyond fp32 (those
 *                rows are computed again, 50 to 150 times as slowly). Where it lies
 *                below fp32's normal numbers, what the block adds is off by up to 2^-125
 *                besides.
 *   C            fp32 [M_cap][N]. Rows at or beyond off[E] are not touched.
 * K is a multiple of 16 and at most GG_MAX_K, N a multiple of 8 and at most
 * GG_MAX_N; all pointers but group_offsets (4) are 16-byte aligned. Offsets, E,
 * M_cap, bm, the stream and the status codes are those of gg_grouped_gemm_bf16.
 * A block's products are summed on the fp8 matrix cores, which align 8 neighbouring
 * products to the largest of them and drop what is 2^-14 of it or smaller; blocks
 * are scaled and added in fp32. A NaN scale makes the row's or the columns'
 * results NaN.
 */
gg_status_t gg_grouped_gemm_fp8_block(const void *Aq, const float *a_scale, const void *Bq,
                                      const float *b_scale, const int32_t *group_offsets, float *C,
                                      int32_t E, int32_t K, int32_t N, int32_t M_cap, int32_t bm,
                                      void *stream);

/*
 * gg_grouped_gemm_fp8_block_bf16out -- the same with C bf16 [M_cap][N], each
 * element the fp32 result rounded once to the nearest bf16 (ties to even).
 */
gg_status_t gg_grouped_gemm_fp8_block_bf16out(const void *Aq, const float *a_scale, const void *Bq,
                                              const float *b_scale, const int32_t *group_offsets,
                                              void *C, int32_t E, int32_t K, int32_t N,
                                              int32_t M_cap, int32_t bm, void *stream);

/*
 * gg_grouped_gemm_fp8_block_swiglu -- gg_grouped_gemm_fp8_block for the gate and
 * up projections, N = 2 I interleaved columns, with the SwiGLU of
 * gg_grouped_gemm_bf16_swiglu in the epilogue: H bf16 [M_cap][N/2].
 */
gg_status_t gg_grouped_gemm_fp8_block_swiglu(const void *Aq, const float *a_scale, const void *Bq,
                                             const float *b_scale, const int32_t *group_offsets,
                                             void *H, int32_t E, int32_t K, int32_t N,
                                             int32_t M_cap, int32_t bm, void *stream);

/*
 * gg_expert_sort -- the choices of a router, T tokens of k experts each, grouped by
 * expert: the row lists that the grouped products take.
 *
 *   experts  int32 [T][k], or int64 where `wide` is not 0: the chosen experts. A
 *            choice outside [0, E) is of no expert here (of another rank, or none)
 *            and gets no row.
 *   weights  fp32 [T][k], or NULL (then row_weights is NULL too).
 *   offsets  int32 [E+1]: expert e has rows offsets[e] .. offsets[e+1]-1, in the
 *            order of its choices (by token, then by place).
 *   rows     int32 [T*k]: each row's token. -1 past offsets[E].
 *   pos      int32 [T][k]: each choice's row, -1 where it has none.
 *   row_weights  fp32 [T*k]: each row's weight. 0 past offsets[E].
 *   workspace  gg_expert_sort_workspace(T * k, E) bytes of device memory, 16-byte
 *            aligned (0 bytes: may be NULL). Its contents are used during the call only.
 * T * k <= 2^31 - 1; k >= 1; E in [1, GG_MAX_EXPERTS]. Pointers are aligned to their
 * elements. (src_rows and, for a combine, dst_rows of gg_grouped_gemm_bf16_gather
 * and _gather_combine are both `rows`, row_weights theirs.)
 */
int64_t gg_expert_sort_workspace(int64_t choices, int32_t E);
gg_status_t gg_expert_sort(const void *experts, int32_t wide, const float *weights, int32_t *offsets,
                           int32_t *rows, int32_t *pos, float *row_weights, void *workspace, int64_t T,
                           int32_t k, int32_t E, void *stream);

/*
 * gg_expert_spread -- each token's row to the rows of its choices:
 * out[pos[t][j]] = X[t] for every pos[t][j] in [0, M_cap); other choices are
 * skipped, and rows that no choice names are not touched. A row that two choices name
 * is undefined, and so are its scales: parts of both tokens', not one of the two.
 *   X, out   [T] and [M_cap] rows of row_bytes bytes, a multiple of 16; 16-byte
 *            aligned. Any type: bytes are moved.
 *   scales, out_scales  block scales that go with the rows, [slices][T] and
 *            [slices][M_cap] elements of scale_bytes: 4 (fp8_block), 8 (mx4), or 0
 *            with slices 0 and both pointers unused. 16-byte aligned.
 * T * ceil(row_bytes / 4096) / 4, and with scales ceil(T / 256) * 8 * ceil(slices /
 * 32) besides, stay below 2^24 (GG_ERR_UNSUPPORTED beyond).
 * Its gradient is gg_expert_combine without weights.
 */
gg_status_t gg_expert_spread(const void *X, const int32_t *pos, void *out, const void *scales,
                             void *out_scales, int32_t scale_bytes, int64_t T, int32_t k,
                             int64_t row_bytes, int32_t slices, int64_t M_cap, void *stream);

/*
 * gg_expert_combine -- each token's rows, weighted and summed:
 *   out[t][n] = sum_j weights[t][j] * Y[pos[t][j]][n]   over the j with pos in [0, M_cap)
 *   Y        [M_cap][N], fp32 where y_fp32 is not 0, else bf16; out [T][N], fp32 where
 *            out_fp32 is not 0, else bf16; both 16-byte aligned. N a multiple of 8.
 *   weights  fp32 [T][k], or NULL for weights of 1.
 * A token with no rows gets zeros. The sum is taken in fp32 in the order of j, one
 * fused multiply-add a term (no atomics: equal inputs give equal bits), and rounded
 * once. N <= GG_MAX_N; T * ceil(N/512) < 2^26.
 */
gg_status_t gg_expert_combine(const void *Y, int32_t y_fp32, const int32_t *pos, const float *weights,
                              void *out, int32_t out_fp32, int64_t T, int32_t k, int32_t N,
                              int64_t M_cap, void *stream);

/*
 * gg_expert_combine_grad -- the gradient of gg_expert_combine: given dO [T][N],
 *   dY[pos[t][j]][n] = weights[t][j] * dO[t][n]
 *   dweights[t][j]   = sum_n dO[t][n] * Y[pos[t][j]][n]     (0 where pos is not in [0, M_cap))
 * dO, Y and dY are all fp32 (fp32 != 0) or all bf16. Rows of dY that no choice names
 * are not touched; a row that two choices name is undefined (parts of both). Products and sums are
 * in fp32, dY is rounded once, dweights is fp32 [T][k] summed in a fixed order.
 * N is a multiple of 8, N <= GG_MAX_N, T < 2^24.
 */
gg_status_t gg_expert_combine_grad(const void *dO, const void *Y, int32_t fp32, const int32_t *pos,
                                   const float *weights, void *dY, float *dweights, int64_t T,
                                   int32_t k, int32_t N, int64_t M_cap, void *stream);

/*
 * gg_rms_norm_fp8 -- root-mean-square norm of X + residual, in 8 bits:
 *   z = bf16(X + residual)  (X where residual is NULL),
 *   y = z / sqrt(mean z^2 + eps) * weight,
 *   q, scales = y by the rule of gg_fp8_quantize, from its fp32 values.
 *   X, residual  bf16 [T][K], residual or NULL; weight bf16 [K].
 *   q, scales    uint8 [T][K], fp32 [ceil(K/128)][T].
 *   sum          bf16 [T][K]: z, the next residual; or NULL. Needs a residual. May be
 *                X or residual itself, from its start.
 *   norm         bf16 [T][K]: y rounded once; or NULL.
 * K is a multiple of 16, at most 16384; T in [0, 2^24 - 2]; eps >= 0; everything
 * 16-byte aligned. Rows and weights may lie anywhere in bf16's range: what leaves fp32
 * on the way does no harm where y does not. A row that holds an infinity or a NaN, or
 * zeros alone with eps = 0, has NaN in the blocks where y is not finite.
 */
gg_status_t gg_rms_norm_fp8(const void *X, const void *residual, const void *weight, void *q,
                            float *scales, void *sum, void *norm, int64_t T, int32_t K, float eps,
                            void *stream);

/*
 * gg_rms_norm_grad -- the gradient of y = z / sqrt(mean z^2 + eps) * weight (for
 * y in 8 bits, that of the values before they were rounded): with r = 1 /
 * sqrt(mean z^2 + eps) and u = weight * dY,
 *   dZ = r * (u - z * r^2 * mean(u * z)) + d_residual,
 *   dweight[c] = sum_t dY[t][c] * z[t][c] * r[t].
 *   dY, Z, d_residual, dZ  bf16 [T][K]; d_residual, the gradient that reaches z
 *            past the norm, or NULL. dZ is rounded once.
 *   weight   bf16 [K];  dweight fp32 [K], overwritten, summed in an order that T and
 *            K fix (no atomics).
 *   workspace  gg_rms_norm_grad_workspace(T, K) bytes of device memory, used during
 *            the call only.
 * Rows, gradients and weights may lie anywhere in bf16's range: squares, products and
 * powers of r that leave fp32 do no harm where the results do not (z * r is an fp32
 * number).
 * Sizes and alignment are those of gg_rms_norm_fp8.
 */
int64_t gg_rms_norm_grad_workspace(int64_t T, int32_t K);
gg_status_t gg_rms_norm_grad(const void *dY, const void *Z, const void *weight, const void *d_residual,
                             void *dZ, float *dweight, void *workspace, int64_t T, int32_t K, float eps,
                             void *stream);

/*
 * gg_tile_schedule -- the flat tile list the product kernel consumes,
 * written out (worklog section 2: one descriptor per output tile of one
 * expert, expert-major order, tiles stopping at expert boundaries, empty
 * experts contributing none).
 *
 * The device builds it from group_offsets with exactly the code the product
 * kernel runs; tile t of the list is written as 5 int32
 *     tiles[5t .. 5t+4] = { expert, row0, rows, col0, bm }
 * in the order the product kernel walks tile ids. The set of descriptors is
 * the worklog's; the order is expert by expert, and inside an expert the M
 * tiles are taken in groups of up to 8 with the N tile outer and the M tile
 * inner in each group (so consecutive tiles share a column slice of the
 * expert's weights). Tiles are 256 columns wide, except when every expert
 * with rows has 16-row tiles: then they are 512 wide. At most
 * max_tiles descriptors are written; *n_tiles (a device int32) receives the
 * full count even when it exceeds max_tiles (0 for malformed offsets whose
 * overlapping groups exceed the bound stated at the top of this file).
 * Arguments E, N, M_cap, bm and the offsets rules are those of
 * gg_grouped_gemm_bf16; tiles may be NULL when max_tiles == 0.
 */
gg_status_t gg_tile_schedule(const int32_t *group_offsets, int32_t E, int32_t N, int32_t M_cap,
                             int32_t bm, int32_t *tiles, int32_t *n_tiles, int32_t max_tiles,
                             void *stream);

/* Static English text for a status code. */
const char *gg_status_string(gg_status_t status);

#ifdef __cplusplus
}
#endif

#endif /* MOE_RAGGED_GROUPED_AMD_GROUPED_GEMM_H */
