/*
 * ts_nvfp4_moe.h: C ABI of the NVFP4 operators (quantise, read back, matrix
 * product) and of the expert-routing operators (token rows sorted by expert,
 * the experts' NVFP4 products, the weighted sum back and its gradient) on one
 * GB300 (sm_103a).
 *
 * They take up where the fused epilogues of ts_fused_norm.h end: patterns 3
 * and 5 there write NVFP4 codes and scale factors, which ts_nvfp4_gemm
 * multiplies; ts_moe_combine writes a partial that the next fused call reduces.
 *
 * Conventions: those of ts_fused_norm.h (caller-owned buffers, host-side
 * checks before any launch, one kernel per call on `stream`, statuses,
 * ts_last_error_detail, TS_FLAG_PDL, no allocation and no synchronisation),
 * with these additions:
 *   - Buffers may be in device memory or in page-locked host memory, except
 *     the operands and the output of ts_nvfp4_gemm and ts_nvfp4_grouped_gemm,
 *     which the tensor copy engine reads and writes and which live in device
 *     memory (alpha and the experts' starts and counts may be in either).
 *   - NVFP4 matrices: codes uint8 [rows, K/2], element 2k in the low nibble of
 *     byte k; one E4M3 scale factor per 16 columns, in the layouts that
 *     ts_outs_t describes.  A matrix has one fp32 global scale g, and stands
 *     for the values  e2m1(code) * e4m3(sf) / g.
 *   - Results are deterministic.  The row-wise operators give a row the same
 *     bits in every call; the two products sum K in an order that depends on
 *     the call's sizes, so there a row's last bits may change with M.
 *   - Row strides (ldx, ldo, ...) are in elements, at most 2^30.
 *   - Index arrays that the kernels read (row_of, row_src, expert_start,
 *     expert_count) are device data that the host cannot check: an entry that
 *     points outside the buffers it refers to is skipped, never followed.
 */
#ifndef TS_NVFP4_MOE_H
#define TS_NVFP4_MOE_H

#include "ts_fused_norm.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * ts_nvfp4_quantize: bf16 rows to NVFP4.  For each block of 16 columns
 *
 *   sf   = e4m3(g * (amax / 6))                    amax the block's largest |x|
 *   code = e2m1(x * (g / value(sf)))               0 for the block if value(sf) == 0
 *
 * every step in fp32 with one rounding, ties to even, saturating (the
 * arithmetic of patterns 3 and 5, on x itself).  An infinite x saturates its
 * block's scale factor; a NaN leaves its block's codes unspecified.
 *
 *   x             bf16 [T, K], row stride ldx (elements, >= K, multiple of 8).
 *   scale_factor  fp32[1], device-accessible: g.
 *   T             rows, >= 0 (T == 0 returns TS_OK).
 *   K             1 <= K <= 65536, multiple of 16.
 *   row_src       int32 [T] or NULL: rows t with row_src[t] < 0 are left
 *                 unread and their codes and scale factors unwritten (the
 *                 unused rows of ts_moe_sort).
 *   quant_out     uint8 [T, K/2].
 *   scale_out     uint8 scale factors in sf_layout (ts_outs_t).  Padding columns
 *                 are written as 0; padding rows too when row_src is NULL.
 *   flags         0 or TS_FLAG_PDL.
 */
TS_API int ts_nvfp4_quantize(const void *x, int64_t T, int64_t K, int64_t ldx, const float *scale_factor,
                             const int32_t *row_src, void *quant_out, void *scale_out, int sf_layout,
                             uint32_t flags, void *stream);

/*
 * ts_nvfp4_dequantize: the values of an NVFP4 matrix,
 *
 *   out[t, j] = bf16(e2m1(code) * (e4m3(sf) / g))              fp32 inside
 *
 * Arguments as for ts_nvfp4_quantize; out is bf16 [T, K] with row stride ldo
 * (>= K, multiple of 8).  Rows with row_src[t] < 0 are left as they were.
 */
TS_API int ts_nvfp4_dequantize(const void *quant, const void *scale, int sf_layout, int64_t T, int64_t K,
                               const float *scale_factor, const int32_t *row_src, void *out, int64_t ldo,
                               uint32_t flags, void *stream);

/*
 * ts_nvfp4_gemm: out[m, n] = bf16(alpha * sum_k A[m, k] B[n, k]), A and B the
 * products e2m1(code) * e4m3(sf) without their global scales, summed in fp32
 * on the tensor cores; alpha = 1 / (g_A * g_B) gives the product of the values.
 *
 *   a, a_scale    codes uint8 [M, K/2] and scale factors of A in SWIZZLED_128x4.
 *   b, b_scale    the same for B, [N, K/2] (weights: one row per output column).
 *   alpha         fp32[1], device-accessible.
 *   M             rows, >= 0 (M == 0 returns TS_OK).
 *   N             multiple of 8, 8 <= N <= 2^24.
 *   K             multiple of 32, 32 <= K <= 65536.  The scale factors' padding
 *                 columns of a K that is not a multiple of 64 are read and must
 *                 be 0, as every writer in this library leaves them.
 *   out           bf16 [M, N], row stride ldo (>= N, multiple of 8).
 *   a, b, a_scale, b_scale, out: 16-byte aligned; out overlaps no input.
 *   flags         0 or TS_FLAG_PDL.
 */
TS_API int ts_nvfp4_gemm(const void *a, const void *a_scale, const void *b, const void *b_scale,
                         const float *alpha, int64_t M, int64_t N, int64_t K, void *out, int64_t ldo,
                         uint32_t flags, void *stream);

/*
 * ts_moe_sort: the stable order of T*k (token, slot) entries by expert.
 *
 *   expert_ids    int32 [T, k]; an id outside 0..E-1 (an expert held by another
 *                 rank, a dropped entry) gets no row.
 *   T             tokens, >= 0.   k: 1..64.   T * k < 2^30.
 *   E             experts, 1..1024.
 *   row_align     each expert's rows start at a multiple of it: 1..256.  The
 *                 NVFP4 products need 128.
 *   rows          length of row_src: at least ts_moe_rows(T, k, E, row_align).
 *   row_of        int32 [T, k]: the entry's row, or -1.
 *   row_src       int32 [rows]: the entry t*k + slot of a row, -1 for the rows
 *                 that no entry has (between the experts and after the last).
 *   expert_start  int32 [E+1]: an expert's first row; [E] is the end of the last
 *                 expert's rows, rounded up to row_align.
 *   expert_count  int32 [E]: an expert's entries.
 * Entries of one expert keep their order (token, then slot).
 */
TS_API int ts_moe_sort(const int32_t *expert_ids, int64_t T, int64_t k, int64_t E, int64_t row_align,
                       int64_t rows, int32_t *row_of, int32_t *row_src, int32_t *expert_start,
                       int32_t *expert_count, uint32_t flags, void *stream);

/* Rows that hold T*k entries of any routing over E experts:
 * T*k + min(E, T*k) * (row_align - 1), rounded up to row_align; -1 for sizes
 * that ts_moe_sort refuses. */
TS_API int64_t ts_moe_rows(int64_t T, int64_t k, int64_t E, int64_t row_align);

/*
 * ts_moe_dispatch: token rows in expert order: row row_of[t, j] of the output
 * is x[t], for every j.  Rows that no entry has are left as they were.  Its
 * gradient is ts_moe_combine without weights, on the gradient of the rows.
 *
 *   x             bf16 [T, H], row stride ldx (>= H, multiple of 8).
 *   H             8 <= H <= 65536, multiple of 8 (16 for NVFP4).
 *   row_of        int32 [T, k] of ts_moe_sort; each row at most once.
 *   rows          rows of the output.
 *   out           bf16 [rows, H], or NULL for the NVFP4 form.
 *   scale_factor, quant_out, scale_out, sf_layout
 *                 NVFP4 form (out NULL): codes uint8 [rows, H/2] and scale
 *                 factors for `rows` rows, the bits ts_nvfp4_quantize gives x[t].
 *                 All NULL with out.
 */
TS_API int ts_moe_dispatch(const void *x, int64_t T, int64_t H, int64_t ldx, const int32_t *row_of, int64_t k,
                           int64_t rows, void *out, const float *scale_factor, void *quant_out,
                           void *scale_out, int sf_layout, uint32_t flags, void *stream);

/*
 * ts_nvfp4_grouped_gemm: each expert's product with its own rows, for
 * i < expert_count[e] and r = expert_start[e] + i:
 *
 *   out[r, n] = bf16(alpha[e] * sum_k A[r, k] B[e, n, k])
 *
 *   a, a_scale    codes uint8 [rows, K/2] and SWIZZLED_128x4 scale factors of the
 *                 sorted rows; rows a multiple of 128.
 *   b, b_scale    codes uint8 [E, N, K/2]; scale factors of each expert's [N, K]
 *                 in SWIZZLED_128x4, one expert after the other
 *                 (ceil(N/128)*128 * ceil(K/64)*4 bytes each).
 *   alpha         fp32 [E].
 *   expert_start  int32 [E+1] and expert_count int32 [E] of ts_moe_sort with
 *                 row_align 128.  An expert whose rows do not start at a
 *                 multiple of 128, or do not lie inside `rows`, is skipped.
 *   entries       an upper bound of the counts' sum (T*k); it only chooses the
 *                 tile size.
 *   E             1..1024;  N, K as for ts_nvfp4_gemm;  rows >= 0.
 *   out           bf16 [rows, N], row stride ldo; other rows are left as they were.
 */
TS_API int ts_nvfp4_grouped_gemm(const void *a, const void *a_scale, const void *b, const void *b_scale,
                                 const float *alpha, const int32_t *expert_start, const int32_t *expert_count,
                                 int64_t E, int64_t rows, int64_t entries, int64_t N, int64_t K, void *out,
                                 int64_t ldo, uint32_t flags, void *stream);

/*
 * ts_moe_combine: the experts' rows back in token order,
 *
 *   out[t] = bf16(sum over j ascending of weights[t, j] * y[row_of[t, j]])    fp32
 *
 * An entry with row_of < 0 adds nothing (its weight is not read as a factor);
 * a token without any gets zeros.
 *
 *   y             bf16 [rows, H], row stride ldy (>= H, multiple of 8).
 *   row_of        int32 [T, k];  k 1..64.
 *   weights       fp32 [T, k], or NULL for 1.
 *   H             8 <= H <= 65536, multiple of 8.
 *   out           bf16 [T, H], row stride ldo (>= H, multiple of 8).
 */
TS_API int ts_moe_combine(const void *y, int64_t rows, int64_t H, int64_t ldy, const int32_t *row_of,
                          const float *weights, int64_t T, int64_t k, void *out, int64_t ldo, uint32_t flags,
                          void *stream);

/*
 * ts_moe_combine_grad: the gradient of ts_moe_combine for dout = dL/dout,
 *
 *   dy[row_of[t, j]] = bf16(weights[t, j] * dout[t])
 *   dweights[t, j]   = sum_h dout[t, h] * y[row_of[t, j], h]     fp32; 0 if row_of < 0
 *
 * Rows of dy that no entry has are left as they were.
 *
 *   dout          bf16 [T, H], row stride ldd;  y bf16 [rows, H], row stride ldy;
 *   dy            bf16 [rows, H], row stride lddy;  strides >= H, multiples of 8.
 *   row_of        int32 [T, k], each row at most once.
 *   weights       fp32 [T, k].
 *   dweights      fp32 [T, k].
 */
TS_API int ts_moe_combine_grad(const void *dout, int64_t ldd, const void *y, int64_t ldy, int64_t rows,
                               int64_t H, const int32_t *row_of, const float *weights, int64_t T, int64_t k,
                               void *dy, int64_t lddy, float *dweights, uint32_t flags, void *stream);

/* Number of waits inside the product kernels of the current device that ran
 * into their time limit since the library was loaded, written to *count (the
 * outputs of such a call are not valid).  It waits for the device. */
TS_API int ts_stalled_waits(uint32_t *count);

#ifdef __cplusplus
}
#endif

#endif /* TS_NVFP4_MOE_H */
