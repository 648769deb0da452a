/*
 * ts_attention.h: C ABI of what an attention layer does around and over a
 * paged 4-bit cache on one GB300 (sm_103a): each head's RMSNorm of queries and
 * keys with the rotation by position in the same pass, its gradient, the keys
 * and values written to the cache as NVFP4 on the way and read back, and the
 * attention of queries over the cache.
 *
 * Conventions: those of ts_fused_norm.h and ts_nvfp4_moe.h (caller-owned
 * buffers, host-side checks before any launch, statuses, ts_last_error_detail,
 * TS_FLAG_PDL, no allocation and no synchronisation, strides in elements and at
 * most 2^30), with these additions:
 *   - ts_qk_norm_rope_grad and ts_nvfp4_attention enqueue two kernels where they need
 *     a workspace: the second joins what the blocks of the first left there.  A
 *     workspace needs no initial contents and holds nothing between calls; two
 *     calls that may run at the same time need one each.
 *   - Buffers may be in device memory or in page-locked host memory, except the
 *     queries, the outputs, the workspace and the cache of ts_nvfp4_attention,
 *     which live in device memory.
 *   - Results are deterministic: the same call gives the same bits.  The rows of
 *     ts_qk_norm_rope and ts_kv_cache_read do not depend on the other rows; the
 *     weights' gradients and the attention sum in an order that depends on the
 *     call's sizes and lengths.
 *   - Positions, slots, lengths and the table of pages are device data that the
 *     host cannot check: an entry that points outside the buffers it refers to is
 *     skipped, never followed.
 */
#ifndef TS_ATTENTION_H
#define TS_ATTENTION_H

#include "ts_nvfp4_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * A paged cache of keys and values in NVFP4.  A slot, page * page_size + offset,
 * holds the keys and values of one token, `heads` rows of head_dim each.
 *
 *   pages      uint8 [num_pages, heads, page_size / 16, 18 * head_dim]: the 16 tokens
 *              of a tile of one head lie in 18 D contiguous bytes (D = head_dim):
 *                [     0,  8 D)  K codes, D/2 bytes a token, element 2j in the low
 *                                nibble of byte j
 *                [   8 D, 16 D)  V codes
 *                [  16 D, 17 D)  K scale factors, E4M3, one per 16 elements, D/16
 *                                bytes a token
 *                [  17 D, 18 D)  V scale factors
 *              so that a step of 16 keys is one contiguous read.
 *   num_pages  0 <= num_pages, num_pages * page_size < 2^31.
 *   page_size  tokens of a page: a multiple of 16 in 16..65536.
 *   heads      1..1024.
 *   head_dim   a multiple of 16 in 16..256 (ts_nvfp4_attention: 64 or 128).
 *   k_scale    fp32[1], device-accessible: the global scale of K.  An element
 *              stands for e2m1(code) * e4m3(sf) / k_scale.
 *   v_scale    the same for V.
 * The struct lives in host memory and is read during the call only.
 */
typedef struct {
    void *pages;
    int64_t num_pages;
    int64_t page_size;
    int64_t heads;
    int64_t head_dim;
    const float *k_scale;
    const float *v_scale;
} ts_kv_cache_t;

/*
 * ts_qk_norm_rope: per-head RMSNorm of queries and keys and rotation by position.
 * For each token t and each head's row x of D elements,
 *
 *   n[j] = (x[j] * rsqrt(sum_i x[i]^2 / D + eps)) * w[j]                     fp32
 *   y    = n with the pairs (a, b) of its first `rot` elements turned by the
 *          position's angles:  (a c - b s,  b c + a s)                        fp32
 *   out  = bf16(y)
 *
 * where pair i is (i, i + rot/2), or (2i, 2i + 1) with `interleaved`, and c, s are
 * cos_sin[positions[t]][i], cos_sin[positions[t]][rot/2 + i].  Products and sums are
 * rounded to fp32 one by one in this order (sum / D as sum * (1 / D)).  The squares of
 * a key's row are summed in 32 sums, column j in sum j mod 32 in ascending order, which
 * are then added in pairs, neighbours first, so that its bits (and those in the cache)
 * can be computed elsewhere; those of a query in an order that depends on D alone.
 *
 *   q             bf16 [T, q_heads * D], row stride ldq.
 *   k             bf16 [T, k_heads * D], row stride ldk.
 *   T             tokens, >= 0 (T == 0 returns TS_OK);  T * (q_heads + 2 k_heads) at
 *                 most 2^30.
 *   q_heads, k_heads  1..1024;  head_dim (D) a multiple of 16 in 16..256.
 *   q_weight, k_weight  bf16 [D]; both NULL leaves the norm out (n = x).
 *   eps           added inside the rsqrt.
 *   positions     int32 [T].  A token whose position is outside 0..max_pos-1
 *                 is left out: its outputs and its slot stay as they were.
 *   cos_sin       fp32 [max_pos, rot]: rot/2 cosines, then rot/2 sines.  Angles of
 *                 far positions want 64 bits where the table is made.
 *   max_pos       1..2^31-1.   rot: a multiple of 16 in 16..D.
 *   q_out         bf16 [T, q_heads * D], row stride ldqo.  May be q (the same
 *                 stride), in place.
 *   k_out         the same for k, row stride ldko; NULL with a cache: not written.
 *   v, ldv, cache, slots   all NULL (0), or the keys' bf16(y) and the rows of v, bf16
 *                 [T, k_heads * D], go into the cache (heads = k_heads) as the bits
 *                 that ts_nvfp4_quantize gives them, token t into slots[t].
 *   slots         int32 [T]; a token with a slot outside the cache is not kept.  Two
 *                 tokens with the same slot leave either's bytes there.
 *   strides       >= heads * D, multiples of 8.  Outputs overlap no input but in
 *                 place, and not each other; rows of the same stride may interleave
 *                 (the q, k and v columns of one matrix).
 *   flags         0 or TS_FLAG_PDL.
 */
TS_API int ts_qk_norm_rope(const void *q, int64_t ldq, const void *k, int64_t ldk, int64_t T, int64_t q_heads,
                           int64_t k_heads, int64_t head_dim, const void *q_weight, const void *k_weight, float eps,
                           const int32_t *positions, const float *cos_sin, int64_t max_pos, int64_t rot,
                           int interleaved, void *q_out, int64_t ldqo, void *k_out, int64_t ldko, const void *v,
                           int64_t ldv, const ts_kv_cache_t *cache, const int32_t *slots, uint32_t flags,
                           void *stream);

/*
 * ts_qk_norm_rope_grad: the gradient of ts_qk_norm_rope (without a cache) for
 * dq_out = dL/dq_out and dk_out: with d the gradient turned back by the angles,
 * r = rsqrt(mean x^2 + eps) and g = d * w,
 *
 *   dx[j] = bf16(r * (g[j] - x[j] * r^2 * sum_i g[i] x[i] / D))               fp32
 *   dw[j] = sum over tokens and heads of d[j] * x[j] * r                      fp32
 *
 *   dq_out, dk_out  bf16, row strides lddqo, lddko.
 *   q, k            the forward call's inputs (which it must not have written in place).
 *   dq, dk          bf16, row strides lddq, lddk; may be dq_out, dk_out in place.
 *   dq_weight, dk_weight  fp32 [D]; NULL exactly where the weights are.  Written
 *                   for T == 0 too (zeros).
 *   workspace       ts_qk_norm_rope_grad_workspace(head_dim) bytes, 16-byte aligned; may
 *                   be NULL without weights.
 * The rows of a token whose position is outside the table are left as they were, and
 * add nothing to the weights' gradients.
 */
TS_API int ts_qk_norm_rope_grad(const void *dq_out, int64_t lddqo, const void *dk_out, int64_t lddko, const void *q,
                                int64_t ldq, const void *k, int64_t ldk, int64_t T, int64_t q_heads,
                                int64_t k_heads, int64_t head_dim, const void *q_weight, const void *k_weight,
                                float eps, const int32_t *positions, const float *cos_sin, int64_t max_pos,
                                int64_t rot, int interleaved, void *dq, int64_t lddq, void *dk, int64_t lddk,
                                float *dq_weight, float *dk_weight, void *workspace, uint32_t flags, void *stream);

/* Bytes of the gradient's workspace, -1 for a head_dim that it refuses. */
TS_API int64_t ts_qk_norm_rope_grad_workspace(int64_t head_dim);

/*
 * ts_kv_cache_read: the values that the cache's slots hold,
 *
 *   k_out[t, h, j] = bf16(e2m1(code) * (e4m3(sf) / k_scale))     fp32 inside
 *
 * and v_out likewise: the bits that ts_nvfp4_dequantize gives.
 *
 *   slots    int32 [T]; a token with a slot outside the cache is left as it was.
 *   T        >= 0;  T * heads at most 2^30.
 *   k_out    bf16 [T, heads * D], row stride ldk;  v_out the same, ldv.
 *            Either may be NULL.
 */
TS_API int ts_kv_cache_read(const ts_kv_cache_t *cache, const int32_t *slots, int64_t T, void *k_out, int64_t ldk,
                            void *v_out, int64_t ldv, uint32_t flags, void *stream);

/*
 * ts_nvfp4_attention: attention of the last queries of each sequence over its
 * keys and values in the cache.  Sequence b has kv_lens[b] keys, of which key j
 * lies in page block_table[b, j / page_size] at offset j % page_size, and
 * n = cu_q[b+1] - cu_q[b] queries, the rows from cu_q[b] on.  Query i stands at
 * position p = kv_lens[b] - n + i; for each of its heads, with the key head
 * q_head / (q_heads / heads),
 *
 *   s[j] = scale * sum_d q[d] K[j, d]
 *   j is seen if  j < kv_lens[b],  j <= p (causal)  and  j > p - window (window > 0)
 *   out  = bf16(sum_j exp(s[j] - lse) V[j]),   lse = log sum_j exp(s[j])    over the seen j
 *
 * A query that sees no key gets zeros and lse = -inf.  Products are exact (a query's
 * row is first scaled by a power of two into fp16, where K and V are exact), sums
 * are in fp32, and exp(s - max) is rounded for the product with V, to 11 bits down to 2^-21 and
 * to multiples of 2^-31 below.  Scale factors of keys that a query of the call sees must not
 * be NaN; those of other slots are not used.
 *
 *   q            bf16 [T, q_heads * D], row stride ldq.
 *   T            rows of q, >= 0 (T == 0 or B == 0 returns TS_OK);  T * q_heads at
 *                most 2^30.  Rows of out and
 *                lse that no sequence has are left as they were.
 *   q_heads      a multiple of cache->heads, at most 1024.
 *   cu_q         int32 [B + 1], ascending from 0, or NULL: one query for each sequence,
 *                T == B.
 *   B            sequences, 0..65536.
 *   max_q        a bound of the queries of a sequence, >= 1.  It chooses the kernel;
 *                the result holds for more.
 *   cache        head_dim 64 or 128.
 *   block_table  int32 [B, max_pages], row stride max_pages; max_pages * page_size at
 *                most 2^30.  A length beyond it counts as max_pages * page_size; the
 *                keys of a page outside the cache are not seen.
 *   kv_lens      int32 [B].
 *   scale        finite, > 0 (1 / sqrt(D) as a rule).
 *   causal       0 or 1.   window: keys that a query sees at most, 0 for all; with
 *                causal only.
 *   out          bf16 [T, q_heads * D], row stride ldo.
 *   lse          fp32 [T, q_heads], natural logarithm, or NULL.
 *   workspace    ts_nvfp4_attention_workspace(...) bytes with max_keys = max_pages *
 *                page_size, 16-byte aligned; may be NULL where that is 0.
 *   strides      >= q_heads * D, multiples of 8.  Outputs overlap no input.
 */
TS_API int ts_nvfp4_attention(const void *q, int64_t ldq, int64_t T, int64_t q_heads, const int32_t *cu_q, int64_t B,
                              int64_t max_q, const ts_kv_cache_t *cache, const int32_t *block_table,
                              int64_t max_pages, const int32_t *kv_lens, float scale, int causal, int64_t window,
                              void *out, int64_t ldo, float *lse, void *workspace, uint32_t flags, void *stream);

/* Bytes of the attention's workspace, whatever the lengths within these bounds (no fewer
 * where a bound is larger, or a window is none); -1 for sizes that it refuses. */
TS_API int64_t ts_nvfp4_attention_workspace(int64_t B, int64_t q_heads, int64_t heads, int64_t head_dim, int64_t max_q,
                                            int64_t max_keys, int64_t window);

#ifdef __cplusplus
}
#endif

#endif /* TS_ATTENTION_H */
