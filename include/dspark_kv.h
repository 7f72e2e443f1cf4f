/*
 * dspark_kv.h -- C ABI of the target side of a verify step (B200 / sm_100a):
 * the paged K/V cache and the attention of the flattened verify rows over it.
 *
 * Between dspark_confidence_prefix, which writes verify_len on the device,
 * and dspark_verify / dspark_verify_lmhead, which read the target's rows,
 * the target model runs its layers on the verify rows.  These calls are the
 * part of a layer that depends on that layout:
 *   dspark_kv_append   norms and rotation of the new rows' queries and keys,
 *                      keys and values written to the cache
 *   dspark_attn_verify attention of the new rows over the cache
 *   dspark_kv_read     rows of the cache read back into contiguous rows
 * They take the row markers of dspark_verify (yage.ai "DSpark speculative
 * decoding hardware scheduling", variable-length verify paragraph: the
 * verify tokens of all requests in one flat tensor, no padding) and read
 * every length on the device, so a whole step (draft, cut, target, verify)
 * captures into one CUDA graph.  A prompt's chunk is the same call with more
 * rows, plain decoding the same call with one row a request.
 *
 * Conventions: those of dspark.h (device pointers owned by the caller,
 * row-major, nothing allocated, no host synchronisation, argument errors
 * before anything is enqueued, data errors as DSPARK_FLAG_* bits readable
 * with dspark_get_device_status / dspark_get_device_flags on the workspace).
 *
 * Rows.  Request b, 0 <= b < B, has verify_len[b] + 1 new tokens (-1: none,
 * an idle slot).  Token p is row row_start[b] + p of the row tensors and
 * stands at position cache_len[b] + p of its sequence.  Requests' rows must
 * not overlap; rows that no request claims are neither read nor written.
 * After the verify accepted n tokens the caller adds n + 1 to cache_len[b];
 * what the rejected tokens left behind it is overwritten by the next append
 * and never read as long as it lies beyond the sequence.
 *
 * Idle slots.  These calls skip a slot with verify_len = -1.  dspark_verify*
 * takes lengths of [0, K] only (it flags a negative one and goes on with 0): give
 * it max(verify_len, 0), so that an idle slot is a request without drafts, whose
 * row row_start[b] must exist and may hold anything finite; ignore what it
 * returns for the slot, and leave cache_len[b] as it is.
 *
 * Cache.  k_cache and v_cache are [n_pages, Hkv, page_size, D]; position j of
 * request b is place j % page_size of page page_table[b, j / page_size]
 * (page_table [B, max_pages] int32; entries behind a sequence's last page are
 * not read).  Two requests may share pages that neither writes.  With
 * DSPARK_KV_E4M3 an element is an e4m3 code, and k_scale / v_scale
 * [n_pages, Hkv, page_size] fp32 hold one scale for each token and head: the
 * element's value is code * scale.  The codes 0x7f and 0xff (NaN) never
 * leave dspark_kv_append, and what the attention makes of them is not
 * defined; a scale that is not finite makes the row's values not finite.
 *
 * Sizes: D 64 or 128; page_size 16, 32, 64, 128 or 256; B <= 4096; Hq a
 * multiple of Hkv, Hq <= 1024; n_pages * Hkv * page_size < 2^31; n_rows at
 * most 2^31 - 2^16, in the attention n_rows * Hq < 2^31; positions below 2^30
 * (later ones: see below).  Everything
 * 16-byte aligned (the workspace 256); row strides (in elements) multiples
 * of 8, the heads of a row contiguous.  Other sizes: DSPARK_ERR_UNSUPPORTED.
 *
 * Data errors.  A request with verify_len outside its range, rows outside
 * [0, n_rows) or positions outside [0, max_pages * page_size) or past 2^30 raises
 * DSPARK_FLAG_BAD_LENGTH and is treated as idle.  A page id outside
 * [0, n_pages) raises DSPARK_FLAG_BAD_PAGE; nothing is written there and
 * reads take page 0 instead.
 */
#ifndef DSPARK_KV_H_
#define DSPARK_KV_H_

#include "dspark.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of these calls: activations (rows) are bf16 or fp16; a cache
 * has its rows' type or e4m3. */
typedef enum { DSPARK_KV_BF16 = 1, DSPARK_KV_F16 = 2, DSPARK_KV_E4M3 = 3 } dspark_kv_dtype;

/* Status flag: a page id outside [0, n_pages). */
#define DSPARK_FLAG_BAD_PAGE 0x40u

/* Workspace bytes of dspark_kv_append and dspark_kv_read (status only). */
size_t dspark_kv_workspace_size(void);

/*
 * The new rows' queries, keys and values, from the projections to the cache:
 *   norm      (q_norm / k_norm given) x <- x / sqrt(mean(x^2) + eps) * w over
 *             the D elements of each head, w [D] fp32
 *   rotation  (rot_dim > 0) of the first rot_dim elements of each query and
 *             key head by the angles a_i = position * inv_freq[i],
 *             i < rot_dim / 2: (x1, x2) <- rope_scale *
 *             (x1 cos a_i - x2 sin a_i, x2 cos a_i + x1 sin a_i), on the
 *             pairs (i, i + rot_dim / 2), or (2i, 2i + 1) if interleaved;
 *             the rest of the head stays as it is
 *   q_out     the query rows, rounded once to their type
 *   cache     the key and value rows, rounded once to the cache's type; e4m3:
 *             scale = max(max|x| / 448, 2^-126) of the row, code = x / scale
 *             to the nearest e4m3 value; a row with an element that is not
 *             finite gets the scale NaN and codes 0
 * Arithmetic is fp32; angles are formed in fp64, so far positions lose
 * nothing.  A model with scaled frequencies for long contexts passes them as
 * inv_freq and its attention factor as rope_scale.
 *
 * Inputs   q [n_rows, Hq, D], k, v [n_rows, Hkv, D] of act_dtype, rows
 *          q_stride / k_stride / v_stride elements apart (slices of one fused
 *          projection); q_norm, k_norm [D] fp32 or NULL; inv_freq
 *          [rot_dim / 2] fp64 (NULL if rot_dim = 0); rot_dim a multiple of
 *          16, at most D; the markers row_start [B] int64, verify_len and
 *          cache_len [B] int32, page_table
 * Outputs  q_out [n_rows, Hq, D] (contiguous; may be q itself where q is
 *          contiguous, else over none of q, k, v), k_cache, v_cache, and with e4m3 k_scale, v_scale
 */
dspark_status dspark_kv_append(
    const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride,
    int64_t v_stride, dspark_kv_dtype act_dtype, int64_t n_rows, int B, int Hq, int Hkv, int D,
    const int64_t *row_start, const int32_t *verify_len, const int32_t *cache_len,
    const int32_t *page_table, int max_pages, void *k_cache, void *v_cache, float *k_scale,
    float *v_scale, dspark_kv_dtype cache_dtype, int64_t n_pages, int page_size,
    const float *q_norm, const float *k_norm, float eps, const double *inv_freq, int rot_dim,
    int interleaved, float rope_scale, void *q_out, void *workspace, size_t ws_bytes,
    void *stream);

/*
 * Cache rows as contiguous rows: row row_start[b] + p of k_out and v_out
 * [n_rows, Hkv, D] (out_dtype bf16 or fp16) is position cache_len[b] + p of
 * request b, p = 0 .. verify_len[b] (the markers that dspark_kv_append wrote
 * them with; cache_len = 0 reads a sequence from its start).  A 16-bit cache
 * has the type out_dtype and is copied; e4m3 gives code * scale rounded once.
 */
dspark_status dspark_kv_read(
    const void *k_cache, const void *v_cache, const float *k_scale, const float *v_scale,
    dspark_kv_dtype cache_dtype, int64_t n_pages, int page_size, const int64_t *row_start,
    const int32_t *verify_len, const int32_t *cache_len, const int32_t *page_table, int max_pages,
    int64_t n_rows, int B, int Hkv, int D, void *k_out, void *v_out, dspark_kv_dtype out_dtype,
    void *workspace, size_t ws_bytes, void *stream);

/* Workspace bytes of dspark_attn_verify: the status, and the partial results
 * of rows whose keys are split over several CTAs: 39 MB at D = 128, 20 at 64,
 * whatever B, Hq, Hkv and max_len are.  Calls that follow one another on a stream
 * (the layers of a step) may share one. */
size_t dspark_attn_workspace_size(int B, int Hq, int Hkv, int D, int max_len);

/*
 * Attention of the new rows over the cache, which already holds the new
 * tokens' keys and values (dspark_kv_append).  For token p of request b, at
 * position i = cache_len[b] + p, and query head h, which reads key/value head
 * h / (Hq / Hkv):
 *   out[row, h, :] = sum_j w_j V_j,  w = softmax_j(sm_scale * q[row, h] . K_j)
 *   over max(0, i - window + 1) <= j <= i   (window = 0: over all j <= i)
 * Scores, softmax statistics and sums are fp32; the weights are rounded to 16
 * bits (the value rows' type; fp16 with an e4m3 cache) for the product with
 * V; out is rounded once.  With an e4m3 cache q enters the scores as a sum of
 * e4m3 parts: elements below 2^-9 (bf16; fp16: 2^-6) of the largest of their row
 * and head are off by up to 2^-17 of it, all others exact.  Positions a row does not see never reach it: K and
 * V there may hold anything, infinities and NaN included.  A row whose result is
 * not finite is formed again by itself: right, but slow.  (Over more than 2^19
 * positions such rows may hold a step's CTA up for longer than its waits' limit
 * of 2 s: the call then ends with DSPARK_FLAG_TIMEOUT.)
 *
 * Inputs   q [n_rows, Hq, D] act_dtype, rows q_stride elements apart;
 *          max_len: an upper bound of verify_len + 1, at least 1 (K + 1 of a
 *          verify step, the longest chunk of a prompt); it chooses the
 *          kernel, and a longer request is a data error; sm_scale > 0
 * Outputs  out [n_rows, Hq, D] act_dtype, contiguous, not over q
 */
dspark_status dspark_attn_verify(
    const void *q, int64_t q_stride, dspark_kv_dtype act_dtype, int64_t n_rows, int B, int Hq,
    int Hkv, int D, int max_len, const int64_t *row_start, const int32_t *verify_len,
    const int32_t *cache_len, const int32_t *page_table, int max_pages, const void *k_cache,
    const void *v_cache, const float *k_scale, const float *v_scale, dspark_kv_dtype cache_dtype,
    int64_t n_pages, int page_size, float sm_scale, int window, void *out, void *workspace,
    size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DSPARK_KV_H_ */
