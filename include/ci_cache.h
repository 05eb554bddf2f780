/*
 * ci_cache.h -- C ABI of the paged key-value cache beside the indexer (libci.so).
 *
 * The indexer (ci.h) picks the positions that sparse attention reads.  The
 * entry points here are what surrounds that read when a model serves tokens:
 *
 *   ci_qk_norm_rope_append  norms and rotates the new tokens' queries and keys
 *                           and writes keys and values into their pages;
 *   ci_attn_decode          attention of each query row over its request's
 *                           whole cache or over the indexer's positions;
 *   ci_pages_alloc, ci_pages_fork, ci_pages_free, ci_pages_compact,
 *   ci_pages_copy           the pages themselves, on the device.
 *
 * The conventions of ci.h hold: device pointers owned by the caller, work
 * enqueued on `stream`, no allocation, no synchronization, host-side argument
 * checks with a negative status, data errors as CI_DEVERR_* bits in the
 * optional *dev_err, the row layouts CI_LAYOUT_* with req_row_start.
 *
 * Cache
 * -----
 *  - head_dim D is 64, 128 or 256; a page holds 64 positions.
 *  - A pool is uint8 [num_pages][num_kv_heads][ci_cache_page_bytes(format, D)],
 *    16-byte aligned; keys and values have one pool each, of the same format:
 *      CI_CACHE_BF16  64 x D bf16;
 *      CI_CACHE_FP8   64 x D e4m3, then 64 fp32 scales (little endian): value
 *                     = scale * e4m3, the shape of the indexer's FP8 page.
 *    num_pages * num_kv_heads * (64 + 256 / D) <= 2^31 - 1.
 *  - page_table int32 [num_req][max_pages]: logical page j of a request is
 *    physical page page_table[req][j]; -1 where there is none.
 *  - Query head h reads key-value head h / (num_q_heads / num_kv_heads).
 *  - ref_count int32 [num_pages]: how many page-table entries name the page;
 *    0 = free.  New pages are always the lowest free ids, so every call's
 *    result is a function of its inputs.
 */
#ifndef CI_CACHE_H_
#define CI_CACHE_H_

#include "ci.h"

#ifdef __cplusplus
extern "C" {
#endif

enum ci_cache_format { CI_CACHE_BF16 = 0, CI_CACHE_FP8 = 1 };

/* Bytes of one (page, key-value head) of a pool, or a negative status. */
CI_API int64_t ci_cache_page_bytes(int32_t cache_format, int32_t head_dim);

/*
 * Attention of `rows` query rows over the paged cache.
 *
 * Row t with length L_t = seq_len[t] reads the positions S_t:
 *   pos == NULL   every s < L_t;
 *   otherwise     the entries pos[t * pos_stride + i], i < npos, that lie in
 *                 [0, L_t), each as often as it occurs; -1 marks an unused
 *                 entry (the indexer's output as it is), any other value
 *                 outside [0, L_t) is skipped and sets CI_DEVERR_POS.
 * With logit[s] = scale * q[t,h] . k[s, h']: lse[t,h] = ln sum_s exp(logit[s])
 * and out[t,h] = sum_s exp(logit[s] - lse) v[s, h'].  A row with no positions
 * gets out = 0 and lse = -inf.  What lies in the cache outside S_t (the rest
 * of a row's last page included) is not read into a result, whatever its bits.
 * A length outside [0, max_len] counts as 0 and sets CI_DEVERR_LEN; a page id
 * outside [0, num_pages) drops its positions and sets CI_DEVERR_PAGE.
 *
 * Products are exact and accumulated in fp32; the softmax statistics are fp32;
 * the probabilities are rounded to bf16 for the product with the values (FP8:
 * with the value's scale in them) and divided by the sum of what they were
 * rounded to, so that the error left is that of their ratios; lse has the sum
 * of the unrounded ones; out is rounded once.  Results do not depend on the
 * order in which blocks run.  Values |v| <= 2^80; FP8 scales: finite, |scale|
 * <= 2^60, and a value's NaN code (0x7F, 0xFF) reads as +-480 * scale.
 *
 * q, out: bf16 [rows][num_q_heads][D] with row strides in elements (multiples
 * of 8); q and out 16-byte aligned.  lse: float [rows][num_q_heads] or NULL.
 * 1 <= num_q_heads / num_kv_heads <= 128, without remainder.
 * max_len <= 64 * max_pages.  With n = max_len, or npos for a list:
 * rows * num_kv_heads * ceil(num_q_heads / num_kv_heads / 64) * (n / 64 + 1) <
 * 2^31.
 * ws: at least ci_attn_workspace_bytes() bytes (the same for any `rows`),
 * 16-byte aligned, of any content; one call's use of it ends with the call's
 * work on the stream.
 */
CI_API int64_t ci_attn_workspace_bytes(int32_t rows, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim);
CI_API int ci_attn_decode(const uint16_t* q, int64_t q_stride, int32_t rows, int32_t num_q_heads,
                          int32_t num_kv_heads, int32_t head_dim, float scale, const uint8_t* k_pool,
                          const uint8_t* v_pool, int64_t num_pages, int32_t cache_format, const int32_t* page_table,
                          int32_t num_req, int32_t max_pages, int32_t layout, const int32_t* req_row_start,
                          const int32_t* seq_len, int32_t max_len, const int32_t* pos, int64_t pos_stride,
                          int32_t npos, uint16_t* out, int64_t out_stride, float* lse, void* ws, int64_t ws_bytes,
                          int32_t* dev_err, void* stream);

/*
 * New tokens' queries, keys and values: norm, rotation, append.
 *
 * For every token t and head of q and k (bf16, [tokens][heads][D], token
 * strides in elements): y = x * rsqrt(mean(x^2) + eps) * w, with w = q_norm or
 * k_norm (float [D]; NULL: y = x), then the rotation of the first rot_dim dims
 * by position p = positions[t]: pairs (i, rot_dim / 2 + i) (is_neox != 0) or
 * (2i, 2i + 1) (is_neox == 0), i < rot_dim / 2, become
 * (a c - b s, b c + a s), c = cos_sin[p][i], s = cos_sin[p][rot_dim / 2 + i];
 * all in fp32.  q_out gets the rotated queries, rounded once to bf16.  The
 * rotated keys and the values as they are go to slot u % 64 of page
 * page_table[request of t][u / 64], u = cache_pos[t] (cache_pos == NULL: u =
 * p): rounded once to bf16, or (CI_CACHE_FP8) as e4m3(x / scale), nearest
 * even, with the position's own fp32 scale = max(amax, 1e-10) / 448 per head
 * (NaN where a value is NaN, so that what reads the entry is NaN too).
 * A negative u writes no cache entry (padding).  p outside [0, max_pos) sets
 * CI_DEVERR_POS, the token's queries are 0 and its cache entry is not written;
 * so is an entry with u >= 64 * max_pages (CI_DEVERR_POS) or with a page id
 * outside [0, num_pages) (CI_DEVERR_PAGE).
 *
 * Tokens are the rows of the layouts: token t is request t (decode), of
 * request 0 (prefill), or of the request that req_row_start says (varlen).
 * Two tokens must not write the same slot.  rot_dim: a multiple of 16,
 * 0 <= rot_dim <= D; cos_sin float [max_pos][rot_dim] (may be NULL for
 * rot_dim == 0; positions still index the cache).  q, k, v, q_out 16-byte
 * aligned with strides that are multiples of 8; cos_sin, q_norm and k_norm
 * 16-byte aligned.
 */
CI_API int ci_qk_norm_rope_append(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride,
                                  const uint16_t* v, int64_t v_stride, int32_t tokens, int32_t num_q_heads,
                                  int32_t num_kv_heads, int32_t head_dim, const float* q_norm, const float* k_norm,
                                  float eps, const float* cos_sin, int32_t max_pos, int32_t rot_dim, int32_t is_neox,
                                  const int32_t* positions, const int32_t* cache_pos, uint16_t* q_out,
                                  int64_t q_out_stride, uint8_t* k_pool, uint8_t* v_pool, int64_t num_pages,
                                  int32_t cache_format, const int32_t* page_table, int32_t num_req, int32_t max_pages,
                                  int32_t layout, const int32_t* req_row_start, int32_t* dev_err, void* stream);

/*
 * Pages.  At most 4096 requests per call (`n`, and num_req of ci_pages_alloc);
 * num_pages <= 2^31 - 1; ref_count 16-byte aligned.
 *
 * ci_pages_alloc: request r grows from old_len[r] to new_len[r] positions: its
 * entries ceil(old / 64) .. ceil(new / 64) - 1 become the lowest free pages (in
 * order of the requests, then of the entries), each with ref_count 1.  new <
 * old or a length outside [0, 64 * max_pages] sets CI_DEVERR_LEN and leaves
 * the request as it is.
 *
 * ci_pages_fork: for i < n request child[i] becomes a copy of the first
 * length[i] positions of request parent[i]: it shares the parent's full pages
 * (ref_count + 1 each); a last page that is only partly filled becomes a page
 * of its own (the lowest free ids, in order of i, ref_count 1), and the pair
 * (copy_src[i], copy_dst[i]) = (the parent's page, the new page) says what is
 * to be copied, (-1, -1) where nothing is.  The rest of the child's row is
 * set to -1; what it held before is not released (ci_pages_free first).  Every
 * child is named once, and no child is a parent in the same call.  A request
 * id outside [0, num_req) or child == parent sets CI_DEVERR_REQ, a length
 * outside [0, 64 * max_pages] CI_DEVERR_LEN: that fork is left out.  An entry
 * of the parent outside [0, num_pages) sets CI_DEVERR_PAGE and becomes -1.
 *
 * In both, entries for which no free page is left become -1 and set
 * CI_DEVERR_PAGE.
 *
 * ci_pages_free: every entry >= 0 of the rows req[i], i < n (each named once)
 * drops one reference; the rows become -1.  An entry >= num_pages or a page
 * without references sets CI_DEVERR_PAGE, a request outside [0, num_req)
 * CI_DEVERR_REQ.
 *
 * ci_pages_compact: with n_live pages of ref_count > 0, moves the live pages
 * with ids >= n_live, ascending, into the free ids < n_live, ascending:
 * (copy_src[i], copy_dst[i]), i < *count, is what is to be copied, and the
 * arrays (int32 [num_pages]) are filled up with -1.  ref_count moves along;
 * remap int32 [num_pages] gets every page's new id, -1 for pages that were
 * free; the entries of page_table (num_req >= 0 rows) are rewritten (an entry
 * that names a free page becomes -1, one >= num_pages too, and sets
 * CI_DEVERR_PAGE).
 *
 * ci_pages_copy: page copy_dst[i] of every pool becomes a copy of page
 * copy_src[i], i < n (and i < *count where count is not NULL); pairs with both
 * ids negative are skipped, other ids outside [0, num_pages) set CI_DEVERR_PAGE
 * and are skipped.  No page that is written may be another pair's source or
 * destination.  pools, page_bytes: HOST arrays of 1 <= num_pools <= 160 device
 * pointers and bytes per page (pools 16-byte aligned, bytes multiples of 16),
 * read before the call returns.
 */
CI_API int ci_pages_alloc(int32_t* page_table, int32_t num_req, int32_t max_pages, int32_t* ref_count,
                          int64_t num_pages, const int32_t* old_len, const int32_t* new_len, int32_t* dev_err,
                          void* stream);
CI_API int ci_pages_fork(int32_t* page_table, int32_t num_req, int32_t max_pages, int32_t* ref_count,
                         int64_t num_pages, const int32_t* parent, const int32_t* child, const int32_t* length,
                         int32_t n, int32_t* copy_src, int32_t* copy_dst, int32_t* dev_err, void* stream);
CI_API int ci_pages_free(int32_t* page_table, int32_t num_req, int32_t max_pages, int32_t* ref_count,
                         int64_t num_pages, const int32_t* req, int32_t n, int32_t* dev_err, void* stream);
CI_API int ci_pages_compact(int32_t* page_table, int32_t num_req, int32_t max_pages, int32_t* ref_count,
                            int64_t num_pages, int32_t* remap, int32_t* copy_src, int32_t* copy_dst, int32_t* count,
                            int32_t* dev_err, void* stream);
CI_API int ci_pages_copy(uint8_t* const* pools, const int64_t* page_bytes, int32_t num_pools, int64_t num_pages,
                         const int32_t* copy_src, const int32_t* copy_dst, int32_t n, const int32_t* count,
                         int32_t* dev_err, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* CI_CACHE_H_ */
