/*
 * ci_draft.h -- C ABI of drafted steps over the paged cache (libci.so).
 *
 * A drafted step runs the model over several guessed tokens per request at
 * once and keeps those that the model agrees with.  The guesses of a request
 * are a tree: nodes 0 .. n - 1, each hanging on an earlier one; a chain is the
 * tree in which node i hangs on node i - 1.  One step, in order:
 *
 *   ci_pages_alloc    (ci_cache.h) pages for positions length .. length + n - 1;
 *   ci_draft_plan     the step's rows, from the lengths and the trees: where
 *                     each request's rows start, every node's position, the
 *                     slot that keeps it, and which nodes it sees;
 *   ci_qk_norm_rope_append  (ci_cache.h, CI_LAYOUT_VARLEN, cache_pos) every
 *                     layer's keys and values into those slots;
 *   ci_attn_draft     every layer's attention: each node over its request's
 *                     cache and its own ancestors;
 *   ci_draft_accept   the path of each tree that the model agrees with;
 *   ci_slots_move     that path's keys and values to where the cache goes on;
 *   ci_pages_trim     the pages behind the new length released.
 *
 * The conventions of ci.h and ci_cache.h hold: device pointers owned by the
 * caller, work enqueued on `stream`, no allocation, no synchronization,
 * host-side argument checks with a negative status, data errors as CI_DEVERR_*
 * bits in the optional *dev_err.
 *
 * Trees and rows
 * --------------
 *  - Request r holds length[r] positions and drafts n_r nodes; node i is kept
 *    at position length[r] + i of its pages until the step ends.
 *  - Its rows are req_start[r] .. req_start[r + 1] - 1, row req_start[r] + i
 *    being node i (req_start int32 [num_req + 1], not descending, within
 *    [0, rows]); 1 <= num_req <= 4096.
 *  - parent int32 [num_req][max_nodes]: the node on which node i hangs, in
 *    [-1, i - 1]; -1 hangs on the cache alone.  parent == NULL: chains.
 *  - Node 0 is the token that the request goes on with: it is always part of
 *    the accepted path.
 *  - A node sees every position below length[r], its ancestors and itself.
 *    mask uint32 [rows][mask_words]: bit j of word w of a row is node 32 w + j.
 */
#ifndef CI_DRAFT_H_
#define CI_DRAFT_H_

#include "ci_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

#define CI_DRAFT_MAX_NODES 256

/*
 * The rows of a drafted step.  count[r], at most max_nodes, is n_r.  Writes
 * req_start [num_req + 1] and, for every node's row,
 *   positions  length[r] + its depth (node 0: 0);
 *   cache_pos  length[r] + i, or -1 where page_table has no page in
 *              [0, num_pages) for it;
 *   mask       its ancestors and itself (NULL: not wanted);
 *   row_token  token[r][i] (both NULL: not wanted).
 * Rows from the last request's end up to `rows` get 0, -1, 0 and 0: `rows` may
 * be more than there are nodes (a captured step).  Where there are more nodes
 * than rows the last ones are left out, and CI_DEVERR_LEN is set.  A count
 * outside [0, max_nodes] or a length for which 0 <= length and length + count
 * <= 64 * max_pages do not hold counts as no nodes and sets CI_DEVERR_LEN.  A
 * parent outside [-1, i - 1] sets CI_DEVERR_POS; the node sees nothing, its
 * cache_pos is -1 and its position length[r].
 * 1 <= max_nodes <= 256; 32 * mask_words >= max_nodes, mask_words <= 8.
 */
CI_API int ci_draft_plan(const int32_t* length, const int32_t* count, const int32_t* parent, const int32_t* token,
                         int32_t num_req, int32_t max_nodes, const int32_t* page_table, int32_t max_pages,
                         int64_t num_pages, int32_t rows, int32_t* req_start, int32_t* positions, int32_t* cache_pos,
                         uint32_t* mask, int32_t mask_words, int32_t* row_token, int32_t* dev_err, void* stream);

/*
 * Attention of every row over its request's positions below length[r] and over
 * the nodes that its mask names, node j at position length[r] + j; bits of
 * nodes that the request does not have are ignored.  mask == NULL: every node
 * up to the row's own, for any number of nodes (a chain, or a prompt's chunk
 * behind what the cache holds).  q, out, lse, scale, the pools and the page
 * table are ci_attn_decode's, and so is what is computed:
 *   logit[s] = scale * q[t,h] . k[s, h'], lse[t,h] = ln sum_s exp(logit[s]),
 *   out[t,h] = sum_s exp(logit[s] - lse) v[s, h'];
 * a row that sees nothing gets out = 0 and lse = -inf.  What a row does not
 * see is not read into its result, whatever its bits.  Rows that belong to no
 * request are left as they are.
 * A request whose length[r] or n_r is not within 0 <= length[r], n_r <=
 * max_rows and length[r] + n_r <= max_len sets CI_DEVERR_LEN, one whose starts
 * are not within [0, rows] or descend CI_DEVERR_REQ: the first gets rows of no
 * positions, the second none.  A page id outside [0, num_pages) drops its
 * positions and sets CI_DEVERR_PAGE.
 *
 * Products are exact and accumulated in fp32; FP8: but for what is left out of a
 * query's elements below 2^-13 m, at most 2^-21 m of each, m being the largest
 * magnitude of its row and head, or 2^-119 if that is larger.  The softmax
 * statistics are fp32; the probabilities are rounded to bf16 for the product with
 * the values (FP8: with the value's scale in them) and divided by the sum of the
 * unrounded ones; out is rounded once.  FP8: a position's part of out is kept in
 * steps of 2^-81, what lies below is lost.  Results do not depend on the order in
 * which blocks run.
 * Any finite logits; values |v| <= 2^80; FP8: scales finite, |scale| <= 2^60,
 * and a value's NaN code (0x7F, 0xFF) reads as +-480 * scale.
 *
 * max_len <= 64 * max_pages; max_rows >= 0: no request has more rows;
 * mask_words >= 1 (ignored for NULL).  rows * G < 2^31, G = num_q_heads /
 * num_kv_heads, and with B = min(num_req * ceil(max_rows * G / 128),
 * ceil(rows * G / 128) + num_req): num_kv_heads * B * (max_len / 128 + 1) < 2^31.
 * ws: at least ci_attn_draft_workspace_bytes() bytes, 16-byte aligned, of any
 * content; one call's use of it ends with the call's work on the stream.  Its size
 * is two blocks of rows' sums per SM, 40 MB for heads of 128 (20 and 40 for 64 and
 * 256), and goes by head_dim alone: max_rows, checked to be >= 0, does not change it.
 */
CI_API int64_t ci_attn_draft_workspace_bytes(int32_t max_rows, int32_t num_q_heads, int32_t num_kv_heads,
                                             int32_t head_dim);
CI_API int ci_attn_draft(const uint16_t* q, int64_t q_stride, int32_t rows, int32_t num_q_heads, int32_t num_kv_heads,
                         int32_t head_dim, float scale, const uint8_t* k_pool, const uint8_t* v_pool, int64_t num_pages,
                         int32_t cache_format, const int32_t* page_table, int32_t num_req, int32_t max_pages,
                         const int32_t* req_start, const int32_t* length, int32_t max_len, int32_t max_rows,
                         const uint32_t* mask, int32_t mask_words, uint16_t* out, int64_t out_stride, float* lse,
                         void* ws, int64_t ws_bytes, int32_t* dev_err, void* stream);

/*
 * What the model agrees with: from node 0 on, the lowest child c of the last
 * accepted node p with row_token[c] == target[p] is accepted, as long as there
 * is one.  row_token, target int32 [rows]: the drafted tokens, and the model's
 * choice behind each row; a row with cache_pos < 0 (NULL: none) is not
 * accepted.  Writes the accepted nodes path [num_req][max_nodes], -1 behind
 * them, their number accepted[r], next[r] = the last one's target (-1 where
 * none is) and new_len[r] = length[r] + accepted[r].
 * A request whose starts are not within [0, rows], descend or hold more than
 * max_nodes rows sets CI_DEVERR_REQ and accepts none.  parent as in
 * ci_draft_plan (values outside [-1, i - 1] belong to no path).
 */
CI_API int ci_draft_accept(const int32_t* req_start, const int32_t* length, const int32_t* parent, int32_t num_req,
                           int32_t max_nodes, int32_t rows, const int32_t* row_token, const int32_t* target,
                           const int32_t* cache_pos, int32_t* path, int32_t* accepted, int32_t* next, int32_t* new_len,
                           int32_t* dev_err, void* stream);

/*
 * In every pool, position length[r] + d of request r becomes what position
 * length[r] + path[r][d] was, for d < count[r].  path int32 [num_req] with
 * rows path_stride apart, count <= path_stride <= 256, ascending without
 * repetition and >= 0; else, or where a position passes 64 * max_pages, the
 * request is left as it is and CI_DEVERR_POS is set.  A page id outside
 * [0, num_pages) sets CI_DEVERR_PAGE and leaves that position as it is.  Pages
 * that hold positions from length[r] on belong to request r alone.
 * A page of pool i is uint8 [heads[i]][64 * row_bytes[i] + 64 * scale_bytes[i]]:
 * the 64 positions' rows, then their scales.  That is every cache pool
 * (row_bytes 2 D and no scales, or D and 4) and every index-K pool (one head;
 * 128 or 64, and 4).  pools, heads, row_bytes, scale_bytes: HOST arrays of
 * 1 <= num_pools <= 160 entries, read before the call returns; pools 16-byte
 * aligned and disjoint (CI_ERR_SHAPE otherwise: a pool that is there twice would be
 * moved twice), row_bytes a multiple of 16 (at most 2^20), scale_bytes 0 or 4.
 */
CI_API int ci_slots_move(uint8_t* const* pools, const int32_t* heads, const int32_t* row_bytes,
                         const int32_t* scale_bytes, int32_t num_pools, int64_t num_pages, const int32_t* page_table,
                         int32_t num_req, int32_t max_pages, const int32_t* length, const int32_t* path,
                         int32_t path_stride, const int32_t* count, int32_t* dev_err, void* stream);

/*
 * The reverse of ci_pages_alloc: request r shrinks from old_len[r] to
 * new_len[r] positions.  Its entries ceil(new / 64) .. ceil(old / 64) - 1 drop
 * one reference each and become -1 (entries that are -1 are passed over).  new
 * > old or a length outside [0, 64 * max_pages] sets CI_DEVERR_LEN and leaves
 * the request as it is; an entry >= num_pages or a page without references
 * sets CI_DEVERR_PAGE.  num_req <= 4096.
 */
CI_API int ci_pages_trim(int32_t* page_table, int32_t num_req, int32_t max_pages, int32_t* ref_count,
                         int64_t num_pages, const int32_t* old_len, const int32_t* new_len, int32_t* dev_err,
                         void* stream);

#ifdef __cplusplus
}
#endif
#endif /* CI_DRAFT_H_ */
