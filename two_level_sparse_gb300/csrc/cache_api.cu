// The C ABI declared in include/ci_cache.h: host-side argument checks, then
// the kernel launches.  No allocation, no synchronization.
#include "../../include/ci_cache.h"
#include "cache_internal.h"
#include "ci_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int launched(cudaError_t e) { return e == cudaSuccess ? CI_OK : CI_ERR_CUDA; }

bool dim_ok(int32_t d) { return d == 64 || d == 128 || d == 256; }

// Heads, dims and format: what needs no data.
int check_heads(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, int32_t cache_format) {
  if (cache_format != CI_CACHE_BF16 && cache_format != CI_CACHE_FP8) return CI_ERR_UNSUPPORTED;
  if (!dim_ok(head_dim)) return CI_ERR_UNSUPPORTED;
  if (num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0) return CI_ERR_SHAPE;
  if (num_q_heads > 65536) return CI_ERR_RANGE;
  return CI_OK;
}

// The pools, the page table and the layout of `rows` > 0 rows.
int check_cache(const uint8_t* k_pool, const uint8_t* v_pool, int64_t num_pages, int32_t num_kv_heads, int32_t head_dim,
                const int32_t* page_table, int32_t num_req, int32_t max_pages, int32_t layout,
                const int32_t* req_row_start, int32_t rows) {
  if (!k_pool || !v_pool || !page_table) return CI_ERR_NULL;
  if (layout == CI_LAYOUT_DECODE && num_req != rows) return CI_ERR_SHAPE;
  if (layout == CI_LAYOUT_PREFILL && num_req != 1) return CI_ERR_SHAPE;
  if (layout == CI_LAYOUT_VARLEN) {
    if (!req_row_start) return CI_ERR_NULL;
    if (num_req < 1 || num_req > ci::kMaxReq) return CI_ERR_RANGE;
  }
  if (num_pages < 1 || num_pages > INT32_MAX || num_pages * num_kv_heads * (CI_PAGE + 256 / head_dim) > INT32_MAX)
    return CI_ERR_RANGE;
  if (!aligned(k_pool, 16) || !aligned(v_pool, 16)) return CI_ERR_ALIGN;
  return CI_OK;
}

bool layout_ok(int32_t layout) {
  return layout == CI_LAYOUT_DECODE || layout == CI_LAYOUT_PREFILL || layout == CI_LAYOUT_VARLEN;
}

// The page table, the counts and the number of requests of a page call.
int check_pages(const int32_t* page_table, int32_t num_req, int32_t max_pages, const int32_t* ref_count,
                int64_t num_pages) {
  if (num_req < 0 || max_pages < 0 || num_pages < 0) return CI_ERR_SHAPE;
  if (num_pages > INT32_MAX || max_pages > INT32_MAX / CI_PAGE) return CI_ERR_RANGE;
  if (num_pages > 0 && !ref_count) return CI_ERR_NULL;
  if (num_req > 0 && max_pages > 0 && !page_table) return CI_ERR_NULL;
  if (!aligned(ref_count, 16)) return CI_ERR_ALIGN;
  return CI_OK;
}

}  // namespace

extern "C" {

int64_t ci_cache_page_bytes(int32_t cache_format, int32_t head_dim) {
  const int st = check_heads(1, 1, head_dim, cache_format);
  if (st != CI_OK) return st;
  return cache_format == CI_CACHE_FP8 ? CI_PAGE * head_dim + CI_PAGE * 4 : CI_PAGE * head_dim * 2;
}

int64_t ci_attn_workspace_bytes(int32_t rows, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim) {
  const int st = check_heads(num_q_heads, num_kv_heads, head_dim, CI_CACHE_BF16);
  if (st != CI_OK) return st;
  if (rows < 0) return CI_ERR_SHAPE;
  if (num_q_heads / num_kv_heads > 128) return CI_ERR_RANGE;
  return ci::attn_workspace_bytes(rows, num_q_heads, num_kv_heads, head_dim);
}

int ci_attn_decode(const uint16_t* q, int64_t q_stride, int32_t rows, int32_t num_q_heads, int32_t num_kv_heads,
                   int32_t head_dim, float scale, const uint8_t* k_pool, const uint8_t* v_pool, int64_t num_pages,
                   int32_t cache_format, const int32_t* page_table, int32_t num_req, int32_t max_pages, int32_t layout,
                   const int32_t* req_row_start, const int32_t* seq_len, int32_t max_len, const int32_t* pos,
                   int64_t pos_stride, int32_t npos, uint16_t* out, int64_t out_stride, float* lse, void* ws,
                   int64_t ws_bytes, int32_t* dev_err, void* stream) {
  if (rows < 0 || max_len < 0 || num_req < 0 || max_pages < 0) return CI_ERR_SHAPE;
  if (!layout_ok(layout)) return CI_ERR_UNSUPPORTED;
  int st = check_heads(num_q_heads, num_kv_heads, head_dim, cache_format);
  if (st != CI_OK) return st;
  if (num_q_heads / num_kv_heads > 128) return CI_ERR_RANGE;
  if (rows == 0) return CI_OK;
  st = check_cache(k_pool, v_pool, num_pages, num_kv_heads, head_dim, page_table, num_req, max_pages, layout,
                   req_row_start, rows);
  if (st != CI_OK) return st;
  if (!q || !seq_len || !out || !ws) return CI_ERR_NULL;
  if (static_cast<int64_t>(max_len) > static_cast<int64_t>(max_pages) * CI_PAGE) return CI_ERR_SHAPE;
  if (pos != nullptr && (npos < 0 || (rows > 1 && pos_stride < npos))) return CI_ERR_SHAPE;
  const int64_t width = static_cast<int64_t>(num_q_heads) * head_dim;
  if (rows > 1 && (q_stride < width || out_stride < width)) return CI_ERR_SHAPE;
  if (q_stride % 8 != 0 || out_stride % 8 != 0) return CI_ERR_ALIGN;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(ws, 16)) return CI_ERR_ALIGN;
  if (ws_bytes < ci::attn_workspace_bytes(rows, num_q_heads, num_kv_heads, head_dim)) return CI_ERR_SHAPE;
  const int64_t tiles = (pos != nullptr ? npos : max_len) / CI_PAGE + 1, blocks = (num_q_heads / num_kv_heads + 63) / 64;
  if (tiles * num_kv_heads * blocks > INT32_MAX / rows) return CI_ERR_RANGE;
  const ci::AttnArgs a{{const_cast<uint8_t*>(k_pool), const_cast<uint8_t*>(v_pool), num_pages,
                        cache_format == CI_CACHE_FP8, num_q_heads, num_kv_heads, head_dim, page_table, max_pages,
                        layout, req_row_start, num_req, dev_err},
                       q, q_stride, rows, scale, seq_len, max_len, pos, pos_stride, npos, out, out_stride, lse, ws};
  return launched(ci::launch_attn(a, static_cast<cudaStream_t>(stream)));
}

int ci_qk_norm_rope_append(const uint16_t* q, int64_t q_stride, const uint16_t* k, int64_t k_stride, const uint16_t* v,
                           int64_t v_stride, int32_t tokens, int32_t num_q_heads, int32_t num_kv_heads,
                           int32_t head_dim, const float* q_norm, const float* k_norm, float eps, const float* cos_sin,
                           int32_t max_pos, int32_t rot_dim, int32_t is_neox, const int32_t* positions,
                           const int32_t* cache_pos, uint16_t* q_out, int64_t q_out_stride, uint8_t* k_pool,
                           uint8_t* v_pool, int64_t num_pages, int32_t cache_format, const int32_t* page_table,
                           int32_t num_req, int32_t max_pages, int32_t layout, const int32_t* req_row_start,
                           int32_t* dev_err, void* stream) {
  if (tokens < 0 || max_pos < 0 || num_req < 0 || max_pages < 0) return CI_ERR_SHAPE;
  if (!layout_ok(layout)) return CI_ERR_UNSUPPORTED;
  int st = check_heads(num_q_heads, num_kv_heads, head_dim, cache_format);
  if (st != CI_OK) return st;
  if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16 != 0) return CI_ERR_UNSUPPORTED;
  if (tokens == 0) return CI_OK;
  st = check_cache(k_pool, v_pool, num_pages, num_kv_heads, head_dim, page_table, num_req, max_pages, layout,
                   req_row_start, tokens);
  if (st != CI_OK) return st;
  if (!q || !k || !v || !positions || !q_out || (rot_dim > 0 && !cos_sin)) return CI_ERR_NULL;
  const int64_t qw = static_cast<int64_t>(num_q_heads) * head_dim, kw = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (tokens > 1 && (q_stride < qw || k_stride < kw || v_stride < kw || q_out_stride < qw)) return CI_ERR_SHAPE;
  if ((q_stride | k_stride | v_stride | q_out_stride) % 8 != 0) return CI_ERR_ALIGN;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(cos_sin, 16) ||
      !aligned(q_norm, 16) || !aligned(k_norm, 16))
    return CI_ERR_ALIGN;
  const ci::AppendArgs a{{k_pool, v_pool, num_pages, cache_format == CI_CACHE_FP8, num_q_heads, num_kv_heads, head_dim,
                          page_table, max_pages, layout, req_row_start, num_req, dev_err},
                         q, k, v, q_stride, k_stride, v_stride, tokens, q_norm, k_norm, eps, cos_sin, max_pos, rot_dim,
                         is_neox != 0, positions, cache_pos, q_out, q_out_stride};
  return launched(ci::launch_append(a, static_cast<cudaStream_t>(stream)));
}

int ci_pages_alloc(int32_t* page_table, int32_t num_req, int32_t max_pages, int32_t* ref_count, int64_t num_pages,
                   const int32_t* old_len, const int32_t* new_len, int32_t* dev_err, void* stream) {
  const int st = check_pages(page_table, num_req, max_pages, ref_count, num_pages);
  if (st != CI_OK) return st;
  if (num_req > ci::kMaxReq) return CI_ERR_RANGE;
  if (num_req == 0) return CI_OK;
  if (!old_len || !new_len) return CI_ERR_NULL;
  const ci::PagesArgs p{page_table, num_req, max_pages, ref_count, num_pages, dev_err};
  return launched(ci::launch_pages_alloc(p, old_len, new_len, static_cast<cudaStream_t>(stream)));
}

int ci_pages_fork(int32_t* page_table, int32_t num_req, int32_t max_pages, int32_t* ref_count, int64_t num_pages,
                  const int32_t* parent, const int32_t* child, const int32_t* length, int32_t n, int32_t* copy_src,
                  int32_t* copy_dst, int32_t* dev_err, void* stream) {
  const int st = check_pages(page_table, num_req, max_pages, ref_count, num_pages);
  if (st != CI_OK) return st;
  if (n < 0) return CI_ERR_SHAPE;
  if (n > ci::kMaxReq) return CI_ERR_RANGE;
  if (n == 0) return CI_OK;
  if (!parent || !child || !length || !copy_src || !copy_dst) return CI_ERR_NULL;
  const ci::ForkArgs a{{page_table, num_req, max_pages, ref_count, num_pages, dev_err}, parent, child, length, n,
                       copy_src, copy_dst};
  return launched(ci::launch_pages_fork(a, static_cast<cudaStream_t>(stream)));
}

int ci_pages_free(int32_t* page_table, int32_t num_req, int32_t max_pages, int32_t* ref_count, int64_t num_pages,
                  const int32_t* req, int32_t n, int32_t* dev_err, void* stream) {
  const int st = check_pages(page_table, num_req, max_pages, ref_count, num_pages);
  if (st != CI_OK) return st;
  if (n < 0) return CI_ERR_SHAPE;
  if (n > ci::kMaxReq) return CI_ERR_RANGE;
  if (n == 0) return CI_OK;
  if (!req) return CI_ERR_NULL;
  const ci::PagesArgs p{page_table, num_req, max_pages, ref_count, num_pages, dev_err};
  return launched(ci::launch_pages_free(p, req, n, static_cast<cudaStream_t>(stream)));
}

int ci_pages_compact(int32_t* page_table, int32_t num_req, int32_t max_pages, int32_t* ref_count, int64_t num_pages,
                     int32_t* remap, int32_t* copy_src, int32_t* copy_dst, int32_t* count, int32_t* dev_err,
                     void* stream) {
  const int st = check_pages(page_table, num_req, max_pages, ref_count, num_pages);
  if (st != CI_OK) return st;
  if (!count || (num_pages > 0 && (!remap || !copy_src || !copy_dst))) return CI_ERR_NULL;
  const ci::CompactArgs a{{page_table, num_req, max_pages, ref_count, num_pages, dev_err}, remap, copy_src, copy_dst,
                          count};
  return launched(ci::launch_pages_compact(a, static_cast<cudaStream_t>(stream)));
}

int ci_pages_copy(uint8_t* const* pools, const int64_t* page_bytes, int32_t num_pools, int64_t num_pages,
                  const int32_t* copy_src, const int32_t* copy_dst, int32_t n, const int32_t* count, int32_t* dev_err,
                  void* stream) {
  if (n < 0 || num_pages < 0) return CI_ERR_SHAPE;
  if (num_pools < 1 || num_pools > ci::kMaxPools || num_pages > INT32_MAX) return CI_ERR_RANGE;
  if (!pools || !page_bytes) return CI_ERR_NULL;
  ci::CopyArgs a{};
  for (int i = 0; i < num_pools; ++i) {
    if (!pools[i]) return CI_ERR_NULL;
    if (page_bytes[i] < 16 || page_bytes[i] > (int64_t{1} << 40)) return CI_ERR_RANGE;
    if (!aligned(pools[i], 16) || page_bytes[i] % 16 != 0) return CI_ERR_ALIGN;
    a.pool[i] = pools[i];
    a.page_bytes[i] = page_bytes[i];
  }
  if (n == 0) return CI_OK;
  if (!copy_src || !copy_dst) return CI_ERR_NULL;
  a.num_pools = num_pools, a.num_pages = num_pages, a.copy_src = copy_src, a.copy_dst = copy_dst, a.n = n,
  a.count = count, a.dev_err = dev_err;
  return launched(ci::launch_pages_copy(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
