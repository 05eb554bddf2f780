// The C ABI declared in include/ci_draft.h: host-side argument checks, then
// the kernel launches.  No allocation, no synchronization.
#include <algorithm>

#include "../../include/ci_draft.h"
#include "ci_internal.h"
#include "draft_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int launched(cudaError_t e) { return e == cudaSuccess ? CI_OK : CI_ERR_CUDA; }

int check_requests(int32_t num_req, int32_t max_pages, int64_t num_pages) {
  if (num_req < 0 || max_pages < 0 || num_pages < 0) return CI_ERR_SHAPE;
  if (num_req > ci::kMaxReq || num_pages > INT32_MAX || max_pages > INT32_MAX / CI_PAGE) return CI_ERR_RANGE;
  return CI_OK;
}

int check_heads(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return CI_ERR_UNSUPPORTED;
  if (num_q_heads < 1 || num_kv_heads < 1 || num_q_heads % num_kv_heads != 0) return CI_ERR_SHAPE;
  if (num_q_heads > 65536 || num_q_heads / num_kv_heads > 128) return CI_ERR_RANGE;
  return CI_OK;
}

struct Span {  // of a pool's bytes
  uint64_t begin, end;
};
Span span_of(const uint8_t* pool, uint64_t page_bytes, uint64_t num_pages) {
  constexpr uint64_t kMost = UINT64_MAX / 2;
  const uint64_t begin = reinterpret_cast<uintptr_t>(pool);
  return {begin, begin + (num_pages > 0 && page_bytes > kMost / num_pages ? kMost : page_bytes * num_pages)};
}
// Whether two of them share bytes.
bool overlap(Span* spans, int n) {
  std::sort(spans, spans + n, [](const Span& x, const Span& y) { return x.begin < y.begin; });
  for (int i = 1; i < n; ++i)
    if (spans[i].begin < spans[i - 1].end) return true;
  return false;
}

}  // namespace

extern "C" {

int ci_draft_plan(const int32_t* length, const int32_t* count, const int32_t* parent, const int32_t* token,
                  int32_t num_req, int32_t max_nodes, const int32_t* page_table, int32_t max_pages, int64_t num_pages,
                  int32_t rows, int32_t* req_start, int32_t* positions, int32_t* cache_pos, uint32_t* mask,
                  int32_t mask_words, int32_t* row_token, int32_t* dev_err, void* stream) {
  const int st = check_requests(num_req, max_pages, num_pages);
  if (st != CI_OK) return st;
  if (rows < 0 || max_nodes < 1) return CI_ERR_SHAPE;
  if (max_nodes > CI_DRAFT_MAX_NODES || num_req < 1) return CI_ERR_RANGE;
  if (mask && (mask_words < 1 || mask_words > CI_DRAFT_MAX_NODES / 32 || 32 * mask_words < max_nodes)) return CI_ERR_SHAPE;
  if (!length || !count || !req_start) return CI_ERR_NULL;
  if (max_pages > 0 && !page_table) return CI_ERR_NULL;
  if (rows > 0 && (!positions || !cache_pos)) return CI_ERR_NULL;
  if (rows > 0 && (token == nullptr) != (row_token == nullptr)) return CI_ERR_NULL;
  const ci::PlanArgs a{length, count, parent, token, num_req, max_nodes, page_table, max_pages, num_pages, rows,
                       req_start, positions, cache_pos, mask, mask_words, row_token, dev_err};
  return launched(ci::launch_draft_plan(a, static_cast<cudaStream_t>(stream)));
}

int64_t ci_attn_draft_workspace_bytes(int32_t max_rows, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim) {
  const int st = check_heads(num_q_heads, num_kv_heads, head_dim);
  if (st != CI_OK) return st;
  if (max_rows < 0) return CI_ERR_SHAPE;
  return ci::attn_draft_workspace_bytes(max_rows, num_q_heads, num_kv_heads, head_dim);
}

int ci_attn_draft(const uint16_t* q, int64_t q_stride, int32_t rows, int32_t num_q_heads, int32_t num_kv_heads,
                  int32_t head_dim, float scale, const uint8_t* k_pool, const uint8_t* v_pool, int64_t num_pages,
                  int32_t cache_format, const int32_t* page_table, int32_t num_req, int32_t max_pages,
                  const int32_t* req_start, const int32_t* length, int32_t max_len, int32_t max_rows,
                  const uint32_t* mask, int32_t mask_words, uint16_t* out, int64_t out_stride, float* lse, void* ws,
                  int64_t ws_bytes, int32_t* dev_err, void* stream) {
  if (rows < 0 || max_len < 0) return CI_ERR_SHAPE;
  if (cache_format != CI_CACHE_BF16 && cache_format != CI_CACHE_FP8) return CI_ERR_UNSUPPORTED;
  int st = check_heads(num_q_heads, num_kv_heads, head_dim);
  if (st != CI_OK) return st;
  st = check_requests(num_req, max_pages, num_pages);
  if (st != CI_OK) return st;
  if (num_req < 1) return CI_ERR_RANGE;
  if (max_rows < 0) return CI_ERR_SHAPE;
  if (rows == 0) return CI_OK;
  if (mask && mask_words < 1) return CI_ERR_SHAPE;
  if (!q || !k_pool || !v_pool || !page_table || !req_start || !length || !out || !ws) return CI_ERR_NULL;
  if (num_pages < 1 || num_pages * num_kv_heads * (CI_PAGE + 256 / head_dim) > INT32_MAX) return CI_ERR_RANGE;
  if (static_cast<int64_t>(max_len) > static_cast<int64_t>(max_pages) * CI_PAGE) return CI_ERR_SHAPE;
  const int64_t width = static_cast<int64_t>(num_q_heads) * head_dim;
  if (rows > 1 && (q_stride < width || out_stride < width)) return CI_ERR_SHAPE;
  if (q_stride % 8 != 0 || out_stride % 8 != 0) return CI_ERR_ALIGN;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(ws, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16))
    return CI_ERR_ALIGN;
  const int64_t group = num_q_heads / num_kv_heads;
  if (rows * group > INT32_MAX) return CI_ERR_RANGE;
  const int64_t each = (max_rows * group + 127) / 128 * num_req, all = (rows * group + 127) / 128 + num_req;
  if (num_kv_heads * (each < all ? each : all) > INT32_MAX / (static_cast<int64_t>(max_len) / 128 + 1)) return CI_ERR_RANGE;
  if (ws_bytes < ci::attn_draft_workspace_bytes(max_rows, num_q_heads, num_kv_heads, head_dim)) return CI_ERR_SHAPE;
  const ci::DraftArgs a{{const_cast<uint8_t*>(k_pool), const_cast<uint8_t*>(v_pool), num_pages,
                         cache_format == CI_CACHE_FP8, num_q_heads, num_kv_heads, head_dim, page_table, max_pages,
                         CI_LAYOUT_VARLEN, req_start, num_req, dev_err},
                        q, q_stride, rows, scale, length, max_len, max_rows, mask, mask_words, out, out_stride, lse, ws};
  return launched(ci::launch_attn_draft(a, static_cast<cudaStream_t>(stream)));
}

int ci_draft_accept(const int32_t* req_start, const int32_t* length, const int32_t* parent, int32_t num_req,
                    int32_t max_nodes, int32_t rows, const int32_t* row_token, const int32_t* target,
                    const int32_t* cache_pos, int32_t* path, int32_t* accepted, int32_t* next, int32_t* new_len,
                    int32_t* dev_err, void* stream) {
  if (num_req < 0 || max_nodes < 1 || rows < 0) return CI_ERR_SHAPE;
  if (num_req > ci::kMaxReq || max_nodes > CI_DRAFT_MAX_NODES) return CI_ERR_RANGE;
  if (num_req == 0) return CI_OK;
  if (!req_start || !length || !path || !accepted || !next || !new_len) return CI_ERR_NULL;
  if (rows > 0 && (!row_token || !target)) return CI_ERR_NULL;
  const ci::AcceptArgs a{req_start, length, parent, num_req, max_nodes, rows, row_token, target, cache_pos,
                         path, accepted, next, new_len, dev_err};
  return launched(ci::launch_draft_accept(a, static_cast<cudaStream_t>(stream)));
}

int ci_slots_move(uint8_t* const* pools, const int32_t* heads, const int32_t* row_bytes, const int32_t* scale_bytes,
                  int32_t num_pools, int64_t num_pages, const int32_t* page_table, int32_t num_req, int32_t max_pages,
                  const int32_t* length, const int32_t* path, int32_t path_stride, const int32_t* count,
                  int32_t* dev_err, void* stream) {
  const int st = check_requests(num_req, max_pages, num_pages);
  if (st != CI_OK) return st;
  if (path_stride < 1) return CI_ERR_SHAPE;
  if (num_pools < 1 || num_pools > ci::kMaxPools || path_stride > CI_DRAFT_MAX_NODES) return CI_ERR_RANGE;
  if (!pools || !heads || !row_bytes || !scale_bytes) return CI_ERR_NULL;
  ci::MoveArgs a{};
  Span spans[ci::kMaxPools];
  for (int i = 0; i < num_pools; ++i) {
    if (!pools[i]) return CI_ERR_NULL;
    if (heads[i] < 1 || row_bytes[i] < 16 || row_bytes[i] > (1 << 20) || heads[i] > (1 << 16)) return CI_ERR_RANGE;
    if (scale_bytes[i] != 0 && scale_bytes[i] != 4) return CI_ERR_UNSUPPORTED;
    if (!aligned(pools[i], 16) || row_bytes[i] % 16 != 0) return CI_ERR_ALIGN;
    a.pool[i] = pools[i], a.heads[i] = heads[i], a.row_bytes[i] = row_bytes[i], a.scale_bytes[i] = scale_bytes[i];
    spans[i] = span_of(pools[i], static_cast<uint64_t>(heads[i]) * CI_PAGE * (row_bytes[i] + scale_bytes[i]), num_pages);
  }
  if (overlap(spans, num_pools)) return CI_ERR_SHAPE;
  if (num_req == 0) return CI_OK;
  if (!length || !path || !count || (max_pages > 0 && !page_table)) return CI_ERR_NULL;
  a.num_pools = num_pools, a.num_pages = num_pages, a.page_table = page_table, a.num_req = num_req,
  a.max_pages = max_pages, a.length = length, a.path = path, a.path_stride = path_stride, a.count = count,
  a.dev_err = dev_err;
  return launched(ci::launch_slots_move(a, static_cast<cudaStream_t>(stream)));
}

int ci_pages_trim(int32_t* page_table, int32_t num_req, int32_t max_pages, int32_t* ref_count, int64_t num_pages,
                  const int32_t* old_len, const int32_t* new_len, int32_t* dev_err, void* stream) {
  const int st = check_requests(num_req, max_pages, num_pages);
  if (st != CI_OK) return st;
  if (num_pages > 0 && !ref_count) return CI_ERR_NULL;
  if (num_req > 0 && max_pages > 0 && !page_table) return CI_ERR_NULL;
  if (num_req == 0) return CI_OK;
  if (!old_len || !new_len) return CI_ERR_NULL;
  const ci::PagesArgs p{page_table, num_req, max_pages, ref_count, num_pages, dev_err};
  return launched(ci::launch_pages_trim(p, old_len, new_len, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
