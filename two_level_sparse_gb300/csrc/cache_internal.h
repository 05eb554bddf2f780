// Host-side interface between the cache's C ABI (cache_api.cu) and its kernel
// launchers (attn.cu, append.cu, pages.cu).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace ci {

constexpr int kMaxPools = 160;

// The two pools of a layer and the way from a row's position to its page.
struct CacheArgs {
  uint8_t* k_pool;
  uint8_t* v_pool;
  int64_t num_pages;
  int32_t fp8;  // 0: bf16 pages, 1: e4m3 pages with fp32 scales
  int32_t num_q_heads, num_kv_heads, head_dim;
  const int32_t* page_table;
  int32_t max_pages;
  int32_t layout;
  const int32_t* req_start;
  int32_t num_req;
  int32_t* dev_err;
};

struct AttnArgs {
  CacheArgs c;
  const uint16_t* q;
  int64_t q_stride;
  int32_t rows;
  float scale;
  const int32_t* seq_len;
  int32_t max_len;
  const int32_t* pos;  // null: every position below the length
  int64_t pos_stride;
  int32_t npos;
  uint16_t* out;
  int64_t out_stride;
  float* lse;
  void* ws;
};

struct AppendArgs {
  CacheArgs c;
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  int32_t tokens;
  const float *q_norm, *k_norm;
  float eps;
  const float* cos_sin;
  int32_t max_pos, rot_dim, neox;
  const int32_t *positions, *cache_pos;
  uint16_t* q_out;
  int64_t q_out_stride;
};

struct PagesArgs {
  int32_t* page_table;
  int32_t num_req, max_pages;
  int32_t* ref_count;
  int64_t num_pages;
  int32_t* dev_err;
};

struct ForkArgs {
  PagesArgs p;
  const int32_t *parent, *child, *length;
  int32_t n;
  int32_t *copy_src, *copy_dst;
};

struct CompactArgs {
  PagesArgs p;
  int32_t *remap, *copy_src, *copy_dst, *count;
};

struct CopyArgs {
  uint8_t* pool[kMaxPools];
  int64_t page_bytes[kMaxPools];
  int32_t num_pools;
  int64_t num_pages;
  const int32_t *copy_src, *copy_dst;
  int32_t n;
  const int32_t* count;
  int32_t* dev_err;
};

// Each returns a cudaError_t from the launch (cudaSuccess when enqueued).
int64_t attn_workspace_bytes(int32_t rows, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim);
cudaError_t launch_attn(const AttnArgs& a, cudaStream_t stream);
cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream);
cudaError_t launch_pages_alloc(const PagesArgs& p, const int32_t* old_len, const int32_t* new_len, cudaStream_t stream);
cudaError_t launch_pages_fork(const ForkArgs& a, cudaStream_t stream);
cudaError_t launch_pages_free(const PagesArgs& p, const int32_t* req, int32_t n, cudaStream_t stream);
cudaError_t launch_pages_compact(const CompactArgs& a, cudaStream_t stream);
cudaError_t launch_pages_copy(const CopyArgs& a, cudaStream_t stream);

}  // namespace ci
