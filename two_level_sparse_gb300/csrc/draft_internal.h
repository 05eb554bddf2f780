// Host-side interface between the drafted step's C ABI (draft_api.cu) and its
// kernel launchers (draft.cu, attn_draft.cu).
#pragma once
#include "cache_internal.h"

namespace ci {

constexpr int kMaxNodes = 256;

struct PlanArgs {
  const int32_t *length, *count, *parent, *token;
  int32_t num_req, max_nodes;
  const int32_t* page_table;
  int32_t max_pages;
  int64_t num_pages;
  int32_t rows;
  int32_t *req_start, *positions, *cache_pos;
  uint32_t* mask;
  int32_t mask_words;
  int32_t* row_token;
  int32_t* dev_err;
};

struct AcceptArgs {
  const int32_t *req_start, *length, *parent;
  int32_t num_req, max_nodes, rows;
  const int32_t *row_token, *target, *cache_pos;
  int32_t *path, *accepted, *next, *new_len;
  int32_t* dev_err;
};

struct MoveArgs {
  uint8_t* pool[kMaxPools];
  int32_t heads[kMaxPools], row_bytes[kMaxPools], scale_bytes[kMaxPools];
  int32_t num_pools;
  int64_t num_pages;
  const int32_t* page_table;
  int32_t num_req, max_pages;
  const int32_t *length, *path;
  int32_t path_stride;
  const int32_t* count;
  int32_t* dev_err;
};

struct DraftArgs {
  CacheArgs c;  // (layout unused; req_start, num_req as in the header)
  const uint16_t* q;
  int64_t q_stride;
  int32_t rows;
  float scale;
  const int32_t* length;
  int32_t max_len, max_rows;
  const uint32_t* mask;  // null: a node sees every one up to itself
  int32_t mask_words;
  uint16_t* out;
  int64_t out_stride;
  float* lse;
  void* ws;
};

// Each returns a cudaError_t from the launch (cudaSuccess when enqueued).
cudaError_t launch_draft_plan(const PlanArgs& a, cudaStream_t stream);
cudaError_t launch_draft_accept(const AcceptArgs& a, cudaStream_t stream);
cudaError_t launch_slots_move(const MoveArgs& a, cudaStream_t stream);
cudaError_t launch_pages_trim(const PagesArgs& p, const int32_t* old_len, const int32_t* new_len, cudaStream_t stream);
int64_t attn_draft_workspace_bytes(int32_t max_rows, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim);
cudaError_t launch_attn_draft(const DraftArgs& a, cudaStream_t stream);

}  // namespace ci
