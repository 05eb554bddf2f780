// A drafted step's bookkeeping over the paged cache: its rows, the accepted
// path, the moves of what is kept, the release of what is not (contract in
// include/ci_draft.h).  All of it is bound by latency: a launch, and a chain of
// dependent loads as long as a tree is deep.  200 requests of up to 64 nodes (8
// of 16), by the kernels' own clock: plan 6.8 us (3.1), accept 2.3 (1.7), trim 1.3
// (1.3), the moves of three tokens a request in 40 pools 10.0 (in 2: 2.5); 30 and
// 45 us for plan and commit as Python calls, which are as long as their host side.
#include "cache_common.cuh"
#include "draft_internal.h"

namespace ci {
namespace {

constexpr int kAll = -1;  // every lane's bit
constexpr int kWarps = 4, kThreads = 32 * kWarps, kWords = kMaxNodes / 32;

// The nodes of request r; 0 (and `bad`) where its count or length is none.
__device__ __forceinline__ int plan_count(const PlanArgs& a, int r, bool& bad) {
  const int n = a.count[r], len = a.length[r];
  bad = n < 0 || n > a.max_nodes || len < 0 || static_cast<int64_t>(len) + n > static_cast<int64_t>(a.max_pages) * kPage;
  return bad ? 0 : n;
}

// A warp per request.  Rows start behind those of the requests before, which
// every CTA adds up for itself (4096 counts at most).  anc(i) = {i} u
// anc(parent(i)), node by node: lane w has word w of every node's set, so a node
// costs a load and a store of shared memory and no exchange; the depth is the
// size of the set less one.
__global__ void __launch_bounds__(kThreads) plan_kernel(const PlanArgs a) {
  __shared__ uint32_t anc[kWarps][kMaxNodes][kWords];
  __shared__ int sum[2][kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r0 = blockIdx.x * kWarps, r = r0 + warp;
  wait_predecessor();
  int before = 0, all = 0;
  bool bad = false;
#pragma unroll 4
  for (int i = threadIdx.x; i < a.num_req; i += kThreads) {
    const int n = plan_count(a, i, bad);
    all += n;
    if (i < r0) before += n;
  }
  before = __reduce_add_sync(kAll, before), all = __reduce_add_sync(kAll, all);
  if (lane == 0) sum[0][warp] = before, sum[1][warp] = all;
  __syncthreads();
  int start = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) start += sum[0][w], total += sum[1][w];
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.req_start[a.num_req] = min(total, a.rows);
    if (total > a.rows) report(a.dev_err, kDevErrLen);
  }
  for (int64_t t = total + static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; t < a.rows;
       t += static_cast<int64_t>(gridDim.x) * kThreads) {  // rows of no request
    a.positions[t] = 0, a.cache_pos[t] = -1;
    if (a.row_token != nullptr) a.row_token[t] = 0;
    if (a.mask != nullptr)
      for (int w = 0; w < a.mask_words; ++w) a.mask[t * a.mask_words + w] = 0;
  }
  if (r >= a.num_req) return;
#pragma unroll 1
  for (int i = r0; i < r; ++i) start += plan_count(a, i, bad);
  int n = plan_count(a, r, bad);
  if (bad && lane == 0) report(a.dev_err, kDevErrLen);
  start = min(start, a.rows);
  n = min(n, a.rows - start);
  if (lane == 0) a.req_start[r] = start;
  const int len = a.length[r];
  const int32_t* table = a.page_table + static_cast<int64_t>(r) * a.max_pages;
  const int32_t* parent = a.parent != nullptr ? a.parent + static_cast<int64_t>(r) * a.max_nodes : nullptr;
  uint32_t(*set)[kWords] = anc[warp];
#pragma unroll 1
  for (int base = 0; base < n; base += 32) {
    const int i = base + lane;
    int up = i - 1;
    if (parent != nullptr && i < n) up = parent[i];
    const bool ok = up >= -1 && up < i;
    if (i < n && !ok) report(a.dev_err, kDevErrPos);
    if (!ok) up = -2;
    const int here = min(32, n - base);
#pragma unroll 4
    for (int j = 0; j < here; ++j) {
      const int p = __shfl_sync(kAll, up, j);
      if (lane >= kWords) continue;
      uint32_t m = p >= 0 ? set[p][lane] : 0;
      if (p != -2 && lane == base / 32) m |= 1u << j;
      set[base + j][lane] = m;
    }
    __syncwarp();
    if (i < n) {
      const int64_t t = start + i;
      int depth = -1;
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        const uint32_t m = set[i][w];
        depth += __popc(m);
        if (a.mask != nullptr && w < a.mask_words) a.mask[t * a.mask_words + w] = m;
      }
      const int at = len + i, page = table[at / kPage];
      a.positions[t] = len + max(depth, 0);
      a.cache_pos[t] = ok && page >= 0 && page < a.num_pages ? at : -1;
      if (a.row_token != nullptr) a.row_token[t] = a.token[static_cast<int64_t>(r) * a.max_nodes + i];
    }
  }
}

// A warp per request, its nodes dealt to the lanes: a step of the path is a
// vote on who is a fitting child of the last node.
template <int kPer>
__global__ void __launch_bounds__(kThreads) accept_kernel(const AcceptArgs a) {
  const int lane = threadIdx.x & 31, r = blockIdx.x * kWarps + (threadIdx.x >> 5);
  wait_predecessor();
  if (r >= a.num_req) return;
  const int first = a.req_start[r], end = a.req_start[r + 1], len = a.length[r];
  int n = end - first;
  if (first < 0 || first > end || end > a.rows || n > a.max_nodes) {
    if (lane == 0) report(a.dev_err, kDevErrReq);
    n = 0;
  }
  int parent[kPer], token[kPer], target[kPer], path[kPer];
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = 32 * k + lane;
    parent[k] = -2, token[k] = target[k] = 0, path[k] = -1;
    if (i >= n) continue;
    const int64_t t = first + i;
    token[k] = a.row_token[t], target[k] = a.target[t];
    parent[k] = a.parent != nullptr ? a.parent[static_cast<int64_t>(r) * a.max_nodes + i] : i - 1;
    if (i == 0) parent[k] = -1;  // (whatever it says)
    if (parent[k] >= i || (a.cache_pos != nullptr && a.cache_pos[t] < 0)) parent[k] = -2;
  }
  const bool begins = __shfl_sync(kAll, parent[0], 0) == -1;
  int node = begins ? 0 : -1, taken = 0, says = -1;
#pragma unroll 1
  while (node >= 0) {
    int up = -1;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (32 * k + lane == taken) path[k] = node;
      const int x = __shfl_sync(kAll, target[k], node & 31);
      if (k == node >> 5) says = x;
    }
    ++taken;
#pragma unroll
    for (int k = kPer - 1; k >= 0; --k) {
      const uint32_t fits = __ballot_sync(kAll, parent[k] == node && token[k] == says);
      if (fits != 0) up = 32 * k + __ffs(fits) - 1;
    }
    node = up;  // (a child is a later node: at most n steps)
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k)
    if (32 * k + lane < a.max_nodes) a.path[static_cast<int64_t>(r) * a.max_nodes + 32 * k + lane] = path[k];
  if (lane == 0) a.accepted[r] = taken, a.next[r] = says, a.new_len[r] = len + taken;
}

// CTA (r, y): request r's moves in every gridDim.y-th pool.  A thread has a
// column, 16 bytes of a head's row or a head's scale, and takes the positions
// in order: path ascends, so position d is written after every read of it
// (path[e] > d for e > d), and four are in flight at a time.
constexpr int kMoveThreads = 128, kFlight = 4;
template <class T>
__device__ __forceinline__ void move_column(uint8_t* base, int64_t page_bytes, int64_t offset, int step,
                                            const int2* from, const int2* to, int first, int n) {
#pragma unroll 1
  for (int d = first; d < n; d += kFlight) {
    T v[kFlight];
#pragma unroll
    for (int j = 0; j < kFlight; ++j)
      if (d + j < n && to[d + j].x >= 0)
        v[j] = *reinterpret_cast<const T*>(base + from[d + j].x * page_bytes + offset + from[d + j].y * step);
#pragma unroll
    for (int j = 0; j < kFlight; ++j)
      if (d + j < n && to[d + j].x >= 0)
        *reinterpret_cast<T*>(base + to[d + j].x * page_bytes + offset + to[d + j].y * step) = v[j];
  }
}

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ MoveArgs a) {
  __shared__ int2 from[kMaxNodes], to[kMaxNodes];  // page (-1: left out) and slot
  __shared__ int begin;
  const int r = blockIdx.x, tid = threadIdx.x;
  wait_predecessor();
  const int n = a.count[r], len = a.length[r];
  if (n == 0) return;
  if (tid == 0) begin = n;
  __syncthreads();
  const int32_t* path = a.path + static_cast<int64_t>(r) * a.path_stride;
  const int32_t* table = a.page_table + static_cast<int64_t>(r) * a.max_pages;
  bool bad = n < 0 || n > a.path_stride || len < 0;
#pragma unroll 1
  for (int d = tid; d < n && !bad; d += kMoveThreads) {
    const int x = path[d];
    bad = x < d || (d > 0 && x <= path[d - 1]) ||
          static_cast<int64_t>(len) + x >= static_cast<int64_t>(a.max_pages) * kPage;
    if (bad || x == d) {
      to[d].x = -1;
      continue;
    }
    atomicMin(&begin, d);
    const int src = table[(len + x) / kPage], dst = table[(len + d) / kPage];
    const bool ok = src >= 0 && src < a.num_pages && dst >= 0 && dst < a.num_pages;
    if (!ok && blockIdx.y == 0) report(a.dev_err, kDevErrPage);
    from[d] = make_int2(src, (len + x) & (kPage - 1));
    to[d] = make_int2(ok ? dst : -1, (len + d) & (kPage - 1));
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0 && blockIdx.y == 0) report(a.dev_err, kDevErrPos);
    return;
  }
#pragma unroll 1
  for (int p = blockIdx.y; p < a.num_pools; p += gridDim.y) {
    const int row = a.row_bytes[p], scale = a.scale_bytes[p], heads = a.heads[p], per = row / 16;
    const int64_t head_bytes = static_cast<int64_t>(kPage) * (row + scale), page_bytes = heads * head_bytes;
    const int64_t columns = static_cast<int64_t>(heads) * per, all = columns + (scale != 0 ? heads : 0);
#pragma unroll 1
    for (int64_t c = tid; c < all; c += kMoveThreads) {
      if (c < columns) {
        const int64_t h = c / per;
        move_column<uint4>(a.pool[p], page_bytes, h * head_bytes + (c - h * per) * 16, row, from, to, begin, n);
      } else {
        move_column<uint32_t>(a.pool[p], page_bytes, (c - columns) * head_bytes + static_cast<int64_t>(kPage) * row, 4, from,
                              to, begin, n);
      }
    }
  }
}

// A warp per request.
__global__ void __launch_bounds__(kThreads) trim_kernel(const PagesArgs p, const int32_t* old_len, const int32_t* new_len) {
  const int lane = threadIdx.x & 31, r = blockIdx.x * kWarps + (threadIdx.x >> 5);
  wait_predecessor();
  if (r >= p.num_req) return;
  const int64_t old = old_len[r], len = new_len[r];
  if (len < 0 || len > old || old > static_cast<int64_t>(p.max_pages) * kPage) {
    if (lane == 0) report(p.dev_err, kDevErrLen);
    return;
  }
  int32_t* row = p.page_table + static_cast<int64_t>(r) * p.max_pages;
#pragma unroll 1
  for (int64_t j = (len + kPage - 1) / kPage + lane; j < (old + kPage - 1) / kPage; j += 32) {
    const int page = row[j];
    if (page < 0) continue;
    row[j] = -1;
    if (page >= p.num_pages) {
      report(p.dev_err, kDevErrPage);
    } else if (atomicSub(p.ref_count + page, 1) <= 0) {
      atomicAdd(p.ref_count + page, 1);
      report(p.dev_err, kDevErrPage);
    }
  }
}

dim3 warp_per_request(int32_t num_req) { return dim3((num_req + kWarps - 1) / kWarps); }

}  // namespace

cudaError_t launch_draft_plan(const PlanArgs& a, cudaStream_t stream) {
  return launch_after(plan_kernel, warp_per_request(a.num_req), kThreads, 0, stream, a);
}

cudaError_t launch_draft_accept(const AcceptArgs& a, cudaStream_t stream) {
  const dim3 grid = warp_per_request(a.num_req);
  const int per = (a.max_nodes + 31) / 32;
  return per <= 2   ? launch_after(accept_kernel<2>, grid, kThreads, 0, stream, a)
         : per <= 4 ? launch_after(accept_kernel<4>, grid, kThreads, 0, stream, a)
                    : launch_after(accept_kernel<kWords>, grid, kThreads, 0, stream, a);
}

cudaError_t launch_slots_move(const MoveArgs& a, cudaStream_t stream) {
  const int want = 8 * device_sm_count() / a.num_req + 1;
  return launch_after(move_kernel, dim3(a.num_req, want < a.num_pools ? want : a.num_pools), kMoveThreads, 0, stream, a);
}

cudaError_t launch_pages_trim(const PagesArgs& p, const int32_t* old_len, const int32_t* new_len, cudaStream_t stream) {
  return launch_after(trim_kernel, warp_per_request(p.num_req), kThreads, 0, stream, p, old_len, new_len);
}

}  // namespace ci
