// The pages of a paged cache, managed on the device: allocation, forking with
// shared pages, release, compaction, and the copies that forks and compaction
// ask for (contract in include/ci_cache.h).
//
// A new page is always the lowest free id, so the results are functions of the
// inputs alone: no free list, only ref_count, scanned in order.  The scan is
// one cluster of eight CTAs: each of its 128 warps counts the free pages of a
// contiguous range of ids, the eight CTAs exchange their totals through
// distributed shared memory, and a second pass over the same range hands the
// pages out by rank.  One launch, no workspace; what bounds it is the latency
// of two passes of loads and a cluster barrier, not bytes (a pool of 2^19
// pages has 2 MB of counts, 16 KB per warp).
//
// Page tables are rewritten by plain grids.  Copies move `page_bytes` per pair
// and pool, read once and written once: a compaction of 6000 pages that moves 1394
// of 8 x 128 KB, 2.92 GB, takes 475-487 us, 452 of them the copy at 6.5 TB/s.  A fork
// of 64 requests of 16k-64k into 256 (81 MB of partly filled pages) takes 28 us with
// the release before it, 12 at the HBM's rate: three launches (release, fork, copy),
// each a chain of loads before the first byte moves.  An allocation of one page for
// each of 64 requests, 2^16 pages of which 64000 are taken: 11 us; for each of 4096: 27
// us; where none needs one: 9 and 13 us (single calls between events).
#include <cooperative_groups.h>

#include "cache_common.cuh"

namespace ci {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32, kCluster = 8;
constexpr int kStep = 128;  // ids per warp and step: one 16-byte load per lane
constexpr int kMaxDemands = kMaxReq;

// ref_count of ids 4 i .. 4 i + 3; -1 past the end (neither free nor live).
__device__ __forceinline__ int4 load_refs(const int32_t* ref, int64_t num_pages, int64_t i) {
  if (i + 3 < num_pages) return *reinterpret_cast<const int4*>(ref + i);
  int4 r = make_int4(-1, -1, -1, -1);
  if (i < num_pages) r.x = ref[i];
  if (i + 1 < num_pages) r.y = ref[i + 1];
  if (i + 2 < num_pages) r.z = ref[i + 2];
  return r;
}
__device__ __forceinline__ int count_free(int4 r) { return (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0); }
__device__ __forceinline__ int count_live(int4 r) { return (r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0); }

__device__ __forceinline__ int warp_inclusive(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The contiguous range of steps of this warp among the cluster's.
struct WarpRange {
  int64_t first, last;
};
__device__ __forceinline__ WarpRange warp_range(int64_t num_pages, int cta, int warp) {
  const int64_t steps = (num_pages + kStep - 1) / kStep;
  const int64_t per = (steps + kCluster * kWarps - 1) / (kCluster * kWarps);
  const int64_t first = per * (cta * kWarps + warp);
  return {min(first, steps), min(first + per, steps)};
}

template <bool kLive>
__device__ __forceinline__ int count_range(const int32_t* ref, int64_t num_pages, WarpRange w, int lane) {
  int n = 0;
#pragma unroll 4
  for (int64_t st = w.first; st < w.last; ++st) {
    const int4 r = load_refs(ref, num_pages, st * kStep + lane * 4);
    n += kLive ? count_live(r) : count_free(r);
  }
  return __reduce_add_sync(0xffffffffu, n);
}

// Exclusive prefix of `mine` (one value per warp) over the cluster's warps, in
// order, and the total.  wsum, ctot: shared memory of this CTA; the caller
// syncs the cluster before it leaves (others read ctot).
struct Scan {
  int before, total;
};
__device__ __forceinline__ Scan cluster_scan(cg::cluster_group& cl, int mine, int* wsum, int* ctot, int warp, int lane) {
  if (lane == 0) wsum[warp] = mine;
  __syncthreads();
  int before = 0, cta = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += wsum[w];
    cta += wsum[w];
  }
  if (threadIdx.x == 0) *ctot = cta;
  cl.sync();
  int total = 0;
  const int me = cl.block_rank();
#pragma unroll
  for (int r = 0; r < kCluster; ++r) {
    const int v = *cl.map_shared_rank(ctot, r);
    if (r < me) before += v;
    total += v;
  }
  return {before, total};
}

// Exclusive prefix of need(i), i < n, into prefix[0 .. n]; returns prefix[n].
// A thread takes as few neighbours as n allows: each is a chain of loads.
template <class Need>
__device__ int64_t demand_prefix(int n, int64_t* prefix, int64_t* wsum, Need need) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (n + kThreads - 1) / kThreads, i0 = min(tid * per, n), i1 = min(i0 + per, n);
  int64_t local = 0;
#pragma unroll 2
  for (int i = i0; i < i1; ++i) {
    const int64_t v = need(i);
    prefix[i] = v;
    local += v;
  }
  int64_t incl = local;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int64_t run = incl - local, total = 0;
#pragma unroll 4
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) run += wsum[w];
    total += wsum[w];
  }
  for (int i = i0; i < i1; ++i) {
    const int64_t v = prefix[i];
    prefix[i] = run;
    run += v;
  }
  if (tid == 0) prefix[n] = total;
  __syncthreads();
  return total;
}

// The demand i with prefix[i] <= rank < prefix[i + 1] (rank < prefix[n]).
__device__ __forceinline__ int demand_of(const int64_t* prefix, int n, int64_t rank) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= rank)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

struct AllocShared {
  int64_t prefix[kMaxDemands + 1];
  int64_t dsum[kWarps];
  int wsum[kWarps];
  int ctot;
};

// Hands the lowest free pages to the demands, in order: give(i, j, page) for
// the j-th page of demand i, with ref_count 1; give(i, j, -1) where none is
// left.  Executed by one cluster.
template <class Give>
__device__ void hand_out(cg::cluster_group& cl, AllocShared& sh, const PagesArgs& p, int n, int64_t wanted, Give give) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const WarpRange w = warp_range(p.num_pages, cl.block_rank(), warp);
  const Scan s = cluster_scan(cl, count_range<false>(p.ref_count, p.num_pages, w, lane), sh.wsum, &sh.ctot, warp, lane);
  int64_t base = s.before;
  for (int64_t st = w.first; st < w.last && base < wanted; ++st) {
    const int64_t id = st * kStep + lane * 4;
    const int4 r = load_refs(p.ref_count, p.num_pages, id);
    const int mine = count_free(r), incl = warp_inclusive(mine, lane);
    int64_t rank = base + incl - mine;
    const int v[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (v[j] != 0 || rank >= wanted) continue;
      const int i = demand_of(sh.prefix, n, rank);
      p.ref_count[id + j] = 1;
      give(i, static_cast<int>(rank - sh.prefix[i]), static_cast<int>(id + j));
      ++rank;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (s.total < wanted && cl.block_rank() == 0) {
    if (tid == 0) report(p.dev_err, kDevErrPage);
    for (int64_t rank = s.total + tid; rank < wanted; rank += kThreads) {
      const int i = demand_of(sh.prefix, n, rank);
      give(i, static_cast<int>(rank - sh.prefix[i]), -1);
    }
  }
  cl.sync();  // the other CTAs have read this one's total
}

__device__ __forceinline__ int pages_of(int len) { return (len + kPage - 1) / kPage; }
__device__ __forceinline__ bool length_ok(const PagesArgs& p, int len) {
  return len >= 0 && len <= static_cast<int64_t>(p.max_pages) * kPage;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    alloc_kernel(const PagesArgs p, const int32_t* old_len, const int32_t* new_len) {
  wait_predecessor();
  __shared__ AllocShared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int64_t wanted = demand_prefix(p.num_req, sh.prefix, sh.dsum, [&](int r) -> int64_t {
    const int a = old_len[r], b = new_len[r];
    if (!length_ok(p, a) || !length_ok(p, b) || b < a) {
      report(p.dev_err, kDevErrLen);
      return 0;
    }
    return pages_of(b) - pages_of(a);
  });
  hand_out(cl, sh, p, p.num_req, wanted, [&](int r, int j, int page) {
    p.page_table[static_cast<int64_t>(r) * p.max_pages + pages_of(old_len[r]) + j] = page;
  });
}

// Whether fork i is carried out; reported where it is not.
__device__ __forceinline__ bool fork_ok(const ForkArgs& a, int i, bool tell) {
  const int s = a.parent[i], c = a.child[i];
  const bool req = s >= 0 && s < a.p.num_req && c >= 0 && c < a.p.num_req && s != c, len = length_ok(a.p, a.length[i]);
  if (tell && !req) report(a.p.dev_err, kDevErrReq);
  if (tell && req && !len) report(a.p.dev_err, kDevErrLen);
  return req && len;
}
// The parent's partly filled last page; -1 where there is none.
__device__ __forceinline__ int fork_tail(const ForkArgs& a, int i, bool tell) {
  const int len = a.length[i];
  if (len % kPage == 0) return -1;
  const int page = a.p.page_table[static_cast<int64_t>(a.parent[i]) * a.p.max_pages + len / kPage];
  const bool ok = page >= 0 && page < a.p.num_pages;
  if (tell && !ok) report(a.p.dev_err, kDevErrPage);
  return ok ? page : -1;
}

// Cluster 0 hands out the pages of the partly filled ends; the other clusters
// share the full pages (references only ever rise there, so a page that is
// free to cluster 0 stays free: no order between the two is needed).
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) fork_kernel(const ForkArgs a) {
  wait_predecessor();
  const PagesArgs& p = a.p;
  if (blockIdx.x < kCluster) {
    __shared__ AllocShared sh;
    cg::cluster_group cl = cg::this_cluster();
    const bool tell = cl.block_rank() == 0;
    const int64_t wanted = demand_prefix(a.n, sh.prefix, sh.dsum, [&](int i) -> int64_t {
      const int tail = fork_ok(a, i, tell) ? fork_tail(a, i, tell) : -1;
      if (tell && tail < 0) a.copy_src[i] = a.copy_dst[i] = -1;
      return tail >= 0;
    });
    hand_out(cl, sh, p, a.n, wanted, [&](int i, int, int page) {
      a.copy_src[i] = page >= 0 ? fork_tail(a, i, false) : -1;
      a.copy_dst[i] = page;
      p.page_table[static_cast<int64_t>(a.child[i]) * p.max_pages + a.length[i] / kPage] = page;
    });
    return;
  }
  const int64_t entries = static_cast<int64_t>(a.n) * p.max_pages;
  const int64_t threads = static_cast<int64_t>(gridDim.x - kCluster) * kThreads;
  for (int64_t e = static_cast<int64_t>(blockIdx.x - kCluster) * kThreads + threadIdx.x; e < entries; e += threads) {
    const int i = static_cast<int>(e / p.max_pages), j = static_cast<int>(e - static_cast<int64_t>(i) * p.max_pages);
    if (!fork_ok(a, i, false)) continue;
    const int full = a.length[i] / kPage;
    int page = -1;
    if (j < full) {
      page = p.page_table[static_cast<int64_t>(a.parent[i]) * p.max_pages + j];
      if (page < 0 || page >= p.num_pages) {
        report(p.dev_err, kDevErrPage);
        page = -1;
      } else {
        atomicAdd(p.ref_count + page, 1);
      }
    } else if (j == full && fork_tail(a, i, false) >= 0) {
      continue;  // cluster 0 writes it
    }
    p.page_table[static_cast<int64_t>(a.child[i]) * p.max_pages + j] = page;
  }
}

__global__ void __launch_bounds__(kThreads) free_kernel(const PagesArgs p, const int32_t* req, int n) {
  wait_predecessor();
  const int64_t entries = static_cast<int64_t>(n) * p.max_pages;
  const int64_t threads = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; e < entries; e += threads) {
    const int i = static_cast<int>(e / p.max_pages), j = static_cast<int>(e - static_cast<int64_t>(i) * p.max_pages);
    const int r = req[i];
    if (r < 0 || r >= p.num_req) {
      if (j == 0) report(p.dev_err, kDevErrReq);
      continue;
    }
    int32_t* at = p.page_table + static_cast<int64_t>(r) * p.max_pages + j;
    const int page = *at;
    if (page < 0) continue;
    *at = -1;
    if (page >= p.num_pages) {
      report(p.dev_err, kDevErrPage);
    } else if (atomicSub(p.ref_count + page, 1) <= 0) {
      atomicAdd(p.ref_count + page, 1);
      report(p.dev_err, kDevErrPage);
    }
  }
}

// With P(i) the number of live ids below i and n the live ids in all: the
// free id i < n is hole i - P(i), the live id i >= n is mover P(i) - P(n).
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) compact_kernel(const CompactArgs a) {
  wait_predecessor();
  __shared__ int wsum[kWarps], ctot, below;  // below: P(n), in the CTA whose range holds id n
  const PagesArgs& p = a.p;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) below = -1;
  const WarpRange w = warp_range(p.num_pages, cl.block_rank(), warp);
  const Scan s = cluster_scan(cl, count_range<true>(p.ref_count, p.num_pages, w, lane), wsum, &ctot, warp, lane);
  const int64_t n = s.total;
  const int64_t step_n = n / kStep;
  if (n < p.num_pages && w.first <= step_n && step_n < w.last) {
    int c = 0;
    for (int64_t st = w.first; st <= step_n; ++st) {
      const int64_t id = st * kStep + lane * 4;
      const int4 r = load_refs(p.ref_count, p.num_pages, id);
      c += (r.x > 0 && id < n) + (r.y > 0 && id + 1 < n) + (r.z > 0 && id + 2 < n) + (r.w > 0 && id + 3 < n);
    }
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) below = s.before + c;
  }
  cl.sync();
  int64_t live_below = n;  // every id is live: P(n) = n
#pragma unroll
  for (int r = 0; r < kCluster; ++r) {
    const int v = *cl.map_shared_rank(&below, r);
    if (v >= 0) live_below = v;
  }
  const int64_t moves = n - live_below;
  int64_t base = s.before;
  for (int64_t st = w.first; st < w.last; ++st) {
    const int64_t id = st * kStep + lane * 4;
    const int4 r = load_refs(p.ref_count, p.num_pages, id);
    const int mine = count_live(r), incl = warp_inclusive(mine, lane);
    int64_t live = base + incl - mine;  // P(id)
    const int v[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t i = id + j;
      if (i >= p.num_pages) continue;
      if (v[j] <= 0 && i < n) a.copy_dst[i - live] = static_cast<int32_t>(i);
      if (v[j] > 0 && i >= n) a.copy_src[live - live_below] = static_cast<int32_t>(i);
      if (v[j] <= 0 || i < n) a.remap[i] = v[j] > 0 ? static_cast<int32_t>(i) : -1;
      live += v[j] > 0;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  cl.sync();  // the pairs are complete, and every count has been read
  const int64_t first = static_cast<int64_t>(cl.block_rank()) * kThreads + tid;
  for (int64_t i = first; i < moves; i += kCluster * kThreads) {
    const int src = a.copy_src[i], dst = a.copy_dst[i];
    a.remap[src] = dst;
    p.ref_count[dst] = p.ref_count[src];
    p.ref_count[src] = 0;
  }
  if (first == 0) *a.count = static_cast<int32_t>(moves);
}

// The second half of a compaction, over the whole card: the page table's
// entries, and the -1 behind the pairs.
__global__ void __launch_bounds__(kThreads) remap_kernel(const CompactArgs a) {
  wait_predecessor();
  const PagesArgs& p = a.p;
  const int64_t entries = static_cast<int64_t>(p.num_req) * p.max_pages, moves = *a.count;
  const int64_t threads = static_cast<int64_t>(gridDim.x) * kThreads;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  for (int64_t e = first; e < entries; e += threads) {
    const int page = p.page_table[e];
    if (page < 0) continue;
    if (page >= p.num_pages) report(p.dev_err, kDevErrPage);
    const int to = page < p.num_pages ? a.remap[page] : -1;
    if (to != page) p.page_table[e] = to;
  }
  for (int64_t i = moves + first; i < p.num_pages; i += threads) a.copy_src[i] = a.copy_dst[i] = -1;
}

constexpr int kCopyThreads = 256, kCopyLoads = 4;
constexpr int64_t kCopyChunk = kCopyThreads * kCopyLoads * 16;  // bytes per CTA and step

// One chunk of one page of one pool at a time.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyArgs a, int64_t chunks_per_pair) {
  wait_predecessor();
  const int64_t n = a.count != nullptr ? min(a.n, *a.count) : a.n;
  for (int64_t c = blockIdx.x; c < n * chunks_per_pair; c += gridDim.x) {
    const int64_t i = c / chunks_per_pair;
    int64_t rest = c - i * chunks_per_pair;
    const int src = a.copy_src[i], dst = a.copy_dst[i];
    if (src < 0 && dst < 0) continue;
    if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages) {
      if (threadIdx.x == 0) report(a.dev_err, kDevErrPage);
      continue;
    }
    int pool = 0;
    for (;; ++pool) {
      const int64_t here = (a.page_bytes[pool] + kCopyChunk - 1) / kCopyChunk;
      if (rest < here) break;
      rest -= here;
    }
    const int64_t bytes = a.page_bytes[pool];
    const uint8_t* from = a.pool[pool] + src * bytes;
    uint8_t* to = a.pool[pool] + dst * bytes;
    const int64_t at = rest * kCopyChunk + threadIdx.x * 16;
    uint4 v[kCopyLoads];
#pragma unroll
    for (int j = 0; j < kCopyLoads; ++j)
      if (at + j * kCopyThreads * 16 < bytes) v[j] = *reinterpret_cast<const uint4*>(from + at + j * kCopyThreads * 16);
#pragma unroll
    for (int j = 0; j < kCopyLoads; ++j)
      if (at + j * kCopyThreads * 16 < bytes) *reinterpret_cast<uint4*>(to + at + j * kCopyThreads * 16) = v[j];
  }
}

// CTAs for `work` items of a grid-stride loop.
unsigned grid_for(int64_t work, int per_cta, int ctas_per_sm) {
  const int64_t most = static_cast<int64_t>(device_sm_count()) * ctas_per_sm;
  const int64_t n = (work + per_cta - 1) / per_cta;
  return static_cast<unsigned>(n < 1 ? 1 : n < most ? n : most);
}

}  // namespace

cudaError_t launch_pages_alloc(const PagesArgs& p, const int32_t* old_len, const int32_t* new_len, cudaStream_t stream) {
  return launch_after(alloc_kernel, dim3(kCluster), kThreads, 0, stream, p, old_len, new_len);
}

cudaError_t launch_pages_fork(const ForkArgs& a, cudaStream_t stream) {
  const unsigned share = grid_for(static_cast<int64_t>(a.n) * a.p.max_pages, kThreads, 2);
  const unsigned clusters = 1 + (share + kCluster - 1) / kCluster;
  return launch_after(fork_kernel, dim3(clusters * kCluster), kThreads, 0, stream, a);
}

cudaError_t launch_pages_free(const PagesArgs& p, const int32_t* req, int32_t n, cudaStream_t stream) {
  return launch_after(free_kernel, dim3(grid_for(static_cast<int64_t>(n) * p.max_pages, kThreads, 2)), kThreads, 0, stream, p,
                      req, n);
}

cudaError_t launch_pages_compact(const CompactArgs& a, cudaStream_t stream) {
  const cudaError_t e = launch_after(compact_kernel, dim3(kCluster), kThreads, 0, stream, a);
  if (e != cudaSuccess) return e;
  const int64_t entries = static_cast<int64_t>(a.p.num_req) * a.p.max_pages;
  return launch_after(remap_kernel, dim3(grid_for(entries > a.p.num_pages ? entries : a.p.num_pages, kThreads, 2)), kThreads, 0,
                      stream, a);
}

cudaError_t launch_pages_copy(const CopyArgs& a, cudaStream_t stream) {
  int64_t per_pair = 0;
  for (int i = 0; i < a.num_pools; ++i) per_pair += (a.page_bytes[i] + kCopyChunk - 1) / kCopyChunk;
  return launch_after(copy_kernel, dim3(grid_for(a.n * per_pair, 1, 8)), kCopyThreads, 0, stream, a, per_pair);
}

}  // namespace ci
