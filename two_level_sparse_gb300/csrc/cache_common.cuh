// Device helpers shared by the cache's kernels.
#pragma once
#include "cache_internal.h"
#include "ci_common.cuh"
#include "ci_internal.h"

namespace ci {

// Every kernel of the cache is launched to begin while its predecessor in the
// stream ends (programmatic dependent launch), and waits here for that one's
// results before it touches global memory.
__device__ __forceinline__ void wait_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the successor's CTAs be scheduled; it still waits for this kernel's end.
__device__ __forceinline__ void release_successor() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// The request of row t; -1 (reported) where the row starts name none.
static __device__ __noinline__ int row_request_varlen(const CacheArgs& c, int t) {
  int lo = 0, hi = c.num_req;  // the last r with req_start[r] <= t
#pragma unroll 1
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (c.req_start[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  if (c.req_start[lo] <= t && t < c.req_start[lo + 1]) return lo;
  report(c.dev_err, kDevErrReq);
  return -1;
}
__device__ __forceinline__ int row_request(const CacheArgs& c, int t) {
  return c.layout == kLayoutDecode ? t : c.layout == kLayoutPrefill ? 0 : row_request_varlen(c, t);
}

template <bool kFp8>
__host__ __device__ constexpr int64_t cache_page_bytes(int d) {
  return kFp8 ? kPage * d + kPage * 4 : kPage * d * 2;
}

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

}  // namespace ci
