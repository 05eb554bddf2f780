// Attention of drafted rows over the paged cache (contract in
// include/ci_draft.h).
//
// A warp per row and query head, 32 positions at a time: a lane computes the
// logit of its position, then the lanes share the dims of the sum.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "cache_common.cuh"
#include "draft_internal.h"

namespace ci {
namespace {

template <int D, bool kFp8>
__global__ void __launch_bounds__(128) draft_kernel(const DraftArgs a) {
  const int lane = threadIdx.x & 31;
  const CacheArgs& c = a.c;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  wait_predecessor();
  if (unit >= static_cast<int64_t>(a.rows) * c.num_q_heads) return;
  const int t = static_cast<int>(unit / c.num_q_heads), h = static_cast<int>(unit % c.num_q_heads);
  const int head = h / (c.num_q_heads / c.num_kv_heads);
  int r = -1;
  for (int x = lane; x < c.num_req; x += 32)
    if (c.req_start[x] < 0 || c.req_start[x] > c.req_start[x + 1] || c.req_start[x + 1] > a.rows)
      report(c.dev_err, kDevErrReq);
    else if (c.req_start[x] <= t && t < c.req_start[x + 1])
      r = x;
  r = __reduce_max_sync(0xffffffffu, r);
  if (r < 0) return;
  const int first = c.req_start[r], n = c.req_start[r + 1] - first;
  int len = a.length[r], all = 0;
  if (len < 0 || n > a.max_rows || static_cast<int64_t>(len) + n > a.max_len) {
    if (lane == 0) report(c.dev_err, kDevErrLen);
  } else {
    all = len + n;
  }
  float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
  for (int j = 0; j < D / 32; ++j) o[j] = 0.f;
  const uint16_t* q = a.q + t * a.q_stride + static_cast<int64_t>(h) * D;
  constexpr int64_t kHead = cache_page_bytes<kFp8>(D);
  auto value = [&](const uint8_t* at, int slot, int dim) {
    if (kFp8) {
      const uint8_t x = at[slot * D + dim];
      const float v = (x & 127) == 127 ? 480.f : __half2float(__half(__nv_cvt_fp8_to_halfraw(x & 127, __NV_E4M3)));
      return (x & 128 ? -v : v) * reinterpret_cast<const float*>(at + kPage * D)[slot];
    }
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(at)[slot * D + dim]);
  };
  for (int s0 = 0; s0 < all; s0 += 32) {
    const int s = s0 + lane, j = s - len;
    bool ok = s < all;
    if (ok && j >= 0) ok = a.mask != nullptr ? j < 32 * a.mask_words && (a.mask[static_cast<int64_t>(t) * a.mask_words + j / 32] >> (j % 32)) & 1 : j <= t - first;
    int page = ok ? c.page_table[static_cast<int64_t>(r) * c.max_pages + s / kPage] : 0;
    if (page < 0 || page >= c.num_pages) {
      report(c.dev_err, kDevErrPage);
      ok = false, page = 0;
    }
    const int64_t at = (static_cast<int64_t>(page) * c.num_kv_heads + head) * kHead;
    float x = -INFINITY;
    if (ok) {
      float dot = 0.f;
      for (int d = 0; d < D; ++d) dot += bf16_lo(q[d]) * value(c.k_pool + at, s % kPage, d);
      x = dot * a.scale;
    }
    float top = m;
    top = fmaxf(top, x);
    for (int b = 16; b > 0; b >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, b));
    const float ref = top == -INFINITY ? 0.f : top, f = expf(m - ref), p = ok ? expf(x - ref) : 0.f;
    m = top;
    l = l * f + p;
#pragma unroll
    for (int k = 0; k < D / 32; ++k) o[k] *= f;
    const uint32_t seen = __ballot_sync(0xffffffffu, ok);
    for (int i = 0; i < 32; ++i) {
      if (!((seen >> i) & 1)) continue;
      const float pi = __shfl_sync(0xffffffffu, p, i);
      const int64_t ai = __shfl_sync(0xffffffffu, at, i);
#pragma unroll
      for (int k = 0; k < D / 32; ++k) o[k] += pi * value(c.v_pool + ai, (s0 + i) % kPage, lane + 32 * k);
    }
  }
  for (int b = 16; b > 0; b >>= 1) l += __shfl_xor_sync(0xffffffffu, l, b);
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int k = 0; k < D / 32; ++k)
    a.out[t * a.out_stride + static_cast<int64_t>(h) * D + lane + 32 * k] = __bfloat16_as_ushort(__float2bfloat16_rn(o[k] * inv));
  if (a.lse != nullptr && lane == 0) a.lse[static_cast<int64_t>(t) * c.num_q_heads + h] = l == 0.f ? -INFINITY : m + logf(l);
}

template <int D>
cudaError_t launch_d(const DraftArgs& a, cudaStream_t stream) {
  const int64_t units = static_cast<int64_t>(a.rows) * a.c.num_q_heads;
  const dim3 grid(static_cast<unsigned>((units + 3) / 4));
  return a.c.fp8 ? launch_after(draft_kernel<D, true>, grid, 128, 0, stream, a)
                 : launch_after(draft_kernel<D, false>, grid, 128, 0, stream, a);
}

}  // namespace

int64_t attn_draft_workspace_bytes(int32_t, int32_t, int32_t, int32_t) { return 16; }

cudaError_t launch_attn_draft(const DraftArgs& a, cudaStream_t stream) {
  return a.c.head_dim == 64 ? launch_d<64>(a, stream) : a.c.head_dim == 128 ? launch_d<128>(a, stream) : launch_d<256>(a, stream);
}

}  // namespace ci
