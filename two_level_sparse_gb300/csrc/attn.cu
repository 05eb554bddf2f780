// Attention of query rows over the paged cache (contract in include/ci_cache.h).
//
// One warp per (row, query head): the positions one after another, the
// softmax's maximum and sum carried along.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "cache_common.cuh"

namespace ci {
namespace {

template <int D, bool kFp8>
__global__ void __launch_bounds__(128) attn_kernel(const AttnArgs a) {
  constexpr int kPer = D / 32;
  const CacheArgs& c = a.c;
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (w >= static_cast<int64_t>(a.rows) * c.num_q_heads) return;
  const int t = static_cast<int>(w / c.num_q_heads), h = static_cast<int>(w % c.num_q_heads);
  const int kvh = h / (c.num_q_heads / c.num_kv_heads);
  int len = a.seq_len[t];
  if (len < 0 || len > a.max_len) {
    if (lane == 0) report(c.dev_err, kDevErrLen);
    len = 0;
  }
  const int req = row_request(c, t);
  if (req < 0) len = 0;
  float q[kPer], o[kPer], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    q[j] = __uint_as_float(static_cast<uint32_t>(a.q[t * a.q_stride + h * D + j * 32 + lane]) << 16);
    o[j] = 0.f;
  }
  const int n = a.pos != nullptr ? a.npos : len;
  for (int i = 0; i < n; ++i) {
    const int s = a.pos != nullptr ? a.pos[t * a.pos_stride + i] : i;
    if (s < 0 || s >= len) {
      if (s != -1 && lane == 0) report(c.dev_err, kDevErrPos);
      continue;
    }
    const int page = c.page_table[static_cast<int64_t>(req) * c.max_pages + s / kPage];
    if (page < 0 || page >= c.num_pages) {
      if (lane == 0) report(c.dev_err, kDevErrPage);
      continue;
    }
    const int64_t at = (static_cast<int64_t>(page) * c.num_kv_heads + kvh) * cache_page_bytes<kFp8>(D);
    const int slot = s % kPage;
    float ks = 1.f, vs = 1.f, k[kPer], v[kPer];
    if (kFp8) {
      ks = reinterpret_cast<const float*>(c.k_pool + at + kPage * D)[slot];
      vs = reinterpret_cast<const float*>(c.v_pool + at + kPage * D)[slot];
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = slot * D + j * 32 + lane;
      if (kFp8) {
        k[j] = static_cast<float>(reinterpret_cast<const __nv_fp8_e4m3*>(c.k_pool + at)[e]);
        v[j] = static_cast<float>(reinterpret_cast<const __nv_fp8_e4m3*>(c.v_pool + at)[e]);
      } else {
        k[j] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(c.k_pool + at)[e]);
        v[j] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(c.v_pool + at)[e]);
      }
    }
    float x = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) x = fmaf(q[j], k[j], x);
#pragma unroll
    for (int b = 16; b > 0; b >>= 1) x += __shfl_xor_sync(0xffffffffu, x, b);
    x *= ks * a.scale;
    const float top = fmaxf(m, x), keep = m == -INFINITY ? 0.f : __expf(m - top);
    const float p = x == -INFINITY ? 0.f : __expf(x - top);
    l = l * keep + p;
#pragma unroll
    for (int j = 0; j < kPer; ++j) o[j] = o[j] * keep + p * vs * v[j];
    m = top;
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    a.out[t * a.out_stride + h * D + j * 32 + lane] =
        __bfloat16_as_ushort(__float2bfloat16_rn(l == 0.f ? 0.f : o[j] / l));
  if (a.lse != nullptr && lane == 0) a.lse[w] = l == 0.f ? -INFINITY : m + logf(l);
}

template <int D>
void launch_d(const AttnArgs& a, unsigned grid, cudaStream_t stream) {
  if (a.c.fp8)
    attn_kernel<D, true><<<grid, 128, 0, stream>>>(a);
  else
    attn_kernel<D, false><<<grid, 128, 0, stream>>>(a);
}

}  // namespace

int64_t attn_workspace_bytes(int32_t, int32_t, int32_t, int32_t) { return 16; }

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(a.rows) * a.c.num_q_heads + 3) / 4);
  if (a.c.head_dim == 64)
    launch_d<64>(a, grid, stream);
  else if (a.c.head_dim == 128)
    launch_d<128>(a, grid, stream);
  else
    launch_d<256>(a, grid, stream);
  return cudaGetLastError();
}

}  // namespace ci
