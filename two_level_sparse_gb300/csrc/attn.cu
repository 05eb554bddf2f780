// Attention over the paged cache: dispatch, the workspace's layout, and the
// join of units that several CTAs worked on (contract in include/ci_cache.h;
// the main kernel is in attn.cuh).
#include "attn.cuh"

namespace ci {
namespace {

using attn::Args;
using attn::Layout;
using attn::Part;

constexpr int kJoinWarps = 16;

// Whether the kernel of attn_wide.cu takes the call.
bool is_wide(const CacheArgs& c) { return !c.fp8 && c.head_dim == 128 && c.num_q_heads / c.num_kv_heads > 16; }

Layout layout_of(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, bool wide) {
  const int group = num_q_heads / num_kv_heads;
  const int heads = wide ? 64 : group <= 8 ? 8 : group <= 16 ? 16 : group <= 32 ? 32 : 64;
  return Layout{device_sm_count() * (head_dim == 256 ? 1 : 2), heads, (group + heads - 1) / heads, group};
}

// With the parts' maxima m_i, sums l_i and unnormalised sums o_i:
//   m = max m_i;  l = sum l_i 2^(m_i - m);  out = sum o_i 2^(m_i - m) / l.
// CTA (x, y) takes the x-th split unit and 16 / ways of its heads; a head's
// parts are dealt to `ways` warps, whose sums are added in order.  Bound by
// the latency of its loads (the parts sit in L2), so few parts per warp.
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const Args k, int ways) {
  constexpr int kPer = D / 32;
  __shared__ float sums[kJoinWarps][D];
  __shared__ int counts[kJoinWarps], starts;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) starts = -1;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the CTA in whose range the x-th split unit starts
  int seen = 0;
  for (int c0 = 0; c0 < k.l.ctas; c0 += 32 * kJoinWarps) {
    const bool one = c0 + tid < k.l.ctas && k.part[c0 + tid].last >= 0;
    const uint32_t b = __ballot_sync(0xffffffffu, one);
    if (lane == 0) counts[warp] = __popc(b);
    __syncthreads();
    int before = seen + __popc(b & lanemask_lt());
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      if (w < warp) before += counts[w];
      seen += counts[w];
    }
    if (one && before == static_cast<int>(blockIdx.x)) starts = c0 + tid;
    __syncthreads();
  }
  const int first = starts;
  if (first < 0) return;
  const Part p = k.part[first];
  const int hw = warp / ways, way = warp - hw * ways;
  const int heads = k.l.heads, h = blockIdx.y * (kJoinWarps / ways) + hw;
  const int head = p.unit / k.l.blocks, hb = p.unit - head * k.l.blocks;
  const bool live = h < heads && hb * heads + h < k.l.group;
  const int n = p.last - first + 1;
  auto slot = [&](int i) -> int64_t { return i == 0 ? 2ll * first + 1 : 2ll * (first + i); };
  float m = -INFINITY, l = 0.f, o[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) o[j] = 0.f;
  if (live) {
    const float2* stat = reinterpret_cast<const float2*>(k.stat) + h;
    for (int i = lane; i < n; i += 32) {
      const float2 st = stat[slot(i) * heads];
      const float top = fmaxf(m, st.x), ref = top == -INFINITY ? 0.f : top;
      l = l * attn::exp2_approx(m - ref) + st.y * attn::exp2_approx(st.x - ref);
      m = top;
    }
    float top = m;
#pragma unroll
    for (int b = 16; b > 0; b >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, b));
    const float ref = top == -INFINITY ? 0.f : top;
    l *= attn::exp2_approx(m - ref);
    m = top;
#pragma unroll
    for (int b = 16; b > 0; b >>= 1) l += __shfl_xor_sync(0xffffffffu, l, b);
#pragma unroll 4
    for (int i = way; i < n; i += ways) {
      const float f = attn::exp2_approx(stat[slot(i) * heads].x - ref);
      const float* src = k.sum + (slot(i) * heads + h) * D + lane;
#pragma unroll
      for (int j = 0; j < kPer; ++j) o[j] += f * src[32 * j];
    }
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) sums[warp][32 * j + lane] = o[j];
  __syncthreads();
  if (!live || way != 0) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t qh = static_cast<int64_t>(head) * k.l.group + hb * heads + h;
  uint16_t* dst = k.a.out + p.row * k.a.out_stride + qh * D;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    float v = 0.f;
    for (int x = 0; x < ways; ++x) v += sums[warp + x][32 * j + lane];
    dst[32 * j + lane] = __bfloat16_as_ushort(__float2bfloat16_rn(v * inv));
  }
  if (k.a.lse != nullptr && lane == 0)
    k.a.lse[static_cast<int64_t>(p.row) * k.a.c.num_q_heads + qh] =
        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

int64_t part_bytes(const Layout& l) { return (static_cast<int64_t>(l.ctas) * sizeof(Part) + 15) / 16 * 16; }
int64_t stat_bytes(const Layout& l) { return 2ll * l.ctas * l.heads * 2 * 4; }

template <int D>
cudaError_t launch_join(const Args& k, cudaStream_t stream) {
  // Units number rows * kv heads * blocks; at most one starts unfinished in a
  // CTA's range.  The fewer units, the more parts each: 16, 4 or 1 warps a head.
  const int64_t units = static_cast<int64_t>(k.a.rows) * k.a.c.num_kv_heads * k.l.blocks;
  const int64_t split = units < k.l.ctas ? units : k.l.ctas, parts = k.l.ctas / split + 1;
  const int ways = parts > 16 ? 16 : parts > 4 ? 4 : 1, per = kJoinWarps / ways;
  const int heads = k.l.heads < k.l.group ? k.l.heads : k.l.group;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(split), (heads + per - 1) / per);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<D>, k, ways);
}

}  // namespace

int64_t attn_workspace_bytes(int32_t, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim) {
  int64_t most = 0;  // either kernel may take the call: the cache's format is not known here
  for (const bool wide : {false, true}) {
    const Layout l = layout_of(num_q_heads, num_kv_heads, head_dim, wide);
    const int64_t n = part_bytes(l) + stat_bytes(l) + 2ll * l.ctas * l.heads * head_dim * 4;
    most = n > most ? n : most;
  }
  return most;
}

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t stream) {
  const CacheArgs& c = a.c;
  const bool wide = is_wide(c);
  Args k{a, layout_of(c.num_q_heads, c.num_kv_heads, c.head_dim, wide), nullptr, nullptr, nullptr};
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  k.part = reinterpret_cast<Part*>(ws);
  k.stat = reinterpret_cast<float*>(ws + part_bytes(k.l));
  k.sum = reinterpret_cast<float*>(ws + part_bytes(k.l) + stat_bytes(k.l));
  const int row = c.fp8 ? c.head_dim : 2 * c.head_dim;
  const int per_page = static_cast<int>((c.fp8 ? cache_page_bytes<true>(c.head_dim) : cache_page_bytes<false>(c.head_dim)) / row);
  CUtensorMap kmap, vmap;
  cudaError_t e = make_rows_tmap(&kmap, c.k_pool, c.num_pages * c.num_kv_heads * per_page, row, a.pos != nullptr ? 1 : attn::kTile);
  if (e == cudaSuccess)
    e = make_rows_tmap(&vmap, c.v_pool, c.num_pages * c.num_kv_heads * per_page, row, attn::kTile);
  if (e == cudaSuccess)
    e = wide ? attn::launch_wide(kmap, vmap, k, stream) : c.fp8 ? attn::launch_fp8(kmap, vmap, k, stream) : attn::launch_bf16(kmap, vmap, k, stream);
  // a unit of one tile has nothing to join
  if (e != cudaSuccess || (a.pos != nullptr ? a.npos : a.max_len) <= (wide ? 2 : 1) * attn::kTile) return e;
  return c.head_dim == 64    ? launch_join<64>(k, stream)
         : c.head_dim == 128 ? launch_join<128>(k, stream)
                             : launch_join<256>(k, stream);
}

}  // namespace ci
