// Attention of drafted rows over the paged cache: dispatch, the workspace's
// layout, and the join of units that several CTAs worked on (contract in
// include/ci_draft.h; the main kernel is in attn_draft.cuh).
#include "attn_draft.cuh"

namespace ci {
namespace {

using draft::Args;
using draft::Layout;
using draft::Part;

constexpr int kJoinWarps = 16, kJoinRows = 8;

int block_rows(int head_dim) { return head_dim == 256 ? 128 : 256; }

Layout layout_of(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim) {
  return Layout{device_sm_count(), num_q_heads / num_kv_heads, block_rows(head_dim)};
}

// With the parts' references m_i, sums l_i and unnormalised sums o_i:
//   m = max m_i;  l = sum l_i 2^(m_i - m);  out = sum o_i 2^(m_i - m) / l.
// CTA (x, y) takes the unit that begins in CTA x and goes on, and every
// gridDim.y-th run of its (row, four dims); neighbouring lanes have neighbouring
// rows.  More than 32 parts are dealt to four warps, whose sums are added in order.
// Bound by latency (the parts sit in L2): a pass over fewer (row, four dims) costs
// more than a few parts one after another.  Whole calls with one warp and with four:
// 4 requests of 16 nodes, 6 parts, 27 and 30 us; one request of 64k of 128 rows, 10,
// 25, 38 and 152 parts, 102 / 104, 62 / 61, 57 / 54 and 71 / 65 us; of 480 rows 219 /
// 226, 106 / 109, 81 / 82 and 86 / 82.  (Of 32 rows four are as fast with 10, 96 / 95,
// and faster from 15 on, 69 / 67; 54 / 26 with 152.)
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ Args k) {
  __shared__ float sums[kJoinWarps][32][7];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  release_successor();
  wait_predecessor();
  const Part p = k.part[blockIdx.x];
  if (p.last < 0) return;
  const int n = p.last - static_cast<int>(blockIdx.x) + 1, ways = n > 32 ? 4 : 1, per = 32 * (kJoinWarps / ways);
  const int way = warp % ways, group = warp / ways;
  const int first = k.a.c.req_start[p.req], row0 = p.block * k.l.block_rows;
  const int rows = min(k.l.block_rows, (k.a.c.req_start[p.req + 1] - first) * k.l.group - row0);
  const float2* stats = reinterpret_cast<const float2*>(k.stat);
  const float4* parts = reinterpret_cast<const float4*>(k.sum);
  auto slot = [&](int i) { return 2ll * (blockIdx.x + i) + (i == 0 ? 1 : 0); };
#pragma unroll 1
  for (int base = blockIdx.y * per; base < rows * (D / 4); base += gridDim.y * per) {
    const int x = base + group * 32 + lane;
    const bool live = x < rows * (D / 4);
    const int c = live ? x / rows : 0, m = live ? x - c * rows : 0;
    // this way's parts: running reference and sums
    float top = -draft::kFar, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = way; i < n; i += ways) {
      const float2 st = stats[slot(i) * k.l.block_rows + m];
      const float4 v = parts[(slot(i) * (D / 4) + c) * k.l.block_rows + m];
      const float up = fmaxf(top, st.x), f = draft::exp2_approx(top - up), g = draft::exp2_approx(st.x - up);
      top = up;
      l = l * f + st.y * g;
      o.x = o.x * f + v.x * g, o.y = o.y * f + v.y * g, o.z = o.z * f + v.z * g, o.w = o.w * f + v.w * g;
    }
    if (ways > 1) {
      float* mine = sums[warp][lane];
      mine[0] = top, mine[1] = l, mine[2] = o.x, mine[3] = o.y, mine[4] = o.z, mine[5] = o.w;
      __syncthreads();
      if (way == 0)
#pragma unroll 1
        for (int y = 1; y < ways; ++y) {
          const float* v = sums[warp + y][lane];
          const float up = fmaxf(top, v[0]), f = draft::exp2_approx(top - up), g = draft::exp2_approx(v[0] - up);
          top = up;
          l = l * f + v[1] * g;
          o.x = o.x * f + v[2] * g, o.y = o.y * f + v[3] * g, o.z = o.z * f + v[4] * g, o.w = o.w * f + v[5] * g;
        }
      __syncthreads();
    }
    if (!live || way != 0) continue;
    const float inv = (l == 0.f ? 0.f : 1.f / l) * (k.a.c.fp8 ? draft::kTwo60 : 1.f);
    const int row = row0 + m, node = row / k.l.group;
    const int64_t t = first + node, qh = static_cast<int64_t>(p.head) * k.l.group + row - node * k.l.group;
    const bool none = l == 0.f;
    *reinterpret_cast<uint2*>(k.a.out + t * k.a.out_stride + qh * D + 4 * c) =
        make_uint2(none ? 0u : draft::bf16x2(o.x * inv, o.y * inv), none ? 0u : draft::bf16x2(o.z * inv, o.w * inv));
    if (k.a.lse != nullptr && c == 0)
      k.a.lse[t * k.a.c.num_q_heads + qh] =
          none ? -INFINITY : (top - (k.a.c.fp8 ? draft::kLift : 0.f) + log2f(l)) * 0.6931471805599453f;
  }
}

int64_t part_bytes(const Layout& l) { return (static_cast<int64_t>(l.ctas) * sizeof(Part) + 15) / 16 * 16; }
int64_t stat_bytes(const Layout& l) { return 2ll * l.ctas * l.block_rows * 2 * 4; }

}  // namespace

int64_t attn_draft_workspace_bytes(int32_t, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim) {
  const Layout l = layout_of(num_q_heads, num_kv_heads, head_dim);
  return part_bytes(l) + stat_bytes(l) + 2ll * l.ctas * l.block_rows * head_dim * 4;
}

cudaError_t launch_attn_draft(const DraftArgs& a, cudaStream_t stream) {
  const CacheArgs& c = a.c;
  Args k{a, layout_of(c.num_q_heads, c.num_kv_heads, c.head_dim), nullptr, nullptr, nullptr};
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  k.part = reinterpret_cast<Part*>(ws);
  k.stat = reinterpret_cast<float*>(ws + part_bytes(k.l));
  k.sum = reinterpret_cast<float*>(ws + part_bytes(k.l) + stat_bytes(k.l));
  const int row = c.fp8 ? c.head_dim : 2 * c.head_dim;
  const int64_t page = c.fp8 ? cache_page_bytes<true>(c.head_dim) : cache_page_bytes<false>(c.head_dim);
  CUtensorMap kmap{}, vmap{};
  const int64_t rows = c.num_pages * c.num_kv_heads * (page / row);
  cudaError_t e = make_rows_tmap(&kmap, c.k_pool, rows, row, kPage);
  if (e == cudaSuccess) e = make_rows_tmap(&vmap, c.v_pool, rows, row, kPage);
  if (e == cudaSuccess) e = c.fp8 ? draft::launch_fp8(kmap, vmap, k, stream) : draft::launch_bf16(kmap, vmap, k, stream);
  if (e != cudaSuccess || a.max_len <= draft::kKeys) return e;  // a unit of one tile has nothing to join
  const dim3 grid(k.l.ctas, kJoinRows);
  return c.head_dim == 64    ? launch_after(join_kernel<64>, grid, 32 * kJoinWarps, 0, stream, k)
         : c.head_dim == 128 ? launch_after(join_kernel<128>, grid, 32 * kJoinWarps, 0, stream, k)
                             : launch_after(join_kernel<256>, grid, 32 * kJoinWarps, 0, stream, k);
}

}  // namespace ci
