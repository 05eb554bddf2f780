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

// Whether the kernel of attn_wide.cu takes the call.  Both measured, in us of calls one
// after another (the warp-level kernel, then the wide one), by heads per key-value head:
//   17 rows of 0-100k, all positions   16: 76.8, 79.3   20: 79.8, 78.6   32: 80.7, 79.8   64: 116.9, 83.3
//   4 rows of 1k-4k, all positions     16: 12.0, 13.4   20: 12.5, 14.2   32: 13.1, 14.5   64: 18.8, 18.3
//   1024 rows over 512 listed          16: 57.9, 60.5   20: 65.5, 61.6   32: 68.3, 62.5   64: 101.8, 66.5
constexpr int kWideListed = 16, kWideAll = 32;
bool is_wide(const CacheArgs& c, bool listed) {
  return !c.fp8 && c.head_dim == 128 && c.num_q_heads / c.num_kv_heads > (listed ? kWideListed : kWideAll);
}

Layout layout_of(int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, bool wide) {
  const int group = num_q_heads / num_kv_heads;
  const int heads = wide ? 64 : group <= 8 ? 8 : group <= 16 ? 16 : group <= 32 ? 32 : 64;
  return Layout{device_sm_count() * (head_dim == 256 ? 1 : 2), heads, (group + heads - 1) / heads, group};
}

// With the parts' maxima m_i, sums l_i and unnormalised sums o_i:
//   m = max m_i;  l = sum l_i 2^(m_i - m);  out = sum o_i 2^(m_i - m) / l.
// CTA (x, y) takes a split unit and 16 / ways of its heads; a head's parts are
// dealt to `ways` warps, whose sums are added in order.  x is a unit, or, where
// units outnumber workers, the worker in whose range one starts and goes on.
// Bound by latency (the parts sit in L2): which parts a unit has is worked out
// before the wait for the main kernel, and sums and statistics are fetched
// together.  (Joining in the main kernel, by the CTA that comes last, took 6 us
// more: its code is cold there.)
template <int D, int kT>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const Args k, int ways, bool by_unit) {
  constexpr int kPer = D / 32, kFetch = 4;
  __shared__ float sums[kJoinWarps][D];
  __shared__ int32_t warp_sum[2][kJoinWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int units = k.a.c.num_kv_heads * k.l.blocks;
  Part p{0, 0, -1, 0};
  int first = blockIdx.x;
  if (by_unit) {  // at most as many units as workers: at most one row per thread
    p.row = blockIdx.x / units;
    p.unit = blockIdx.x - p.row * units;
    const int mine = tid < k.a.rows ? attn::row_tiles<kT>(k.a, tid) : 0;
    const int all = __reduce_add_sync(0xffffffffu, mine), before = __reduce_add_sync(0xffffffffu, tid < p.row ? mine : 0);
    if (lane == 0) warp_sum[0][warp] = all, warp_sum[1][warp] = before;
    __syncthreads();
    int total = 0, start = 0;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) total += warp_sum[0][w], start += warp_sum[1][w];
    const int n = attn::row_tiles<kT>(k.a, p.row);
    if (n > 0) {
      attn::Range r{};
      r.total = total * units;
      r.workers = min(k.l.ctas, r.total);
      start = start * units + p.unit * n;
      first = attn::worker_of(start, r);
      p.last = attn::worker_of(start + n - 1, r);
      if (p.last == first) p.last = -1;  // one worker had it all, and has written the result
    }
  }
  release_successor();
  wait_predecessor();  // (every CTA: this kernel must not end before the main one)
  if (!by_unit) p = k.part[first];
  if (p.last < 0) return;
  const int hw = warp / ways, way = warp - hw * ways;
  const int heads = k.l.heads, h = blockIdx.y * (kJoinWarps / ways) + hw;
  const int head = p.unit / k.l.blocks, hb = p.unit - head * k.l.blocks;
  const bool live = h < heads && hb * heads + h < k.l.group;
  const int n = p.last - first + 1;
  auto slot = [&](int i) { return attn::slot_of(first + i, i == 0); };
  float m = -INFINITY, l = 0.f, o[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) o[j] = 0.f;
  if (live) {
    const float2* stat = reinterpret_cast<const float2*>(k.stat) + h;
    // the warp's first parts, under way before the statistics are needed
    float x[kFetch][kPer], mx[kFetch];
#pragma unroll
    for (int f = 0; f < kFetch; ++f) {
      const int i = way + f * ways;
      mx[f] = -INFINITY;
      if (i >= n) continue;
      mx[f] = stat[slot(i) * heads].x;
#pragma unroll
      for (int j = 0; j < kPer; ++j) x[f][j] = k.sum[(slot(i) * heads + h) * D + lane + 32 * j];
    }
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
#pragma unroll
    for (int f = 0; f < kFetch; ++f) {
      if (way + f * ways >= n) continue;
      const float g = attn::exp2_approx(mx[f] - ref);
#pragma unroll
      for (int j = 0; j < kPer; ++j) o[j] += g * x[f][j];
    }
#pragma unroll 4
    for (int i = way + kFetch * ways; i < n; i += ways) {
      const float f = attn::exp2_approx(stat[slot(i) * heads].x - ref);
      const float* src = k.sum + (slot(i) * heads + h) * D + lane;
#pragma unroll
      for (int j = 0; j < kPer; ++j) o[j] += f * src[32 * j];
    }
  }
  if (ways > 1) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) sums[warp][32 * j + lane] = o[j];
    __syncthreads();
    if (!live || way != 0) return;
#pragma unroll 1
    for (int x = 1; x < ways; ++x)
#pragma unroll
      for (int j = 0; j < kPer; ++j) o[j] += sums[warp + x][32 * j + lane];
  }
  if (!live) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t qh = static_cast<int64_t>(head) * k.l.group + hb * heads + h;
  uint16_t* dst = k.a.out + p.row * k.a.out_stride + qh * D;
#pragma unroll
  for (int j = 0; j < kPer; ++j) dst[32 * j + lane] = __bfloat16_as_ushort(__float2bfloat16_rn(o[j] * inv));
  if (k.a.lse != nullptr && lane == 0)
    k.a.lse[static_cast<int64_t>(p.row) * k.a.c.num_q_heads + qh] =
        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

int64_t part_bytes(const Layout& l) { return (static_cast<int64_t>(l.ctas) * sizeof(Part) + 15) / 16 * 16; }
int64_t stat_bytes(const Layout& l) { return 2ll * l.ctas * l.heads * 2 * 4; }

template <int D, int kT>
cudaError_t launch_join(const Args& k, cudaStream_t stream) {
  // The fewer units, the more parts each: 16, 4 or 1 warps a head.  Both kernels with 1, 4 and 16 (us of calls one
  // after another): one row of 256k, 77 parts a unit: 95.2, 90.1, 87.8; 16 rows of 10k-20k, 5 parts: 81.5, 80.5, 83.9;
  // 64 rows of 512 listed, at most 2 parts: 33.8, 36.1, 46.6.
  const int64_t units = static_cast<int64_t>(k.a.rows) * k.a.c.num_kv_heads * k.l.blocks;
  const bool by_unit = units <= k.l.ctas && k.a.rows <= 32 * kJoinWarps;
  const int64_t split = by_unit ? units : k.l.ctas, parts = k.l.ctas / (units < k.l.ctas ? units : k.l.ctas) + 1;
  const int ways = parts > 32 ? 16 : parts > 4 ? 4 : 1, per = kJoinWarps / ways;
  const int heads = k.l.heads < k.l.group ? k.l.heads : k.l.group;
  return launch_after(join_kernel<D, kT>, dim3(static_cast<unsigned>(split), (heads + per - 1) / per), 32 * kJoinWarps, 0,
                      stream, k, ways, by_unit);
}

}  // namespace

int64_t attn_workspace_bytes(int32_t, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim) {
  // Where the wide kernel takes calls of so many heads, either may take this one: neither the cache's format nor
  // whether positions are listed is known here.
  const bool may_be_wide = head_dim == 128 && num_q_heads / num_kv_heads > kWideListed;
  int64_t most = 0;
  for (const bool wide : {false, true}) {
    if (wide && !may_be_wide) continue;
    const Layout l = layout_of(num_q_heads, num_kv_heads, head_dim, wide);
    const int64_t n = part_bytes(l) + stat_bytes(l) + 2ll * l.ctas * l.heads * head_dim * 4;
    most = n > most ? n : most;
  }
  return most;
}

cudaError_t launch_attn(const AttnArgs& a, cudaStream_t stream) {
  const CacheArgs& c = a.c;
  const bool wide = is_wide(c, a.pos != nullptr);
  Args k{a, layout_of(c.num_q_heads, c.num_kv_heads, c.head_dim, wide), nullptr, nullptr, nullptr};
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  k.part = reinterpret_cast<Part*>(ws);
  k.stat = reinterpret_cast<float*>(ws + part_bytes(k.l));
  k.sum = reinterpret_cast<float*>(ws + part_bytes(k.l) + stat_bytes(k.l));
  const int row = c.fp8 ? c.head_dim : 2 * c.head_dim;
  const int per_page = static_cast<int>((c.fp8 ? cache_page_bytes<true>(c.head_dim) : cache_page_bytes<false>(c.head_dim)) / row);
  CUtensorMap kmap{}, vmap{};  // listed rows use none
  cudaError_t e = cudaSuccess;
  if (a.pos == nullptr) {
    const int64_t rows = c.num_pages * c.num_kv_heads * per_page;
    e = make_rows_tmap(&kmap, c.k_pool, rows, row, attn::kTile);
    if (e == cudaSuccess) e = make_rows_tmap(&vmap, c.v_pool, rows, row, attn::kTile);
  }
  if (e == cudaSuccess)
    e = wide ? attn::launch_wide(kmap, vmap, k, stream) : c.fp8 ? attn::launch_fp8(kmap, vmap, k, stream) : attn::launch_bf16(kmap, vmap, k, stream);
  // a unit of one tile has nothing to join
  if (e != cudaSuccess || (a.pos != nullptr ? a.npos : a.max_len) <= (wide ? 2 : 1) * attn::kTile) return e;
  if (wide) return launch_join<128, 2 * attn::kTile>(k, stream);
  return c.head_dim == 64    ? launch_join<64, attn::kTile>(k, stream)
         : c.head_dim == 128 ? launch_join<128, attn::kTile>(k, stream)
                             : launch_join<256, attn::kTile>(k, stream);
}

}  // namespace ci
