// New tokens' queries, keys and values: per-head RMS norm, rotation, and the
// append of keys and values to their pages (contract in include/ci_cache.h).
//
//   y = x * rsqrt(mean(x^2) + eps) * w;  (a, b) -> (a c - b s, b c + a s);
//   bf16 once, or e4m3(x / scale) with scale = max(amax, 1e-10) / 448.
//
// Memory-bound: every head is read once and written once.  D / 8 lanes hold a
// head, eight dims each, as two runs of four that are chosen so that both
// elements of every rotated pair sit in one lane (half layout: dims 4m.. and
// rot/2 + 4m..; interleaved and unrotated dims: 8m..8m + 7): the rotation needs
// no exchange between lanes, only the norm's sum and the FP8 maximum do.  A
// warp's task is a token and a few of its heads; the next task's loads are in
// flight while one is worked on, and the norm weights stay in registers.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "cache_common.cuh"

namespace ci {
namespace {

constexpr int kWarps = 4, kCtasPerSm = 5;
constexpr int kBatch = 4;  // groups of heads per task

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t e4m3_quad(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// The heads of a task: kBatch groups of 32 / (D / 8) heads, all of q, then of k,
// then of v (a group holds heads of one kind).
struct Groups {
  int q, k, all, chunks;  // groups of q; of q and k; of all; tasks per token
};

// A task's raw heads and position.
struct Loaded {
  uint2 lo[kBatch], hi[kBatch];
  int p, u;
};

template <int D>
__device__ __forceinline__ void load_task(const AppendArgs& a, const Groups& n, int t, int chunk, int o0, int o1, int sub,
                                          Loaded& x) {
  constexpr int kPer = 32 / (D / 8);
  x.p = a.positions[t];
  x.u = a.cache_pos != nullptr ? a.cache_pos[t] : x.p;
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int g = chunk * kBatch + i;
    const bool isq = g < n.q, isk = g < n.k;
    const int h = (isq ? g : isk ? g - n.q : g - n.k) * kPer + sub;
    const uint16_t* src = (isq ? a.q + t * a.q_stride : isk ? a.k + t * a.k_stride : a.v + t * a.v_stride) + h * D;
    x.lo[i] = x.hi[i] = make_uint2(0, 0);
    if (g < n.all && h < (isq ? a.c.num_q_heads : a.c.num_kv_heads)) {
      x.lo[i] = *reinterpret_cast<const uint2*>(src + o0);
      x.hi[i] = *reinterpret_cast<const uint2*>(src + o1);
    }
  }
}

template <int D, bool kFp8, bool kNeox>
__global__ void __launch_bounds__(32 * kWarps) append_kernel(const AppendArgs a, const Groups n) {
  constexpr int kLanes = D / 8, kPer = 32 / kLanes;  // lanes per head, heads per group
  const CacheArgs& c = a.c;
  const int lane = threadIdx.x & 31, m = lane % kLanes, sub = lane / kLanes;
  const int half = a.rot_dim / 2;
  const bool turns = 8 * m < a.rot_dim;
  const int o0 = kNeox && turns ? 4 * m : 8 * m, o1 = kNeox && turns ? half + 4 * m : 8 * m + 4;
  const int64_t tasks = static_cast<int64_t>(a.tokens) * n.chunks, step = static_cast<int64_t>(gridDim.x) * kWarps;
  int64_t task = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (task >= tasks) return;
  int t = static_cast<int>(task / n.chunks), chunk = static_cast<int>(task - static_cast<int64_t>(t) * n.chunks);
  Loaded now;
  load_task<D>(a, n, t, chunk, o0, o1, sub, now);
  float wq[8], wk[8];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float4 one = make_float4(1.f, 1.f, 1.f, 1.f);
    const float4 x = a.q_norm != nullptr ? *reinterpret_cast<const float4*>(a.q_norm + (j ? o1 : o0)) : one;
    const float4 y = a.k_norm != nullptr ? *reinterpret_cast<const float4*>(a.k_norm + (j ? o1 : o0)) : one;
    wq[4 * j] = x.x, wq[4 * j + 1] = x.y, wq[4 * j + 2] = x.z, wq[4 * j + 3] = x.w;
    wk[4 * j] = y.x, wk[4 * j + 1] = y.y, wk[4 * j + 2] = y.z, wk[4 * j + 3] = y.w;
  }
  while (true) {
    // ---- this task's rotation and page; the next task's heads
    const int p = now.p, u = now.u, g0 = chunk * kBatch, tok = t;
    const bool ok = p >= 0 && p < a.max_pos;
    if (!ok && lane == 0 && chunk == 0) report(c.dev_err, kDevErrPos);
    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    if (ok && turns && g0 < n.k) {
      const float* at = a.cos_sin + static_cast<int64_t>(p) * a.rot_dim + 4 * m;
      const float4 x = *reinterpret_cast<const float4*>(at), y = *reinterpret_cast<const float4*>(at + half);
      cs[0] = x.x, cs[1] = x.y, cs[2] = x.z, cs[3] = x.w;
      sn[0] = y.x, sn[1] = y.y, sn[2] = y.z, sn[3] = y.w;
    }
    int page = -1;
    if (ok && u >= 0 && g0 + kBatch > n.q) {
      const int r = row_request(c, tok);
      if (u >= static_cast<int64_t>(c.max_pages) * kPage) {
        if (lane == 0) report(c.dev_err, kDevErrPos);
      } else if (r >= 0) {
        page = c.page_table[static_cast<int64_t>(r) * c.max_pages + u / kPage];
        if (page < 0 || page >= c.num_pages) {
          if (lane == 0) report(c.dev_err, kDevErrPage);
          page = -1;
        }
      }
    }
    const Loaded cur = now;
    task += step;
    const bool more = task < tasks;
    if (more) {
      t = static_cast<int>(task / n.chunks);
      chunk = static_cast<int>(task - static_cast<int64_t>(t) * n.chunks);
      load_task<D>(a, n, t, chunk, o0, o1, sub, now);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int g = g0 + i;
      if (g >= n.all) break;
      const bool isq = g < n.q, isk = !isq && g < n.k;
      const int h = (isq ? g : isk ? g - n.q : g - n.k) * kPer + sub;
      const bool live = h < (isq ? c.num_q_heads : c.num_kv_heads);
      float x[8] = {bf16_lo(cur.lo[i].x), bf16_hi(cur.lo[i].x), bf16_lo(cur.lo[i].y), bf16_hi(cur.lo[i].y),
                    bf16_lo(cur.hi[i].x), bf16_hi(cur.hi[i].x), bf16_lo(cur.hi[i].y), bf16_hi(cur.hi[i].y)};
      if (isq || isk) {
        if ((isq ? a.q_norm : a.k_norm) != nullptr) {
          float ss = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
          for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float r = rsqrtf(ss * (1.f / D) + a.eps);
          if (isq) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = x[j] * r * wq[j];
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = x[j] * r * wk[j];
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // dims past rot_dim turn by (1, 0)
          const int e = kNeox ? j : 2 * j, f = kNeox ? j + 4 : 2 * j + 1;
          const float va = x[e], vb = x[f];
          if (turns) x[e] = va * cs[j] - vb * sn[j], x[f] = vb * cs[j] + va * sn[j];
        }
      }
      if (isq) {
        uint16_t* dst = a.q_out + tok * a.q_out_stride + h * D;
        if (live) {
          const uint2 lo = make_uint2(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]));
          const uint2 hi = make_uint2(bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
          *reinterpret_cast<uint2*>(dst + o0) = ok ? lo : make_uint2(0, 0);
          *reinterpret_cast<uint2*>(dst + o1) = ok ? hi : make_uint2(0, 0);
        }
        continue;
      }
      const bool store = live && page >= 0;
      const int slot = u & (kPage - 1);
      uint8_t* at = (isk ? c.k_pool : c.v_pool) +
                    (static_cast<int64_t>(page) * c.num_kv_heads + h) * cache_page_bytes<kFp8>(D);
      if (kFp8) {
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = max_nan(amax, fabsf(x[j]));
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float scale = __fdiv_rn(max_nan(amax, 1e-10f), 448.f);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __fdiv_rn(x[j], scale);
        if (store) {
          *reinterpret_cast<uint32_t*>(at + slot * D + o0) = e4m3_quad(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<uint32_t*>(at + slot * D + o1) = e4m3_quad(x[4], x[5], x[6], x[7]);
          if (m == 0) reinterpret_cast<float*>(at + kPage * D)[slot] = scale;
        }
      } else if (store) {
        uint16_t* dst = reinterpret_cast<uint16_t*>(at) + slot * D;
        *reinterpret_cast<uint2*>(dst + o0) = make_uint2(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]));
        *reinterpret_cast<uint2*>(dst + o1) = make_uint2(bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
      }
    }
    if (!more) break;
  }
}

template <int D>
void launch_d(const AppendArgs& a, cudaStream_t stream) {
  constexpr int kPer = 32 / (D / 8);
  const int qg = (a.c.num_q_heads + kPer - 1) / kPer, kg = (a.c.num_kv_heads + kPer - 1) / kPer;
  const Groups n{qg, qg + kg, qg + 2 * kg, (qg + 2 * kg + kBatch - 1) / kBatch};
  const int64_t ctas = (static_cast<int64_t>(a.tokens) * n.chunks + kWarps - 1) / kWarps;
  const int64_t most = static_cast<int64_t>(device_sm_count()) * kCtasPerSm;
  const unsigned grid = static_cast<unsigned>(ctas < most ? ctas : most);
  if (a.c.fp8) {
    if (a.neox)
      append_kernel<D, true, true><<<grid, 32 * kWarps, 0, stream>>>(a, n);
    else
      append_kernel<D, true, false><<<grid, 32 * kWarps, 0, stream>>>(a, n);
  } else {
    if (a.neox)
      append_kernel<D, false, true><<<grid, 32 * kWarps, 0, stream>>>(a, n);
    else
      append_kernel<D, false, false><<<grid, 32 * kWarps, 0, stream>>>(a, n);
  }
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream) {
  if (a.c.head_dim == 64)
    launch_d<64>(a, stream);
  else if (a.c.head_dim == 128)
    launch_d<128>(a, stream);
  else
    launch_d<256>(a, stream);
  return cudaGetLastError();
}

}  // namespace ci
