// New tokens' queries, keys and values: per-head RMS norm, rotation, and the
// append of keys and values to their pages (contract in include/ci_cache.h).
//
//   y = x * rsqrt(mean(x^2) + eps) * w;  (a, b) -> (a c - b s, b c + a s);
//   bf16 once, or e4m3(x / scale) with scale = max(amax, 1e-10) / 448.
//
// Memory-bound: every head is read once and written once.  A CTA takes whole
// tokens, so the token's rotation is read once per warp and its page is looked
// up once; the norm weights stay in registers over the CTA's tokens.  D / 8
// lanes hold a head, eight dims each, as two runs of four that are chosen so
// that both elements of every rotated pair sit in one lane (half layout: dims
// 4m.. and rot/2 + 4m..; interleaved and unrotated dims: 8m..8m + 7): the
// rotation needs no exchange between lanes, only the norm's sum and the FP8
// maximum do.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "cache_common.cuh"

namespace ci {
namespace {

constexpr int kWarps = 8;
constexpr int kBatch = 4;  // heads per lane group whose loads are in flight together

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

template <int D, bool kFp8, bool kNeox>
__global__ void __launch_bounds__(32 * kWarps) append_kernel(const AppendArgs a) {
  constexpr int kLanes = D / 8, kPer = 32 / kLanes;  // lanes per head, heads per warp
  const CacheArgs& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, m = lane % kLanes, sub = lane / kLanes;
  const int half = a.rot_dim / 2;
  const bool turns = 8 * m < a.rot_dim;
  const int o0 = kNeox && turns ? 4 * m : 8 * m, o1 = kNeox && turns ? half + 4 * m : 8 * m + 4;
  float wq[8], wk[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int d = j < 4 ? o0 + j : o1 + j - 4;
    wq[j] = a.q_norm != nullptr ? a.q_norm[d] : 1.f;
    wk[j] = a.k_norm != nullptr ? a.k_norm[d] : 1.f;
  }
  const int qg = (c.num_q_heads + kPer - 1) / kPer, kg = (c.num_kv_heads + kPer - 1) / kPer, groups = qg + 2 * kg;
  for (int t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const int p = a.positions[t], u = a.cache_pos != nullptr ? a.cache_pos[t] : p;
    const bool ok = p >= 0 && p < a.max_pos;
    if (!ok && threadIdx.x == 0) report(c.dev_err, kDevErrPos);
    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    if (ok && turns) {
      const float4 x = *reinterpret_cast<const float4*>(a.cos_sin + static_cast<int64_t>(p) * a.rot_dim + 4 * m);
      const float4 y = *reinterpret_cast<const float4*>(a.cos_sin + static_cast<int64_t>(p) * a.rot_dim + half + 4 * m);
      cs[0] = x.x, cs[1] = x.y, cs[2] = x.z, cs[3] = x.w;
      sn[0] = y.x, sn[1] = y.y, sn[2] = y.z, sn[3] = y.w;
    }
    int page = -1;
    if (ok && u >= 0) {
      const int r = row_request(c, t);
      if (u >= static_cast<int64_t>(c.max_pages) * kPage) {
        if (threadIdx.x == 0) report(c.dev_err, kDevErrPos);
      } else if (r >= 0) {
        page = c.page_table[static_cast<int64_t>(r) * c.max_pages + u / kPage];
        if (page < 0 || page >= c.num_pages) {
          if (threadIdx.x == 0) report(c.dev_err, kDevErrPage);
          page = -1;
        }
      }
    }
    for (int g0 = warp; g0 < groups; g0 += kWarps * kBatch) {
      uint2 lo[kBatch], hi[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int g = g0 + i * kWarps;
        const bool isq = g < qg, isk = g < qg + kg;
        const int h = (isq ? g : isk ? g - qg : g - qg - kg) * kPer + sub;
        const bool live = g < groups && h < (isq ? c.num_q_heads : c.num_kv_heads);
        const uint16_t* src = isq ? a.q + t * a.q_stride : isk ? a.k + t * a.k_stride : a.v + t * a.v_stride;
        lo[i] = hi[i] = make_uint2(0, 0);
        if (live) {
          lo[i] = *reinterpret_cast<const uint2*>(src + h * D + o0);
          hi[i] = *reinterpret_cast<const uint2*>(src + h * D + o1);
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int g = g0 + i * kWarps;
        if (g >= groups) break;
        const bool isq = g < qg, isk = !isq && g < qg + kg;
        const int h = (isq ? g : isk ? g - qg : g - qg - kg) * kPer + sub;
        const bool live = h < (isq ? c.num_q_heads : c.num_kv_heads);
        float x[8] = {bf16_lo(lo[i].x), bf16_hi(lo[i].x), bf16_lo(lo[i].y), bf16_hi(lo[i].y),
                      bf16_lo(hi[i].x), bf16_hi(hi[i].x), bf16_lo(hi[i].y), bf16_hi(hi[i].y)};
        if (isq || isk) {
          if ((isq ? a.q_norm : a.k_norm) != nullptr) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float r = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = x[j] * r * (isq ? wq[j] : wk[j]);
          }
          if (turns) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int e = kNeox ? j : 2 * j, f = kNeox ? j + 4 : 2 * j + 1;
              const float va = x[e], vb = x[f];
              x[e] = va * cs[j] - vb * sn[j];
              x[f] = vb * cs[j] + va * sn[j];
            }
          }
        }
        if (isq) {
          if (!ok) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = 0.f;
          }
          uint16_t* dst = a.q_out + t * a.q_out_stride + h * D;
          if (live) {
            *reinterpret_cast<uint2*>(dst + o0) = make_uint2(bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3]));
            *reinterpret_cast<uint2*>(dst + o1) = make_uint2(bf16_pair(x[4], x[5]), bf16_pair(x[6], x[7]));
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
    }
  }
}

template <int D>
void launch_d(const AppendArgs& a, unsigned grid, cudaStream_t stream) {
  if (a.c.fp8) {
    if (a.neox)
      append_kernel<D, true, true><<<grid, 32 * kWarps, 0, stream>>>(a);
    else
      append_kernel<D, true, false><<<grid, 32 * kWarps, 0, stream>>>(a);
  } else {
    if (a.neox)
      append_kernel<D, false, true><<<grid, 32 * kWarps, 0, stream>>>(a);
    else
      append_kernel<D, false, false><<<grid, 32 * kWarps, 0, stream>>>(a);
  }
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream) {
  const int64_t most = static_cast<int64_t>(device_sm_count()) * 8;
  const unsigned grid = static_cast<unsigned>(a.tokens < most ? a.tokens : most);
  if (a.c.head_dim == 64)
    launch_d<64>(a, grid, stream);
  else if (a.c.head_dim == 128)
    launch_d<128>(a, grid, stream);
  else
    launch_d<256>(a, grid, stream);
  return cudaGetLastError();
}

}  // namespace ci
