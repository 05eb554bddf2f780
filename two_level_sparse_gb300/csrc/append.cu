// New tokens' queries, keys and values: per-head RMS norm, rotation, and the
// append of keys and values to their pages (contract in include/ci_cache.h).
//
//   y = x * rsqrt(mean(x^2) + eps) * w;  (a, b) -> (a c - b s, b c + a s);
//   bf16 once, or e4m3(x / scale) with scale = max(amax, 1e-10) / 448.
//
// Memory-bound: every head is read once and written once: 16384 tokens of 64 + 16
// heads of 128 into FP8 pages move 647 MB in 110 us, 5.9 TB/s of a copy's 6.8 (IEEE
// divisions by the FP8 scale took it to 248 us; the scale's reciprocal and one
// correction give the same codes, as a test compares).  A call with few tokens is as
// long as its host side: 18-19 us for 8 tokens.
//
// D / 8 lanes hold a head, eight dims each, as two runs of four that are chosen so
// that both elements of every rotated pair sit in one lane (half layout: dims 4m..
// and rot/2 + 4m..; interleaved and unrotated dims: 8m..8m + 7): the rotation needs
// no exchange between lanes, only the norm's sum and the FP8 maximum do.  A warp's
// task is a token and a few of its heads of one kind: norm weight and rotation
// become two factors per element once for all of them, and the next task's loads
// are in flight while one is worked on (a task per head took 164 us, these 113).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "cache_common.cuh"

namespace ci {
namespace {

constexpr int kWarps = 4, kCtasPerSm = 6;
constexpr int kBatch = 4;  // groups of 32 / (D / 8) heads per task

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

// The tasks of a token: chunks of kBatch * 32 / (D / 8) heads, of q, then of k,
// then of v.
struct Chunks {
  int q, k, all;              // chunks of q; of q and k; of all
  int step_tok, step_chunk;   // a warp's stride over the tasks
};

// A task's raw heads and position.
struct Loaded {
  uint2 lo[kBatch], hi[kBatch];
  int p, u;
};

template <int D>
__device__ __forceinline__ void load_task(const AppendArgs& a, const Chunks& n, int t, int chunk, int o0, int o1, int sub,
                                          Loaded& x) {
  constexpr int kPer = 32 / (D / 8);
  x.p = a.positions[t];
  x.u = a.cache_pos != nullptr ? a.cache_pos[t] : x.p;
  const bool isq = chunk < n.q, isk = chunk < n.k;
  const int h = (chunk - (isq ? 0 : isk ? n.q : n.k)) * kBatch * kPer + sub;
  const int left = (isq ? a.c.num_q_heads : a.c.num_kv_heads) - h;
  const uint16_t* src = (isq ? a.q + t * a.q_stride : isk ? a.k + t * a.k_stride : a.v + t * a.v_stride) + h * D;
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    x.lo[i] = x.hi[i] = make_uint2(0, 0);
    if (i * kPer < left) {
      x.lo[i] = *reinterpret_cast<const uint2*>(src + i * kPer * D + o0);
      x.hi[i] = *reinterpret_cast<const uint2*>(src + i * kPer * D + o1);
    }
  }
}

__device__ __forceinline__ void unpack8(uint2 lo, uint2 hi, float2 (&x)[4]) {
  x[0] = make_float2(bf16_lo(lo.x), bf16_hi(lo.x)), x[1] = make_float2(bf16_lo(lo.y), bf16_hi(lo.y));
  x[2] = make_float2(bf16_lo(hi.x), bf16_hi(hi.x)), x[3] = make_float2(bf16_lo(hi.y), bf16_hi(hi.y));
}

// Two fp32 operations per instruction, each rounded as its scalar form is.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\t"
      "mov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// A lane's share of norm and rotation, as two factors per element:
//   out_j = r (x_j own_j + x_j' other_j),  j' the pair's other element,
// own = w cos, other = -+ w' sin, r = rsqrt(mean(x^2) + eps).  Pairs of elements
// (2i, 2i + 1); j' is j +- 4 in the half layout, j ^ 1 in the interleaved one.
struct Factors {
  float2 own[4], other[4];
};

template <int D, bool kNeox>
__device__ __forceinline__ Factors factors_of(const float* w, int o0, int o1, const float* cos_sin, int half, int m) {
  const float4 one = make_float4(1.f, 1.f, 1.f, 1.f);
  const float4 wl = w != nullptr ? *reinterpret_cast<const float4*>(w + o0) : one;
  const float4 wh = w != nullptr ? *reinterpret_cast<const float4*>(w + o1) : one;
  float4 c = one, s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (cos_sin != nullptr) {
    c = *reinterpret_cast<const float4*>(cos_sin + 4 * m);
    s = *reinterpret_cast<const float4*>(cos_sin + half + 4 * m);
  }
  Factors f;
  if (kNeox) {  // elements j and j + 4 are a pair, turned by angle j
    f.own[0] = make_float2(wl.x * c.x, wl.y * c.y), f.own[1] = make_float2(wl.z * c.z, wl.w * c.w);
    f.own[2] = make_float2(wh.x * c.x, wh.y * c.y), f.own[3] = make_float2(wh.z * c.z, wh.w * c.w);
    f.other[0] = make_float2(-wh.x * s.x, -wh.y * s.y), f.other[1] = make_float2(-wh.z * s.z, -wh.w * s.w);
    f.other[2] = make_float2(wl.x * s.x, wl.y * s.y), f.other[3] = make_float2(wl.z * s.z, wl.w * s.w);
  } else {  // elements 2i and 2i + 1 are a pair, turned by angle i
    f.own[0] = make_float2(wl.x * c.x, wl.y * c.x), f.own[1] = make_float2(wl.z * c.y, wl.w * c.y);
    f.own[2] = make_float2(wh.x * c.z, wh.y * c.z), f.own[3] = make_float2(wh.z * c.w, wh.w * c.w);
    f.other[0] = make_float2(-wl.y * s.x, wl.x * s.x), f.other[1] = make_float2(-wl.w * s.y, wl.z * s.y);
    f.other[2] = make_float2(-wh.y * s.z, wh.x * s.z), f.other[3] = make_float2(-wh.w * s.w, wh.z * s.w);
  }
  return f;
}

// `whole`: every dim turns.  Where one does not, its `other` is 0 and must not
// meet an infinity of the pair's other element.
template <int D, bool kNeox>
__device__ __forceinline__ void norm_turn(float2 (&x)[4], const Factors& f, bool norm, float eps, bool whole, bool turns) {
  float r = 1.f;
  if (norm) {
    float2 ss = mul2(x[0], x[0]);
#pragma unroll
    for (int j = 1; j < 4; ++j) ss = fma2(x[j], x[j], ss);
    float s = ss.x + ss.y;
#pragma unroll
    for (int o = 1; o < D / 8; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    r = rsqrtf(s * (1.f / D) + eps);
  }
  const float2 rr = make_float2(r, r);
  float2 y[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 mate = kNeox ? x[j ^ 2] : make_float2(x[j].y, x[j].x);
    y[j] = mul2(fma2(mate, f.other[j], mul2(x[j], f.own[j])), rr);
    if (!whole && !turns) y[j] = mul2(mul2(x[j], f.own[j]), rr);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = y[j];
}

__device__ __forceinline__ void store_bf16(uint16_t* dst, int o0, int o1, const float2 (&x)[4]) {
  *reinterpret_cast<uint2*>(dst + o0) = make_uint2(bf16_pair(x[0].x, x[0].y), bf16_pair(x[1].x, x[1].y));
  *reinterpret_cast<uint2*>(dst + o1) = make_uint2(bf16_pair(x[2].x, x[2].y), bf16_pair(x[3].x, x[3].y));
}

// One position's entry of a (page, head) at `at`; all lanes of the head take part.
template <int D, bool kFp8>
__device__ __forceinline__ void store_entry(uint8_t* at, int slot, int o0, int o1, int m, bool store, float2 (&x)[4]) {
  if (!kFp8) {
    if (store) store_bf16(reinterpret_cast<uint16_t*>(at) + slot * D, o0, o1, x);
    return;
  }
  float amax = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) amax = max_nan(max_nan(amax, fabsf(x[j].x)), fabsf(x[j].y));
#pragma unroll
  for (int o = 1; o < D / 8; o <<= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float scale = __fdiv_rn(max_nan(amax, 1e-10f), 448.f), inv = __frcp_rn(scale);
  // (an infinite scale has an exact reciprocal, 0, and nothing to correct)
  const float back = scale == INFINITY ? 0.f : -scale;
  const float2 inv2 = make_float2(inv, inv), minus = make_float2(back, back);
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // x / scale: a product with the reciprocal, and Markstein's correction of it
    const float2 y = mul2(x[j], inv2);
    x[j] = fma2(fma2(y, minus, x[j]), inv2, y);
  }
  if (store) {
    *reinterpret_cast<uint32_t*>(at + slot * D + o0) = e4m3_quad(x[0].x, x[0].y, x[1].x, x[1].y);
    *reinterpret_cast<uint32_t*>(at + slot * D + o1) = e4m3_quad(x[2].x, x[2].y, x[3].x, x[3].y);
    if (m == 0) reinterpret_cast<float*>(at + kPage * D)[slot] = scale;
  }
}

template <int D, bool kFp8, bool kNeox>
__global__ void __launch_bounds__(32 * kWarps, kCtasPerSm) append_kernel(const AppendArgs a, const Chunks n) {
  constexpr int kLanes = D / 8, kPer = 32 / kLanes;  // lanes per head, heads per group
  const CacheArgs& c = a.c;
  const int lane = threadIdx.x & 31, m = lane % kLanes, sub = lane / kLanes;
  const int half = a.rot_dim / 2;
  const bool turns = 8 * m < a.rot_dim;
  const int o0 = kNeox && turns ? 4 * m : 8 * m, o1 = kNeox && turns ? half + 4 * m : 8 * m + 4;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  int t = static_cast<int>(task / n.all), chunk = static_cast<int>(task - static_cast<int64_t>(t) * n.all);
  wait_predecessor();
  if (t >= a.tokens) return;
  Loaded now;
  load_task<D>(a, n, t, chunk, o0, o1, sub, now);
  const bool whole = a.rot_dim == D;
  bool more = true;
  while (more) {
    // ---- this task's rotation and page
    const int p = now.p, u = now.u, tok = t, mine = chunk;
    const bool isq = mine < n.q, isk = !isq && mine < n.k;
    const bool ok = p >= 0 && p < a.max_pos;
    if (!ok && lane == 0 && mine == 0) report(c.dev_err, kDevErrPos);
    Factors f;
    if (isq || isk)
      f = factors_of<D, kNeox>(isq ? a.q_norm : a.k_norm, o0, o1,
                               ok && turns ? a.cos_sin + static_cast<int64_t>(p) * a.rot_dim : nullptr, half, m);
    int page = -1;
    if (ok && u >= 0 && !isq) {
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
    // ---- the next task's heads
    const Loaded cur = now;
    t += n.step_tok;
    chunk += n.step_chunk;
    if (chunk >= n.all) chunk -= n.all, ++t;
    more = t < a.tokens;
    if (more) load_task<D>(a, n, t, chunk, o0, o1, sub, now);
    // ---- this task's heads
    const int h = (mine - (isq ? 0 : isk ? n.q : n.k)) * kBatch * kPer + sub;
    if (isq) {
      uint16_t* dst = a.q_out + tok * a.q_out_stride + h * D;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        float2 x[4];
        unpack8(cur.lo[i], cur.hi[i], x);
        norm_turn<D, kNeox>(x, f, a.q_norm != nullptr, a.eps, whole, turns);
        if (!ok) x[0] = x[1] = x[2] = x[3] = make_float2(0.f, 0.f);
        if (h + i * kPer < c.num_q_heads) store_bf16(dst + i * kPer * D, o0, o1, x);
      }
    } else {
      uint8_t* at = (isk ? c.k_pool : c.v_pool) +
                    (static_cast<int64_t>(max(page, 0)) * c.num_kv_heads + h) * cache_page_bytes<kFp8>(D);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        float2 x[4];
        unpack8(cur.lo[i], cur.hi[i], x);
        if (isk) norm_turn<D, kNeox>(x, f, a.k_norm != nullptr, a.eps, whole, turns);
        store_entry<D, kFp8>(at + i * kPer * cache_page_bytes<kFp8>(D), u & (kPage - 1), o0, o1, m,
                             page >= 0 && h + i * kPer < c.num_kv_heads, x);
      }
    }
  }
}

template <int D>
cudaError_t launch_d(const AppendArgs& a, cudaStream_t stream) {
  constexpr int kHeads = kBatch * (32 / (D / 8));  // of a task
  const int qc = (a.c.num_q_heads + kHeads - 1) / kHeads, kc = (a.c.num_kv_heads + kHeads - 1) / kHeads;
  const int all = qc + 2 * kc;
  const int64_t ctas = (static_cast<int64_t>(a.tokens) * all + kWarps - 1) / kWarps;
  const int64_t most = static_cast<int64_t>(device_sm_count()) * kCtasPerSm;
  const unsigned grid = static_cast<unsigned>(ctas < most ? ctas : most);
  const int warps = static_cast<int>(grid) * kWarps;
  const Chunks n{qc, qc + kc, all, warps / all, warps % all};
  const dim3 ctas3(grid);
  constexpr int kThreads = 32 * kWarps;
  if (a.c.fp8)
    return a.neox ? launch_after(append_kernel<D, true, true>, ctas3, kThreads, 0, stream, a, n)
                  : launch_after(append_kernel<D, true, false>, ctas3, kThreads, 0, stream, a, n);
  return a.neox ? launch_after(append_kernel<D, false, true>, ctas3, kThreads, 0, stream, a, n)
                : launch_after(append_kernel<D, false, false>, ctas3, kThreads, 0, stream, a, n);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, cudaStream_t stream) {
  return a.c.head_dim == 64 ? launch_d<64>(a, stream) : a.c.head_dim == 128 ? launch_d<128>(a, stream) : launch_d<256>(a, stream);
}

}  // namespace ci
