// Attention over a paged bf16 cache where many query heads (more than 32, or more
// than 16 where positions are listed) share a key-value head of 128 dims (contract
// in include/ci_cache.h; the list of tiles, its split over the CTAs and the join are
// those of attn.cuh).
//
// With G = 64 heads the products cost 64 flop per byte of cache: at the HBM's
// rate 435 TFLOP/s, half of what the warp-level MMA instructions reach (attn.cu
// has both kernels' times), so here the fifth-generation tensor cores compute, a
// tile of 128 positions at a time:
//
//   S^T [128 positions x 64 heads] = K Q^T    A = K (rows of dims), B = Q, both
//                                             from shared memory, S in tensor memory
//   P = 2^(S c - m)                           a thread per position and half of the heads
//   O^T [128 dims x 64 heads] += V^T P^T      A = V and B = P with the positions
//                                             as the reduced rows (MN-major), O in tensor memory
//
// One CTA per SM, two workers per CTA: each has its own range of the list, eight
// softmax warps, references, sums and O, a warp that issues its products and warps
// that fetch, so that one's exponentials and results run beside the other's
// products.  A worker has one K slot (a tile, 32 KB), filled again while the tile's
// probabilities are computed, and three V slots of half a tile.  Scores are issued
// before the values of the tile before where their keys are there.
//
// What bounds it.  17 rows of 0-100k, one key-value head: 436 MB in 83 us with the
// join, 5.2 TB/s of a copy's 6.8; the start (4 us until the first tile arrives) and
// an uneven end are 10 us of it.  4096 rows over 512 listed positions each, of one
// request: 1.07 GB of rows from L2 in 214 us, 5.0 TB/s; a worker's tile takes 5500
// cycles, of which its keys' arrival is 3900 and the softmax 2700, and a row's end
// 8000 every four tiles.  (Four softmax warps per worker instead of eight: 266 us.
// Spilled registers cost more than they seem to: a reload that misses waits behind
// the cache's own reads, 115 us instead of 85 for the 17 rows.)
//
// The reference m of a head is not the running maximum but 24 above the logit (in
// base 2) of the segment's first position; once a tile has a logit 16 above a
// reference, 24 above each head's largest of that tile, where that is more.  fp32 and
// bf16 have the exponents for that: probabilities from 2^-24 to 2^16 are as exact as
// those below one, and maxima across the positions (across lanes, here) and the
// rescaling of O happen only where a logit lies 40 above the one that set the
// reference.  Values of 2^80 under probabilities of 2^16 add up to less than 2^128
// over 2^31 positions.
#include "attn.cuh"

namespace ci {
namespace attn {
namespace {

constexpr int kD = 128, kH = 64, kPos = 128;
constexpr int kKSlot = kPos * kD * 2, kVSlot = kKSlot / 2;  // K: a tile; V: half of one (a page)
constexpr int kVSlots = 3;                                 // per worker
constexpr int kSlotBytes = 2 * (kKSlot + kVSlots * kVSlot);  // the workers' K slots, then their V slots
constexpr int kPBytes = kPos * kH * 2, kQBytes = kH * kD * 2;
constexpr int kSoftmaxWarps = 8;  // per worker: a quarter of a tile's positions and half of the heads each
constexpr int kGroup = 32 * kSoftmaxWarps, kWideThreads = 256 + 2 * kGroup;
// of worker g, at + 64 g: S, O, the sums of P, those of P as it is rounded
constexpr int kTmem = 512, kColS = 0, kColO = 128, kColL = 256, kColR = 384;
constexpr float kFar = 3.0e38f;                     // a first logit's reference lies in [-kFar, kFar]
constexpr float kLead = 24.f, kSlack = 16.f;       // a reference over its logit; a logit over its reference

struct WideShared {
  uint64_t k_full[2], k_empty[2], v_full[2][kVSlots], v_empty[2][kVSlots], s_full[2], p_full[2], pv_done[2], drain[2];
  alignas(16) uint32_t mask[2][4][4];  // of each worker's last four tiles: which positions count
  uint32_t first[2][4];                // and whether they begin a segment
  alignas(16) float ref[2][kH], alpha[2][kH];
  RangeShared<2> r;
  uint32_t tmem;
  int32_t abort;
};
constexpr int kWideSmem = 1024 + kSlotBytes + 2 * kPBytes + 2 * kQBytes + static_cast<int>(sizeof(WideShared));
static_assert(kWideSmem <= 227 * 1024, "");

// 128-byte swizzled operand: K-major (rows of 64 elements of the reduced
// dimension; groups of 8 rows 1024 bytes apart), or MN-major (rows of 64
// elements of the other dimension, one per element of the reduced one; the next
// 64 elements `next` bytes further, groups of 8 rows 1024 bytes apart).
__device__ __forceinline__ uint64_t desc128(uint32_t addr, uint32_t next) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | static_cast<uint64_t>((next >> 4) & 0x3FFFu) << 16 |
         static_cast<uint64_t>(1024u >> 4) << 32 | static_cast<uint64_t>(1u) << 46 | static_cast<uint64_t>(2u) << 61;
}
// Instruction descriptor: bf16 x bf16 -> fp32, M = 128, N = 64; `mn`: both operands MN-major.
__host__ __device__ constexpr uint32_t idesc(bool mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (mn ? 3u << 15 : 0u) | ((kH >> 3) << 17) | ((128u >> 4) << 24);
}
// Eight products along the reduced dimension, issued by one lane: step j reads
// the operands at a + A_j, b + B_j (in 16 bytes), with A_j = A1 (j % 4) + A4 (j / 4).
template <int A1, int A4, int B1, int B4>
__device__ __forceinline__ void mma8(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e, o;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 o, %4, %4;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "add.s64 x, %1, %5;\n\tadd.s64 y, %2, %12;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %6;\n\tadd.s64 y, %2, %13;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %7;\n\tadd.s64 y, %2, %14;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %8;\n\tadd.s64 y, %2, %15;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %9;\n\tadd.s64 y, %2, %16;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %10;\n\tadd.s64 y, %2, %17;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %11;\n\tadd.s64 y, %2, %18;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(accumulate), "n"(A1), "n"(2 * A1), "n"(3 * A1), "n"(A4), "n"(A4 + A1), "n"(A4 + 2 * A1),
      "n"(A4 + 3 * A1), "n"(B1), "n"(2 * B1), "n"(3 * B1), "n"(B4), "n"(B4 + B1), "n"(B4 + 2 * B1), "n"(B4 + 3 * B1)
      : "memory");
}
// Four of them, the operands `step` (in 16 bytes) apart.
template <int kStep>
__device__ __forceinline__ void mma4(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, o, e;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 o, 0, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "add.s64 x, %1, %5;\n\tadd.s64 y, %2, %5;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %6;\n\tadd.s64 y, %2, %6;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %7;\n\tadd.s64 y, %2, %7;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(accumulate), "n"(kStep), "n"(2 * kStep), "n"(3 * kStep)
      : "memory");
}
__device__ __forceinline__ void stmatrix4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}
// `bytes` (a multiple of 16) from shared memory to global memory; what was read
// may be overwritten after the wait (of the same thread).
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;\n\tcp.async.bulk.commit_group;" ::"l"(dst), "r"(src),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// Whether any of a softmax group's threads says so (a barrier of the group).
__device__ __forceinline__ bool group_any(int id, bool mine) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(mine ? 1u : 0u), "r"(id), "n"(kGroup)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}
// 16 rows x 32 columns as matrix fragments: per 8 columns, the lane's row lane / 4
// (r[4 i], r[4 i + 1]) and the one 8 further (r[4 i + 2], r[4 i + 3]), at columns
// 8 i + 2 (lane % 4) and the next.
__device__ __forceinline__ void tmem_ld_frag4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// A score's logit in base 2, rounded by itself: the reference is made of rounded
// logits, and the distance to it would otherwise be off by half of their last place,
// more than any slack from logits of 2^30 on.
__device__ __forceinline__ float logit_of(uint32_t score, float factor) { return __fmul_rn(__uint_as_float(score), factor); }
// Two logits less their references.  (Packed products are fused with the packed
// differences, so these are scalar.)
__device__ __forceinline__ float2 over_ref(uint32_t s0, uint32_t s1, float factor, float r0, float r1) {
  float2 d;
  asm("{\n\t.reg .b64 x, r;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 r, {%4, %5};\n\tsub.rn.f32x2 x, x, r;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(logit_of(s0, factor)), "f"(logit_of(s1, factor)), "f"(r0), "f"(r1));
  return d;
}
struct Buffers {
  uint32_t slots, p, q;  // shared-memory addresses
};
using WideWalk = Walk<kPos>;

// One role's waits: false once anything has given up; the role then goes on
// through its loop without touching memory.
struct Waiter {
  WideShared& sh;
  int32_t* dev_err;
  bool alive = true;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) {
    alive = alive && wait_warp(bar, parity, &sh.abort, dev_err);
    return alive;
  }
};
// A worker's V slots in turn: the halves of its tiles, one after another.
struct VPlace {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void advance() {
    if (++slot == kVSlots) slot = 0, phase ^= 1;
  }
};
__device__ __forceinline__ uint32_t k_slot(const Buffers& b, int g) { return b.slots + g * kKSlot; }
__device__ __forceinline__ uint32_t v_slot(const Buffers& b, int g, int slot) {
  return b.slots + 2 * kKSlot + (g * kVSlots + slot) * kVSlot;
}

// ------------------------------------------------------------------ producers
// The heads [p0, p0 + n) of a unit's queries; zeros past the last one.
struct Queries {
  const uint16_t* src;
  int there;
};
__device__ __forceinline__ Queries queries_of(const Args& k, const WideWalk& w) {
  const int head = w.unit / k.l.blocks, h0 = (w.unit - head * k.l.blocks) * kH;
  return {k.a.q + w.row * k.a.q_stride + (static_cast<int64_t>(head) * k.l.group + h0) * kD, min(kH, k.l.group - h0)};
}
__device__ __forceinline__ void copy_queries(const Queries& q, uint32_t dst, int p0, int n, int lane) {
  const int chunk = lane & 15, odd = lane >> 4;
#pragma unroll 2
  for (int p = p0; p < p0 + n; p += 2) {
    const int h = p + odd;
    copy16(dst + (chunk >> 3) * (kQBytes / 2) + h * 128 + (((chunk & 7) ^ (h & 7)) << 4),
           reinterpret_cast<const uint8_t*>(q.src) + (h < q.there ? h : 0) * (kD * 2) + chunk * 16, h < q.there);
  }
}

// Worker g's pages, by TMA: a tile is two pages.  The K slot of a segment's first
// tile is free once the last product with the segment before is done, and so is
// the worker's query buffer: the queries are fetched with it.
template <bool kValues>
__device__ __forceinline__ void wide_pages(const Args& k, WideShared& sh, WideWalk w, const Buffers& b,
                                           const CUtensorMap* map, int g) {
  const AttnArgs& a = k.a;
  const CacheArgs& c = a.c;
  const int lane = threadIdx.x & 31;
  Waiter wait{sh, c.dev_err};
  VPlace vs;
  uint32_t n = 0;  // tiles so far
#pragma unroll 1
  while (w.next(a)) {
    const int req = row_request(c, w.row), head = w.unit / k.l.blocks;
    const int32_t* table = req >= 0 ? c.page_table + static_cast<int64_t>(req) * c.max_pages : nullptr;
    const int len = table != nullptr ? a.seq_len[w.row] : 0;
    int lo = -1, hi = -1;
#pragma unroll 1
    for (int i = w.i0; i < w.i1; ++i, ++n) {
      const int j = (i - w.i0) & 31;
      if (j == 0) {  // the next 32 tiles' pages, two per lane
        const int64_t at = static_cast<int64_t>(i + lane) * kPos;
        const bool in = i + lane < w.i1;
        lo = in && at < len ? table[at / kPage] : -1;
        hi = in && at + kPage < len ? table[at / kPage + 1] : -1;
        if (!kValues && in && ((at < len && (lo < 0 || lo >= c.num_pages)) || (at + kPage < len && (hi < 0 || hi >= c.num_pages))))
          report(c.dev_err, kDevErrPage);
        if (lo >= c.num_pages) lo = -1;
        if (hi >= c.num_pages) hi = -1;
      }
      const int page0 = __shfl_sync(0xffffffffu, lo, j), page1 = __shfl_sync(0xffffffffu, hi, j);
      if constexpr (kValues) {
#pragma unroll 1
        for (int x = 0; x < 2; ++x, vs.advance()) {
          if (!wait(&sh.v_empty[g][vs.slot], vs.phase ^ 1)) continue;
          const int page = x ? page1 : page0;
          uint64_t* full = &sh.v_full[g][vs.slot];
          if (lane == 0) {
            if (page >= 0)
              mbar_arrive_expect_tx(full, kVSlot);
            else
              mbar_arrive(full);
          }
          __syncwarp();
          if (lane < 2 && page >= 0)
            tma_box(v_slot(b, g, vs.slot) + lane * (kVSlot / 2), map, lane * 128, (page * c.num_kv_heads + head) * kPage, smem_u32(full));
        }
      } else if (wait(&sh.k_empty[g], (n + 1) & 1)) {
        const int pages = (page0 >= 0) + (page1 >= 0);
        const int mine = lane & 2 ? page1 : page0;  // lane 0..3: page lane / 2, dims 64 (lane % 2) ..
        uint64_t* full = &sh.k_full[g];
        if (lane < 4) {
          const int left = mine >= 0 ? len - i * kPos - lane * 32 : 0;
          sh.mask[g][n & 3][lane] = left >= 32 ? ~0u : left > 0 ? (1u << left) - 1 : 0;
          if (lane == 0) sh.first[g][n & 3] = i == w.i0;
        }
        __syncwarp();
        if (lane == 0) {
          if (pages > 0)
            mbar_arrive_expect_tx(full, pages * (kKSlot / 2));
          else
            mbar_arrive(full);
        }
        __syncwarp();
        if (lane < 4 && mine >= 0)
          tma_box(k_slot(b, g) + (lane & 1) * (kKSlot / 2) + (lane >> 1) * (kKSlot / 4), map, (lane & 1) * 128,
                  (mine * c.num_kv_heads + head) * kPage, smem_u32(full));
        if (i == w.i0) {
          copy_queries(queries_of(k, w), b.q + g * kQBytes, 0, kH, lane);
          cp_async_arrive_noinc(full);
        } else {
          mbar_arrive(full);
        }
      }
    }
  }
  cp_async_wait<0>();
}

// 32 listed rows of 256 bytes of a pool, the lane's one (-1: zeros), by 16-byte
// asynchronous copies to dst and behind it, 64 dims there and the others `other`
// further.  (Gathers by TMA: 221 us for 4096 rows over 512 positions, these 210.)
__device__ __forceinline__ void copy_listed(uint32_t dst, uint32_t other, const uint8_t* pool, int row, int lane) {
  const int chunk = lane & 15, odd = lane >> 4;
  dst += (chunk >> 3) * other;
  pool += chunk * 16;
#pragma unroll 4
  for (int p = 0; p < 32; p += 2) {  // rows p and p + 1
    const int at = p + odd, r = __shfl_sync(0xffffffffu, row, at);
    copy16(dst + at * 128 + (((chunk & 7) ^ (at & 7)) << 4), pool + static_cast<int64_t>(max(r, 0)) * (kD * 2), r >= 0);
  }
}

// Worker g's listed rows: two warps fetch K, 64 positions each, which the next
// scores wait for, and one V.  The list entries of the second next tile and the
// page ids of the next one are on their way while a tile is copied.
template <bool kValues>
__device__ __forceinline__ void wide_list(const Args& k, WideShared& sh, WideWalk w, const Buffers& b, int g, int part) {
  constexpr int N = kValues ? 4 : 2;  // positions per lane
  struct Entry {
    const int32_t* table;  // null: the row has no request
    int head, len, s[N];
    bool live, first;
    Queries q;
  };
  const AttnArgs& a = k.a;
  const CacheArgs& c = a.c;
  const int lane = threadIdx.x & 31, first = part * 32 * N + lane;
  Waiter wait{sh, c.dev_err};
  Entry seg{}, now{}, next{};
  int i = 0, end = 0, page[N];
  auto fetch = [&]() {
    Entry x{};
    if (i >= end) {
      if (!w.next(a)) return x;
      i = w.i0, end = w.i1;
      const int req = row_request(c, w.row);
      seg.table = req >= 0 ? c.page_table + static_cast<int64_t>(req) * c.max_pages : nullptr;
      seg.len = seg.table != nullptr ? a.seq_len[w.row] : 0;
      seg.head = w.unit / k.l.blocks;
      if (!kValues) seg.q = queries_of(k, w);
    }
    x = seg;
    x.live = true;
    x.first = i == w.i0;
    const int at = i * kPos + first;
    const int32_t* list = a.pos + static_cast<int64_t>(w.row) * a.pos_stride + at;
#pragma unroll
    for (int j = 0; j < N; ++j) x.s[j] = at + 32 * j < a.npos ? list[32 * j] : -1;
    ++i;
    return x;
  };
  VPlace vs;
  // steps -2 and -1 fill the look-ahead
#pragma unroll 1
  for (int n = -2; n < 0 || now.live; ++n) {
    const bool live = n >= 0 && now.live;
    int row[N];  // -1: an entry that does not count
    uint32_t m[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int s = now.s[j];
      const bool in = live && s >= 0 && s < now.len, ok = in && page[j] >= 0 && page[j] < c.num_pages;
      if (!kValues) {
        if (live && now.table != nullptr && !in && s != -1) report(c.dev_err, kDevErrPos);
        if (ok != in) report(c.dev_err, kDevErrPage);
        m[j] = __ballot_sync(0xffffffffu, ok);
      }
      row[j] = ok ? (page[j] * c.num_kv_heads + now.head) * kPage + (s & (kPage - 1)) : -1;
    }
    const bool begins = now.first;
    const Queries q = now.q;
    // the look-ahead moves on: its loads land while the tile is copied
#pragma unroll
    for (int j = 0; j < N; ++j) page[j] = next.live && next.s[j] >= 0 && next.s[j] < next.len ? next.table[next.s[j] / kPage] : 0;
    const Entry after = fetch();
    now = next, next = after;
    if constexpr (!kValues) {
      if (!live || !wait(&sh.k_empty[g], (n + 1) & 1)) continue;
      uint64_t* full = &sh.k_full[g];
      if (lane == 0) {
        sh.mask[g][n & 3][2 * part] = m[0], sh.mask[g][n & 3][2 * part + 1] = m[1];
        if (part == 0) sh.first[g][n & 3] = begins;
        mbar_arrive(full);
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 2; ++j) copy_listed(k_slot(b, g) + (64 * part + 32 * j) * 128, kKSlot / 2, c.k_pool, row[j], lane);
      if (begins) copy_queries(q, b.q + g * kQBytes, part * (kH / 2), kH / 2, lane);
      cp_async_arrive_noinc(full);
    } else if (live) {
#pragma unroll 1
      for (int x = 0; x < 2; ++x, vs.advance()) {
        if (!wait(&sh.v_empty[g][vs.slot], vs.phase ^ 1)) continue;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          copy_listed(v_slot(b, g, vs.slot) + 32 * j * 128, kVSlot / 2, c.v_pool, x ? row[N - 2 + j] : row[j], lane);
        cp_async_arrive_noinc(&sh.v_full[g][vs.slot]);
      }
    }
  }
  cp_async_wait<0>();
}

// What the copies in flight write lands before the CTA's memory goes (after a
// role has given up): both parities of a barrier, whichever is the last fill's.
__device__ __forceinline__ void drain_copies(WideShared& sh) {
#pragma unroll 1
  for (int i = 0; i < 4 * (1 + kVSlots); ++i) {
    const int g = (i >> 1) & 1, s = i >> 2;
    mbar_wait(s == 0 ? &sh.k_full[g] : &sh.v_full[g][s - 1], i & 1, nullptr, 1000000ull);
  }
}

// ------------------------------------------------------------------ products
// Worker g's: the scores of a tile, as soon as those of the tile before have been
// read, then the values of the tile before.
__device__ __forceinline__ void wide_products(const Args& k, WideShared& sh, const Buffers& b, uint32_t tmem, int g) {
  const AttnArgs& a = k.a;
  const int lane = threadIdx.x & 31, tiles = sh.r.range[g].end - sh.r.range[g].first;
  const uint32_t pb = b.p + g * kPBytes;
  Waiter wait{sh, a.c.dev_err};
  VPlace vs;
#pragma unroll 1
  for (int n = 0; n <= tiles; ++n) {
    if (n > 0) wait(&sh.p_full[g], (n - 1) & 1);
    // the scores come first where their keys are there, so that the softmax goes on beside the values' product
    const bool early = n < tiles && __all_sync(0xffffffffu, mbar_try_wait(&sh.k_full[g], n & 1));
#pragma unroll 1
    for (int step = 0; step < 3; ++step) {
      if (step != 1) {
        if (n == tiles || early != (step == 0) || !wait(&sh.k_full[g], n & 1)) continue;
        fence_proxy_async_smem();  // queries are written through the generic proxy
        tc_fence_after();
        mma8<2, kKSlot / 2 / 16, 2, kQBytes / 2 / 16>(tmem + kColS + kH * g, desc128(k_slot(b, g), 16),
                                                      desc128(b.q + g * kQBytes, 16), idesc(false), 0);
        mma_commit_elect(&sh.s_full[g]);
        mma_commit_elect(&sh.k_empty[g]);
        continue;
      }
      if (n == 0) continue;
      const uint32_t* mask = sh.mask[g][(n - 1) & 3];
      uint32_t more = sh.first[g][(n - 1) & 3] ^ 1;  // adds to the segment's earlier tiles
#pragma unroll 1
      for (int x = 0; x < 2; ++x, vs.advance(), more = 1) {
        if (!wait(&sh.v_full[g][vs.slot], vs.phase)) continue;
        const uint32_t vb = v_slot(b, g, vs.slot);
        if (a.pos == nullptr && (mask[2 * x] & mask[2 * x + 1]) != ~0u) {
          // values that do not count must not reach a product with 0
#pragma unroll 1
          for (int e = lane; e < 64 * 16; e += 32) {
            const int p = e >> 4, c = e & 15;
            if ((mask[2 * x + (p >> 5)] >> (p & 31)) & 1) continue;
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(vb + (c >> 3) * (kVSlot / 2) + p * 128 + (c & 7) * 16), "r"(0)
                         : "memory");
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        fence_proxy_async_smem();  // listed rows and probabilities are written through the generic proxy
        tc_fence_after();
        mma4<128>(tmem + kColO + kH * g, desc128(vb, kVSlot / 2), desc128(pb + x * 64 * 128, 16), idesc(true), more);
        mma_commit_elect(&sh.v_empty[g][vs.slot]);
      }
      if (wait.alive) mma_commit_elect(&sh.pv_done[g]);
    }
  }
  if (!wait.alive) {  // the products in flight end before the CTA's memory goes
    mma_commit_elect(&sh.drain[g]);
    mbar_wait(&sh.drain[g], 0, nullptr, 1000000ull);
  }
}

// ------------------------------------------------------------------ softmax
// Halves the columns that a lane keeps and adds the partner's share of them.
template <int kHalf, int kBit>
__device__ __forceinline__ void fold(float (&l)[8], int lane) {
  const bool up = (lane & kBit) != 0;
#pragma unroll
  for (int j = 0; j < kHalf; ++j) {
    const float give = up ? l[j] : l[j + kHalf], keep = up ? l[j + kHalf] : l[j];
    l[j] = keep + __shfl_xor_sync(0xffffffffu, give, kBit);
  }
}
// The sum over the warp's 32 rows of tensor memory of 32 columns; the lane gets
// that of column sum_column(lane).  Read as matrix fragments (a lane has four
// rows and eight columns), so that three exchanges are left.
__device__ __forceinline__ int sum_column(int lane) { return 8 * (lane >> 3) + 2 * (lane & 3) + ((lane >> 2) & 1); }
__device__ __forceinline__ float sum_rows(uint32_t taddr, int lane) {
  uint32_t x[16], y[16];
  tmem_ld_frag4(taddr, x);
  tmem_ld_frag4(taddr + (16u << 16), y);
  tmem_ld_wait();
  float l[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {  // column block j / 2, column j % 2 of the lane's pair: rows r and r + 8
    const int i = 4 * (j >> 1) + (j & 1);
    l[j] = (__uint_as_float(x[i]) + __uint_as_float(x[i + 2])) + (__uint_as_float(y[i]) + __uint_as_float(y[i + 2]));
  }
  fold<4, 16>(l, lane);
  fold<2, 8>(l, lane);
  fold<1, 4>(l, lane);
  return l[0];
}

__device__ __forceinline__ void wide_softmax(const Args& k, WideShared& sh, WideWalk w, const Buffers& b, uint8_t* pmem, uint32_t tmem,
                             int g) {
  const AttnArgs& a = k.a;
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, row = quad * 32 + lane;
  const int in_group = threadIdx.x & (kGroup - 1), half = (in_group >> 7) * 32;  // the warp's heads: half .. half + 31
  const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16) + kH * g + half;  // this warp's, at its columns
  float* scratch = reinterpret_cast<float*>(pmem + g * kPBytes);  // [2][4][kH], while no product reads the probabilities
  float *group_ref = sh.ref[g], *group_alpha = sh.alpha[g], *ref = group_ref + half, *alpha = group_alpha + half;
  Waiter wait{sh, a.c.dev_err};
  uint32_t mine = 0;  // tiles so far
#pragma unroll 1
  while (w.next(a)) {
    bool set = false;  // whether there are references
#pragma unroll 1
    for (int i = w.i0; i < w.i1; ++i) {
      const float factor = a.scale * kLog2e;
      wait(&sh.s_full[g], mine & 1);
      tc_fence_after();
      const uint4 m = *reinterpret_cast<const uint4*>(sh.mask[g][mine & 3]);
      const bool valid = ((quad == 0 ? m.x : quad == 1 ? m.y : quad == 2 ? m.z : m.w) >> lane) & 1;
      // (asked of the group: after a role has given up, its warps may see different masks, and must still meet)
      if (!set && group_any(1 + g, (m.x | m.y | m.z | m.w) != 0)) {  // the first position's logits
        const int first = m.x ? __ffs(m.x) - 1 : m.y ? 31 + __ffs(m.y) : m.z ? 63 + __ffs(m.z) : 95 + __ffs(m.w);
#pragma unroll 1
        for (int h = 0; h < 32; h += 8) {
          uint32_t s[8];
          tmem_ld8(lanes + kColS + h, s);
          tmem_ld_wait();
          if (row == first) {
#pragma unroll
            for (int j = 0; j < 8; ++j) ref[h + j] = fmaxf(fminf(logit_of(s[j], factor) + kLead, kFar), -kFar);
          }
        }
        named_sync(1 + g, kGroup);
        set = true;
      }
      float over = -INFINITY;
      {
        uint32_t s[16];
#pragma unroll 1
        for (int h = 0; h < 32; h += 16) {
        tmem_ld16(lanes + kColS + h, s);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 r = *reinterpret_cast<const float4*>(ref + h + j);
          const float2 a = over_ref(s[j], s[j + 1], factor, r.x, r.y), b = over_ref(s[j + 2], s[j + 3], factor, r.z, r.w);
          over = fmaxf(over, fmaxf(a.x, a.y));
          over = fmaxf(over, fmaxf(b.x, b.y));
        }}
      }
      const bool raise = group_any(1 + g, valid && over > kSlack);
      if (mine > 0) wait(&sh.pv_done[g], (mine - 1) & 1);  // the probabilities' buffer is free, O is complete
      if (raise) {
#pragma unroll 1
        for (int h = 0; h < 32; h += 4) {
          uint32_t x[4];
          tmem_ld4(lanes + kColS + h, x);
          tmem_ld_wait();
#pragma unroll 1
          for (int j = 0; j < 4; ++j) {
            const float r = warp_max(valid ? logit_of(j == 0 ? x[0] : j == 1 ? x[1] : j == 2 ? x[2] : x[3], factor) : -INFINITY);
            if (lane == 0) scratch[quad * kH + half + h + j] = r;
          }
        }
        named_sync(1 + g, kGroup);
        if (in_group < kH) {
          const float old = group_ref[in_group];
          float top = old;
#pragma unroll
          for (int x = 0; x < 4; ++x) top = fmaxf(top, scratch[x * kH + in_group] + kLead);
          group_alpha[in_group] = exp2_approx(old - top);
          group_ref[in_group] = top;
        }
        named_sync(1 + g, kGroup);
        if (i > w.i0) {  // what the segment has so far
          tc_fence_after();
#pragma unroll 1
          for (int x = 0; x < 96; x += 8) {  // O and both sums: 2 kH columns apart
            uint32_t o[8];
            const int h = x & 31;
            const uint32_t at = lanes + kColO + (x >> 5) * 2 * kH + h;
            tmem_ld8(at, o);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha[h + j]);
            tmem_st8(at, o);
          }
          tmem_st_wait();
        }
      }
      uint8_t* prow = pmem + g * kPBytes + row * 128;
      const bool fresh = i == w.i0;
#pragma unroll 1
      for (int j0 = 0; j0 < 32; j0 += 8) {
        uint32_t s[8], l[8], lr[8], v[4];
        tmem_ld8(lanes + kColS + j0, s);
        tmem_ld8(lanes + kColL + j0, l);
        tmem_ld8(lanes + kColR + j0, lr);
        tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 8; x += 2) {
          const float2 r = *reinterpret_cast<const float2*>(ref + j0 + x);
          const float2 d = over_ref(s[x], s[x + 1], factor, r.x, r.y);
          float p0 = exp2_approx(d.x), p1 = exp2_approx(d.y);
          if (!valid) p0 = p1 = 0.f;
          v[x / 2] = bf16x2(p0, p1);
          const float r0 = bf16_lo(v[x / 2]), r1 = bf16_hi(v[x / 2]);
          l[x] = __float_as_uint(fresh ? p0 : __uint_as_float(l[x]) + p0);
          l[x + 1] = __float_as_uint(fresh ? p1 : __uint_as_float(l[x + 1]) + p1);
          lr[x] = __float_as_uint(fresh ? r0 : __uint_as_float(lr[x]) + r0);
          lr[x + 1] = __float_as_uint(fresh ? r1 : __uint_as_float(lr[x + 1]) + r1);
        }
        *reinterpret_cast<uint4*>(prow + ((((half + j0) >> 3) ^ (row & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
        tmem_st8(lanes + kColL + j0, l);
        tmem_st8(lanes + kColR + j0, lr);
      }
      tmem_st_wait();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_full[g]);
      ++mine;
    }
    // ---- the segment's end: sums over the positions, the result
    const float sum_p = sum_rows(lanes + kColL, lane), sum_r = sum_rows(lanes + kColR, lane);
    wait(&sh.pv_done[g], (mine - 1) & 1);  // the products that read the probabilities are done, O is complete
    tc_fence_after();
    scratch[quad * kH + half + sum_column(lane)] = sum_p;
    scratch[(4 + quad) * kH + half + sum_column(lane)] = sum_r;
    named_sync(1 + g, kGroup);
    const bool whole = w.i0 == 0 && w.i1 == w.n;
    const int64_t slot = slot_of(sh.r.range[g].worker, w.i0 == 0);
    const int head = w.unit / k.l.blocks, h0 = (w.unit - head * k.l.blocks) * kH, live = min(kH, k.l.group - h0);
    if (in_group < kH) {
      const int h = in_group;
      const float *sp = scratch + h, *sr = sp + 4 * kH;
      const float total = (sp[0] + sp[kH]) + (sp[2 * kH] + sp[3 * kH]);
      const float rounded = (sr[0] + sr[kH]) + (sr[2 * kH] + sr[3 * kH]);  // 0 only with the other
      const float top = total != 0.f ? group_ref[h] : -kFar;
      group_alpha[h] = rounded == 0.f ? 0.f : (whole ? 1.f : total) / rounded;  // (attn.cuh says why)
      if (!whole) {
        *reinterpret_cast<float2*>(k.stat + (slot * kH + h) * 2) = make_float2(top, total);
      } else if (a.lse != nullptr && h < live) {
        a.lse[static_cast<int64_t>(w.row) * a.c.num_q_heads + static_cast<int64_t>(head) * k.l.group + h0 + h] =
            total == 0.f ? -INFINITY : (top + log2f(total)) * 0.6931471805599453f;
      }
    }
    named_sync(1 + g, kGroup);
    // O's fragments: the lane has dims quad * 32 + 16 d + lane / 4 (+ 8) of heads 8 x + 2 (lane % 4) (+ 1)
    uint16_t* turned = reinterpret_cast<uint16_t*>(pmem + g * kPBytes);  // [kH][kD]
    const uint32_t row0 = smem_u32(turned) + (half + (lane & 7)) * (kD * 2) + (quad * 32 + (lane & 8)) * 2 + (lane >> 4) * 8 * (kD * 2);
#pragma unroll 1
    for (int d = 0; d < 2; ++d) {
      uint32_t o[16];
      tmem_ld_frag4(lanes + kColO + (static_cast<uint32_t>(d * 16) << 16), o);
      tmem_ld_wait();
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float2 f = *reinterpret_cast<const float2*>(alpha + 8 * x + 2 * (lane & 3));
#pragma unroll
        for (int y = 0; y < 4; ++y) o[4 * x + y] = __float_as_uint(__uint_as_float(o[4 * x + y]) * (y & 1 ? f.y : f.x));
      }
      if (whole) {
#pragma unroll
        for (int x = 0; x < 4; x += 2)  // heads 8 x .. 8 x + 15: matrices of 8 dims and 8 heads, turned
          stmatrix4_trans(row0 + x * 8 * (kD * 2) + d * 32, bf16x2(__uint_as_float(o[4 * x]), __uint_as_float(o[4 * x + 1])),
                          bf16x2(__uint_as_float(o[4 * x + 2]), __uint_as_float(o[4 * x + 3])),
                          bf16x2(__uint_as_float(o[4 * x + 4]), __uint_as_float(o[4 * x + 5])),
                          bf16x2(__uint_as_float(o[4 * x + 6]), __uint_as_float(o[4 * x + 7])));
      } else {
        float* sum = k.sum + (slot * kH + half + 2 * (lane & 3)) * kD + quad * 32 + d * 16 + (lane >> 2);
#pragma unroll
        for (int x = 0; x < 16; ++x)
          if (half + 8 * (x >> 2) + 2 * (lane & 3) + (x & 1) < live)
            sum[(8 * (x >> 2) + (x & 1)) * kD + (x & 2) * 4] = __uint_as_float(o[x]);
      }
    }
    if (whole) {
      fence_proxy_async_smem();
      named_sync(1 + g, kGroup);
      if (in_group == 0) {
        uint16_t* out = a.out + w.row * a.out_stride + (static_cast<int64_t>(head) * k.l.group + h0) * kD;
        bulk_store(out, smem_u32(turned), live * kD * 2);
        bulk_store_wait_read();
      }
    } else if (in_group == 0 && w.i0 == 0) {
      k.part[sh.r.range[g].worker] = part_of(w, sh.r.range[g]);
    }
    tc_fence_before();
    // the next writes to references, factors and probabilities come behind a barrier of the group's next tile
  }
}

__global__ void __launch_bounds__(kWideThreads, 1)
    attn_wide_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const Args k) {
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;  // the swizzle is one of address bits
  uint8_t* mem = raw + (base - smem_u32(raw));
  const Buffers b{base, base + kSlotBytes, base + kSlotBytes + 2 * kPBytes};
  uint8_t* pmem = mem + kSlotBytes;
  WideShared& sh = *reinterpret_cast<WideShared*>(mem + kSlotBytes + 2 * kPBytes + 2 * kQBytes);
  const AttnArgs& a = k.a;
  const int tid = threadIdx.x, warp = tid >> 5;
  if (warp == 1) {
    tmem_alloc(&sh.tmem, kTmem);
    tmem_relinquish();
  }
  if (tid == 0) {
    // K: per producer warp the bytes, and every lane (a segment's first tile: its copies of the queries); listed V: every lane
    for (int g = 0; g < 2; ++g) {
      mbar_init(&sh.k_full[g], a.pos != nullptr ? 2 * 33 : 33);
      mbar_init(&sh.k_empty[g], 1);
      mbar_init(&sh.s_full[g], 1);
      mbar_init(&sh.p_full[g], kSoftmaxWarps);
      mbar_init(&sh.pv_done[g], 1);
      mbar_init(&sh.drain[g], 1);
      for (int s = 0; s < kVSlots; ++s) mbar_init(&sh.v_full[g][s], a.pos != nullptr ? 32 : 1), mbar_init(&sh.v_empty[g][s], 1);
    }
    fence_mbar_init();
    sh.abort = 0;
  }
  wait_predecessor();
  // each CTA its own workers' records: nothing orders it with the CTAs that write the others
  if (tid < 2) k.part[blockIdx.x + tid * gridDim.x].last = -1;
  if (tid < 2 * kH) sh.ref[tid / kH][tid % kH] = 0.f;
  tc_fence_before();
  const int units = a.c.num_kv_heads * k.l.blocks;
  const bool none = find_ranges<kWideThreads, kPos, 2>(k, sh.r, units);
  tc_fence_after();
  if (none) write_empty_rows<kD, kWideThreads>(a);
  const uint32_t tmem = sh.tmem;
  if (warp < 8) {
    const int g = warp & 1;
    const WideWalk w = walk_of<kPos>(a, sh.r.range[g], units);
    if (warp < 2) {
      wide_products(k, sh, b, tmem, g);
    } else if (warp < 4) {
      if (a.pos != nullptr)
        wide_list<true>(k, sh, w, b, g, 0);
      else
        wide_pages<true>(k, sh, w, b, &vmap, g);
    } else if (a.pos != nullptr) {
      wide_list<false>(k, sh, w, b, g, (warp >> 1) & 1);
    } else if (warp < 6) {
      wide_pages<false>(k, sh, w, b, &kmap, g);
    }
  } else {
    const int g = (warp - 8) >> 3;
    wide_softmax(k, sh, walk_of<kPos>(a, sh.r.range[g], units), b, pmem, tmem, g);
  }
  tc_fence_before();
  __syncthreads();
  if (sh.abort != 0 && warp == 0) drain_copies(sh);
  if (warp == 1) tmem_dealloc(tmem, kTmem);
  release_successor();
}

}  // namespace

cudaError_t launch_wide(const CUtensorMap& kmap, const CUtensorMap& vmap, const Args& k, cudaStream_t stream) {
  static bool set[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !set[dev]) {
    e = cudaFuncSetAttribute(attn_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kWideSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) set[dev] = true;
  }
  return launch_after(attn_wide_kernel, dim3(k.l.ctas / 2), kWideThreads, kWideSmem, stream, kmap, vmap, k);
}

}  // namespace attn
}  // namespace ci
