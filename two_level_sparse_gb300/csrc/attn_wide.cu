// Attention over a paged bf16 cache where many query heads (more than 16)
// share a key-value head of 128 dims (contract in include/ci_cache.h; the
// list of tiles, its split over the CTAs and the join are those of attn.cuh).
//
// With G = 64 heads the products cost 64 flop per byte of cache: at the HBM's
// rate 435 TFLOP/s, half of what the warp-level MMA instructions reached
// (their kernel: 108 us for 436 MB, 47% of that pipe), so here the
// fifth-generation tensor cores compute, a tile of 128 positions at a time:
//
//   S^T [128 positions x 64 heads] = K Q^T    A = K (rows of dims), B = Q, both
//                                             from shared memory, S in tensor memory
//   P = 2^(S c - m)                           one thread per position
//   O^T [128 dims x 64 heads] += V^T P^T      A = V and B = P with the positions
//                                             as the reduced rows (MN-major), O in tensor memory
//
// One CTA per SM, two workers per CTA: each has its own range of the list, a
// group of four softmax warps, references, sums and O, so that one's
// exponentials and results run beside the other's products.  Tile t is worker
// (t % 2)'s tile t / 2.  A K tile (32 KB) has the worker's own slot, V tiles
// share three.  One warp issues the products with K, one those with V (a single
// one took 2800 cycles for the two and their waits, as long as the HBM for the
// tile); each worker has a warp per K and V that fetches pages, and listed rows
// are fetched by four warps (K) and two (V) for both.
//
// The reference m of a head is not the running maximum but the logit of the
// segment's first position, kept until another one passes it by 2^40.  fp32 and
// bf16 have the exponents for that: probabilities up to 2^40 are as exact as
// those below one, the reference's own is 1, and maxima across the positions
// (across lanes, here) and the rescaling of O happen only where a logit is
// further off.
#include "attn.cuh"

namespace ci {
namespace attn {
namespace {

constexpr int kD = 128, kH = 64, kPos = 128;
constexpr int kVSlots = 3, kSlots = 2 + kVSlots, kSlot = kPos * kD * 2;  // a K slot per worker, then V's
constexpr int kPBytes = kPos * kH * 2, kQBytes = kH * kD * 2;
constexpr int kWideThreads = 512;
// of worker g, at + 64 g: S, O, the sums of P, those of P as it is rounded
constexpr int kTmem = 512, kColS = 0, kColO = 128, kColL = 256, kColR = 384;
constexpr float kFar = 1.0e30f;                     // references lie in [-kFar, kFar]
constexpr float kSlack = 40.f;

struct WideShared {
  uint64_t k_full[2], k_empty[2], v_full[kVSlots], v_empty[kVSlots], s_full[2], p_full[2], pv_done[2], drain[2];
  alignas(16) uint32_t mask[8][4];  // of the last eight tiles: which positions count
  uint32_t first[8];                // and whether they begin a segment
  alignas(16) float ref[2][kH], alpha[2][kH];
  RangeShared<2> r;
  uint32_t tmem;
  int32_t abort;
};
constexpr int kWideSmem = 1024 + kSlots * kSlot + 2 * kPBytes + 2 * kQBytes + static_cast<int>(sizeof(WideShared));
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
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
// Whether any of a softmax group's 128 threads says so (a barrier of the group).
__device__ __forceinline__ bool group_any(int id, bool mine) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(mine ? 1u : 0u), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
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
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
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
// Tile t's V slot, t % 3, and the parity of its t / 3-th use.  (Where one worker
// has a tile more than the other, the last tile's number has a gap before it;
// nothing follows that, so the gap's slot is not used again.)
struct VPlace {
  int slot;
  uint32_t phase;
  __device__ __forceinline__ explicit VPlace(int t) : slot(t), phase(0) {}
  __device__ __forceinline__ void advance(int tiles) {
    slot += tiles;
    if (slot >= kVSlots) slot -= kVSlots, phase ^= 1;
  }
};

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
  VPlace vs(g);
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
      const int pages = (page0 >= 0) + (page1 >= 0);
      const int mine = lane & 2 ? page1 : page0;  // lane 0..3: page lane / 2, dims 64 (lane % 2) ..
      uint64_t* full = kValues ? &sh.v_full[vs.slot] : &sh.k_full[g];
      if (kValues ? wait(&sh.v_empty[vs.slot], vs.phase ^ 1) : wait(&sh.k_empty[g], (n + 1) & 1)) {
        if (!kValues && lane < 4) {
          const int left = mine >= 0 ? len - i * kPos - lane * 32 : 0;
          const int at = (2 * n + g) & 7;
          sh.mask[at][lane] = left >= 32 ? ~0u : left > 0 ? (1u << left) - 1 : 0;
          if (lane == 0) sh.first[at] = i == w.i0;
        }
        __syncwarp();
        if (lane == 0) {
          if (pages > 0)
            mbar_arrive_expect_tx(full, pages * (kSlot / 2));
          else
            mbar_arrive(full);
        }
        __syncwarp();
        if (lane < 4 && mine >= 0)
          tma_box(b.slots + (kValues ? 2 + vs.slot : g) * kSlot + (lane & 1) * (kSlot / 2) + (lane >> 1) * (kSlot / 4), map,
                  (lane & 1) * 128, (mine * c.num_kv_heads + head) * kPage, smem_u32(full));
        if (!kValues) {
          if (i == w.i0) {
            copy_queries(queries_of(k, w), b.q + g * kQBytes, 0, kH, lane);
            cp_async_arrive_noinc(full);
          } else {
            mbar_arrive(full);
          }
        }
      }
      vs.advance(2);
    }
  }
  cp_async_wait<0>();
}

// Listed rows of both workers' tiles in turn: four warps gather K by TMA, 32
// positions each, and two copy V by 16-byte asynchronous copies, 64 each
// (produce_list in attn.cuh says why).  Of each worker, the list entries of the
// second next tile and the page ids of the next one are on their way while a
// tile is copied.
template <int N>  // positions per warp: 32 N
struct ListStream {
  struct Entry {
    const int32_t* table;  // null: the row has no request
    int head, len, s[N];
    bool live, first;
    Queries q;
  };
  WideWalk w;
  int i, end, page[N];
  Entry seg, now, next;

  __device__ __forceinline__ ListStream(const AttnArgs& a, const Range& r, int units)
      : w(walk_of<kPos>(a, r, units)), i(0), end(0), seg{}, now{}, next{} {}
  __device__ __forceinline__ Entry fetch(const Args& k, int first) {
    const AttnArgs& a = k.a;
    Entry x{};
    if (i >= end) {
      if (!w.next(a)) return x;
      i = w.i0, end = w.i1;
      const int req = row_request(a.c, w.row);
      seg.table = req >= 0 ? a.c.page_table + static_cast<int64_t>(req) * a.c.max_pages : nullptr;
      seg.len = seg.table != nullptr ? a.seq_len[w.row] : 0;
      seg.head = w.unit / k.l.blocks;
      if (N == 1) seg.q = queries_of(k, w);
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
  }
  // The look-ahead moves on: the next tile becomes the current one.  first: the
  // lane's first position in a tile.
  __device__ __forceinline__ void step(const Args& k, int first) {
#pragma unroll
    for (int j = 0; j < N; ++j) page[j] = next.live && next.s[j] >= 0 && next.s[j] < next.len ? next.table[next.s[j] / kPage] : 0;
    const Entry after = fetch(k, first);
    now = next, next = after;
  }
};

template <bool kValues>
__device__ __forceinline__ void wide_list(const Args& k, WideShared& sh, const Buffers& b, const CUtensorMap* kmap, int part,
                                          int units) {
  constexpr int N = kValues ? 2 : 1;
  const AttnArgs& a = k.a;
  const CacheArgs& c = a.c;
  const int lane = threadIdx.x & 31, chunk = lane & 15, odd = lane >> 4, first = part * 32 * N + lane;
  Waiter wait{sh, c.dev_err};
  ListStream<N> cur(a, sh.r.range[0], units), other(a, sh.r.range[1], units);
  VPlace vs(0);
  // steps -4 .. -1 fill both streams' look-ahead
#pragma unroll 1
  for (int t = -4; t < 0 || cur.now.live || other.now.live; ++t) {
    const bool live = t >= 0 && cur.now.live;
    int row[N];  // -1: an entry that does not count (row 0 of K, zeros of V)
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int s = cur.now.s[j];
      const bool in = live && s >= 0 && s < cur.now.len, ok = in && cur.page[j] >= 0 && cur.page[j] < c.num_pages;
      if (!kValues) {
        if (live && cur.now.table != nullptr && !in && s != -1) report(c.dev_err, kDevErrPos);
        if (ok != in) report(c.dev_err, kDevErrPage);
        m = __ballot_sync(0xffffffffu, ok);
      }
      row[j] = ok ? (cur.page[j] * c.num_kv_heads + cur.now.head) * kPage + (s & (kPage - 1)) : -1;
    }
    const bool begins = cur.now.first;
    const Queries q = cur.now.q;
    cur.step(k, first);  // its loads land while the tile is copied
    const int g = t & 1;
    if (live && (kValues ? wait(&sh.v_empty[vs.slot], vs.phase ^ 1) : wait(&sh.k_empty[g], ((t >> 1) + 1) & 1))) {
      if constexpr (!kValues) {
        uint64_t* full = &sh.k_full[g];
        const uint32_t dst = b.slots + g * kSlot + part * 32 * 128;
        if (lane == 0) {
          sh.mask[t & 7][part] = m;
          if (part == 0) sh.first[t & 7] = begins;
          mbar_arrive_expect_tx(full, kSlot / 4);
        }
        __syncwarp();
        const int mine = max(row[0], 0);
#pragma unroll 2
        for (int p = 0; p < 32; p += 4) {
          const int r0 = __shfl_sync(0xffffffffu, mine, p), r1 = __shfl_sync(0xffffffffu, mine, p + 1);
          const int r2 = __shfl_sync(0xffffffffu, mine, p + 2), r3 = __shfl_sync(0xffffffffu, mine, p + 3);
          gather4_elect(dst + p * 128, kmap, 0, r0, r1, r2, r3, smem_u32(full));
          gather4_elect(dst + kSlot / 2 + p * 128, kmap, 128, r0, r1, r2, r3, smem_u32(full));
        }
        if (begins) {
          copy_queries(q, b.q + g * kQBytes, part * (kH / 4), kH / 4, lane);
          cp_async_arrive_noinc(full);
        } else {
          mbar_arrive(full);
        }
      } else {
        uint64_t* full = &sh.v_full[vs.slot];
        const uint32_t dst = b.slots + (2 + vs.slot) * kSlot + (chunk >> 3) * (kSlot / 2) + part * 64 * 128;
        const uint8_t* base = c.v_pool + chunk * 16;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll 4
          for (int p = 0; p < 32; p += 2) {  // positions p and p + 1
            const int at = p + odd, r = __shfl_sync(0xffffffffu, row[j], at);
            copy16(dst + (32 * j + at) * 128 + (((chunk & 7) ^ (at & 7)) << 4), base + static_cast<int64_t>(max(r, 0)) * (kD * 2),
                   r >= 0);
          }
        cp_async_arrive_noinc(full);
      }
    }
    if (t >= 0) vs.advance(1);
    const ListStream<N> turn = cur;
    cur = other, other = turn;
  }
  cp_async_wait<0>();
}

// What the copies in flight write lands before the CTA's memory goes (after a
// role has given up): both parities of a barrier, whichever is the last fill's.
__device__ __forceinline__ void drain_copies(WideShared& sh) {
#pragma unroll 1
  for (int i = 0; i < 2 * (2 + kVSlots); ++i) {
    const int s = i >> 1;
    mbar_wait(s < 2 ? &sh.k_full[s] : &sh.v_full[s - 2], i & 1, nullptr, 1000000ull);
  }
}

// ------------------------------------------------------------------ products
__device__ __forceinline__ int tiles_of(const WideShared& sh, int g) {
  return sh.r.range[g].end - sh.r.range[g].first;
}

__device__ __forceinline__ void wide_scores(const Args& k, WideShared& sh, const Buffers& b, uint32_t tmem) {
  Waiter wait{sh, k.a.c.dev_err};
  const int n0 = tiles_of(sh, 0), n1 = tiles_of(sh, 1), steps = 2 * max(n0, n1);
#pragma unroll 1
  for (int t = 0; t < steps; ++t) {
    const int g = t & 1, n = t >> 1;
    if (n >= (g ? n1 : n0)) continue;
    if (n > 0) wait(&sh.p_full[g], (n - 1) & 1);  // the last tile's scores have been read
    if (!wait(&sh.k_full[g], n & 1)) continue;
    fence_proxy_async_smem();  // queries are written through the generic proxy
    tc_fence_after();
    mma8<2, kSlot / 2 / 16, 2, kQBytes / 2 / 16>(tmem + kColS + kH * g, desc128(b.slots + g * kSlot, 16),
                                                 desc128(b.q + g * kQBytes, 16), idesc(false), 0);
    mma_commit_elect(&sh.s_full[g]);
    mma_commit_elect(&sh.k_empty[g]);
  }
  if (!wait.alive) {  // the products in flight end before the CTA's memory goes
    mma_commit_elect(&sh.drain[0]);
    mbar_wait(&sh.drain[0], 0, nullptr, 1000000ull);
  }
}

__device__ __forceinline__ void wide_values(const Args& k, WideShared& sh, const Buffers& b, uint32_t tmem) {
  const AttnArgs& a = k.a;
  const int lane = threadIdx.x & 31;
  Waiter wait{sh, a.c.dev_err};
  const int n0 = tiles_of(sh, 0), n1 = tiles_of(sh, 1), steps = 2 * max(n0, n1);
  VPlace vs(0);
#pragma unroll 1
  for (int t = 0; t < steps; ++t, vs.advance(1)) {
    const int g = t & 1, n = t >> 1;
    if (n >= (g ? n1 : n0)) continue;
    wait(&sh.v_full[vs.slot], vs.phase);
    if (!wait(&sh.p_full[g], n & 1)) continue;
    const uint32_t vb = b.slots + (2 + vs.slot) * kSlot, pb = b.p + g * kPBytes;
    const uint4 m = *reinterpret_cast<const uint4*>(sh.mask[t & 7]);
    const uint32_t more = sh.first[t & 7] ^ 1;  // adds to the segment's earlier tiles
    if (a.pos == nullptr && (m.x & m.y & m.z & m.w) != ~0u) {
      // values that do not count must not reach a product with 0
#pragma unroll 1
      for (int e = lane; e < kPos * 16; e += 32) {
        const int p = e >> 4, c = e & 15;
        if ((sh.mask[t & 7][p >> 5] >> (p & 31)) & 1) continue;
        asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(vb + (c >> 3) * (kSlot / 2) + p * 128 + (c & 7) * 16), "r"(0)
                     : "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
    }
    fence_proxy_async_smem();  // listed rows and probabilities are written through the generic proxy
    tc_fence_after();
    mma8<128, 512, 128, 512>(tmem + kColO + kH * g, desc128(vb, kSlot / 2), desc128(pb, 16), idesc(true), more);
    mma_commit_elect(&sh.pv_done[g]);
    mma_commit_elect(&sh.v_empty[vs.slot]);
  }
  if (!wait.alive) {
    mma_commit_elect(&sh.drain[1]);
    mbar_wait(&sh.drain[1], 0, nullptr, 1000000ull);
  }
}

// ------------------------------------------------------------------ softmax
// S, the sums and O are read from tensor memory half of the heads at a time, in
// loops that are not unrolled: with every role's code straight-line, the roles
// together outgrew the instruction cache, and a row of 512 positions (four tiles)
// took twice as long.
//
// Halves the heads that a lane keeps and adds the partner's share of them.
template <int kHalf, int kBit>
__device__ __forceinline__ void fold(uint32_t (&l)[32], int lane) {
  const bool up = (lane & kBit) != 0;
#pragma unroll
  for (int j = 0; j < kHalf; ++j) {
    const uint32_t give = up ? l[j] : l[j + kHalf], keep = up ? l[j + kHalf] : l[j];
    l[j] = __float_as_uint(__uint_as_float(keep) + __uint_as_float(__shfl_xor_sync(0xffffffffu, give, kBit)));
  }
}

__device__ __forceinline__ void wide_softmax(const Args& k, WideShared& sh, WideWalk w, const Buffers& b, uint8_t* pmem, uint32_t tmem,
                             int g) {
  const AttnArgs& a = k.a;
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, row = quad * 32 + lane;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16) + kH * g;  // this warp's, at the worker's columns
  const float factor = a.scale * kLog2e;
  const Range range = sh.r.range[g];
  float* scratch = reinterpret_cast<float*>(pmem + g * kPBytes);  // [4][2 kH], while no product reads the probabilities
  float *ref = sh.ref[g], *alpha = sh.alpha[g];
  const int worker = range.worker;
  Waiter wait{sh, a.c.dev_err};
  uint32_t mine = 0;  // tiles so far: the CTA's tile 2 mine + g
#pragma unroll 1
  while (w.next(a)) {
    const int head = w.unit / k.l.blocks, h0 = (w.unit - head * k.l.blocks) * kH, live = min(kH, k.l.group - h0);
    bool set = false;  // whether there are references
#pragma unroll 1
    for (int i = w.i0; i < w.i1; ++i) {
      wait(&sh.s_full[g], mine & 1);
      tc_fence_after();
      const uint4 m = *reinterpret_cast<const uint4*>(sh.mask[(2 * mine + g) & 7]);
      const bool valid = ((quad == 0 ? m.x : quad == 1 ? m.y : quad == 2 ? m.z : m.w) >> lane) & 1;
      if (!set && (m.x | m.y | m.z | m.w) != 0) {  // the first position's logits
        const int first = m.x ? __ffs(m.x) - 1 : m.y ? 31 + __ffs(m.y) : m.z ? 63 + __ffs(m.z) : 95 + __ffs(m.w);
#pragma unroll 1
        for (int h = 0; h < kH; h += 8) {
          uint32_t s[8];
          tmem_ld8(lanes + kColS + h, s);
          tmem_ld_wait();
          if (row == first) {
#pragma unroll
            for (int j = 0; j < 8; ++j) ref[h + j] = fmaxf(fminf(__uint_as_float(s[j]) * factor, kFar), -kFar);
          }
        }
        named_sync(1 + g, 128);
        set = true;
      }
      float over = -INFINITY;
#pragma unroll 1
      for (int h = 0; h < kH; h += 32) {
        uint32_t s[32];
        tmem_ld32(lanes + kColS + h, s);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 r = *reinterpret_cast<const float4*>(ref + h + j);
          over = fmaxf(over, fmaxf(fmaf(__uint_as_float(s[j]), factor, -r.x), fmaf(__uint_as_float(s[j + 1]), factor, -r.y)));
          over = fmaxf(over, fmaxf(fmaf(__uint_as_float(s[j + 2]), factor, -r.z), fmaf(__uint_as_float(s[j + 3]), factor, -r.w)));
        }
      }
      const bool raise = group_any(1 + g, valid && over > kSlack);
      if (mine > 0) wait(&sh.pv_done[g], (mine - 1) & 1);  // the probabilities' buffer is free, O is complete
      if (raise) {
#pragma unroll 1
        for (int h = 0; h < kH; h += 4) {
          uint32_t x[4];
          tmem_ld4(lanes + kColS + h, x);
          tmem_ld_wait();
#pragma unroll 1
          for (int j = 0; j < 4; ++j) {
            const float r = warp_max(valid ? __uint_as_float(j == 0 ? x[0] : j == 1 ? x[1] : j == 2 ? x[2] : x[3]) * factor : -INFINITY);
            if (lane == 0) scratch[quad * kH + h + j] = r;
          }
        }
        named_sync(1 + g, 128);
        if (row < kH) {
          const float old = ref[row];
          float top = old;
#pragma unroll
          for (int x = 0; x < 4; ++x) top = fmaxf(top, scratch[x * kH + row]);
          alpha[row] = exp2_approx(old - top);
          ref[row] = top;
        }
        named_sync(1 + g, 128);
        if (i > w.i0) {  // what the segment has so far
          tc_fence_after();
#pragma unroll 1
          for (int h = 0; h < 3 * kH; h += 8) {  // O and both sums: 2 kH columns apart
            uint32_t o[8];
            const uint32_t at = lanes + kColO + h + (h / kH) * kH;
            tmem_ld8(at, o);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha[(h & (kH - 1)) + j]);
            tmem_st8(at, o);
          }
          tmem_st_wait();
        }
      }
      uint8_t* prow = pmem + g * kPBytes + row * 128;
#pragma unroll 1
      for (int h = 0; h < kH; h += 32) {
        uint32_t s[32];
        tmem_ld32(lanes + kColS + h, s);
        tmem_ld_wait();
        const bool fresh = i == w.i0;
#pragma unroll
        for (int j0 = 0; j0 < 32; j0 += 16) {
          uint32_t l[16], lr[16];
          tmem_ld16(lanes + kColL + h + j0, l);
          tmem_ld16(lanes + kColR + h + j0, lr);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; j += 8) {
            uint32_t v[4];
#pragma unroll
            for (int x = 0; x < 8; x += 2) {
              const float2 r = *reinterpret_cast<const float2*>(ref + h + j0 + j + x);
              float p0 = exp2_approx(fmaf(__uint_as_float(s[j0 + j + x]), factor, -r.x));
              float p1 = exp2_approx(fmaf(__uint_as_float(s[j0 + j + x + 1]), factor, -r.y));
              if (!valid) p0 = p1 = 0.f;
              v[x / 2] = bf16x2(p0, p1);
              const float r0 = bf16_lo(v[x / 2]), r1 = bf16_hi(v[x / 2]);
              l[j + x] = __float_as_uint(fresh ? p0 : __uint_as_float(l[j + x]) + p0);
              l[j + x + 1] = __float_as_uint(fresh ? p1 : __uint_as_float(l[j + x + 1]) + p1);
              lr[j + x] = __float_as_uint(fresh ? r0 : __uint_as_float(lr[j + x]) + r0);
              lr[j + x + 1] = __float_as_uint(fresh ? r1 : __uint_as_float(lr[j + x + 1]) + r1);
            }
            *reinterpret_cast<uint4*>(prow + ((((h + j0 + j) >> 3) ^ (row & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
          }
          tmem_st16(lanes + kColL + h + j0, l);
          tmem_st16(lanes + kColR + h + j0, lr);
        }
      }
      tmem_st_wait();
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_full[g]);
      ++mine;
    }
    // ---- the segment's end: sums over the positions, the result
#pragma unroll 1
    for (int h = 0; h < 2 * kH; h += 32) {  // the sums of P, then those of P as it is rounded
      uint32_t l[32];
      tmem_ld32(lanes + kColL + h + (h & kH), l);
      tmem_ld_wait();
      fold<16, 16>(l, lane);
      fold<8, 8>(l, lane);
      fold<4, 4>(l, lane);
      fold<2, 2>(l, lane);
      fold<1, 1>(l, lane);
      if (h == 0) {  // (the products that read the probabilities are done before the buffer is written)
        wait(&sh.pv_done[g], (mine - 1) & 1);
        tc_fence_after();
      }
      scratch[quad * 2 * kH + h + lane] = __uint_as_float(l[0]);  // lane bits 16 .. 1 chose heads + 16 .. + 1
    }
    named_sync(1 + g, 128);
    const bool whole = w.i0 == 0 && w.i1 == w.n;
    const int64_t slot = 2ll * worker + (w.i0 == 0 ? 1 : 0);
    if (row < kH) {
      const int h = row;
      const float total = (scratch[h] + scratch[2 * kH + h]) + (scratch[4 * kH + h] + scratch[6 * kH + h]);
      const float* sr = scratch + kH;
      const float rounded = (sr[h] + sr[2 * kH + h]) + (sr[4 * kH + h] + sr[6 * kH + h]);  // 0 only with the other
      const float top = total != 0.f ? ref[h] : -kFar;
      alpha[h] = rounded == 0.f ? 0.f : (whole ? 1.f : total) / rounded;  // (attn.cuh says why)
      if (!whole) {
        *reinterpret_cast<float2*>(k.stat + (slot * kH + h) * 2) = make_float2(top, total);
      } else if (a.lse != nullptr && h < live) {
        a.lse[static_cast<int64_t>(w.row) * a.c.num_q_heads + static_cast<int64_t>(head) * k.l.group + h0 + h] =
            total == 0.f ? -INFINITY : (top + log2f(total)) * 0.6931471805599453f;
      }
    }
    named_sync(1 + g, 128);
    // a thread holds one dim of all heads; whole results are turned in shared memory
    uint16_t* turned = reinterpret_cast<uint16_t*>(pmem + g * kPBytes);  // [kH][kD]
    float* sum = k.sum + slot * kH * kD + row;
#pragma unroll 1
    for (int h = 0; h < live; h += 16) {
      uint32_t o[16];
      tmem_ld16(lanes + kColO + h, o);
      tmem_ld_wait();
      if (whole) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          turned[(h + j) * kD + row] = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(o[j]) * alpha[h + j]));
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (h + j < live) sum[(h + j) * kD] = __uint_as_float(o[j]) * alpha[h + j];
      }
    }
    if (whole) {
      named_sync(1 + g, 128);
      uint16_t* out = a.out + w.row * a.out_stride + (static_cast<int64_t>(head) * k.l.group + h0) * kD;
#pragma unroll 2
      for (int e = row; e < live * (kD / 8); e += 128)
        *reinterpret_cast<uint4*>(out + e * 8) = *reinterpret_cast<const uint4*>(turned + e * 8);
    } else if (row == 0 && w.i0 == 0) {
      k.part[worker] = part_of(w, range);
    }
    tc_fence_before();
    named_sync(1 + g, 128);  // O, the factors and the shared buffer have been read
  }
}

__global__ void __launch_bounds__(kWideThreads, 1)
    attn_wide_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const Args k) {
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;  // the swizzle is one of address bits
  uint8_t* mem = raw + (base - smem_u32(raw));
  const Buffers b{base, base + kSlots * kSlot, base + kSlots * kSlot + 2 * kPBytes};
  uint8_t* pmem = mem + kSlots * kSlot;
  WideShared& sh = *reinterpret_cast<WideShared*>(mem + kSlots * kSlot + 2 * kPBytes + 2 * kQBytes);
  const AttnArgs& a = k.a;
  const int tid = threadIdx.x, warp = tid >> 5;
  if (warp == 1) {
    tmem_alloc(&sh.tmem, kTmem);
    tmem_relinquish();
  }
  if (tid == 0) {
    // K: per producer warp the bytes, and every lane (a segment's first tile: its copies of the queries); listed V: every lane
    for (int g = 0; g < 2; ++g) {
      mbar_init(&sh.k_full[g], a.pos != nullptr ? 4 * 33 : 33);
      mbar_init(&sh.k_empty[g], 1);
      mbar_init(&sh.s_full[g], 1);
      mbar_init(&sh.p_full[g], 4);
      mbar_init(&sh.pv_done[g], 1);
      mbar_init(&sh.drain[g], 1);
    }
    for (int s = 0; s < kVSlots; ++s) mbar_init(&sh.v_full[s], a.pos != nullptr ? 64 : 1), mbar_init(&sh.v_empty[s], 1);
    fence_mbar_init();
    sh.abort = 0;
  }
  wait_predecessor();
  if (tid < 2) k.part[2 * blockIdx.x + tid].last = -1;
  if (tid < 2 * kH) sh.ref[tid / kH][tid % kH] = 0.f;
  tc_fence_before();
  const int units = a.c.num_kv_heads * k.l.blocks;
  const bool none = find_ranges<kWideThreads, kPos, 2>(k, sh.r, units);
  tc_fence_after();
  if (none) write_empty_rows<kD, kWideThreads>(a);
  const uint32_t tmem = sh.tmem;
  if (warp < 8) {
    if (warp == 0) wide_scores(k, sh, b, tmem);
    if (warp == 1) wide_values(k, sh, b, tmem);
    if (a.pos != nullptr) {
      if (warp == 2 || warp == 3) wide_list<true>(k, sh, b, &kmap, warp - 2, units);
      if (warp >= 4) wide_list<false>(k, sh, b, &kmap, warp - 4, units);
    } else if (warp >= 4) {
      const int g = warp & 1;
      const WideWalk w = walk_of<kPos>(a, sh.r.range[g], units);
      if (warp < 6)
        wide_pages<false>(k, sh, w, b, &kmap, g);
      else
        wide_pages<true>(k, sh, w, b, &vmap, g);
    }
  } else {
    const int g = (warp - 8) >> 2;
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
