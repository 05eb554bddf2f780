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
// One CTA per SM, 16 warps: TMA producer, MMA issuer, query loader, four warps
// that copy listed rows, and two groups of four softmax warps that take tiles
// in turn, each with its own reference maxima, sums and O (joined at the
// segment's end), so that one group's exponentials run beside the other's
// products.  K and V tiles share a ring of five 32 KB slots.
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
constexpr int kSlots = 5, kSlot = kPos * kD * 2;
constexpr int kPBytes = kPos * kH * 2, kQBytes = kH * kD * 2;
constexpr int kWideThreads = 512;
constexpr int kTmem = 256, kColS = 0, kColO = 128;  // S and O of softmax group w at + 64 w
constexpr float kFar = 1.0e30f;                     // references lie in [-kFar, kFar]
constexpr float kSlack = 40.f;

struct WideShared {
  uint64_t full[kSlots], empty[kSlots], s_full[2], p_full[2], pv_done[2], q_full[2], q_empty[2], drain;
  alignas(16) uint32_t mask[4][4];  // of the last four tiles: which positions count
  alignas(16) float ref[2][kH], alpha[2][kH];  // read four at a time
  RangeShared r;
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
// A role's place in the ring of slots: K and V of the tiles, in turn.
struct Place {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void advance(int by = 1) {
    slot += by;
    if (slot >= kSlots) slot -= kSlots, phase ^= 1;
  }
};

// ------------------------------------------------------------------ producers
__device__ __forceinline__ void wide_pages(const Args& k, WideShared& sh, WideWalk w, const Buffers& b,
                                           const CUtensorMap* kmap, const CUtensorMap* vmap) {
  const AttnArgs& a = k.a;
  const CacheArgs& c = a.c;
  const int lane = threadIdx.x & 31;
  Waiter wait{sh, c.dev_err};
  Place at_slot;
  int tile = 0;
  while (w.next(a)) {
    const int req = row_request(c, w.row), head = w.unit / k.l.blocks;
    const int32_t* table = req >= 0 ? c.page_table + static_cast<int64_t>(req) * c.max_pages : nullptr;
    const int len = table != nullptr ? a.seq_len[w.row] : 0;
    int lo = -1, hi = -1;
    for (int i = w.i0; i < w.i1; ++i, ++tile) {
      const int j = (i - w.i0) & 31;
      if (j == 0) {  // the next 32 tiles' pages, two per lane
        const int64_t at = static_cast<int64_t>(i + lane) * kPos;
        lo = at < len ? table[at / kPage] : -1;
        hi = at + kPage < len ? table[at / kPage + 1] : -1;
        const bool bad = (at < len && (lo < 0 || lo >= c.num_pages)) || (at + kPage < len && (hi < 0 || hi >= c.num_pages));
        if (bad && i + lane < w.i1) report(c.dev_err, kDevErrPage);
        if (lo >= c.num_pages) lo = -1;
        if (hi >= c.num_pages) hi = -1;
      }
      const int page0 = __shfl_sync(0xffffffffu, lo, j), page1 = __shfl_sync(0xffffffffu, hi, j);
      const int pages = (page0 >= 0) + (page1 >= 0);
      const int mine = lane & 2 ? page1 : page0;  // lane 0..3: page lane / 2, dims 64 (lane % 2) ..
#pragma unroll 1
      for (int v = 0; v < 2; ++v, at_slot.advance()) {  // K, then V
        uint64_t* bar = &sh.full[at_slot.slot];
        if (!wait(&sh.empty[at_slot.slot], at_slot.phase ^ 1)) continue;
        if (v == 0 && lane < 4) {
          const int left = (lane & 2 ? page1 : page0) >= 0 ? len - i * kPos - lane * 32 : 0;
          sh.mask[tile & 3][lane] = left >= 32 ? ~0u : left > 0 ? (1u << left) - 1 : 0;
        }
        __syncwarp();
        if (lane == 0) {
          if (pages > 0)
            mbar_arrive_expect_tx(bar, pages * (kSlot / 2));
          else
            mbar_arrive(bar);
        }
        __syncwarp();
        if (lane < 4 && mine >= 0)
          tma_box(b.slots + at_slot.slot * kSlot + (lane & 1) * (kSlot / 2) + (lane >> 1) * (kSlot / 4), v == 0 ? kmap : vmap,
                  (lane & 1) * 128, (mine * c.num_kv_heads + head) * kPage, smem_u32(bar));
      }
    }
  }
  if (!wait.alive)  // what is in flight lands before the CTA's memory goes
    for (int s = 0; s < kSlots; ++s) {
      const uint32_t last = s < at_slot.slot ? at_slot.phase : at_slot.phase ^ 1;  // parity of the slot's last fill
      if (2 * tile > s) mbar_wait(&sh.full[s], last, nullptr, 1000000ull);
    }
}

// Warp `part` of four copies positions 32 part .. 32 part + 31 of every tile.
// The entries of the second next tile and the page ids of the next one are on
// their way while a tile is copied.
__device__ __forceinline__ void wide_list(const Args& k, WideShared& sh, WideWalk w, const Buffers& b, int part) {
  const AttnArgs& a = k.a;
  const CacheArgs& c = a.c;
  const int lane = threadIdx.x & 31, chunk = lane & 15, odd = lane >> 4;
  const uint8_t *kbase = c.k_pool + chunk * 16, *vbase = c.v_pool + chunk * 16;
  Waiter wait{sh, c.dev_err};
  struct Entry {
    const int32_t* table;  // null: the row has no request
    int head, len, s;
    bool live;
  };
  int i = 0, end = 0;
  Entry seg{nullptr, 0, 0, -1, false};
  auto fetch = [&]() {
    Entry x{nullptr, 0, 0, -1, false};
    if (i >= end) {
      if (!w.next(a)) return x;
      i = w.i0, end = w.i1;
      const int req = row_request(c, w.row);
      seg.table = req >= 0 ? c.page_table + static_cast<int64_t>(req) * c.max_pages : nullptr;
      seg.len = seg.table != nullptr ? a.seq_len[w.row] : 0;
      seg.head = w.unit / k.l.blocks;
    }
    x = seg;
    x.live = true;
    const int at = i * kPos + part * 32 + lane;
    if (at < a.npos) x.s = a.pos[static_cast<int64_t>(w.row) * a.pos_stride + at];
    ++i;
    return x;
  };
  auto look_up = [&](const Entry& x) { return x.s >= 0 && x.s < x.len ? x.table[x.s / kPage] : 0; };
  Entry now = seg, next = seg;
  int page = 0, tile = 0;
  Place at_slot;
  while (true) {
    const int page_next = look_up(next);
    const Entry after = fetch();
    if (!now.live) {  // the pipeline fills, or is empty
      if (!next.live && !after.live) break;
      now = next, next = after, page = page_next;
      continue;
    }
    const bool in = now.s >= 0 && now.s < now.len;
    if (now.table != nullptr && !in && now.s != -1) report(c.dev_err, kDevErrPos);
    const bool ok = in && page >= 0 && page < c.num_pages;
    if (ok != in) report(c.dev_err, kDevErrPage);
    const int row = ok ? (page * c.num_kv_heads + now.head) * kPage + (now.s & (kPage - 1)) : -1;
    const uint32_t m = __ballot_sync(0xffffffffu, ok);
#pragma unroll 1
    for (int v = 0; v < 2; ++v, at_slot.advance()) {  // K, then V
      if (!wait(&sh.empty[at_slot.slot], at_slot.phase ^ 1)) continue;
      uint64_t* bar = &sh.full[at_slot.slot];
      if (v == 0 && lane == 0) sh.mask[tile & 3][part] = m;
      const uint8_t* base = v == 0 ? kbase : vbase;
      const uint32_t dst = b.slots + at_slot.slot * kSlot + (chunk >> 3) * (kSlot / 2) + part * 32 * 128;
#pragma unroll
      for (int p = 0; p < 32; p += 2) {  // positions p and p + 1
        const int at = p + odd, r = __shfl_sync(0xffffffffu, row, at);
        copy16(dst + at * 128 + (((chunk & 7) ^ (at & 7)) << 4), base + static_cast<int64_t>(max(r, 0)) * (kD * 2), r >= 0);
      }
      cp_async_arrive_noinc(bar);
      if (lane == 0) mbar_arrive(bar);  // the mask
    }
    ++tile;
    now = next, next = after, page = page_next;
  }
  cp_async_wait<0>();
}

__device__ __forceinline__ void wide_queries(const Args& k, WideShared& sh, WideWalk w, const Buffers& b) {
  const AttnArgs& a = k.a;
  const int lane = threadIdx.x & 31, chunk = lane & 15, odd = lane >> 4;
  Waiter wait{sh, a.c.dev_err};
  for (int seg = 0; w.next(a); ++seg) {
    const int head = w.unit / k.l.blocks, h0 = (w.unit - head * k.l.blocks) * kH, live = min(kH, k.l.group - h0);
    const uint8_t* src = reinterpret_cast<const uint8_t*>(a.q + w.row * a.q_stride + (static_cast<int64_t>(head) * k.l.group + h0) * kD) + chunk * 16;
    if (!wait(&sh.q_empty[seg & 1], ((seg >> 1) + 1) & 1)) continue;
    const uint32_t dst = b.q + (seg & 1) * kQBytes + (chunk >> 3) * (kQBytes / 2);
#pragma unroll 8
    for (int p = 0; p < kH; p += 2) {
      const int h = p + odd;
      copy16(dst + h * 128 + (((chunk & 7) ^ (h & 7)) << 4), src + (h < live ? h : 0) * (kD * 2), h < live);
    }
    cp_async_arrive_noinc(&sh.q_full[seg & 1]);
  }
  cp_async_wait<0>();
}

// ------------------------------------------------------------------ products
__device__ __forceinline__ void wide_mma(const Args& k, WideShared& sh, const WideWalk& w0, const Buffers& b, uint32_t tmem) {
  const AttnArgs& a = k.a;
  const int lane = threadIdx.x & 31;
  Waiter wait{sh, a.c.dev_err};
  // two walks over the same tiles: the products with K run two tiles ahead
  WideWalk ws = w0, wp = w0;
  int s_i = 0, s_end = 0, seg = -1, p_i = 0, p_end = 0, first = 0;  // first: the first tile of wp's segment
  Place ks, vs{1, 0};
  bool more = true;
  for (int t = 0;; ++t) {
    const int tp = t - 2;
    if (tp >= 0) {
      if (p_i >= p_end) {
        if (!wp.next(a)) break;
        p_i = wp.i0, p_end = wp.i1, first = tp;
      }
      const int g = tp & 1;
      wait(&sh.p_full[g], (tp >> 1) & 1);
      if (wait(&sh.full[vs.slot], vs.phase)) {
        const uint32_t vb = b.slots + vs.slot * kSlot, pb = b.p + g * kPBytes;
        if (a.pos == nullptr && (sh.mask[tp & 3][0] & sh.mask[tp & 3][1] & sh.mask[tp & 3][2] & sh.mask[tp & 3][3]) != ~0u) {
          // values that do not count must not reach a product with 0
#pragma unroll 1
          for (int e = lane; e < kPos * 16; e += 32) {
            const int p = e >> 4, c = e & 15;
            if ((sh.mask[tp & 3][p >> 5] >> (p & 31)) & 1) continue;
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(vb + (c >> 3) * (kSlot / 2) + p * 128 + (c & 7) * 16),
                         "r"(0)
                         : "memory");
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        fence_proxy_async_smem();
        tc_fence_after();
        mma8<128, 512, 128, 512>(tmem + kColO + kH * g, desc128(vb, kSlot / 2), desc128(pb, 16), idesc(true), tp > first + 1);
        mma_commit_elect(&sh.empty[vs.slot]);
        mma_commit_elect(&sh.pv_done[g]);
      }
      vs.advance(2);
      ++p_i;
    }
    if (more) {
      bool start = false;
      if (s_i >= s_end) {
        more = ws.next(a);
        s_i = ws.i0, s_end = ws.i1, ++seg, start = true;
      }
      if (more) {
        if (start) wait(&sh.q_full[seg & 1], (seg >> 1) & 1);
        if (wait(&sh.full[ks.slot], ks.phase)) {
          fence_proxy_async_smem();  // queries and listed rows are written through the generic proxy
          tc_fence_after();
          mma8<2, kSlot / 2 / 16, 2, kQBytes / 2 / 16>(tmem + kColS + kH * (t & 1), desc128(b.slots + ks.slot * kSlot, 16),
                                                       desc128(b.q + (seg & 1) * kQBytes, 16), idesc(false), 0);
          mma_commit_elect(&sh.empty[ks.slot]);
          mma_commit_elect(&sh.s_full[t & 1]);
          if (s_i + 1 == s_end) mma_commit_elect(&sh.q_empty[seg & 1]);
        }
        ks.advance(2);
        ++s_i;
      }
    }
  }
  if (!wait.alive) {  // the products in flight end before the CTA's memory goes
    mma_commit_elect(&sh.drain);
    mbar_wait(&sh.drain, 0, nullptr, 1000000ull);
  }
}

// ------------------------------------------------------------------ softmax
// Halves the heads that a lane keeps and adds the partner's share of them.
template <int kHalf, int kBit>
__device__ __forceinline__ void fold(float (&l)[kH], int lane) {
  const bool up = (lane & kBit) != 0;
#pragma unroll
  for (int j = 0; j < kHalf; ++j) {
    const float give = up ? l[j] : l[j + kHalf];
    l[j] = (up ? l[j + kHalf] : l[j]) + __shfl_xor_sync(0xffffffffu, give, kBit);
  }
}

__device__ __forceinline__ void wide_softmax(const Args& k, WideShared& sh, WideWalk w, const Buffers& b, uint8_t* pmem, uint32_t tmem,
                             int g) {
  const AttnArgs& a = k.a;
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, row = quad * 32 + lane;
  const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
  const float factor = a.scale * kLog2e;
  const Range range = sh.r.range;
  float* scratch = reinterpret_cast<float*>(pmem + g * kPBytes);  // [4][kH], while no product reads the probabilities
  float *ref = sh.ref[g], *alpha = sh.alpha[g];
  Waiter wait{sh, a.c.dev_err};
  int tile = 0;
  uint32_t mine = 0;  // tiles of this group so far
  while (w.next(a)) {
    const int head = w.unit / k.l.blocks, h0 = (w.unit - head * k.l.blocks) * kH, live = min(kH, k.l.group - h0);
    const int end = tile + (w.i1 - w.i0);
    const bool had[2] = {tile + (tile & 1) < end, tile + 1 - (tile & 1) < end};  // whether group 0, 1 has a tile
    float l[kH];
#pragma unroll
    for (int h = 0; h < kH; ++h) l[h] = 0.f;
    bool begun = false, set = false;  // this group has had a tile; its references are set
    for (; tile < end; ++tile) {
      if ((tile & 1) != g) continue;
      float s[kH];
      wait(&sh.s_full[g], mine & 1);
      tc_fence_after();
      {
        uint32_t(&lo)[32] = *reinterpret_cast<uint32_t(*)[32]>(&s[0]);
        uint32_t(&hi)[32] = *reinterpret_cast<uint32_t(*)[32]>(&s[32]);
        tmem_ld32(tmem + lanes + kColS + kH * g, lo);
        tmem_ld32(tmem + lanes + kColS + kH * g + 32, hi);
        tmem_ld_wait();
      }
      const uint4 m = *reinterpret_cast<const uint4*>(sh.mask[tile & 3]);
      const bool valid = ((quad == 0 ? m.x : quad == 1 ? m.y : quad == 2 ? m.z : m.w) >> lane) & 1;
      if (!set && (m.x | m.y | m.z | m.w) != 0) {  // the first position's logits
        const int first = m.x ? __ffs(m.x) - 1 : m.y ? 31 + __ffs(m.y) : m.z ? 63 + __ffs(m.z) : 95 + __ffs(m.w);
        if (row == first) {
#pragma unroll
          for (int h = 0; h < kH; ++h) ref[h] = fmaxf(fminf(s[h] * factor, kFar), -kFar);
        }
        named_sync(1 + g, 128);
        set = true;
      }
      float over = -INFINITY;
#pragma unroll
      for (int h = 0; h < kH; h += 4) {
        const float4 r = *reinterpret_cast<const float4*>(ref + h);
        over = fmaxf(over, fmaxf(fmaf(s[h], factor, -r.x), fmaf(s[h + 1], factor, -r.y)));
        over = fmaxf(over, fmaxf(fmaf(s[h + 2], factor, -r.z), fmaf(s[h + 3], factor, -r.w)));
      }
      const bool raise = group_any(1 + g, valid && over > kSlack);
      if (mine > 0) wait(&sh.pv_done[g], (mine - 1) & 1);  // the probabilities' buffer is free, O is complete
      if (raise) {
#pragma unroll 1
        for (int h = 0; h < kH; h += 4) {  // (rare: short code rather than fast)
          uint32_t x[4];
          tmem_ld4(tmem + lanes + kColS + kH * g + h, x);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float r = warp_max(valid ? __uint_as_float(x[j]) * factor : -INFINITY);
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
#pragma unroll
        for (int h = 0; h < kH; ++h) l[h] *= alpha[h];
        if (begun) {
          tc_fence_after();
#pragma unroll 1
          for (int h = 0; h < kH; h += 8) {
            uint32_t o[8];
            tmem_ld8(tmem + lanes + kColO + kH * g + h, o);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha[h + j]);
            tmem_st8(tmem + lanes + kColO + kH * g + h, o);
          }
          tmem_st_wait();
        }
      }
      uint8_t* prow = pmem + g * kPBytes + row * 128;
#pragma unroll
      for (int h = 0; h < kH; h += 8) {
        uint32_t v[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float2 r = *reinterpret_cast<const float2*>(ref + h + 2 * x);
          float p0 = exp2_approx(fmaf(s[h + 2 * x], factor, -r.x)), p1 = exp2_approx(fmaf(s[h + 2 * x + 1], factor, -r.y));
          if (!valid) p0 = p1 = 0.f;
          l[h + 2 * x] += p0;
          l[h + 2 * x + 1] += p1;
          v[x] = bf16x2(p0, p1);
        }
        *reinterpret_cast<uint4*>(prow + (((h >> 3) ^ (row & 7)) << 4)) = make_uint4(v[0], v[1], v[2], v[3]);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_full[g]);
      ++mine;
      begun = true;
    }
    // ---- the segment's end: sums over the positions, the two groups joined
    if (begun) wait(&sh.pv_done[g], (mine - 1) & 1);
    tc_fence_after();
    fold<32, 16>(l, lane);
    fold<16, 8>(l, lane);
    fold<8, 4>(l, lane);
    fold<4, 2>(l, lane);
    fold<2, 1>(l, lane);
    // lane bits 16, 8, 4, 2, 1 chose heads + 32, 16, 8, 4, 2
    *reinterpret_cast<float2*>(scratch + quad * kH + 2 * lane) = make_float2(l[0], l[1]);
    named_sync(3, 256);
    const bool whole = w.i0 == 0 && w.i1 == w.n;
    const int64_t slot = 2ll * blockIdx.x + (w.i0 == 0 ? 1 : 0);
    if (g == 0 && row < kH) {
      const int h = row;
      float sum[2], m[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float* sc = reinterpret_cast<const float*>(pmem + x * kPBytes);
        sum[x] = had[x] ? (sc[h] + sc[kH + h]) + (sc[2 * kH + h] + sc[3 * kH + h]) : 0.f;
        m[x] = sum[x] != 0.f ? sh.ref[x][h] : -kFar;
      }
      const float top = fmaxf(m[0], m[1]), f0 = exp2_approx(m[0] - top), f1 = exp2_approx(m[1] - top);
      const float total = sum[0] * f0 + sum[1] * f1;
      const float inv = !whole ? 1.f : total == 0.f ? 0.f : 1.f / total;
      sh.alpha[0][h] = f0 * inv;
      sh.alpha[1][h] = f1 * inv;
      if (!whole) {
        float* st = k.stat + (slot * kH + h) * 2;
        st[0] = top;
        st[1] = total;
      } else if (a.lse != nullptr && h < live) {
        a.lse[static_cast<int64_t>(w.row) * a.c.num_q_heads + static_cast<int64_t>(head) * k.l.group + h0 + h] =
            total == 0.f ? -INFINITY : (top + log2f(total)) * 0.6931471805599453f;
      }
    }
    named_sync(3, 256);
    tc_fence_after();
    // group g writes heads 32 g .. 32 g + 31; a thread holds one dim
    {
      uint16_t* out = a.out + w.row * a.out_stride + (static_cast<int64_t>(head) * k.l.group + h0) * kD + row;
      float* sum = k.sum + slot * kH * kD + row;
#pragma unroll 1
      for (int h = 32 * g; h < 32 * g + 32 && h < live; h += 8) {
        uint32_t v[2][8];
        tmem_ld8(tmem + lanes + kColO + h, v[0]);
        tmem_ld8(tmem + lanes + kColO + kH + h, v[1]);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float o = 0.f;
          if (had[0]) o = __uint_as_float(v[0][j]) * sh.alpha[0][h + j];
          if (had[1]) o = fmaf(__uint_as_float(v[1][j]), sh.alpha[1][h + j], o);
          if (h + j >= live) break;
          if (whole)
            out[(h + j) * kD] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
          else
            sum[(h + j) * kD] = o;
        }
      }
    }
    if (g == 0 && row == 0 && !whole && w.i0 == 0) k.part[blockIdx.x] = part_of(w, range);
    tc_fence_before();
    named_sync(3, 256);  // O, the factors and the scratch have been read
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
    const uint32_t fills = a.pos != nullptr ? 4 * 33 : 1;  // listed rows: every lane's copies, and one for the mask
    for (int s = 0; s < kSlots; ++s) mbar_init(&sh.full[s], fills), mbar_init(&sh.empty[s], 1);
    for (int g = 0; g < 2; ++g) {
      mbar_init(&sh.s_full[g], 1);
      mbar_init(&sh.p_full[g], 4);
      mbar_init(&sh.pv_done[g], 1);
      mbar_init(&sh.q_full[g], 32);
      mbar_init(&sh.q_empty[g], 1);
    }
    mbar_init(&sh.drain, 1);
    fence_mbar_init();
    sh.abort = 0;
    k.part[blockIdx.x].last = -1;
  }
  if (tid < 2 * kH) sh.ref[tid / kH][tid % kH] = 0.f;
  tc_fence_before();
  const int units = a.c.num_kv_heads * k.l.blocks;
  find_range<kWideThreads, kPos>(k, sh.r, units);
  tc_fence_after();
  write_empty_rows<kD, kWideThreads>(a);
  const Range r = sh.r.range;
  const uint32_t tmem = sh.tmem;
  if (r.first < r.end) {
    const WideWalk w = walk_of<kPos>(a, r, units);
    if (warp < 8) {
      regs_dec<64>();
      if (warp == 0 && a.pos == nullptr) wide_pages(k, sh, w, b, &kmap, &vmap);
      if (warp == 1) wide_mma(k, sh, w, b, tmem);
      if (warp == 2) wide_queries(k, sh, w, b);
      if (warp >= 4 && a.pos != nullptr) wide_list(k, sh, w, b, warp - 4);
    } else {
      regs_inc<192>();
      wide_softmax(k, sh, w, b, pmem, tmem, (warp - 8) >> 2);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, kTmem);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
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
  attn_wide_kernel<<<k.l.ctas, kWideThreads, kWideSmem, stream>>>(kmap, vmap, k);
  return cudaGetLastError();
}

}  // namespace attn
}  // namespace ci
