// Attention of drafted rows over the paged cache (contract in
// include/ci_draft.h): the main kernel; instances per cache format in
// attn_draft_bf16.cu and attn_draft_fp8.cu, dispatch and the join in
// attn_draft.cu.
//
// Work.  The rows of a request that share a key-value head, n nodes times G
// query heads, are one matrix Q of n G rows (row m is node m / G, head m % G).
// A unit is (request, key-value head, block of 128 or 256 of those rows); it
// reads the request's positions in tiles of 128.  The units' tiles, in order,
// are one list, split evenly by weight over the CTAs, one per SM.  A unit that several
// worked on is joined in a second launch, in order.  (CTAs that take a request's
// neighbouring blocks in step read each tile once from HBM, which is 2 to 3% of
// the time where all requests have as many blocks, and loses a fifth where they
// have not.)
//
// A tile, on the fifth-generation tensor cores:
//   S [128 rows x 128 positions] = Q K^T   both from shared memory, S in tensor memory
//   P = 2^(S c - m), a thread per row      over S, as bf16
//   O [128 rows x D] += P V                A = P from tensor memory, V positions-major
// Two streams of such steps run in turn, so that one's exponentials are beside
// the other's products: the two halves of a block of 256 rows over the same
// tiles, or, where the block has no more than 128 rows, even and odd tiles with
// sums of their own that are put together at the end.  With D = 256 tensor
// memory holds one O: one stream with two score buffers.
//
// The reference m of a row is the largest logit of its first tile, raised where
// a later one passes it by 8 (in base 2): probabilities are at most 2^8, and O
// is rescaled only then.  P is rounded to bf16, an error of its size of 2^-9 for
// the positions that carry a row, and divided by the sum of the unrounded ones (by
// that of the rounded ones, in bf16: error against 64 bits, two norms, 0.00198 for
// 0.00205, of which 0.00166 is the result's own rounding, and 1 to 4% more time; FP8:
// a probability is rounded with its value's scale in it, and the sum is without).
//
// What bounds it.  Few rows in bf16: the HBM (32 requests of 16k, 4 nodes, 64
// heads over 8 of 128: 2.15 GB in 330 to 335 us, 6.4 to 6.5 TB/s of a
// copy's 6.7).  Many rows: a
// step's chain of softmax and products (64 trees of 64 nodes over 4k-16k: 1.10 ms in
// short runs, 1.21 where the clock settles under load, 1130 TFLOP/s; a chunk of 2048
// behind 16k: 0.85 and 0.90 ms, 1300 TFLOP/s).  A pair of steps takes 3700 cycles, of
// which the tensor cores work half: a softmax of 128 columns is 2000 (500 the largest,
// 1130 the exponentials, the rest waits and stores), P V and the next Q K^T behind it
// 1500.  Neither shared memory (40%) nor exponentials (27%) nor issue slots (39%) are
// full.  FP8: V's widening and the issuing warp's waits, 1950 cycles a tile where the HBM's rate is 1460 (64 chains
// of 4 over 16k-64k: 1.16 to 1.23 ms, 4.5 TB/s); with many rows the scales, 96 reads
// of 16 bytes from shared memory per row and tile that bf16 has not (a chunk of 1024
// behind 8192: 1.6 times bf16's instructions, shared memory at 71%, where bf16 has
// 40, and 1.35 times its time).  Short calls: the start, 8000 cycles until the first
// tile arrives, cold code, and the join (4 requests of 16 nodes over 1k-4k: 27 us; one
// row over 16 positions: 10 us).  Chains of many rows: the search for the CTA's range
// walks a request's blocks one after another, 28 us of 0.86 ms with the 64 blocks of
// 2048 tokens of 8 heads, 0.82 of 2.1 ms with the 2048 of 8192 tokens of 64 heads.
//
// Where FP8's loops come to lie counts, too: 64 to 256 instructions that never run,
// put in front of V's widening, took up to 7% more time, 512 none.
//
// Masks.  Only tiles that reach past the positions that all rows of a block see
// have any: there a row's 128 bits come from its mask words, shifted to the
// tile, and a warp leaves out 32 positions that none of its rows sees and takes 32
// that all see as any other (64 trees of 64 nodes: 5% less time).  Values that some
// rows do not see must not meet their zeros as NaN or infinities: in those tiles
// everything that is not finite becomes 0 in shared memory before the product, and at
// the end the rows that do see it add it.
//
// FP8 pages.  Keys are multiplied as they are: the query, each row scaled by a
// power of two, is the sum of an e4m3 and an e5m2 number, exactly where an element is
// no smaller than 2^-13 of the row's largest, else within 2^-21 of that.  Values widen
// to bf16 (x 2^-120) on the way from a ring of raw tiles to the operands.  A
// position's scales join its logit and its probability.
#pragma once
#include <cuda_fp16.h>

#include "attn.cuh"
#include "draft_internal.h"

namespace ci {
namespace draft {

using attn::bf16x2;
using attn::exp2_approx;

constexpr int kKeys = 128;               // positions of a tile
constexpr float kFar = 3.0e38f;          // references lie in [-kFar, kFar]
constexpr float kSlack = 8.f;            // a logit over its reference
constexpr int kTmem = 512, kColO = 256;  // score buffers at columns 0 and 128, then O
// FP8: probabilities carry 2^52, so that with values of 2^-120 O is no smaller than the values by more than 2^-68.  A
// probability is at most 2^8 and a value 480 x 2^60, so O stays below 2^9 per position and 2^40 for any number of them.
// Only divided by the sum does it take all of 2^120: what several CTAs' parts are joined from carries 2^60 of it, too
// little for an overflow and enough that nothing of O gets lost.
constexpr float kLift = 52.f, kTwo120 = 1329227995784915872903807060280344576.f, kTwo60 = 1152921504606846976.f;

struct Part {  // the unit that goes on past the end of a CTA's range; last < 0: none
  int32_t req, head, block, last;
};
struct Layout {
  int32_t ctas;
  int32_t group;       // query heads per key-value head
  int32_t block_rows;  // rows of a block: 128 or 256
};
struct Args {
  DraftArgs a;
  Layout l;
  Part* part;   // [ctas]
  float* stat;  // [2 ctas][block_rows][2]: reference (base 2) and sum
  float* sum;   // [2 ctas][D / 4][block_rows][4]: neighbouring rows are neighbouring lanes; FP8: x 2^-60
};

template <int D_, bool kFp8_>
struct Config {
  static constexpr int D = D_;
  static constexpr bool kFp8 = kFp8_, kTwo = D < 256;     // kTwo: two streams
  static constexpr int kTiles = kTwo ? 2 : 1;             // of 128 rows in a block
  static constexpr int kBlockRows = 128 * kTiles;
  static constexpr int kParts = D == 256 ? 2 : 1;         // slots of a tile's K or V
  static constexpr int kSlotKeys = kKeys / kParts;
  static constexpr int kOperand = kSlotKeys * D * 2;      // bytes of a slot
  static constexpr int kQ = 128 * D * 2;                  // of a tile of Q
  static constexpr int kRow = kFp8 ? D : 2 * D;           // of a cached position
  static constexpr int kBox = kRow < 128 ? kRow : 128;
  static constexpr int kBoxes = kRow / kBox;
  static constexpr int kRaw = kSlotKeys * kRow;           // of a loaded slot
  // K is read from the loaded slots, and so is V in bf16; FP8: V from operand slots
  static constexpr int kLoads = kFp8 ? (D == 64 ? 10 : 5) : (D == 64 ? 8 : 4);
  static constexpr int kOps = kFp8 ? (D == 64 ? 4 : 2) : 0;
  static constexpr int kPrepWarps = kTwo ? 4 : 8;  // (one stream: those of the other one, too)
  static constexpr int kStreamThreads = kTwo ? 256 : 128;  // of the softmax
  static constexpr int kPageBytes = kFp8 ? 64 * D + 256 : 128 * D;
};

constexpr int kMaxSlots = 10;
struct Shared {
  // Loaded slots, with barriers of their own for keys and values: a role that waited for some phases of a barrier only,
  // or that is not waited for by those that free the slot, would take one phase for another.
  uint64_t full[kMaxSlots], v_full[kMaxSlots], empty[kMaxSlots];
  uint64_t ready[kMaxSlots], op_empty[kMaxSlots];  // values looked over (bf16), operands (FP8)
  // pv_done: two streams: of a segment's last step (a score buffer that is full says that what was issued before is done,
  // the stream's last product among it); one stream: of every step
  uint64_t s_full[2], p_full[2], pv_done[2], q_full, q_empty, drain;
  float ref[2][128], sums[2][128];  // the streams' references and sums, when they are put together
  float fold[2][8][96];              // and eight dims of the copies of rows
  uint32_t pages[16];                // of the last sixteen tiles: which of the two pages are there
  int32_t odd[4];                    // of the last four segments: the one where a value was not finite
  int64_t warp_sum[2][16];
  int32_t tile_at[2];                // the CTA's range of the list
  int32_t end, total, ctas;          // where its share of the weight ends, the weight of all, how many share it
  int32_t weighted, skip;            // whether a tile weighs more than 1; the first one behind the range begins `skip` behind `end`
  int32_t req, head, block, tile;    // where it starts
  int32_t row0, n, len, limit;       // and that request
  uint32_t tmem;
  int32_t abort;
};
struct Scales {  // FP8
  alignas(16) float k[8][kKeys], v[8][kKeys];  // of the last eight tiles
  float factor[2][2][128];                     // of the last two segments: what the rows of Q were divided by
};

template <class C>
constexpr int smem_bytes() {
  return C::kTiles * C::kQ + C::kLoads * C::kRaw + C::kOps * C::kOperand +
         (C::kFp8 ? static_cast<int>(sizeof(Scales)) : 0) + static_cast<int>(sizeof(Shared));
}

// ------------------------------------------------------------------ the list
struct Request {
  int first, n, len;  // rows first .. first + n - 1
  int limit;          // positions that there are: len + n, or 0
  int blocks;
};
enum { kGood = 0, kBadLen = 1, kBadReq = 2 };
__device__ __forceinline__ int blocks_of(const Args& k, int n) {  // (the host has checked that rows * G fit)
  return static_cast<int>((static_cast<int64_t>(n) * k.l.group + k.l.block_rows - 1) / k.l.block_rows);
}
__device__ __forceinline__ Request request_of(const Args& k, int r, int& bad) {
  const DraftArgs& a = k.a;
  Request q;
  q.first = a.c.req_start[r];
  const int end = a.c.req_start[r + 1];
  q.len = a.length[r];
  bad = kGood;
  if (q.first < 0 || end < q.first || end > a.rows) {
    bad = kBadReq;
    q.n = 0;
  } else {
    q.n = end - q.first;
  }
  q.limit = q.len + q.n;
  if (q.n > 0 && (q.len < 0 || q.n > a.max_rows || q.n > a.max_len - q.len)) {
    bad = kBadLen;
    q.len = q.limit = 0;
  }
  q.blocks = blocks_of(k, q.n);
  return q;
}
// The last node of block b.
__device__ __forceinline__ int last_node(const Args& k, const Request& q, int b) {
  return static_cast<int>(min(static_cast<int64_t>(q.n), (static_cast<int64_t>(b + 1) * k.l.block_rows - 1) / k.l.group + 1)) - 1;
}
// Tiles of block b.
__device__ __forceinline__ int block_tiles(const Args& k, const Request& q, int b) {
  const int keys = q.limit == 0 ? 1 : k.a.mask != nullptr ? q.limit : q.len + last_node(k, q, b) + 1;
  return (keys - 1) / kKeys + 1;
}
// Tiles of one key-value head.
__device__ __forceinline__ int head_tiles(const Args& k, const Request& q) {
  if (k.a.mask != nullptr || q.limit == 0) return q.n == 0 ? 0 : q.blocks * block_tiles(k, q, 0);
  int n = 0;
#pragma unroll 1
  for (int b = 0; b < q.blocks; ++b) n += block_tiles(k, q, b);
  return n;
}

// Whether block b, a request's last, has no more than 128 rows (of 256).
__device__ __forceinline__ bool is_light(const Args& k, const Request& q, int b) {
  return static_cast<int64_t>(q.n) * k.l.group - static_cast<int64_t>(b) * k.l.block_rows <= 128;
}
// Tiles of such a block of one key-value head.
__device__ __forceinline__ int light_tiles(const Args& k, const Request& q) {
  return q.n > 0 && is_light(k, q, q.blocks - 1) ? block_tiles(k, q, q.blocks - 1) : 0;
}
// What a tile weighs in the split of the list: where some blocks are light, 2 in
// those and 3 in others, else 1.  (bf16, without, with, and with weights of 1 and 2:
// 60 requests of one row behind 8192 beside two chunks of 1024 behind 4096, 64 / 8
// heads of 128, 641, 534 and 536 us; 17 trees of 1 to 20 nodes, 64 heads over one,
// 272, 264 and 305; 9 chains of 1 to 1024 behind 16k, 1460, 1505 and 1479.)
constexpr int kLight = 2, kHeavy = 3;
__device__ __forceinline__ int weight_of(const Args& k, const Request& q, int b, bool weighted) {
  return !weighted ? 1 : is_light(k, q, b) ? kLight : kHeavy;
}

// A CTA's way through its range: tiles [i0, i1) of a unit at a time.
struct Walk {
  int left;                         // tiles of the range behind the segment
  int r, head, block, tile, tiles;  // where the next segment starts
  Request q;
  int i0, i1;
  __device__ __forceinline__ bool next(const Args& k) {
    if (left == 0) return false;
    if (tile == tiles) {
      tile = 0;
      if (++block == q.blocks) {
        block = 0;
        if (++head == k.a.c.num_kv_heads) {
          head = 0;
          int bad;
#pragma unroll 1
          do q = request_of(k, ++r, bad);
          while (q.n == 0);
        }
      }
      tiles = block_tiles(k, q, block);
    }
    i0 = tile;
    i1 = min(tiles, i0 + left);
    left -= i1 - i0;
    tile = i1;
    return true;
  }
};

__device__ __forceinline__ int share_start(int cta, int per, int rest) { return cta * per + min(cta, rest); }
// The CTA that has tile x of the list.
__device__ __forceinline__ int cta_of(int x, int total, int ctas) {
  const int per = total / ctas, rest = total - per * ctas, longer = rest * (per + 1);
  return x < longer ? x / (per + 1) : rest + (x - longer) / per;
}

// The range of this CTA: every thread adds up a run of requests, a scan
// over the threads gives the total, and the thread whose run holds the range's
// first tile walks to it.  Split by weight, a range has the tiles that begin in its
// share of the whole weight, and the one that holds the share's end counts to it.
template <int kThreads, bool kTwo>
__device__ __forceinline__ void find_range(const Args& k, Shared& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, heads = k.a.c.num_kv_heads;
  const int per_thread = (k.a.c.num_req + kThreads - 1) / kThreads;
  const int r0 = min(tid * per_thread, k.a.c.num_req), r1 = min(r0 + per_thread, k.a.c.num_req);
  int64_t mine = 0, light = 0;  // tiles
  int bits = 0;
#pragma unroll 1
  for (int r = r0; r < r1; ++r) {
    int bad;
    const Request q = request_of(k, r, bad);
    bits |= bad;
    mine += static_cast<int64_t>(head_tiles(k, q)) * heads;
    if (kTwo) light += static_cast<int64_t>(light_tiles(k, q)) * heads;
  }
  if (bits != 0 && blockIdx.x == 0)
    report(k.a.c.dev_err, (bits & kBadLen ? kDevErrLen : 0) | (bits & kBadReq ? kDevErrReq : 0));
  int64_t incl = mine, light_incl = light;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o), y = kTwo ? __shfl_up_sync(0xffffffffu, light_incl, o) : 0;
    if (lane >= o) incl += v, light_incl += y;
  }
  if (lane == 31) sh.warp_sum[0][warp] = incl, sh.warp_sum[1][warp] = light_incl;
  __syncthreads();
  int64_t before = incl - mine, sum = 0, light_before = light_incl - light, light_sum = 0;
#pragma unroll 1
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sh.warp_sum[0][w], light_before += sh.warp_sum[1][w];
    sum += sh.warp_sum[0][w], light_sum += sh.warp_sum[1][w];
  }
  if (sum > INT32_MAX) {  // starts that descend: requests with the same rows
    if (blockIdx.x == 0 && tid == 0) report(k.a.c.dev_err, kDevErrReq);
    sum = 0;
  }
  // by weight where tiles differ and every CTA's share weighs a tile, so that one begins in each
  const int tiles = static_cast<int>(sum), tiles_before = static_cast<int>(before);
  const int64_t weights = kHeavy * sum - (kHeavy - kLight) * light_sum;
  const bool weighted =
      kTwo && 0 < light_sum && light_sum < sum && weights >= static_cast<int64_t>(kHeavy) * k.l.ctas && weights <= INT32_MAX;
  if (weighted) {
    sum = weights;
    mine = kHeavy * mine - (kHeavy - kLight) * light;
    before = kHeavy * before - (kHeavy - kLight) * light_before;
  }
  const int total = static_cast<int>(sum);
  const int ctas = min(k.l.ctas, total), per = ctas > 0 ? total / ctas : 0, rest = total - per * ctas;
  const int cta = static_cast<int>(blockIdx.x);
  const int first = share_start(min(cta, ctas), per, rest), end = share_start(min(cta + 1, ctas), per, rest);
  if (tid == 0) {
    sh.end = end, sh.total = total, sh.ctas = ctas, sh.weighted = weighted;
    if (!weighted || end == total) sh.tile_at[1] = weighted ? tiles : end, sh.skip = 0;
  }
#pragma unroll 1
  for (int e = 0; e <= weighted; ++e) {
    const int pos = e ? end : first;
    if (first == end || pos < before || pos >= before + mine) continue;
    int at = static_cast<int>(pos - before), r = r0, bad, index = tiles_before;
    Request q;
    int of_head, n;  // a head's tiles and their weight
#pragma unroll 1
    for (;; ++r) {
      q = request_of(k, r, bad);
      n = of_head = head_tiles(k, q);
      if (weighted) n = kHeavy * of_head - (kHeavy - kLight) * light_tiles(k, q);
      if (at < static_cast<int64_t>(n) * heads) break;
      at -= n * heads, index += of_head * heads;
    }
    const int head = at / n;
    at -= head * n, index += head * of_head;
    int b = 0;
    if (k.a.mask != nullptr || q.limit == 0) {  // (the light block is the last)
      const int t = block_tiles(k, q, 0), weight = t * weight_of(k, q, 0, weighted);
      b = at / weight;
      at -= b * weight;
      index += b * t;
    } else {
#pragma unroll 1
      for (;; ++b) {
        const int t = block_tiles(k, q, b), weight = t * weight_of(k, q, b, weighted);
        if (at < weight) break;
        at -= weight;
        index += t;
      }
    }
    const int weight = weight_of(k, q, b, weighted), tile = (at + weight - 1) / weight;
    sh.tile_at[e] = weighted ? index + tile : first;
    if (e) sh.skip = tile * weight - at;
    if (e) continue;
    sh.req = r, sh.head = head, sh.block = b, sh.tile = tile;
    sh.row0 = q.first, sh.n = q.n, sh.len = q.len, sh.limit = q.limit;
  }
  if (first == end && tid == 0) sh.tile_at[0] = sh.tile_at[1] = 0;
  __syncthreads();
}
__device__ __forceinline__ Walk walk_of(const Args& k, const Shared& sh) {
  Walk w{};
  w.left = sh.tile_at[1] - sh.tile_at[0];
  if (w.left == 0) return w;
  w.r = sh.req, w.head = sh.head, w.block = sh.block, w.tile = sh.tile;
  w.q = Request{sh.row0, sh.n, sh.len, sh.limit, blocks_of(k, sh.n)};
  w.tiles = block_tiles(k, w.q, w.block);
  return w;
}

struct Segment {
  int rows;         // of its block
  int row0;         // its first row of the request's matrix
  bool two;         // two tiles of rows, over the same positions
  int span;         // else rows are there 128 / span times, each copy for its own span positions of a tile
  int tiles, steps;
  int lag;          // by how many tiles V's loads are behind K's
  int seen;         // positions that every row of the block sees
};
template <class C>
__device__ __forceinline__ Segment segment_of(const Args& k, const Walk& w) {
  Segment s;
  s.row0 = w.block * C::kBlockRows;
  s.rows = min(C::kBlockRows, w.q.n * k.l.group - s.row0);
  s.two = C::kTwo && s.rows > 128;
  s.lag = C::kFp8 || s.two ? 0 : 1;
  // Copies: FP8 alone, where a tile's softmax and scales are what counts (32 requests of 16k, 4 nodes of 8 heads: without
  // 311 us, with 258); in bf16 they are slower (338 and 476 us), as a copy's zeros may not meet values that are not
  // finite, so that every tile's would have to be looked over.  (A copy's span holds at least one of the rows, so that
  // every warp of a stream is busy where there are copies: they meet at barriers.)
  s.span = !C::kFp8 || s.rows > 64 ? 128 : s.rows > 32 ? 64 : 32;
  s.tiles = w.i1 - w.i0;
  s.steps = s.two ? 2 * s.tiles : s.tiles;
  s.seen = w.q.limit == 0 ? 0 : w.q.len + (k.a.mask != nullptr ? 0 : s.row0 / k.l.group + 1);
  return s;
}

// ------------------------------------------------------------------ small things
// One role's waits: false once anything has given up; the role then goes on
// through its loop without touching memory.  (By one lane and a shuffle instead of
// all: 1.4 times the time of the whole.)
struct Waiter {
  Shared& sh;
  int32_t* dev_err;
  bool alive = true;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) {
    alive = alive && attn::wait_warp(bar, parity, &sh.abort, dev_err);
    return alive;
  }
};
template <int N>
struct Place {  // a ring's slot
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void advance() {
    if (++slot == N) slot = 0, phase ^= 1;
  }
};

// 128-byte swizzled operands: K-major (rows of 64 elements of the reduced
// dimension), or MN-major (rows of 64 elements of the other dimension, one per
// element of the reduced one; the next 64 elements `next` bytes further).
__device__ __forceinline__ uint64_t desc128(uint32_t addr, uint32_t next) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | static_cast<uint64_t>((next >> 4) & 0x3FFFu) << 16 |
         static_cast<uint64_t>(1024u >> 4) << 32 | static_cast<uint64_t>(1u) << 46 | static_cast<uint64_t>(2u) << 61;
}
// Rows of 64 bytes (64 e4m3 dims), 64-byte swizzle; K-major.
__device__ __forceinline__ uint64_t desc_rows(uint32_t addr, int row_bytes) {
  return row_bytes == 64 ? sdesc_k64_sw64(addr) : desc128(addr, 16);
}
// Instruction descriptor: M = 128, fp32 sums; bf16 or e4m3 operands, B MN-major or not.  kE5m2: A is e5m2.
constexpr uint32_t kE5m2 = 1u << 7;
__host__ __device__ constexpr uint32_t idesc(int n, bool bf16, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         ((128u >> 4) << 24);
}
// N products issued by one lane (one election for all of them: the warp shares its
// scheduler with the softmax's); step j reads the operands at a + S::a(j) and b +
// S::b(j), in 16 bytes, or columns for an A in tensor memory.  kFp8: the second half's
// instruction descriptor is id2.
template <class S, int N, bool kFp8>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t id2, uint32_t accumulate) {
  static_assert(N == 8 || N == 4, "");
  if constexpr (kFp8 && N == 8)
    asm volatile(
      "{\n\t.reg .pred p, e, o;\n\t.reg .b64 x;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 o, %4, %4;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
      "add.s64 x, %1, %5;\n\tadd.s64 y, %2, %12;\n\t@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %6;\n\tadd.s64 y, %2, %13;\n\t@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %7;\n\tadd.s64 y, %2, %14;\n\t@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %8;\n\tadd.s64 y, %2, %15;\n\t@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %19, o;\n\t"
      "add.s64 x, %1, %9;\n\tadd.s64 y, %2, %16;\n\t@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %19, o;\n\t"
      "add.s64 x, %1, %10;\n\tadd.s64 y, %2, %17;\n\t@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %19, o;\n\t"
      "add.s64 x, %1, %11;\n\tadd.s64 y, %2, %18;\n\t@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %19, o;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(accumulate), "n"(S::a(1)), "n"(S::a(2)), "n"(S::a(3)), "n"(S::a(4)), "n"(S::a(5)), "n"(S::a(6)), "n"(S::a(7)), "n"(S::b(1)), "n"(S::b(2)), "n"(S::b(3)), "n"(S::b(4)), "n"(S::b(5)), "n"(S::b(6)), "n"(S::b(7)), "r"(id2)
      : "memory");
  else if constexpr (kFp8)
    asm volatile(
      "{\n\t.reg .pred p, e, o;\n\t.reg .b64 x;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 o, %4, %4;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t"
      "add.s64 x, %1, %5;\n\tadd.s64 y, %2, %8;\n\t@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %6;\n\tadd.s64 y, %2, %9;\n\t@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %11, o;\n\t"
      "add.s64 x, %1, %7;\n\tadd.s64 y, %2, %10;\n\t@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], x, y, %11, o;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(accumulate), "n"(S::a(1)), "n"(S::a(2)), "n"(S::a(3)), "n"(S::b(1)), "n"(S::b(2)), "n"(S::b(3)), "r"(id2)
      : "memory");
  else if constexpr (N == 8)
    asm volatile(
      "{\n\t.reg .pred p, e, o;\n\t.reg .b64 x;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 o, %4, %4;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "add.s64 x, %1, %5;\n\tadd.s64 y, %2, %12;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %6;\n\tadd.s64 y, %2, %13;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %7;\n\tadd.s64 y, %2, %14;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %8;\n\tadd.s64 y, %2, %15;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %9;\n\tadd.s64 y, %2, %16;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %10;\n\tadd.s64 y, %2, %17;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %11;\n\tadd.s64 y, %2, %18;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(accumulate), "n"(S::a(1)), "n"(S::a(2)), "n"(S::a(3)), "n"(S::a(4)), "n"(S::a(5)), "n"(S::a(6)), "n"(S::a(7)), "n"(S::b(1)), "n"(S::b(2)), "n"(S::b(3)), "n"(S::b(4)), "n"(S::b(5)), "n"(S::b(6)), "n"(S::b(7))
      : "memory");
  else
    asm volatile(
      "{\n\t.reg .pred p, e, o;\n\t.reg .b64 x;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 o, %4, %4;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "add.s64 x, %1, %5;\n\tadd.s64 y, %2, %8;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %6;\n\tadd.s64 y, %2, %9;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t"
      "add.s64 x, %1, %7;\n\tadd.s64 y, %2, %10;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, o;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(accumulate), "n"(S::a(1)), "n"(S::a(2)), "n"(S::a(3)), "n"(S::b(1)), "n"(S::b(2)), "n"(S::b(3))
      : "memory");
}
template <class S, int N>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t accumulate) {
  static_assert(N == 8 || N == 4, "");
  if constexpr (N == 8)
    asm volatile(
      "{\n\t.reg .pred p, e, o;\n\t.reg .b32 x;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 o, %4, %4;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "add.s32 x, %1, %5;\n\tadd.s64 y, %2, %12;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, o;\n\t"
      "add.s32 x, %1, %6;\n\tadd.s64 y, %2, %13;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, o;\n\t"
      "add.s32 x, %1, %7;\n\tadd.s64 y, %2, %14;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, o;\n\t"
      "add.s32 x, %1, %8;\n\tadd.s64 y, %2, %15;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, o;\n\t"
      "add.s32 x, %1, %9;\n\tadd.s64 y, %2, %16;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, o;\n\t"
      "add.s32 x, %1, %10;\n\tadd.s64 y, %2, %17;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, o;\n\t"
      "add.s32 x, %1, %11;\n\tadd.s64 y, %2, %18;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, o;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(accumulate), "n"(S::a(1)), "n"(S::a(2)), "n"(S::a(3)), "n"(S::a(4)), "n"(S::a(5)), "n"(S::a(6)), "n"(S::a(7)), "n"(S::b(1)), "n"(S::b(2)), "n"(S::b(3)), "n"(S::b(4)), "n"(S::b(5)), "n"(S::b(6)), "n"(S::b(7))
      : "memory");
  else
    asm volatile(
      "{\n\t.reg .pred p, e, o;\n\t.reg .b32 x;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.eq.b32 o, %4, %4;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "add.s32 x, %1, %5;\n\tadd.s64 y, %2, %8;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, o;\n\t"
      "add.s32 x, %1, %6;\n\tadd.s64 y, %2, %9;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, o;\n\t"
      "add.s32 x, %1, %7;\n\tadd.s64 y, %2, %10;\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], y, %3, o;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(accumulate), "n"(S::a(1)), "n"(S::a(2)), "n"(S::a(3)), "n"(S::b(1)), "n"(S::b(2)), "n"(S::b(3))
      : "memory");
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
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\t"
      "mov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\t"
      "mov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
// Chunk `chunk` of 16 bytes of row p of an operand with `rows` rows.
__device__ __forceinline__ uint32_t operand_offset(int rows, int p, int chunk) {
  return (chunk >> 3) * (rows * 128) + p * 128 + (((chunk & 7) ^ (p & 7)) << 4);
}

struct Buffers {
  uint32_t q, load, op;  // shared-memory addresses
  Scales* sc;            // FP8
};
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_all;" ::: "memory"); }


// ------------------------------------------------------------------ loads
// K and V of the tiles, in the order in which they are taken: with two tiles of
// rows K and V of a tile, else V a tile behind K; FP8: K and V of a tile, as V is
// prepared while the tile's scores are computed.
template <class C>
__device__ __forceinline__ void load_tiles(const Args& k, Shared& sh, Walk w, const Buffers& b, const CUtensorMap* kmap,
                                           const CUtensorMap* vmap) {
  const CacheArgs& c = k.a.c;
  const int lane = threadIdx.x & 31;
  constexpr int kPages = C::kSlotKeys / kPage, kPerPage = C::kPageBytes / C::kRow;
  Waiter wait{sh, c.dev_err};
  Place<C::kLoads> at;
  uint32_t base = 0;  // tiles so far
#pragma unroll 1
  while (w.next(k)) {
    const Segment s = segment_of<C>(k, w);
    const int32_t* table = c.page_table + static_cast<int64_t>(w.r) * c.max_pages;
    const int lag = s.lag;
    // the pages of 32 tiles, two per lane; those of the 32 before, for V
    int lo = -1, hi = -1, lo0 = -1, hi0 = -1;
#pragma unroll 1
    for (int j = 0; j < s.tiles + lag; ++j) {
      if ((j & 31) == 0) {
        const int64_t pos = static_cast<int64_t>(w.i0 + j + lane) * kKeys;
        const bool in = j + lane < s.tiles, in0 = in && pos < w.q.limit, in1 = in && pos + kPage < w.q.limit;
        lo0 = lo, hi0 = hi;
        lo = in0 ? table[pos / kPage] : -1;
        hi = in1 ? table[pos / kPage + 1] : -1;
        const bool out0 = lo < 0 || lo >= c.num_pages, out1 = hi < 0 || hi >= c.num_pages;
        if ((in0 && out0) || (in1 && out1)) report(c.dev_err, kDevErrPage);
        if (out0) lo = -1;
        if (out1) hi = -1;
      }
#pragma unroll 1
      for (int v = 0; v < 2; ++v) {
        const int t = v ? j - lag : j;
        if (t < 0 || t >= s.tiles) continue;
        const bool old = (t >> 5) != (j >> 5);
        const int page0 = __shfl_sync(0xffffffffu, old ? lo0 : lo, t & 31), page1 = __shfl_sync(0xffffffffu, old ? hi0 : hi, t & 31);
        if (v == 0 && lane == 0) sh.pages[(base + t) & 15] = (page0 >= 0 ? 1u : 0u) | (page1 >= 0 ? 2u : 0u);
#pragma unroll 1
        for (int x = 0; x < C::kParts; ++x, at.advance()) {
          if (!wait(&sh.empty[at.slot], at.phase ^ 1)) continue;
          uint64_t* full = v ? &sh.v_full[at.slot] : &sh.full[at.slot];
          // a lane per box: page lane / boxes of the slot, box lane % boxes; a lane per page's scales
          const int which = lane / C::kBoxes, box = lane % C::kBoxes;
          const int page = (kPages == 1 ? x : which) ? page1 : page0;
          const int there = kPages == 1 ? page >= 0 : (page0 >= 0) + (page1 >= 0);
          __syncwarp();
          if (lane == 0) {
            if (there > 0)
              mbar_arrive_expect_tx(full, there * (kPage * C::kRow + (C::kFp8 && v == 0 ? 512 : 0)));
            else
              mbar_arrive(full);
          }
          __syncwarp();
          const uint32_t dst = b.load + at.slot * C::kRaw;
          if (which < kPages && page >= 0) {
            const int row = page * c.num_kv_heads + w.head;
            attn::tma_box(dst + box * (C::kSlotKeys * C::kBox) + which * (kPage * C::kBox), v ? vmap : kmap, box * 128,
                          row * kPerPage, smem_u32(full));
            if (C::kFp8 && v == 0 && box == 0) {
              // (the tile's eighth predecessor has been read: its slots have been filled again since)
              const int64_t from = static_cast<int64_t>(row) * C::kPageBytes + kPage * C::D;
              const int first = x * C::kSlotKeys + which * kPage;
              attn::bulk_load(smem_u32(&b.sc->k[(base + t) & 7][first]), c.k_pool + from, 256, smem_u32(full));
              attn::bulk_load(smem_u32(&b.sc->v[(base + t) & 7][first]), c.v_pool + from, 256, smem_u32(full));
            }
          }
        }
      }
    }
    base += s.tiles;
  }
}

// ------------------------------------------------------------------ preparation
__device__ __forceinline__ uint32_t f16x2_to_e4m3(uint32_t x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_to_e5m2(uint32_t x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ __half2 e4m3x2_to_f16(uint32_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(x)));
  return *reinterpret_cast<const __half2*>(&r);
}
// The rows of Q: row m of the request's matrix is node m / G.  FP8: each row
// scaled by a power of two, 1 / factor, and split into an e4m3 and an e5m2 number
// per element, one tile of each.  A bf16 element has eight bits: e4m3 has the leading
// four, and what is left is at most eight of its last place, three bits and a sign,
// which is what e5m2 has, with a smallest step of 2^-16 where e4m3's is 2^-9.  With the
// largest in [2^7, 2^8) that is exact from 2^-13 of the largest on, else within 2^-21
// of it (all bf16 values tried; with e4m3 for both, from 2^-9 on, and 2^-17).  Larger
// elements' leading bits in e5m2 would allow a largest in [2^11, 2^12), exact from 2^-17
// on and within 2^-25: seven operations per pair more, and 3 to 12% of a call's time
// (32 requests of 16k, 64 nodes 1085 -> 1135 us, a prompt of 9001 1.95 -> 2.19 ms).
template <class C>
__device__ __forceinline__ void prep_queries(const Args& k, const Walk& w, const Segment& s, const Buffers& b,
                                             float (*factor)[128], int tid) {
  constexpr int kChunks = C::D / 8, kRowsAtOnce = 32 * C::kPrepWarps / kChunks;
  const int chunk = tid % kChunks;
  const int rows = s.two ? 256 : 128, group = k.l.group;
  // y / group = y inv / 2^16 rounded down, for y < 384 and group <= 128
  const uint32_t inv = (65535u + group) / group;
  const int node0 = s.row0 / group, rest0 = s.row0 - node0 * group;
  const uint16_t* first = k.a.q + (w.q.first + node0) * k.a.q_stride + static_cast<int64_t>(w.head) * group * C::D + chunk * 8;
  auto row_of = [&](int m, bool& there) {
    const int of = s.two ? m : m & (s.span - 1);
    there = of < s.rows;
    const uint32_t y = there ? rest0 + of : 0, node = (y * inv) >> 16;
    return first + node * k.a.q_stride + (y - node * group) * C::D;
  };
  if (!C::kFp8) {
#pragma unroll 4
    for (int m = tid / kChunks; m < rows; m += kRowsAtOnce) {
      bool there;
      const uint16_t* src = row_of(m, there);
      attn::copy16(b.q + (m >> 7) * C::kQ + operand_offset(128, m & 127, chunk), reinterpret_cast<const uint8_t*>(src), there);
    }
    wait_copies();
  }
  // four rows at a time, so that their steps fill each other's waits, and the next four on their way
  constexpr int kAtOnce = 4, kStep = kAtOnce * kRowsAtOnce;
  static_assert(128 % kStep == 0, "");
  uint4 next[kAtOnce];
  auto load = [&](int m0) {
#pragma unroll
    for (int x = 0; x < kAtOnce; ++x) {
      bool there;
      const uint16_t* src = row_of(m0 + x * kRowsAtOnce, there);
      next[x] = make_uint4(0, 0, 0, 0);
      if (there) next[x] = *reinterpret_cast<const uint4*>(src);
    }
  };
  if (C::kFp8) load(tid / kChunks);
#pragma unroll 1
  for (int m0 = tid / kChunks; C::kFp8 && m0 < rows; m0 += kStep) {
    uint32_t u[kAtOnce][4], top[kAtOnce];  // top: the largest magnitudes' bits, of even and of odd dims
#pragma unroll
    for (int x = 0; x < kAtOnce; ++x) {
      u[x][0] = next[x].x, u[x][1] = next[x].y, u[x][2] = next[x].z, u[x][3] = next[x].w;
      top[x] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) top[x] = __vmaxu2(top[x], u[x][i] & 0x7FFF7FFFu);
      top[x] = max(top[x] & 0xFFFFu, top[x] >> 16);
    }
    if (m0 + kStep < rows) load(m0 + kStep);
#pragma unroll
    for (int o = 1; o < kChunks; o <<= 1) {
#pragma unroll
      for (int x = 0; x < kAtOnce; ++x) top[x] = max(top[x], __shfl_xor_sync(0xffffffffu, top[x], o));
    }
    uint32_t hi[kAtOnce][2] = {}, lo[kAtOnce][2] = {};
    float down[kAtOnce];
#pragma unroll
    for (int x = 0; x < kAtOnce; ++x) {
      const int e = static_cast<int>(top[x] >> 7);  // biased; 255: not finite
      const int up = e == 255 || top[x] == 0 ? 0 : min(7 - (e - 127), 126);
      const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);  // 2^up, -120 <= up <= 126
      down[x] = __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // (f16 has the scaled elements exactly, down to 2^-32 of the largest, and the differences)
        const uint32_t y = attn::f16x2(bf16_lo(u[x][i]) * f, bf16_hi(u[x][i]) * f);
        uint32_t h = f16x2_to_e4m3(y);
        const __half2 less = __hsub2(*reinterpret_cast<const __half2*>(&y), e4m3x2_to_f16(h));
        const uint32_t l = f16x2_to_e5m2(*reinterpret_cast<const uint32_t*>(&less));
        if (e == 255) h = 0x7F7F;  // a row that is not finite: NaN
        hi[x][i >> 1] |= h << (16 * (i & 1)), lo[x][i >> 1] |= l << (16 * (i & 1));
      }
    }
#pragma unroll
    for (int x = 0; x < kAtOnce; ++x) {
      const int m = m0 + x * kRowsAtOnce, row = m & 127, c16 = chunk >> 1;
      const uint32_t at = b.q + (m >> 7) * C::kQ + (chunk & 1) * 8 +
                          (C::D == 64 ? row * 64 + ((c16 ^ ((row >> 1) & 3)) << 4)
                                      : (c16 >> 3) * (128 * 128) + row * 128 + (((c16 & 7) ^ (row & 7)) << 4));
      sts64(at, hi[x][0], hi[x][1]);
      sts64(at + 128 * C::D, lo[x][0], lo[x][1]);
      if (chunk == 0) factor[m >> 7][row] = down[x];
    }
  }
  fence_proxy_async_smem();
}

// Values of a slot that not every row of the block sees (positions from s.seen
// on): zeros where there are none or where they are not finite, which is noted.
template <class C>
__device__ __forceinline__ void prep_values(Shared& sh, const Walk& w, const Segment& s, uint32_t slot, int64_t pos0,
                                            uint32_t pages, int x, int warp, int lane, int segment) {
  constexpr int kChunks = C::D / 8, kPer = C::kSlotKeys / C::kPrepWarps;
  bool odd = false;
#pragma unroll 4
  for (int e = lane; e < kPer * kChunks; e += 32) {
    const int p = warp * kPer + e / kChunks;
    const int64_t pos = pos0 + p;
    const bool page = (pages >> (C::kParts == 1 ? p / kPage : x)) & 1;
    if (page && pos < s.seen) continue;
    const uint32_t at = slot + operand_offset(C::kSlotKeys, p, e % kChunks);
    if (!page || pos >= w.q.limit) {
      sts128(at, make_uint4(0, 0, 0, 0));
      continue;
    }
    const uint4 v = lds128(at);
    uint32_t u[4] = {v.x, v.y, v.z, v.w}, any = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) any |= ((u[i] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;  // an exponent of ones carries
    if (any == 0) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((u[i] & 0x7F80u) == 0x7F80u) u[i] &= 0xFFFF0000u;
      if ((u[i] & 0x7F800000u) == 0x7F800000u) u[i] &= 0xFFFFu;
    }
    sts128(at, make_uint4(u[0], u[1], u[2], u[3]));
    odd = true;
  }
  if (odd) sh.odd[segment & 3] = segment;
  fence_proxy_async_smem();
}

// Bytes 0 .. 3 of r (e4m3) as two bf16 pairs of the value x 2^-120, in order.
__device__ __forceinline__ uint2 widen_bf16(uint32_t r) {
  const uint32_t a = __byte_perm(r, 0, 0x1404), b = __byte_perm(r, 0, 0x3424);  // bytes to the upper half of each 16 bits
  return make_uint2((a & 0x80008000u) | ((a >> 4) & 0x07F007F0u), (b & 0x80008000u) | ((b >> 4) & 0x07F007F0u));
}
// A raw slot of V into an operand, bf16 x 2^-120.  A warp takes 8
// positions of 64 dims at a time, 16 codes per lane: eight neighbouring lanes have
// positions q and q ^ 5, which the swizzles of both layouts put on different banks.
template <class C>
__device__ __forceinline__ void widen(uint32_t raw, uint32_t op, int warp, int lane) {
  constexpr int kBlocks = C::D / 64, kCount = C::kSlotKeys / 8 * kBlocks / C::kPrepWarps;
  static_assert(C::kPrepWarps % kBlocks == 0, "");
  const int u = lane & 3, p = (lane >> 3) ^ ((lane & 4) ? 5 : 0), block = warp % kBlocks;
  raw += C::kBox == 128 ? (block >> 1) * (C::kSlotKeys * 128) + p * 128 + (((4 * (block & 1) + u) ^ p) << 4)
                        : p * 64 + ((u ^ ((p >> 1) & 3)) << 4);
  const uint32_t row = op + block * (C::kSlotKeys * 128) + p * 128;
  const uint32_t op0 = row + (((2 * u) ^ p) << 4), op1 = row + (((2 * u + 1) ^ p) << 4);
  const int first = warp / kBlocks;
#pragma unroll
  for (int j = 0; j < kCount; j += 4) {
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = lds128(raw + (first + (j + i) * (C::kPrepWarps / kBlocks)) * (8 * C::kBox));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      uint2 r[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) r[x] = widen_bf16(c[x]);
      const uint32_t at = (first + (j + i) * (C::kPrepWarps / kBlocks)) * 1024;
      sts128(op0 + at, make_uint4(r[0].x, r[0].y, r[1].x, r[1].y));
      sts128(op1 + at, make_uint4(r[2].x, r[2].y, r[3].x, r[3].y));
    }
  }
}

template <class C>
__device__ __forceinline__ void prepare(const Args& k, Shared& sh, Walk w, const Buffers& b) {
  const int tid = threadIdx.x - (384 - 32 * C::kPrepWarps), lane = tid & 31, warp = tid >> 5;
  Waiter wait{sh, k.a.c.dev_err};
  Place<C::kLoads> at;
  Place<C::kFp8 ? C::kOps : 1> op;
  uint32_t segments = 0, base = 0, v_turn = 0;  // v_turn: parities of the slots' values
#pragma unroll 1
  while (w.next(k)) {
    const Segment s = segment_of<C>(k, w);
    if (wait(&sh.q_empty, (segments & 1) ^ 1)) {
      prep_queries<C>(k, w, s, b, C::kFp8 ? b.sc->factor[(segments + 1) & 1] : nullptr, tid);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full);
    }
    ++segments;
    const int lag = s.lag;
#pragma unroll 1
    for (int j = 0; j < s.tiles + lag; ++j) {
#pragma unroll 1
      for (int v = 0; v < 2; ++v) {
        const int t = v ? j - lag : j;
        if (t < 0 || t >= s.tiles) continue;
#pragma unroll 1
        for (int x = 0; x < C::kParts; ++x, at.advance()) {
          const uint32_t raw = b.load + at.slot * C::kRaw;
          const int64_t pos0 = static_cast<int64_t>(w.i0 + t) * kKeys + x * C::kSlotKeys;
          if (v == 0) continue;
          const uint32_t turn = (v_turn >> at.slot) & 1;
          v_turn ^= 1u << at.slot;
          if (!C::kFp8) {
            if (!wait(&sh.v_full[at.slot], turn)) continue;
            const uint32_t pages = sh.pages[(base + t) & 15];
            if (pages != 3 || pos0 + C::kSlotKeys > s.seen)
              prep_values<C>(sh, w, s, raw, pos0, pages, x, warp, lane, static_cast<int>(segments));
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.ready[at.slot]);
            continue;
          }
          if (wait(&sh.v_full[at.slot], turn) && wait(&sh.op_empty[op.slot], op.phase ^ 1)) {
            widen<C>(raw, b.op + op.slot * C::kOperand, warp, lane);
            fence_proxy_async_smem();
          }
          named_sync(4, 32 * C::kPrepWarps);
          if (tid == 0 && wait.alive) mbar_arrive(&sh.ready[op.slot]), mbar_arrive(&sh.empty[at.slot]);
          op.advance();
        }
      }
    }
    base += s.tiles;
  }
}

// ------------------------------------------------------------------ products
// Steps of Q K^T: 32 bytes of the rows at a time, blocks of 128 bytes of all rows;
// FP8: with the query's e4m3 parts, then with its e5m2 parts.
template <class C>
struct ScoreSteps {
  static constexpr int kCount = C::D / 16;  // FP8: half as many, twice
  __host__ __device__ static constexpr int e(int j) { return C::kFp8 ? j % (kCount / 2) : j; }
  __host__ __device__ static constexpr int a(int j) {
    return (C::kFp8 && j >= kCount / 2 ? 128 * C::D / 16 : 0) + (e(j) >> 2) * (128 * 128 / 16) + (e(j) & 3) * 2;
  }
  __host__ __device__ static constexpr int b(int j) { return (e(j) >> 2) * (C::kSlotKeys * 128 / 16) + (e(j) & 3) * 2; }
};
// Steps of P V: 16 positions at a time.
struct ValueSteps {
  __host__ __device__ static constexpr int a(int j) { return 8 * j; }
  __host__ __device__ static constexpr int b(int j) { return 128 * j; }
};
// Step i is Q K^T into score buffer i % 2, the softmax, then P V.  A wait costs some
// 200 cycles even where it is for something done, so a step's keys and values are
// waited for before its probabilities: P V and, as the buffer is free then, the
// scores of the step after next follow at once.
template <class C>
__device__ __forceinline__ void products(const Args& k, Shared& sh, Walk w, const Buffers& b, uint32_t tmem) {
  constexpr uint32_t kIdQ = idesc(C::kSlotKeys, !C::kFp8, false), kIdP = idesc(C::D, true, true);
  Waiter wait{sh, k.a.c.dev_err};
  Place<C::kLoads> at;              // of the next item
  Place<C::kFp8 ? C::kOps : 1> op;  // FP8: of the next values
  int k_slot = 0, v_slot = 0;       // of the present tiles' first parts
  uint32_t k_turn = 0, v_turn = 0;  // parities of the slots' keys and values
  uint32_t p_turn = 0, segments = 0;
#pragma unroll 1
  while (w.next(k)) {
    const Segment s = segment_of<C>(k, w);
    auto keys = [&](int i) {  // waits for step i's keys
      if (i >= s.steps || (s.two && (i & 1))) return;
      k_slot = at.slot;
#pragma unroll 1
      for (int x = 0; x < C::kParts; ++x, at.advance()) {
        wait(&sh.full[at.slot], (k_turn >> at.slot) & 1);
        k_turn ^= 1u << at.slot;
      }
      if (C::kFp8)  // (the values' slots are the preparation's)
        for (int x = 0; x < C::kParts; ++x) at.advance();
    };
    auto scores = [&](int i) {
      if (i >= s.steps || !wait.alive) return;
      const bool last = !s.two || (i & 1);  // of the tile's
      const uint32_t q = b.q + (s.two ? (i & 1) * C::kQ : 0);
      tc_fence_after();
#pragma unroll 1
      for (int x = 0, slot = k_slot; x < C::kParts; ++x) {
        constexpr int kBytes = C::kRow < 128 ? C::kRow : 128;  // of an operand's rows; 32 of them per product
        const uint64_t da = desc_rows(q, kBytes), db = desc_rows(b.load + slot * C::kRaw, kBytes);
        const uint32_t d = tmem + 128 * (i & 1) + x * C::kSlotKeys;
        using S = ScoreSteps<C>;
        constexpr int kSteps = S::kCount > 8 ? 8 : S::kCount;
        constexpr uint32_t kId2 = C::kFp8 ? kIdQ | kE5m2 : kIdQ;
        mma_ss<S, kSteps, C::kFp8>(d, da, db, kIdQ, S::kCount > 8 ? kIdQ : kId2, 0);
        if (S::kCount > 8) mma_ss<S, kSteps, C::kFp8>(d, da + S::a(8), db + S::b(8), kId2, kId2, 1);  // (a step's offsets repeat)
        if (x == C::kParts - 1) mma_commit_elect(&sh.s_full[i & 1]);
        if (last) mma_commit_elect(&sh.empty[slot]);
        if (++slot == C::kLoads) slot = 0;
      }
      if (i == s.steps - 1) mma_commit_elect(&sh.q_empty);
    };
    keys(0);
    wait(&sh.q_full, segments & 1);
    ++segments;
    scores(0);
    keys(1);
    scores(1);
#pragma unroll 1
    for (int i = 0; i < s.steps; ++i) {
      const int o = C::kTwo ? i & 1 : 0;
      const bool fresh = !s.two || (i & 1) == 0, last = !s.two || (i & 1) == 1;
      if (fresh) {
        v_slot = C::kFp8 ? op.slot : at.slot;
#pragma unroll 1
        for (int x = 0; x < C::kParts; ++x) {
          if (C::kFp8) {
            wait(&sh.ready[op.slot], op.phase);
            op.advance();
          } else {
            const uint32_t turn = (v_turn >> at.slot) & 1;
            if (wait(&sh.v_full[at.slot], turn)) wait(&sh.ready[at.slot], turn);
            v_turn ^= 1u << at.slot;
            at.advance();
          }
        }
      }
      if (C::kTwo) keys(i + 2);
      wait(&sh.p_full[i & 1], (p_turn >> (i & 1)) & 1);
      p_turn ^= 1u << (i & 1);
      if (wait.alive) tc_fence_after();
#pragma unroll 1
      for (int x = 0, slot = v_slot; wait.alive && x < C::kParts; ++x) {
        const uint64_t db = desc128(C::kFp8 ? b.op + slot * C::kOperand : b.load + slot * C::kRaw, C::kSlotKeys * 128);
        mma_ts<ValueSteps, C::kSlotKeys / 16>(tmem + kColO + o * C::D, tmem + 128 * (i & 1) + x * (C::kSlotKeys / 2), db, kIdP,
                                              x > 0 || i >= (C::kTwo ? 2 : 1));
        if (last) mma_commit_elect(C::kFp8 ? &sh.op_empty[slot] : &sh.empty[slot]);
        if (++slot == (C::kFp8 ? C::kOps : C::kLoads)) slot = 0;
      }
      if (wait.alive && (!C::kTwo || i + 2 >= s.steps)) mma_commit_elect(&sh.pv_done[o]);
      if (!C::kTwo) keys(i + 2);  // (its slots may be those that this product frees)
      scores(i + 2);
    }
  }
  if (!wait.alive) {  // the products in flight end before the CTA's memory goes
    mma_commit_elect(&sh.drain);
    mbar_wait(&sh.drain, 0, nullptr, 1000000ull);
  }
}

// ------------------------------------------------------------------ softmax
// Which of the 32 positions from pos on a row sees.
struct RowMask {
  const uint32_t* words;  // null: a chain
  int node, n, len, limit, count;
};
__device__ __forceinline__ uint32_t mask_word(const RowMask& m, int i) {
  if (i >= m.count || 32 * i >= m.n) return 0;
  const uint32_t v = m.words[i];
  return 32 * i + 32 > m.n ? v & ((1u << (m.n - 32 * i)) - 1) : v;
}
__device__ __forceinline__ uint32_t seen_of(const RowMask& m, int64_t pos) {
  if (m.limit == 0) return 0;
  const int64_t rel = pos - m.len;
  if (m.words == nullptr) {
    const int64_t c = m.node + 1 - rel;
    return c >= 32 ? ~0u : c <= 0 ? 0 : (1u << c) - 1;
  }
  if (rel <= -32) return ~0u;
  if (rel < 0) return (mask_word(m, 0) << -rel) | ((1u << -rel) - 1);
  if (rel >= m.n) return 0;
  const int i = static_cast<int>(rel) >> 5;
  return __funnelshift_r(mask_word(m, i), mask_word(m, i + 1), static_cast<int>(rel) & 31);
}

// What a row sees that is not finite, of the nodes and of 16 dims from d0 on: added
// as it is.
template <class C>
__device__ __noinline__ void add_odd(const Args& k, const Walk& w, const RowMask& m, int d0, float (&o)[16]) {
  const CacheArgs& c = k.a.c;
  const int64_t end = min(static_cast<int64_t>(w.i1) * kKeys, static_cast<int64_t>(w.q.limit));
#pragma unroll 1
  for (int64_t pos = max(static_cast<int64_t>(w.q.len), static_cast<int64_t>(w.i0) * kKeys); pos < end; ++pos) {
    if ((seen_of(m, pos) & 1) == 0) continue;
    const int page = c.page_table[static_cast<int64_t>(w.r) * c.max_pages + pos / kPage];
    if (page < 0 || page >= c.num_pages) continue;
    const uint4* v = reinterpret_cast<const uint4*>(
        c.v_pool + (static_cast<int64_t>(page) * c.num_kv_heads + w.head) * C::kPageBytes + ((pos & (kPage - 1)) * C::D + d0) * 2);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 x = v[i];
      const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float &lo = o[8 * i + 2 * j], &hi = o[8 * i + 2 * j + 1];
        if ((u[j] & 0x7F80u) == 0x7F80u) lo += bf16_lo(u[j]);
        if ((u[j] & 0x7F800000u) == 0x7F800000u) hi += bf16_hi(u[j]);
      }
    }
  }
}

// A row's 128 scores, 32 columns at a time, the next ones on their way.
template <class F>
__device__ __forceinline__ void over_scores(uint32_t at, F f) {
  uint32_t x[2][32];
  tmem_ld32(at, x[0]);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    tmem_ld_wait();
    if (c < 3) tmem_ld32(at + 32 * (c + 1), x[(c + 1) & 1]);
    f(c, x[c & 1]);
  }
}
// n times 32 of them, one after another: the code is a quarter, and a call's first
// tiles and its masked ones run it cold.  bits(c) are those that the row sees: where
// no row of the warp sees any, none(c); where some see some or `careful` asks for
// it, part(c, j, x, bits) for 16 from j on.
template <class B, class F, class P, class N>
__device__ __forceinline__ void over_some_scores(uint32_t at, int n, bool masked, bool careful, B bits, F all, P part, N none) {
#pragma unroll 1
  for (int c = 0; c < n; ++c) {
    const uint32_t seen = masked ? bits(c) : ~0u;
    if (masked && !__any_sync(0xffffffffu, seen != 0)) {
      none(c);
    } else if (!careful && (!masked || __all_sync(0xffffffffu, seen == ~0u))) {
      uint32_t x[32];
      tmem_ld32(at + 32 * c, x);
      tmem_ld_wait();
      all(c, x);
    } else {
#pragma unroll 1
      for (int j = 0; j < 32; j += 16) {
        uint32_t x[16];
        tmem_ld16(at + 32 * c + j, x);
        tmem_ld_wait();
        part(c, j, x, seen >> j);
      }
    }
  }
}
// Two scores, times their keys' scales.
template <class C>
__device__ __forceinline__ float2 scores_of(uint32_t s0, uint32_t s1, float k0, float k1) {
  const float2 x = make_float2(__uint_as_float(s0), __uint_as_float(s1));
  return C::kFp8 ? mul2(x, make_float2(k0, k1)) : x;
}
__device__ __forceinline__ bool bit(uint32_t bits, int j) { return (bits >> j) & 1; }

// The largest of N scores and `top` (kDown: the smallest).
template <class C, bool kCareful, bool kDown, int N>
__device__ __forceinline__ float top_of(const uint32_t (&x)[N], uint32_t bits, const float* ks, float top) {
  float other = top;
#pragma unroll
  for (int j = 0; j < N; j += 4) {
    float4 f = make_float4(1.f, 1.f, 1.f, 1.f);
    if (C::kFp8) f = *reinterpret_cast<const float4*>(ks + j);
    float2 y = scores_of<C>(x[j], x[j + 1], f.x, f.y), z = scores_of<C>(x[j + 2], x[j + 3], f.z, f.w);
    if (kCareful) {
      const float none = kDown ? INFINITY : -INFINITY;
      y.x = bit(bits, j) ? y.x : none, y.y = bit(bits, j + 1) ? y.y : none;
      z.x = bit(bits, j + 2) ? z.x : none, z.y = bit(bits, j + 3) ? z.y : none;
    }
    top = kDown ? fminf(top, fminf(y.x, y.y)) : fmaxf(top, fmaxf(y.x, y.y));
    other = kDown ? fminf(other, fminf(z.x, z.y)) : fmaxf(other, fmaxf(z.x, z.y));
  }
  return kDown ? fminf(top, other) : fmaxf(top, other);
}

// N probabilities, over their scores, and their sum.  kCareful: masked, or
// logits that are rounded by themselves, as the reference is (a product and a
// difference in one step are off by half of the reference's last place, which
// only counts where logits pass 2^22).
template <class C, bool kCareful, int N>
__device__ __forceinline__ void probabilities_of(const uint32_t (&x)[N], uint32_t to, uint32_t bits, const float* ks,
                                                 const float* vs, float factor, float ref, float2& sum, float2& other) {
  const float up = C::kFp8 ? kLift - ref : -ref;
  const float2 less = make_float2(up, up), by = make_float2(factor, factor);
  uint32_t p[N / 2];
#pragma unroll
  for (int j = 0; j < N; j += 4) {
    float4 f = make_float4(1.f, 1.f, 1.f, 1.f), h = f;
    if (C::kFp8) {
      f = *reinterpret_cast<const float4*>(ks + j);
      h = *reinterpret_cast<const float4*>(vs + j);
    }
    float2 y = scores_of<C>(x[j], x[j + 1], f.x, f.y), z = scores_of<C>(x[j + 2], x[j + 3], f.z, f.w);
    if (kCareful) {
      y = add2(make_float2(__fmul_rn(y.x, factor), __fmul_rn(y.y, factor)), make_float2(-ref, -ref));
      z = add2(make_float2(__fmul_rn(z.x, factor), __fmul_rn(z.y, factor)), make_float2(-ref, -ref));
      if (C::kFp8) y = add2(y, make_float2(kLift, kLift)), z = add2(z, make_float2(kLift, kLift));
    } else {
      y = fma2(y, by, less), z = fma2(z, by, less);
    }
    y = make_float2(exp2_approx(y.x), exp2_approx(y.y));
    z = make_float2(exp2_approx(z.x), exp2_approx(z.y));
    if (kCareful) {
      y.x = bit(bits, j) ? y.x : 0.f, y.y = bit(bits, j + 1) ? y.y : 0.f;
      z.x = bit(bits, j + 2) ? z.x : 0.f, z.y = bit(bits, j + 3) ? z.y : 0.f;
    }
    sum = add2(sum, y), other = add2(other, z);
    if (C::kFp8) {
      y = mul2(y, make_float2(h.x, h.y)), z = mul2(z, make_float2(h.z, h.w));
      if (kCareful) {  // (a scale that is not finite must not meet a 0)
        y.x = bit(bits, j) ? y.x : 0.f, y.y = bit(bits, j + 1) ? y.y : 0.f;
        z.x = bit(bits, j + 2) ? z.x : 0.f, z.y = bit(bits, j + 3) ? z.y : 0.f;
      }
    }
    p[j / 2] = bf16x2(y.x, y.y), p[j / 2 + 1] = bf16x2(z.x, z.y);
  }
  if constexpr (N == 32)
    tmem_st16(to, p);
  else
    tmem_st8(to, p);
}

// A step of the softmax for a warp that has the 32 n columns of the buffer `at` from
// 32 c0 on: reference, rescaling of O, probabilities; zeros in the other columns.
struct Row {
  float factor, ref;
  float2 sum;
  bool far;  // whether a reference of the warp's rows is too large for a product and a difference in one step
};
template <class C>
__device__ __forceinline__ void softmax_step(Shared& sh, Waiter& wait, const RowMask& mask, int64_t pos0, uint32_t pages,
                                             int seen, const float* ks, const float* vs, uint32_t at, uint32_t own, int c0,
                                             int n, bool first, uint32_t done, Row& r) {
  const bool masked = pages != 3 || pos0 + kKeys > seen, plain = !masked, down = r.factor < 0.f;
  const uint32_t scores = at + 32 * c0, to = at + 16 * c0;
  if (C::kFp8) ks += 32 * c0, vs += 32 * c0;
  auto bits_of = [&](int c) { return (pages >> ((c0 + c) >> 1)) & 1 ? seen_of(mask, pos0 + 32 * (c0 + c)) : 0; };
  // the largest logit (base 2): of the scores, as rounding keeps their order
  float top = down ? INFINITY : -INFINITY;
  if (plain && n == 4 && !down)
    over_scores(scores, [&](int c, const uint32_t (&x)[32]) { top = top_of<C, false, false>(x, 0, ks + 32 * c, top); });
  else
    over_some_scores(
        scores, n, masked, down, bits_of,
        [&](int c, const uint32_t (&x)[32]) { top = top_of<C, false, false>(x, 0, ks + 32 * c, top); },
        [&](int c, int j, const uint32_t (&x)[16], uint32_t bits) {
          top = down ? top_of<C, true, true>(x, bits, ks + 32 * c + j, top) : top_of<C, true, false>(x, bits, ks + 32 * c + j, top);
        },
        [](int) {});
  top = r.factor == 0.f && fabsf(top) == INFINITY ? -INFINITY : top * r.factor;
  if (C::kFp8) top = ceilf(top);  // so that kLift less a reference is exact
  if (first) {
    r.ref = fmaxf(fminf(top, kFar), -kFar);
    r.far = __any_sync(0xffffffffu, fabsf(r.ref) >= 4194304.f);
  } else if (__any_sync(0xffffffffu, top > r.ref + kSlack)) {
    const float up = fmaxf(r.ref, fminf(top, kFar)), by = exp2_approx(r.ref - up);
    r.ref = up;
    r.far = __any_sync(0xffffffffu, fabsf(up) >= 4194304.f);
    r.sum = mul2(r.sum, make_float2(by, by));
    if (C::kTwo || wait(&sh.pv_done[0], (done - 1) & 1)) {
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < C::D; c += 32) {
        uint32_t o[32];
        tmem_ld32(own + c, o);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * by);
        tmem_st32(own + c, o);
      }
      tmem_st_wait();
    }
  }
  float2 other = make_float2(0.f, 0.f);
  auto zeros = [&](int c) {
    uint32_t none[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) none[j] = 0;
    tmem_st16(at + 16 * ((c0 + c) & 3), none);
  };
  if (plain && !r.far && n == 4)
    over_scores(scores, [&](int c, const uint32_t (&x)[32]) {
      probabilities_of<C, false>(x, to + 16 * c, 0, ks + 32 * c, vs + 32 * c, r.factor, r.ref, r.sum, other);
    });
  else
    over_some_scores(
        scores, n, masked, r.far, bits_of,
        [&](int c, const uint32_t (&x)[32]) {
          probabilities_of<C, false>(x, to + 16 * c, 0, ks + 32 * c, vs + 32 * c, r.factor, r.ref, r.sum, other);
        },
        [&](int c, int j, const uint32_t (&x)[16], uint32_t bits) {
          probabilities_of<C, true>(x, to + 16 * c + j / 2, bits, ks + 32 * c + j, vs + 32 * c + j, r.factor, r.ref, r.sum, other);
        },
        zeros);
  r.sum = add2(r.sum, other);
#pragma unroll 1
  for (int c = n; c < 4; ++c) zeros(c);
  tmem_st_wait();
}

template <class C>
__device__ __forceinline__ void softmax(const Args& k, Shared& sh, Walk w, const Scales* sc, uint32_t tmem, int g) {
  const DraftArgs& a = k.a;
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, row = quad * 32 + lane;
  const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16), own = lanes + kColO + (C::kTwo ? g * C::D : 0);
  constexpr int kStride = C::kTwo ? 2 : 1;
  Waiter wait{sh, a.c.dev_err};
  uint32_t turn = 0, done = 0, base = 0, segment = 0;  // done: products with this stream's probabilities
#pragma unroll 1
  while (w.next(k)) {
    const Segment s = segment_of<C>(k, w);
    ++segment;
    // this thread's row of the block, and its copy's first 32 columns of a tile
    const int m0 = s.two ? g * 128 + row : row & (s.span - 1), c0 = s.two ? 0 : (row & ~(s.span - 1)) >> 5;
    const bool live = m0 < s.rows && c0 == 0;
    const int x0 = s.row0 + (m0 < s.rows ? m0 : 0), node = x0 / k.l.group;
    const RowMask mask{a.mask != nullptr ? a.mask + static_cast<int64_t>(w.q.first + node) * a.mask_words : nullptr,
                       node, w.q.n, w.q.len, w.q.limit, a.mask_words};
    const int seen = C::kTwo && s.two && g == 1 && a.mask == nullptr && w.q.limit > 0
                         ? w.q.len + (s.row0 + 128) / k.l.group + 1 : s.seen;
    Row r{a.scale * attn::kLog2e, -kFar, make_float2(0.f, 0.f), false};
    const int span = s.two ? 128 : s.span;
    const bool busy = (m0 & ~31) < s.rows;  // whether the warp has rows
#pragma unroll 1
    for (int i = C::kTwo ? g : 0; i < s.steps; i += kStride) {
      const int buf = i & 1, t = s.two ? i >> 1 : i;
      const bool first = i < kStride;
      wait(&sh.s_full[buf], (turn >> buf) & 1);
      turn ^= 1u << buf;
      tc_fence_after();
      if (C::kFp8 && first) r.factor = a.scale * attn::kLog2e * sc->factor[segment & 1][s.two ? g : 0][row];
      const uint32_t at = lanes + 128 * buf;
      const uint32_t pages = sh.pages[(base + t) & 15];
      const int64_t pos0 = static_cast<int64_t>(w.i0 + t) * kKeys;
      const float *ks = C::kFp8 ? sc->k[(base + t) & 7] : nullptr, *vs = C::kFp8 ? sc->v[(base + t) & 7] : nullptr;
      if (busy)
        softmax_step<C>(sh, wait, mask, pos0, pages, seen, ks, vs, at, own, c0, span >> 5, first, done, r);
      // every phase is waited for in turn, as a wait tells only the present one from the one before
      if (!C::kTwo && !first) wait(&sh.pv_done[0], (done - 1) & 1);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_full[buf]);
      if (!C::kTwo || i + kStride >= s.steps) ++done;
    }
    base += s.tiles;
    // ---- the segment's end
    const int mine = s.two ? s.tiles : C::kTwo ? (s.steps + 1 - g) / 2 : s.steps;  // steps of this stream
    if (mine > 0) wait(&sh.pv_done[C::kTwo ? g : 0], (done - 1) & 1);
    tc_fence_after();
    float ref = r.ref, total = r.sum.x + r.sum.y;
    const bool both = C::kTwo && !s.two;  // both streams have the same rows
    const bool joined = both || span < 128;
    float fa = 1.f, fb = 0.f;
    int d0 = 0, d1 = C::D;
    if (joined) {
      sh.ref[g][row] = ref, sh.sums[g][row] = total;
      tc_fence_before();
      named_sync(1, C::kStreamThreads);
      tc_fence_after();
      const int streams = both && s.steps > 1 ? 2 : 1;  // (of one step the second stream has nothing)
      float top = -kFar;
      for (int x = 0; x < streams; ++x)
        for (int y = row & (span - 1); y < 128; y += span) top = fmaxf(top, sh.ref[x][y]);
      total = 0.f;
      for (int x = 0; x < streams; ++x)
        for (int y = row & (span - 1); y < 128; y += span) total += sh.sums[x][y] * exp2_approx(sh.ref[x][y] - top);
      fa = exp2_approx(sh.ref[0][row] - top), fb = streams > 1 ? exp2_approx(sh.ref[1][row] - top) : 0.f;
      ref = top;
      if (both) d0 = g * (C::D / 2), d1 = d0 + C::D / 2;  // a half of the dims each
    }
    const bool whole = w.i0 == 0 && w.i1 == w.tiles;
    const float by = (whole && total != 0.f ? 1.f / total : 1.f) * (!C::kFp8 ? 1.f : whole ? kTwo120 : kTwo60);  // O is 0 where the sum is
    const int64_t slot = 2ll * blockIdx.x + (w.i0 == 0 ? 1 : 0), qh = static_cast<int64_t>(w.head) * k.l.group + x0 - node * k.l.group;
    const int64_t t = w.q.first + node;
    const bool odd = !C::kFp8 && sh.odd[segment & 3] == static_cast<int>(segment);
    const uint32_t from = both ? lanes + kColO : own;
#pragma unroll 1
    for (int c = busy ? d0 : d1; c < d1; c += 16) {
      uint32_t o[16], y[16];
      tmem_ld16(from + c, o);
      if (both && s.steps > 1) tmem_ld16(from + C::D + c, y);
      tmem_ld_wait();
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        v[j] = __uint_as_float(o[j]);
        if (joined) v[j] *= fa;
        if (both && s.steps > 1) v[j] += __uint_as_float(y[j]) * fb;
      }
      if (span < 128) {  // the copies' sums, eight dims at a time (all of the stream's warps are busy)
#pragma unroll
        for (int j0 = 0; j0 < 16; j0 += 8) {
          if (c0 != 0) {
#pragma unroll
            for (int j = 0; j < 8; ++j) sh.fold[g][j][row - span] = v[j0 + j];
          }
          named_sync(2 + g, 128);
          if (c0 == 0) {
#pragma unroll 1
            for (int x = row; x < 128 - span; x += span) {
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j0 + j] += sh.fold[g][j][x];
            }
          }
          named_sync(2 + g, 128);
        }
      }
      if (live) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = total == 0.f ? 0.f : v[j] * by;
        if (odd) {
          float z[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) z[j] = v[j];
          add_odd<C>(k, w, mask, c, z);
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = z[j];
        }
        if (whole) {
          uint16_t* dst = a.out + t * a.out_stride + qh * C::D + c;
#pragma unroll
          for (int j = 0; j < 16; j += 8)
            *reinterpret_cast<uint4*>(dst + j) = make_uint4(bf16x2(v[j], v[j + 1]), bf16x2(v[j + 2], v[j + 3]),
                                                            bf16x2(v[j + 4], v[j + 5]), bf16x2(v[j + 6], v[j + 7]));
        } else {
          float4* dst = reinterpret_cast<float4*>(k.sum) + (slot * (C::D / 4) + c / 4) * C::kBlockRows + m0;
#pragma unroll
          for (int j = 0; j < 16; j += 4) dst[j / 4 * C::kBlockRows] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
        }
      }
      __syncwarp();
    }
    tc_fence_before();
    if (live && d0 == 0) {
      if (!whole)
        *reinterpret_cast<float2*>(k.stat + (slot * C::kBlockRows + m0) * 2) = make_float2(ref, total);
      else if (a.lse != nullptr)
        a.lse[t * a.c.num_q_heads + qh] = total == 0.f ? -INFINITY : (ref - (C::kFp8 ? kLift : 0.f) + log2f(total)) * 0.6931471805599453f;
    }
    if (!whole && w.i0 == 0 && g == 0 && row == 0)  // (the segment ends where the range does)
      k.part[blockIdx.x] = Part{w.r, w.head, w.block, cta_of(sh.end + sh.skip + (w.tiles - 1 - w.i1) * weight_of(k, w.q, w.block, sh.weighted != 0), sh.total, sh.ctas)};
    if (joined) named_sync(1, C::kStreamThreads);  // all have read the sums
  }
}

// What the copies in flight write lands before the CTA's memory goes (after a
// role has given up): both parities of a barrier, whichever is the last fill's.
template <class C>
__device__ __forceinline__ void drain_copies(Shared& sh) {
#pragma unroll 1
  for (int i = 0; i < 4 * C::kLoads; ++i)
    mbar_wait(i & 1 ? &sh.v_full[i >> 2] : &sh.full[i >> 2], (i >> 1) & 1, nullptr, 1000000ull);
}

// 14 warps of 128 registers: 8 softmax, 4 preparation, products, loads.  (A split by
// setmaxnreg, 160 and 96, spilled in the products' and loads' warps: 8% more time.)
constexpr int kThreads = 448;

template <class C>
__global__ void __launch_bounds__(kThreads, 1)
    draft_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Args k) {
  extern __shared__ __align__(1024) uint8_t raw[];
  const uint32_t mem = smem_u32(raw);  // (checked below: the swizzle is one of address bits)
  constexpr int kOpAt = C::kTiles * C::kQ, kLoadAt = kOpAt + C::kOps * C::kOperand,
                kEnd = kLoadAt + C::kLoads * C::kRaw, kSharedAt = kEnd + (C::kFp8 ? static_cast<int>(sizeof(Scales)) : 0);
  const Buffers b{mem, mem + kLoadAt, mem + kOpAt, C::kFp8 ? reinterpret_cast<Scales*>(raw + kEnd) : nullptr};
  Shared& sh = *reinterpret_cast<Shared*>(raw + kSharedAt);
  const int tid = threadIdx.x, warp = tid >> 5;
  if (warp == 12) {
    tmem_alloc(&sh.tmem, kTmem);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < C::kLoads; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.v_full[i], 1);
      mbar_init(&sh.empty[i], 1);
      mbar_init(&sh.ready[i], C::kFp8 ? 1 : C::kPrepWarps);
      mbar_init(&sh.op_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&sh.s_full[i], 1), mbar_init(&sh.p_full[i], 4), mbar_init(&sh.pv_done[i], 1);
    mbar_init(&sh.q_full, C::kPrepWarps);
    mbar_init(&sh.q_empty, 1);
    mbar_init(&sh.drain, 1);
    fence_mbar_init();
    sh.abort = 0;
    for (int i = 0; i < 4; ++i) sh.odd[i] = 0;
  }
  wait_predecessor();
  if (tid == 0) k.part[blockIdx.x].last = -1;
  tc_fence_before();
  find_range<kThreads, C::kTwo>(k, sh);
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  if ((mem & 1023u) != 0) {  // not by the launch's rules: nothing is read
    if (tid == 0) report(k.a.c.dev_err, kDevErrTimeout);
  } else if (warp < C::kStreamThreads / 32) {
    softmax<C>(k, sh, walk_of(k, sh), b.sc, tmem, warp >> 2);
  } else if (warp < 12) {
    prepare<C>(k, sh, walk_of(k, sh), b);
  } else if (warp == 12) {
    products<C>(k, sh, walk_of(k, sh), b, tmem);
  } else if (warp == 13) {
    load_tiles<C>(k, sh, walk_of(k, sh), b, &kmap, &vmap);
  }
  tc_fence_before();
  __syncthreads();
  if (sh.abort != 0 && warp == 0) drain_copies<C>(sh);
  if (warp == 12) tmem_dealloc(tmem, kTmem);
  release_successor();
}

template <class C>
cudaError_t launch_config(const CUtensorMap& kmap, const CUtensorMap& vmap, const Args& k, cudaStream_t stream) {
  static_assert(smem_bytes<C>() <= 227 * 1024, "");
  static bool set[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !set[dev]) {
    e = cudaFuncSetAttribute(draft_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<C>());
    if (e != cudaSuccess) return e;
    if (dev < 64) set[dev] = true;
  }
  return launch_after(draft_kernel<C>, dim3(k.l.ctas), kThreads, smem_bytes<C>(), stream, kmap, vmap, k);
}

cudaError_t launch_bf16(const CUtensorMap& kmap, const CUtensorMap& vmap, const Args& k, cudaStream_t stream);
cudaError_t launch_fp8(const CUtensorMap& kmap, const CUtensorMap& vmap, const Args& k, cudaStream_t stream);

}  // namespace draft
}  // namespace ci
