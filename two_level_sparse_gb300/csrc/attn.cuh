// The attention kernel over a paged cache (contract in include/ci_cache.h);
// instances per cache format in attn_bf16.cu and attn_fp8.cu, dispatch and the
// join in attn.cu.
//
// Work.  A row's positions are cut into tiles of 64 (a page, or 64 entries of
// its list); a unit is (row, key-value head, block of up to 64 query heads).
// The units' tiles, in order, are one long list that is split evenly over the
// CTAs of one wave, so ragged batches and a single long row fill the card
// alike.  A CTA whose range covers a whole unit writes its result; where a
// range ends inside a unit, each part leaves its unnormalised sum and softmax
// statistics in the workspace (two parts per CTA at most), and the join kernel
// adds them in order.
//
// A tile.  A producer warp fetches K and V into a ring of stages, pages by TMA
// (128-byte swizzled rows); listed positions take two (produce_list).  WP x WH
// consumer warps compute, WP along the positions and WH along the heads:
//   S^T = K Q^T   A = K from shared memory (ldmatrix), B = Q in registers;
//   online softmax per head, a column of S^T: its maximum over the warp's
//                 positions is a reduction over registers and three shuffles;
//   O^T += V^T P^T  A = V transposed by ldmatrix, B = P transposed in
//                 registers (movmatrix).
// P is rounded to bf16 for the second product, an error of its size of 2^-9 for
// the positions that carry a row.  The sum that divides O is that of the rounded
// P, so that it cancels for a position that carries the row alone; the one that
// the row's statistics keep is of the unrounded P, and O is scaled from the one
// to the other at a segment's end.
// Positions sit on the 16-wide side of the MMA and heads on the 8-wide one, so
// that a group of 8 query heads wastes nothing.
//
// What bounds it: the HBM, where a row reads its whole cache.  64 rows of 16k-64k
// in FP8, 64 heads over 8, D = 128: 5.54 GB in 820 us, 6.75 TB/s, a copy's rate;
// one row of 256k in bf16, 28 heads over 4: 537 MB in 87 us with the join, 6.15
// TB/s.  There the warps' arithmetic is half of what the SM issues, most of it the
// softmax and FP8's conversions, tensor instructions a sixth; two CTAs per SM keep
// the loads going while one reduces.  Short calls are bound by latency: 4 rows of
// 1k-4k (42 MB) take 17 us, 6 of them at the HBM's rate, two launches and their
// starts the rest.  64 rows of 512 listed positions over 8 heads (137 MB) take 35
// us: 8 tiles a unit, whose rows (256 bytes) are fetched at 3.9 TB/s.
//
// FP8 pages.  K: e4m3 widens to f16 exactly, one conversion per pair; the
// query becomes f16 exactly too once each head is scaled by a power of two to
// a largest magnitude in [2^14, 2^15) (what it loses lies 2^-39 below that).
// V: the probabilities carry the value's scale, whose range f16 does not have,
// so this product is bf16: an e4m3 code's exponent and mantissa, moved into the
// low bits of a bf16's, are the value x 2^-120, subnormals included.  The
// powers of two come back in the logit's factor and the final division.
#pragma once
#include <cuda_bf16.h>

#include "cache_common.cuh"

namespace ci {
namespace attn {

constexpr int kTile = 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTwo60 = 1152921504606846976.f;

// What the main kernel and the join agree on.
struct Part {  // the unit that goes on past the end of a CTA's range; last < 0: none
  int32_t row, unit, last, pad;
};
struct Layout {
  int32_t ctas;      // workers (CTAs, or halves of them) that share the list of tiles
  int32_t heads;     // query heads of a unit, padded (HB)
  int32_t blocks;    // head blocks per key-value head
  int32_t group;     // query heads per key-value head
};
struct Args {
  AttnArgs a;
  Layout l;
  Part* part;    // [ctas]
  float* stat;   // [2 ctas][heads][2]: maximum (base 2) and sum
  float* sum;    // [2 ctas][heads][D]
};

template <int D, bool kFp8, int NT, int WP, int WH>
struct Config {
  static constexpr int kRow = kFp8 ? D : 2 * D;           // bytes of a position
  static constexpr int kBox = kRow < 128 ? kRow : 128;    // bytes of a TMA box's rows
  static constexpr int kBoxes = kRow / kBox;
  static constexpr int kSub = kTile * kBox;               // bytes of one box in shared memory
  static constexpr int kMat = kTile * kRow;               // K or V of a tile
  static constexpr int kScale = kFp8 ? kTile * 4 : 0;
  static constexpr int kStage = 2 * kMat;                 // a multiple of the swizzle's 1024 bytes
  static constexpr int kHeadsU = 8 * NT * WH;
  static constexpr int kAccStride = D + 4;                // floats; the pad spreads the heads over the banks
  static constexpr int kAcc = kHeadsU * kAccStride * 4;
  static constexpr int kStat = WP * kHeadsU * 2 * 4;
  static constexpr int kMisc = 1024;                      // barriers, masks, the range
  static constexpr int kCtasPerSm = D == 256 ? 1 : 2;
  static constexpr int kBudget = kCtasPerSm == 1 ? 226 * 1024 : 112 * 1024;
  static constexpr int kFit = (kBudget - 1024 - kAcc - kStat - kMisc) / (kStage + 2 * kScale);
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static_assert(kStages >= 2, "a ring needs two stages");
  static constexpr int kSmem = 1024 + kStages * (kStage + 2 * kScale) + kAcc + kStat + kMisc;
  static constexpr int kConsumers = 32 * WP * WH;
  static constexpr int kThreads = kConsumers + 64;  // and two producer warps
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 2^x and 1 / x to within about 2^-22 of their values, results below 2^-126 as 0: as
// good as the fp32 sums that they go into.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Bytes 0, 1 and bytes 2, 3 of r (e4m3) as f16 pairs.
__device__ __forceinline__ void e4m3_to_f16(uint32_t r, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(r));
}
// Bytes 0, 2 and bytes 1, 3 of r (e4m3) as bf16 pairs of the value x 2^-120.
__device__ __forceinline__ void e4m3_to_bf16(uint32_t r, uint32_t& even, uint32_t& odd) {
  even = ((r << 8) & 0x80008000u) | ((r << 4) & 0x07F007F0u);
  odd = (r & 0x80008000u) | ((r >> 4) & 0x07F007F0u);
}

// Byte offset of 16-byte chunk `chunk` of position `p` in a matrix of a tile:
// boxes of 128-byte (64-byte) rows, the chunk index XOR-ed as the TMA swizzle does.
template <class C>
__device__ __forceinline__ uint32_t tile_offset(int p, int chunk) {
  constexpr int kPer = C::kBox / 16;
  const int box = chunk / kPer, c = chunk % kPer;
  const int x = C::kBox == 128 ? c ^ (p & 7) : c ^ ((p >> 1) & 3);
  return box * C::kSub + p * C::kBox + x * 16;
}

__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int x, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(row), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// 16 bytes to shared memory, asynchronously: from src, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src, bool read) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}

__device__ __forceinline__ void cp_async4_to(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// The tiles (of kT positions) of row t (0: nothing to read).
template <int kT>
__device__ __forceinline__ int row_tiles(const AttnArgs& a, int t) {
  const int len = a.seq_len[t];
  if (len <= 0 || len > a.max_len) return 0;
  return static_cast<int>((static_cast<uint32_t>(a.pos != nullptr ? a.npos : len) + kT - 1) / kT);
}

// A worker's range of the list (the host has checked that its indices fit in 31
// bits) and where it starts.
struct Range {
  int32_t first, end, total, workers;  // workers: how many share the list (every one has a tile)
  int32_t row, unit, tile, worker;
};

// A worker's way through its range: segment by segment (tiles [i0, i1) of a unit).
template <int kT>
struct Walk {
  int left;                       // tiles of the range behind the segment
  int row, unit, tile, n, units;  // where the next segment starts; n: tiles of the row
  int i0, i1;
  __device__ __forceinline__ bool next(const AttnArgs& a) {
    if (left == 0) return false;
    if (tile == n) {
      tile = 0;
      if (++unit == units) {
        unit = 0;
#pragma unroll 1
        do n = row_tiles<kT>(a, ++row);
        while (n == 0);
      }
    }
    i0 = tile;
    i1 = min(n, i0 + left);
    left -= i1 - i0;
    tile = i1;
    return true;
  }
};

template <int N>
struct RangeShared {
  Range range[N];
  int32_t warp_sum[24];
};

struct Shared {
  uint64_t full[8], empty[8];
  uint32_t mask[8][2];  // per stage: which of the 64 positions count
  RangeShared<1> r;
  int32_t abort;
};
static_assert(sizeof(Shared) <= 1024, "");

// The list's first worker-th share: total / workers tiles each, the first total %
// workers one more.
__device__ __forceinline__ int share_start(int worker, int per, int rest) { return worker * per + min(worker, rest); }

// The ranges of this CTA's N workers: every thread adds up a run of rows, a scan
// over the threads gives the total, and the thread whose run holds a range's
// first tile walks to it.  True where some row has nothing to read.
template <int kThreads, int kT, int N>
__device__ __forceinline__ bool find_ranges(const Args& k, RangeShared<N>& sh, int units) {
  const AttnArgs& a = k.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per_thread = (a.rows + kThreads - 1) / kThreads;
  const int r0 = min(tid * per_thread, a.rows), r1 = min(r0 + per_thread, a.rows);
  int mine = 0;
  bool none = false, bad = false;
#pragma unroll 4
  for (int r = r0; r < r1; ++r) {
    const int n = row_tiles<kT>(a, r), len = a.seq_len[r];
    bad |= len < 0 || len > a.max_len;
    none |= n == 0;
    mine += n;
  }
  if (bad && blockIdx.x == 0) report(a.c.dev_err, kDevErrLen);
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sh.warp_sum[warp] = incl;
  none = __syncthreads_or(none);
  int before = incl - mine, total = 0;
#pragma unroll 1
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sh.warp_sum[w];
    total += sh.warp_sum[w];
  }
  total *= units;
  const int workers = min(k.l.ctas, total), per = workers > 0 ? total / workers : 0, rest = total - per * workers;
#pragma unroll 1
  for (int i = 0; i < N; ++i) {
    const int worker = blockIdx.x + i * gridDim.x;
    const int first = share_start(min(worker, workers), per, rest), end = share_start(min(worker + 1, workers), per, rest);
    Range& range = sh.range[i];
    if (tid == 0) range.first = first, range.end = end, range.total = total, range.workers = workers, range.worker = worker;
    int at = before * units;
    if (first < end && at <= first && first < at + mine * units) {
      int r = r0, n = row_tiles<kT>(a, r);
#pragma unroll 1
      while (first >= at + n * units) {
        at += n * units;
        n = row_tiles<kT>(a, ++r);
      }
      range.row = r;
      range.unit = (first - at) / n;
      range.tile = (first - at) - range.unit * n;
    }
  }
  __syncthreads();
  return none;
}
template <int kT>
__device__ __forceinline__ Walk<kT> walk_of(const AttnArgs& a, const Range& r, int units) {
  return Walk<kT>{r.end - r.first, r.row, r.unit, r.tile, r.first < r.end ? row_tiles<kT>(a, r.row) : 0, units, 0, 0};
}
// The worker that has tile x of the list.
__device__ __forceinline__ int worker_of(int x, const Range& r) {
  const int per = r.total / r.workers, rest = r.total - per * r.workers, longer = rest * (per + 1);
  return x < longer ? x / (per + 1) : rest + (x - longer) / per;
}
// What a worker leaves behind for the unit that goes on past its range: the
// unit, and the worker that has its last tile.
template <int kT>
__device__ __forceinline__ Part part_of(const Walk<kT>& w, const Range& r) {
  return Part{w.row, w.unit, worker_of(r.end - 1 + w.n - w.i1, r), 0};  // (the segment ends where the range does)
}
// Where a worker keeps its part of a unit: the unit's first part is the last
// segment of its worker's range, every other one a first segment.
__host__ __device__ __forceinline__ int64_t slot_of(int worker, bool begins) { return 2ll * worker + (begins ? 1 : 0); }

// A bounded wait of a whole warp for phase `parity`; false once it, or another
// warp of the CTA, has given up (reported once).
static __device__ __noinline__ bool wait_warp_slow(uint64_t* bar, uint32_t parity, int32_t* abort, int32_t* dev_err) {
  const uint64_t t0 = globaltimer_ns();
  bool ok = false;
  while (!ok && *static_cast<volatile int32_t*>(abort) == 0 && globaltimer_ns() - t0 < 2000000000ull)
    ok = mbar_try_wait_sleep(bar, parity);
  ok = __all_sync(0xffffffffu, ok);
  if (!ok && (threadIdx.x & 31) == 0 && atomicExch(abort, 1) == 0) report(dev_err, kDevErrTimeout);
  return ok;
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int32_t* abort, int32_t* dev_err) {
  // (the second probe sleeps in the barrier for a while)
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  if (__all_sync(0xffffffffu, mbar_try_wait_sleep(bar, parity))) return true;
  return wait_warp_slow(bar, parity, abort, dev_err);
}

// Rows with nothing to read.
template <int D, int kThreads>
__device__ __forceinline__ void write_empty_rows(const AttnArgs& a) {
#pragma unroll 1
  for (int t = blockIdx.x; t < a.rows; t += gridDim.x) {
    if (row_tiles<kTile>(a, t) != 0) continue;
#pragma unroll 1
    for (int e = threadIdx.x; e < a.c.num_q_heads * (D / 8); e += kThreads)
      *reinterpret_cast<uint4*>(a.out + t * a.out_stride + e * 8) = make_uint4(0, 0, 0, 0);
    if (a.lse == nullptr) continue;
#pragma unroll 1
    for (int h = threadIdx.x; h < a.c.num_q_heads; h += kThreads)
      a.lse[static_cast<int64_t>(t) * a.c.num_q_heads + h] = -INFINITY;
  }
}

// ------------------------------------------------------------------ producers
// The ring as the producer sees it.
template <class C>
struct Ring {
  Shared& sh;
  const Args& k;
  int stage = 0;
  uint32_t phase = 1;  // the first round of stages is free
  uint32_t used = 0;
  bool alive = true;

  __device__ __forceinline__ bool acquire() {
    alive = alive && wait_warp(&sh.empty[stage], phase, &sh.abort, k.a.c.dev_err);
    return alive;
  }
  __device__ __forceinline__ void advance() {
    used |= 1u << stage;
    if (++stage == C::kStages) stage = 0, phase ^= 1;
  }
  // Gave up: what is in flight lands before the CTA's memory goes.
  __device__ __forceinline__ void drain() {
    if (alive) return;
    for (int st = 0; st < C::kStages; ++st) {
      const uint32_t last = st < stage ? phase ^ 1 : phase;  // parity of the stage's last fill
      if ((used >> st) & 1) mbar_wait(&sh.full[st], last, nullptr, 1000000ull);
    }
  }
};

// Every position below the length: a tile is a page, fetched by TMA.
template <class C, int D, bool kFp8>
__device__ void produce_pages(const Args& k, Shared& sh, Walk<kTile> w, const CUtensorMap* kmap, const CUtensorMap* vmap,
                              uint32_t stages) {
  const AttnArgs& a = k.a;
  const CacheArgs& c = a.c;
  constexpr int kRowsPerPage = cache_page_bytes<kFp8>(D) / C::kRow;
  const int lane = threadIdx.x & 31;
  Ring<C> ring{sh, k};
#pragma unroll 1
  while (w.next(a)) {
    const int req = row_request(c, w.row);
    const int head = w.unit / k.l.blocks;
    const int32_t* table = req >= 0 ? c.page_table + static_cast<int64_t>(req) * c.max_pages : nullptr;
    const int len = table != nullptr ? a.seq_len[w.row] : 0;
    int ids = 0;
#pragma unroll 1
    for (int i = w.i0; i < w.i1; ++i) {
      const int j = (i - w.i0) & 31;
      if (j == 0) {  // the next 32 tiles' pages, one per lane
        ids = -1;
        if (i + lane < w.i1 && table != nullptr) ids = table[i + lane];
      }
      const int page = __shfl_sync(0xffffffffu, ids, j);
      const bool ok = page >= 0 && page < c.num_pages;
      if (!ok && lane == 0 && table != nullptr) report(c.dev_err, kDevErrPage);
      const int left = ok ? len - i * kTile : 0;
      const uint32_t m0 = left >= 32 ? ~0u : left > 0 ? (1u << left) - 1 : 0;
      const uint32_t m1 = left >= 64 ? ~0u : left > 32 ? (1u << (left - 32)) - 1 : 0;
      if (ring.acquire()) {
        const int stage = ring.stage;
        const uint32_t bar = smem_u32(&sh.full[stage]);
        const uint32_t kdst = stages + stage * C::kStage, vdst = kdst + C::kMat;
        const uint32_t sdst = stages + C::kStages * C::kStage + stage * 2 * C::kScale;
        if (lane == 0) {
          sh.mask[stage][0] = m0;
          sh.mask[stage][1] = m1;
          if (left > 0)
            mbar_arrive_expect_tx(&sh.full[stage], C::kStage + 2 * C::kScale);
          else
            mbar_arrive(&sh.full[stage]);
        }
        __syncwarp();
        if (left > 0) {
          const int row = (page * c.num_kv_heads + head) * kRowsPerPage;
          if (lane < 2 * C::kBoxes) {
            const int b = lane % C::kBoxes;
            tma_box((lane < C::kBoxes ? kdst : vdst) + b * C::kSub, lane < C::kBoxes ? kmap : vmap, b * C::kBox, row,
                    bar);
          }
          if (kFp8 && (lane == 16 || lane == 17)) {
            const int64_t at = (static_cast<int64_t>(page) * c.num_kv_heads + head) * cache_page_bytes<kFp8>(D) + kPage * D;
            bulk_load(sdst + (lane - 16) * C::kScale, (lane == 16 ? c.k_pool : c.v_pool) + at, C::kScale, bar);
          }
        }
      }
      ring.advance();
    }
  }
  ring.drain();
}

// Listed positions, by two warps side by side: one copies K, the other V and the
// FP8 scales, by 16-byte asynchronous copies whose chunks are put where the TMA
// swizzle would have put them.  (K gathered by TMA, four rows per instruction:
// 300 rows over 512 positions of 4 heads of 64 in bf16 63 us, these 58; FP8 70, 66;
// 64 rows of 8 heads of 128 45.7, 46.7; cold caches.)  Two tiles of look-ahead: the
// list entries of the second next tile and the page ids of the next one are on
// their way while a tile is copied.
struct ListTile {
  const int32_t* table;  // null: the row has no request
  int head, len;
  int s0, s1;  // the list's entries lane and 32 + lane of the tile
  bool live;
};

template <class C, int D, bool kFp8, bool kValues>
__device__ void produce_list(const Args& k, Shared& sh, Walk<kTile> w, uint32_t stages) {
  const AttnArgs& a = k.a;
  const CacheArgs& c = a.c;
  constexpr int64_t kPageBytes = cache_page_bytes<kFp8>(D);
  constexpr int kChunks = C::kRow / 16, kRows = 32 / kChunks;  // 16-byte chunks of a row; rows per warp and copy
  constexpr int kRowsPerPage = kPageBytes / C::kRow;
  const int lane = threadIdx.x & 31, chunk = lane % kChunks;
  Ring<C> ring{sh, k};
  int i = 0, end = 0;  // the next tile of the walk's segment
  ListTile seg{nullptr, 0, 0, -1, -1, false};
  auto fetch = [&]() {  // the next tile, its list entries under way
    ListTile x{nullptr, 0, 0, -1, -1, false};
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
    const int at = i * kTile + lane;
    const int32_t* list = a.pos + static_cast<int64_t>(w.row) * a.pos_stride + at;
    if (at < a.npos) x.s0 = list[0];
    if (at + 32 < a.npos) x.s1 = list[32];
    ++i;
    return x;
  };
  ListTile now = seg, next = seg;
  int p0 = 0, p1 = 0;
#pragma unroll 1
  while (true) {
    // page ids of the next tile's entries (0 where an entry does not count)
    const int n0 = next.s0 >= 0 && next.s0 < next.len ? next.table[next.s0 / kPage] : 0;
    const int n1 = next.s1 >= 0 && next.s1 < next.len ? next.table[next.s1 / kPage] : 0;
    const ListTile after = fetch();
    if (!now.live) {  // the pipeline fills, or is empty
      if (!next.live && !after.live) break;
      now = next, next = after, p0 = n0, p1 = n1;
      continue;
    }
    const bool in0 = now.s0 >= 0 && now.s0 < now.len, in1 = now.s1 >= 0 && now.s1 < now.len;
    const bool ok0 = in0 && p0 >= 0 && p0 < c.num_pages, ok1 = in1 && p1 >= 0 && p1 < c.num_pages;
    if (!kValues) {
      if (now.table != nullptr && ((!in0 && now.s0 != -1) || (!in1 && now.s1 != -1))) report(c.dev_err, kDevErrPos);
      if (ok0 != in0 || ok1 != in1) report(c.dev_err, kDevErrPage);
    }
    // rows of the pool (of kRow bytes); -1: an entry that does not count, zeros
    const int row0 = ok0 ? (p0 * c.num_kv_heads + now.head) * kRowsPerPage + (now.s0 & (kPage - 1)) : -1;
    const int row1 = ok1 ? (p1 * c.num_kv_heads + now.head) * kRowsPerPage + (now.s1 & (kPage - 1)) : -1;
    if (ring.acquire()) {
      const int stage = ring.stage;
      const uint32_t kdst = stages + stage * C::kStage;
      if constexpr (!kValues) {
        const uint32_t m0 = __ballot_sync(0xffffffffu, ok0), m1 = __ballot_sync(0xffffffffu, ok1);
        if (lane == 0) {
          sh.mask[stage][0] = m0;
          sh.mask[stage][1] = m1;
          mbar_arrive(&sh.full[stage]);
        }
        __syncwarp();
        const uint8_t* kbase = c.k_pool + chunk * 16;
#pragma unroll
        for (int p = 0; p < kTile; p += kRows) {  // positions p .. p + kRows - 1
          const int row = __shfl_sync(0xffffffffu, p < 32 ? row0 : row1, (p + lane / kChunks) & 31);
          copy16(kdst + tile_offset<C>(p + lane / kChunks, chunk), kbase + static_cast<int64_t>(max(row, 0)) * C::kRow, row >= 0);
        }
        cp_async_arrive_noinc(&sh.full[stage]);
      } else {
        const uint8_t* vbase = c.v_pool + chunk * 16;
#pragma unroll
        for (int p = 0; p < kTile; p += kRows) {  // positions p .. p + kRows - 1
          const int row = __shfl_sync(0xffffffffu, p < 32 ? row0 : row1, (p + lane / kChunks) & 31);
          copy16(kdst + C::kMat + tile_offset<C>(p + lane / kChunks, chunk),
                 vbase + static_cast<int64_t>(max(row, 0)) * C::kRow, row >= 0);
        }
        if (kFp8) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int row = hh ? row1 : row0;
            if (row < 0) continue;
            const int64_t page = row / kRowsPerPage;
            const int64_t at = page * kPageBytes + kPage * D + (row - page * kRowsPerPage) * 4;
            const uint32_t to = stages + C::kStages * C::kStage + stage * 2 * C::kScale + (hh * 32 + lane) * 4;
            cp_async4_to(to, c.k_pool + at);
            cp_async4_to(to + C::kScale, c.v_pool + at);
          }
        }
        cp_async_arrive_noinc(&sh.full[stage]);
      }
    }
    ring.advance();
    now = next, next = after, p0 = n0, p1 = n1;
  }
  cp_async_wait<0>();
}

// ------------------------------------------------------------------ consumers
template <class C, int D, bool kFp8, int NT, int WP, int WH>
__device__ void consume(const Args& k, Shared& sh, Walk<kTile> w, uint32_t stages, float* acc, float* stat) {
  constexpr int kM = D / 16, kK = D / 16, MT = 4 / WP;
  // How many of its 16-position tiles a warp has in registers at once: all, or half
  // where that spills 192 bytes (FP8, D = 128, 64 heads: 17 rows of 0-100k 166 -> 156
  // us, 1024 rows over 512 listed 161 -> 128; elsewhere all is as fast or faster).
  constexpr int MS = kFp8 && D == 128 && MT == 4 ? 2 : MT;
  const AttnArgs& a = k.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const int wp = warp % WP, wh = warp / WP, p0 = wp * 16 * MT;
  const int tid = threadIdx.x;
  const float factor = a.scale * kLog2e;
  const Range range = sh.r.range[0];
  int stage = 0;
  uint32_t phase = 0;
  bool alive = true;
#pragma unroll 1
  while (w.next(a)) {
    const int head = w.unit / k.l.blocks, hb = w.unit - head * k.l.blocks;
    const int h0 = hb * C::kHeadsU;                                // first head of the unit, within its group
    const int live = min(C::kHeadsU, k.l.group - h0);              // heads of the unit that exist
    // ---- the queries, as B fragments
    uint32_t qf[NT][kK][2];
    float qs[NT][2];  // FP8: what undoes the scaling of heads 2q and 2q + 1
    {
      const uint16_t* row = a.q + w.row * a.q_stride + (static_cast<int64_t>(head) * k.l.group + h0) * D;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int h = wh * 8 * NT + nt * 8 + g;
        const uint16_t* src = row + static_cast<int64_t>(h < live ? h : 0) * D;
#pragma unroll
        for (int kk = 0; kk < kK; ++kk) {
          uint2 v;
          if (kFp8) {  // the order of the 16 dims that the widened codes come in: 4q, 4q + 1 | 4q + 2, 4q + 3
            v = *reinterpret_cast<const uint2*>(src + kk * 16 + 4 * q);
          } else {
            v.x = *reinterpret_cast<const uint32_t*>(src + kk * 16 + 2 * q);
            v.y = *reinterpret_cast<const uint32_t*>(src + kk * 16 + 8 + 2 * q);
          }
          qf[nt][kk][0] = h < live ? v.x : 0;
          qf[nt][kk][1] = h < live ? v.y : 0;
        }
        if (kFp8) {
          uint32_t most = 0;  // the largest magnitude's bits, of both halves
#pragma unroll
          for (int kk = 0; kk < kK; ++kk) most = __vmaxu2(most, __vmaxu2(qf[nt][kk][0] & 0x7FFF7FFFu, qf[nt][kk][1] & 0x7FFF7FFFu));
          most = max(most & 0xFFFFu, most >> 16);
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
          most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
          const int e = most >> 7;  // biased exponent; 0: zeros and subnormals, 255: not finite
          const int up = e == 0 || e == 255 ? 0 : 127 + 14 - e;  // times 2^up
          // 2^up lies in [2^-113, 2^140]: in two steps, each a normal number
          const float f0 = __uint_as_float((127 + up / 2) << 23), f1 = __uint_as_float((127 + up - up / 2) << 23);
          const float back = __uint_as_float((127 - up / 2) << 23) * __uint_as_float((127 - (up - up / 2)) << 23);
          qs[nt][0] = __shfl_sync(0xffffffffu, back, 8 * q);
          qs[nt][1] = __shfl_sync(0xffffffffu, back, 8 * q + 4);
#pragma unroll
          for (int kk = 0; kk < kK; ++kk)
#pragma unroll
            for (int e2 = 0; e2 < 2; ++e2)
              qf[nt][kk][e2] = f16x2(bf16_lo(qf[nt][kk][e2]) * f0 * f1, bf16_hi(qf[nt][kk][e2]) * f0 * f1);
        }
      }
    }
    float o[NT][kM][4], top[NT][2], l[NT][2], lr[NT][2];  // lr: the sums of P as it is rounded
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][m][e] = 0.f;
      top[nt][0] = top[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = lr[nt][0] = lr[nt][1] = 0.f;
    }
#pragma unroll 1
    for (int i = w.i0; i < w.i1; ++i) {
      alive = alive && wait_warp(&sh.full[stage], phase, &sh.abort, a.c.dev_err);
      const uint32_t kbase = stages + stage * C::kStage, vbase = kbase + C::kMat;
      const uint32_t sbase = stages + C::kStages * C::kStage + stage * 2 * C::kScale;
      const uint64_t mask = static_cast<uint64_t>(sh.mask[stage][1]) << 32 | sh.mask[stage][0];
      constexpr uint64_t kOnes = MS == 4 ? ~0ull : (1ull << (16 * MS & 63)) - 1;
#pragma unroll 1
      for (int part = 0; part < MT / MS; ++part) {
        const int pp = p0 + part * 16 * MS;
        const uint64_t here = (mask >> pp) & kOnes;  // these positions
        if (!alive || here == 0) continue;
        // ---- S^T
        float s[MS][NT][4];
#pragma unroll
        for (int mt = 0; mt < MS; ++mt) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.f;
          const int p = pp + mt * 16;
          if (kFp8) {
#pragma unroll
            for (int kk = 0; kk < kK; kk += 2) {
              uint32_t r[4];  // positions 0-7 | 8-15 of dims 0-15, then of dims 16-31
              ldsm4(r, kbase + tile_offset<C>(p + (lane & 15), kk + (lane >> 4)));
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
                const uint32_t x = r[2 * hh], y = r[2 * hh + 1];
                uint32_t a0, a1, a2, a3;
                e4m3_to_f16(x, a0, a2);
                e4m3_to_f16(y, a1, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16(s[mt][nt], a0, a1, a2, a3, qf[nt][kk + hh][0], qf[nt][kk + hh][1]);
              }
            }
          } else {
#pragma unroll
            for (int kk = 0; kk < kK; ++kk) {
              uint32_t r[4];
              ldsm4(r, kbase + tile_offset<C>(p + (lane & 15), 2 * kk + (lane >> 4)));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_bf16(s[mt][nt], r[0], r[1], r[2], r[3], qf[nt][kk][0], qf[nt][kk][1]);
            }
          }
        }
        // ---- logits in base 2, the new maxima
        const bool all = here == kOnes;
        float now[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) now[nt][0] = top[nt][0], now[nt][1] = top[nt][1];
#pragma unroll
        for (int mt = 0; mt < MS; ++mt) {
          const int pa = pp + mt * 16 + g;
          float fa = factor, fb = factor;
          if (kFp8) {
            fa *= lds_f32(sbase + pa * 4);
            fb *= lds_f32(sbase + (pa + 8) * 4);
          }
          const bool ina = all || ((mask >> pa) & 1), inb = all || ((mask >> (pa + 8)) & 1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float(&v)[4] = s[mt][nt];
            if (kFp8) v[0] *= qs[nt][0], v[1] *= qs[nt][1], v[2] *= qs[nt][0], v[3] *= qs[nt][1];
            v[0] = ina ? v[0] * fa : -INFINITY;
            v[1] = ina ? v[1] * fa : -INFINITY;
            v[2] = inb ? v[2] * fb : -INFINITY;
            v[3] = inb ? v[3] * fb : -INFINITY;
            now[nt][0] = fmaxf(now[nt][0], fmaxf(v[0], v[2]));
            now[nt][1] = fmaxf(now[nt][1], fmaxf(v[1], v[3]));
          }
        }
        bool grew = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int b = 4; b < 32; b <<= 1) now[nt][e] = fmaxf(now[nt][e], __shfl_xor_sync(0xffffffffu, now[nt][e], b));
            grew |= now[nt][e] > top[nt][e];
          }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float keep[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              keep[e] = now[nt][e] > top[nt][e] ? exp2_approx(top[nt][e] - now[nt][e]) : 1.f;
              top[nt][e] = now[nt][e];
              l[nt][e] *= keep[e];
              lr[nt][e] *= keep[e];
            }
#pragma unroll
            for (int m = 0; m < kM; ++m) {
              o[nt][m][0] *= keep[0], o[nt][m][1] *= keep[1];
              o[nt][m][2] *= keep[0], o[nt][m][3] *= keep[1];
            }
          }
        }
        if (!kFp8 && !all && a.pos == nullptr) {  // what follows a row's last position must not reach a product with 0
#pragma unroll 1
          for (int e = lane; e < 16 * MS * (C::kRow / 16); e += 32) {
            const int p = pp + e / (C::kRow / 16);
            if ((mask >> p) & 1) continue;
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(vbase + tile_offset<C>(p, e % (C::kRow / 16))),
                         "r"(0)
                         : "memory");
          }
          fence_proxy_async_smem();  // before the stage's next TMA write
          __syncwarp();
        }
        // ---- probabilities; O^T += V^T P^T
#pragma unroll
        for (int mt = 0; mt < MS; ++mt) {
          const int p = pp + mt * 16;
          float va = 1.f, vb = 1.f;
          if (kFp8) {
            va = kTwo60 * lds_f32(sbase + C::kScale + (p + g) * 4);
            vb = kTwo60 * lds_f32(sbase + C::kScale + (p + g + 8) * 4);
            if (!all) {
              if (!((mask >> (p + g)) & 1)) va = 0.f;
              if (!((mask >> (p + g + 8)) & 1)) vb = 0.f;
            }
          }
          // FP8: P is rounded with the value's scale in it
          const float ia = !kFp8 || va == 0.f ? 0.f : rcp_approx(va), ib = !kFp8 || vb == 0.f ? 0.f : rcp_approx(vb);
          uint32_t b0[NT], b1[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float(&v)[4] = s[mt][nt];
            // top is -inf only while every logit of the head so far is: exp2(-inf) = 0 either way
            const float t0 = top[nt][0] == -INFINITY ? 0.f : top[nt][0], t1 = top[nt][1] == -INFINITY ? 0.f : top[nt][1];
            v[0] = exp2_approx(v[0] - t0);
            v[1] = exp2_approx(v[1] - t1);
            v[2] = exp2_approx(v[2] - t0);
            v[3] = exp2_approx(v[3] - t1);
            l[nt][0] += v[0] + v[2];
            l[nt][1] += v[1] + v[3];
            if (kFp8) {
              const float w0 = v[0] * va, w1 = v[1] * va, w2 = v[2] * vb, w3 = v[3] * vb;
              b0[nt] = bf16x2(w0, w1);
              b1[nt] = bf16x2(w2, w3);
              lr[nt][0] += fmaf(bf16_lo(b0[nt]) - w0, ia, v[0]) + fmaf(bf16_lo(b1[nt]) - w2, ib, v[2]);
              lr[nt][1] += fmaf(bf16_hi(b0[nt]) - w1, ia, v[1]) + fmaf(bf16_hi(b1[nt]) - w3, ib, v[3]);
            } else {
              b0[nt] = bf16x2(v[0], v[1]);
              b1[nt] = bf16x2(v[2], v[3]);
              lr[nt][0] += bf16_lo(b0[nt]) + bf16_lo(b1[nt]);
              lr[nt][1] += bf16_hi(b0[nt]) + bf16_hi(b1[nt]);
            }
            b0[nt] = transpose8x8(b0[nt]);
            b1[nt] = transpose8x8(b1[nt]);
          }
          if (kFp8) {
#pragma unroll
            for (int m = 0; m < kM; m += 2) {
              uint32_t r[4];  // positions 0-7 | 8-15 of dims 0-15, then of dims 16-31; pairs of dims move together
              ldsm4_t(r, vbase + tile_offset<C>(p + (lane & 15), m + (lane >> 4)));
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {  // row g of the product is dim 2g, row g + 8 dim 2g + 1
                const uint32_t x = r[2 * hh], y = r[2 * hh + 1];
                uint32_t a0, a1, a2, a3;
                e4m3_to_bf16(x, a0, a1);
                e4m3_to_bf16(y, a2, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_bf16(o[nt][m + hh], a0, a1, a2, a3, b0[nt], b1[nt]);
              }
            }
          } else {
#pragma unroll
            for (int m = 0; m < kM; ++m) {
              uint32_t r[4];
              ldsm4_t(r, vbase + tile_offset<C>(p + (lane & 7) + ((lane >> 4) << 3), 2 * m + ((lane >> 3) & 1)));
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma_bf16(o[nt][m], r[0], r[1], r[2], r[3], b0[nt], b1[nt]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[stage]);
      if (++stage == C::kStages) stage = 0, phase ^= 1;
    }
    // ---- the warps' parts of the segment into one
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int b = 4; b < 32; b <<= 1) {
          l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], b);
          lr[nt][e] += __shfl_xor_sync(0xffffffffu, lr[nt][e], b);
        }
        if (g == 0) {
          const int h = wh * 8 * NT + nt * 8 + 2 * q + e;
          stat[(wp * C::kHeadsU + h) * 2] = top[nt][e];
          stat[(wp * C::kHeadsU + h) * 2 + 1] = l[nt][e];
        }
      }
    named_sync(1, C::kConsumers);
    const bool whole = w.i0 == 0 && w.i1 == w.n;
    float keep[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = wh * 8 * NT + nt * 8 + 2 * q + e;
        float m = -INFINITY, sum = 0.f;
#pragma unroll
        for (int x = 0; x < WP; ++x) m = fmaxf(m, stat[(x * C::kHeadsU + h) * 2]);
        const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int x = 0; x < WP; ++x)
          sum += stat[(x * C::kHeadsU + h) * 2 + 1] * exp2_approx(stat[(x * C::kHeadsU + h) * 2] - ref);
        // (lr is 0 only with l)
        keep[nt][e] = exp2_approx(top[nt][e] - ref) * (kFp8 ? kTwo60 : 1.f) * (lr[nt][e] == 0.f ? 1.f : l[nt][e] / lr[nt][e]);
        if (whole) keep[nt][e] *= sum == 0.f ? 0.f : 1.f / sum;
        if (wp == 0 && g == 0) {
          if (!whole) {
            const int64_t slot = slot_of(blockIdx.x, w.i0 == 0);
            float* st = k.stat + (slot * C::kHeadsU + h) * 2;
            st[0] = m;
            st[1] = sum;
          } else if (a.lse != nullptr && h < live) {
            a.lse[static_cast<int64_t>(w.row) * a.c.num_q_heads + static_cast<int64_t>(head) * k.l.group + h0 + h] =
                sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
          }
        }
      }
#pragma unroll 1
    for (int x = 0; x < WP; ++x) {
      if (wp == x) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int m = 0; m < kM; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int h = wh * 8 * NT + nt * 8 + 2 * q + (e & 1);
              const int d = m * 16 + (kFp8 ? 2 * g + (e >> 1) : g + 8 * (e >> 1));
              float* at = acc + h * C::kAccStride + d;
              const float v = o[nt][m][e] * keep[nt][e & 1];
              *at = x == 0 ? v : *at + v;
            }
      }
      named_sync(1, C::kConsumers);
    }
    if (whole) {
      uint16_t* dst = a.out + w.row * a.out_stride + (static_cast<int64_t>(head) * k.l.group + h0) * D;
#pragma unroll 1
      for (int e = tid; e < live * (D / 8); e += C::kConsumers) {
        const int h = e / (D / 8), d = e % (D / 8) * 8;
        const float4 x = *reinterpret_cast<const float4*>(acc + h * C::kAccStride + d);
        const float4 y = *reinterpret_cast<const float4*>(acc + h * C::kAccStride + d + 4);
        *reinterpret_cast<uint4*>(dst + h * D + d) = make_uint4(bf16x2(x.x, x.y), bf16x2(x.z, x.w), bf16x2(y.x, y.y), bf16x2(y.z, y.w));
      }
    } else {
      float* dst = k.sum + slot_of(blockIdx.x, w.i0 == 0) * C::kHeadsU * D;
#pragma unroll 1
      for (int e = tid; e < live * (D / 4); e += C::kConsumers) {
        const int h = e / (D / 4), d = e % (D / 4) * 4;
        *reinterpret_cast<float4*>(dst + h * D + d) = *reinterpret_cast<const float4*>(acc + h * C::kAccStride + d);
      }
      if (tid == 0 && w.i0 == 0) {
        k.part[blockIdx.x] = part_of(w, range);
      }
    }
  }
}

template <int D, bool kFp8, int NT, int WP, int WH>
__global__ void __launch_bounds__(Config<D, kFp8, NT, WP, WH>::kThreads, Config<D, kFp8, NT, WP, WH>::kCtasPerSm)
    attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap, const Args k) {
  using C = Config<D, kFp8, NT, WP, WH>;
  extern __shared__ uint8_t raw[];
  const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u;  // the swizzle is one of address bits
  uint8_t* mem = raw + (base - smem_u32(raw));
  float* acc = reinterpret_cast<float*>(mem + C::kStages * (C::kStage + 2 * C::kScale));
  float* stat = acc + C::kAcc / 4;
  Shared& sh = *reinterpret_cast<Shared*>(reinterpret_cast<uint8_t*>(stat) + C::kStat);
  const AttnArgs& a = k.a;
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sh.full[s], a.pos != nullptr ? 65 : 1);
      mbar_init(&sh.empty[s], WP * WH);
    }
    fence_mbar_init();
    sh.abort = 0;
  }
  wait_predecessor();
  if (tid == 0) k.part[blockIdx.x].last = -1;
  const int units = a.c.num_kv_heads * k.l.blocks;
  if (find_ranges<C::kThreads, kTile, 1>(k, sh.r, units)) write_empty_rows<D, C::kThreads>(a);
  const Range r = sh.r.range[0];
  if (r.first < r.end) {
    const Walk<kTile> w = walk_of<kTile>(a, r, units);
    if (warp < WP * WH)
      consume<C, D, kFp8, NT, WP, WH>(k, sh, w, base, acc, stat);
    else if (a.pos != nullptr && warp == WP * WH)
      produce_list<C, D, kFp8, false>(k, sh, w, base);
    else if (a.pos != nullptr)
      produce_list<C, D, kFp8, true>(k, sh, w, base);
    else if (warp == WP * WH)
      produce_pages<C, D, kFp8>(k, sh, w, &kmap, &vmap, base);
  }
  release_successor();
}

template <int D, bool kFp8, int NT, int WP, int WH>
cudaError_t launch(const CUtensorMap& kmap, const CUtensorMap& vmap, const Args& k, cudaStream_t stream) {
  using C = Config<D, kFp8, NT, WP, WH>;
  auto fn = attn_kernel<D, kFp8, NT, WP, WH>;
  static bool set[64] = {false};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !set[dev]) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) set[dev] = true;
  }
  return launch_after(fn, dim3(k.l.ctas), C::kThreads, C::kSmem, stream, kmap, vmap, k);
}

// The instance for a head size and a padded number of heads per unit.  A thread
// keeps NT D / 4 sums of O, which registers bound to 64: NT = 2 heads of eight, or 1
// for D = 256.  The positions go to the warps that the heads leave of four (of eight
// for D = 256, one CTA per SM).  More heads cost more, as each of WH warps reads the
// whole tile from shared memory (and widens it, in FP8): 17 rows of 0-100k, one
// key-value head, 8, 16, 32 and 64 query heads, us (floor: the bytes):
//   D =  64  bf16  43.6,  46.5,  49.0,  69.9 (32)    FP8  36.4,  42.7,  59.2,  92.7 (17)
//   D = 128  bf16  73.0,  77.0,  80.7, wide  (64)    FP8  47.7,  58.9,  92.7, 151.8 (33)
//   D = 256  bf16 135.8, 139.1, 157.0, 263.5 (128)   FP8  84.3, 126.1, 210.1, 363.8 (65)
template <bool kFp8>
cudaError_t launch_format(const CUtensorMap& kmap, const CUtensorMap& vmap, const Args& k, cudaStream_t s) {
  const int d = k.a.c.head_dim, h = k.l.heads;
  if (d == 64) {
    if (h == 8) return launch<64, kFp8, 1, 4, 1>(kmap, vmap, k, s);
    if (h == 16) return launch<64, kFp8, 2, 4, 1>(kmap, vmap, k, s);
    if (h == 32) return launch<64, kFp8, 2, 2, 2>(kmap, vmap, k, s);
    return launch<64, kFp8, 2, 1, 4>(kmap, vmap, k, s);
  }
  if (d == 128) {
    if (h == 8) return launch<128, kFp8, 1, 4, 1>(kmap, vmap, k, s);
    if (h == 16) return launch<128, kFp8, 2, 4, 1>(kmap, vmap, k, s);
    if (h == 32) return launch<128, kFp8, 2, 2, 2>(kmap, vmap, k, s);
    if constexpr (kFp8) return launch<128, kFp8, 2, 1, 4>(kmap, vmap, k, s);
    return cudaErrorInvalidValue;  // bf16: more than 32 heads are the wide kernel's
  }
  if (h == 8) return launch<256, kFp8, 1, 4, 1>(kmap, vmap, k, s);
  if (h == 16) return launch<256, kFp8, 1, 4, 2>(kmap, vmap, k, s);
  if (h == 32) return launch<256, kFp8, 1, 2, 4>(kmap, vmap, k, s);
  return launch<256, kFp8, 1, 1, 8>(kmap, vmap, k, s);
}

cudaError_t launch_bf16(const CUtensorMap& kmap, const CUtensorMap& vmap, const Args& k, cudaStream_t s);
cudaError_t launch_fp8(const CUtensorMap& kmap, const CUtensorMap& vmap, const Args& k, cudaStream_t s);
cudaError_t launch_wide(const CUtensorMap& kmap, const CUtensorMap& vmap, const Args& k, cudaStream_t s);  // attn_wide.cu

}  // namespace attn
}  // namespace ci
