// Softmax attention of many query rows per request over its paged cache
// (is_attend with prompts), on the 5th-generation tensor cores.
//
// With n new tokens every key is used by up to n * G rows (G query heads share
// a KV head), so the time is that of the two products, 4 * D flops per (row,
// key) pair.  An item is (request, KV head, run of tokens whose rows fill two
// 128-row tiles A and B); per 128 keys
//   S = Q K^T   M 128 x N 128 keys x K D      (operands in shared memory)
//   O += P V    M 128 x N D x K 128 keys      (P in tensor memory, over S)
// Tile A's softmax runs while the tensor core works on tile B and the other way
// round.  12 warps, each with one job:
//   warps 0-3   softmax of tile A: one thread per row, so the row's maximum and
//               sum need no exchange between threads
//   warps 4-7   softmax of tile B
//   warps 8-10  bring Q, K and V tiles into shared memory: with bulk tensor
//               copies, a block of the paged cache at a time; where those do not
//               fit the block size with 16-byte asynchronous copies, row by row;
//               FP8 rows likewise, as bytes, and widened to fp16 from there
//               (exactly).  Rows of no key are zero
//   warp 11     one elected thread issues the MMAs
// Tensor memory (512 columns): S_A, S_B (128 each; P takes the first half of
// its S as 16-bit pairs), O_A, O_B (D each).  Shared memory: Q (2 x 128 rows),
// then a ring of 128-key tiles, K and V in turn.  Rows are stored as 64-element
// halves of 128 bytes with the 128-byte swizzle: K-major for Q and K; V's
// rows are keys, so it is the MN-major operand of the second product.
//
// As in the split kernel the items' keys are numbered in units of 128 over
// the call and every CTA of a persistent grid (one per SM) takes one run of
// them, so ragged and causal batches are balanced; items cut by a run's end
// are joined from the workspace.  The running maximum moves only when a logit
// passes it by 2^8 (see kRaise); moving it rescales O in tensor memory, which the wait for
// S already made safe: the MMA thread issued the previous O += P V before it.
// Every wait is bounded (2 s, or the call's limit): on time-out the CTA latches
// IS_ST_TIMEOUT, lets its own work in flight end, for which it waits 2 s whatever
// the limit, frees its tensor memory and returns.
//
// At head_dim 256 an item is one 128-row tile: O takes 256 columns, and tile
// B's place.
//
// Over a scaled cache (is_attend_scaled) there are 16 warps.  One finds the tiles'
// blocks and scales, two tiles at a time, and hands them on through a ring; six bring
// the codes as they are, a thread its own chunks, and widen them to fp16.  An item's
// tiles follow the last item's in that ring, so that codes are on their way across
// items.  What a softmax warp does differently is at ScaledTile.
//
// Measured (H = 8, G = 4, D = 128, bf16): two prompts of 2000-2500 tokens
// behind up to 8192, 538 GFLOP, 385 us = 1.40 PFLOP/s, 74 % of the burst rate of
// a plain library product.  128 keys of a pair of tiles are 2048 clocks of MMAs
// (64 each for M 128, N 128, K 16) and take 2900.  Leaving out the exponentials
// changes nothing; half the S products save 3 %, half the O products 2 %, half
// of the loaded bytes 8 %: shared memory feeds the MMAs (S alone reads 128
// bytes a clock) while it takes in the next tiles, and a tile's next S waits
// for its softmax (1400 clocks) and the other tile's products.  16 requests with
// 20-100 new tokens over 900-2000: 51.6 us; the start and end of an item (its first
// tiles, 64 KB of output or 128 KB of partial) cost as much as about six key
// tiles.  One request, 100 new tokens over 400: 19.5 us, the latency of this kernel
// (1 us to its run, 4 to the first S, 2 for the tiles, 2 of output) and the join.
// Over an FP8 cache the two long prompts take 560 us, 0.96 PFLOP/s: the three
// loader warps that widen the rows are the limit.  At head_dim 256 (bf16, twice
// the operations) 947 us, 1.14 PFLOP/s: with one tile, its products and its softmax
// take turns.  Over a scaled cache 606 us (INT8) and 574 us (E4M3), 0.89 and 0.94
// PFLOP/s: instructions, about 10,000 a pair of tiles at half of the issue slots, two
// thirds of them the softmax (what a group of keys shares costs as much as two of its
// weights), one third the loaders; 16 requests' prompts 67.5 us.
#pragma once

#include <cuda.h>

#include <algorithm>
#include <cfloat>
#include <cstddef>
#include <cstring>
#include <type_traits>

#include "attend.cuh"
#include "block_scan.cuh"
#include "tcgen05.cuh"

namespace isk {

namespace prompt {

constexpr int kThreads = 384;
constexpr int kKeys = 128;               // keys of a tile, and of a unit
constexpr int kLoaderWarp = 8, kLoaders = 96;
// Registers a thread: 168 at launch (65,536 / 384); the softmax warps take what
// a row of S needs, the other four give it: 2 * 192 + 120 = 3 * 168.  (208 and 88:
// the loaders and the MMA thread spill, and the long prompts take 426 us, not 406.)
constexpr int kSoftmaxRegs = 192, kOtherRegs = 120;
// Units of a CTA's run, at least.  4: one request's 100 tokens over 400 take 23.1
// us, not 21.7, over 1313 26.6, not 26.0; larger batches have longer runs anyway.
constexpr int kMinRun = 2;
// Starting and ending an item costs a CTA about as much as this many units, so
// an item counts as so many more, before its first.  Over a scaled cache a unit
// takes twice as long (3: 16 requests' prompts 68.7 us; 2: 70.0, 4 and 6: 71.9).
constexpr int kItemCost = 6, kScaledItemCost = 3;
constexpr int kMaskRing = 8;
// The form over a scaled cache has 16 warps: 0-7 softmax, 8 finds the tiles'
// blocks and scales, 9-11 bring K, 12-14 V, 15 issues the MMAs; 128 registers a thread.
constexpr int kScaledThreads = 512;
constexpr int kCodeWarps = 3;            // that bring K, and that bring V
constexpr int kCodeThreads = 2 * 32 * kCodeWarps;
// The exponents are x * sc - m in one rounding, so that they keep the error of
// the product that m was rounded by: half a step of m.  That passes a weight's
// range where m is past 2^24 (fp16) or 2^30: past this, far_weights rounds the
// product first, as it was for m.
constexpr float kFar = 4194304.f;
constexpr uint32_t kTmemAll = 512;

template <int D, bool F8, bool SCALED = false>
struct Shape {
  // Rows of an item, at most: tiles A and B; at head_dim 256 tensor memory has room for O of one.
  static constexpr int kRows = D == 256 ? 128 : 256;
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kHalves = D / 64;
  // A tile is 16 groups of 8 rows; a group holds the 64-element parts of its
  // rows one after the other, 1024 bytes each (one swizzle atom).
  static constexpr uint32_t kGroupBytes = kHalves * 1024;
  static constexpr uint32_t kTileBytes = 16 * kGroupBytes;
  static constexpr int kRing =           // K and V tiles in shared memory
      D == 256 ? 2 : SCALED ? (D == 128 ? 3 : 8) : F8 ? (D == 128 ? 3 : 5) : D == 128 ? 5 : 8;
  // FP8 rows are copied as they are, kRaw tiles ahead, and widened from there.
  static constexpr int kRaw = D == 128 ? 3 : 4;
  static constexpr uint32_t kRawBytes = F8 && !SCALED ? 128 * D : 0;
  // Scaled cache: batches of four chunks that bring a thread's part of a tile, and the place of two tiles of them.
  static constexpr int kBatches = D == 128 ? 3 : 2;
  static constexpr size_t kCodeBytes = SCALED ? 2 * kBatches * 4 * 32 * kCodeWarps * 16 : 0;
  // A tile's mask is written when its K has a place, that is once load 2 t - kRing has been released; the mask it
  // replaces has been read once V of tile t - kMaskRing, load 2 (t - kMaskRing) + 1, has been released.
  static_assert(2 * kMaskRing >= kRing + 1, "a mask is read before its place is used again");
  static constexpr size_t kSmem = 1024 + kQBytes + kRing * (size_t)kTileBytes + kRaw * (size_t)kRawBytes +
                                  kCodeBytes + (SCALED ? 0 : F8 ? 2 : 1) * 128 * 8;
  static constexpr uint32_t kOCol = 256;                      // first column of O_A; O_B follows D columns on
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// Waits for this thread's loads from tensor memory, r's among them.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24])
               :
               : "memory");
  asm volatile("" : "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
}
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32], uint32_t (&s)[32]) {
  tmem_wait_ld32(r);
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile("" : "+r"(s[i]), "+r"(s[i + 1]), "+r"(s[i + 2]), "+r"(s[i + 3]), "+r"(s[i + 4]), "+r"(s[i + 5]), "+r"(s[i + 6]), "+r"(s[i + 7]));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float max3(float x, float y, float z) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
  return r;
}
__device__ __forceinline__ unsigned long long add2_rn(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Groups of 8 tokens from group t8 on, all of head h (make_rows_map).
__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, int h, int t8, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3, %4}], "
      "[%5];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(h), "r"(t8), "r"(bar)
      : "memory");
}

// Both operands in shared memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A in tensor memory (lane = row, a column = two consecutive 16-bit elements of K).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Descriptors of 128-byte-swizzled tiles (version 1, layout type 2).  Q and K
// are K-major: groups of 8 rows follow one another (stride byte offset).  For
// O += P V the keys are K: again 8 to a group (stride byte offset), and N runs
// over the 64 elements of a row and then the halves (leading byte offset).
template <int D, bool F8>
__device__ __forceinline__ uint64_t tile_desc(uint32_t saddr, uint32_t leading) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)leading << 16) |
         ((uint64_t)(Shape<D, F8>::kGroupBytes >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// kind::f16 instruction descriptor: D fp32 (bit 4), A and B fp16 or bf16
// (bits 7, 10), B MN-major (bit 16) for V, N >> 3 at 17, M >> 4 at 24.
template <typename T>
__device__ constexpr uint32_t idesc_of(int n, bool mn_major_b) {
  constexpr uint32_t fmt = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | ((mn_major_b ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(128 >> 4) << 24);
}

// Tile t of a request: its tokens, the positions its rows see, its units.
struct Tile {
  int32_t tok0, toks;
  int32_t see;           // first position that some row sees
  int32_t kb, ke, units;
};
template <int COST>
__device__ __forceinline__ Tile tile_of(const AttendArgs& a, const Req& q, int per, int t) {
  Tile x;
  x.tok0 = t * per;
  x.toks = min(per, q.n - x.tok0);
  const int32_t p0 = q.seq - q.n + x.tok0;           // position of the first token
  x.ke = min(q.ke, p0 + x.toks);
  // whole tiles from position 0 on, so that tiles line up with the cache's blocks
  x.see = a.window > 0 ? (int32_t)max((int64_t)p0 - a.window + 1, (int64_t)0) : 0;
  x.kb = x.see / kKeys * kKeys;
  x.units = COST + max(1, (x.ke - x.kb + kKeys - 1) / kKeys);
  return x;
}
template <int COST>
__device__ __forceinline__ int64_t units_of_request(const AttendArgs& a, const Req& q, int per) {
  int64_t sum = 0;
  for (int t = 0; t * per < q.n; ++t) sum += tile_of<COST>(a, q, per, t).units;
  return sum * a.H;
}

// One segment (a run's share of one item) as its workers need it, handed from
// one loader thread to all warps through a ring in shared memory: the walk costs
// the others no registers, and the CTA agrees on its segments whatever happens
// to the caller's arrays meanwhile.
struct Segment {
  int32_t tiles;         // -1: the run has ended
  int32_t k_lo, k_hi, rows;
  int32_t k_see;         // first key that some row of the item sees
  int32_t r;
  int32_t lim0;          // position of the item's first token
  int32_t head;
  int32_t row0;          // first query row
  int32_t slot;          // of the partial result; -1: the item is whole
};
constexpr int kSegments = 4;

// The segments of a CTA's run, walked by one thread.
template <int COST>
struct Walk {
  int64_t u, u_end, u_first, run, base;  // base: first unit of tile (r, t)
  int r, t;
  Req q;
  Tile x;
  // of the current segment
  int head, k_lo, k_hi, rows, parts;
  bool whole, begins, at_start;
  bool crosses;                          // the run's last item began here and goes on in the next CTA

  // From the first tile of request `req`, whose first unit is number `first`.
  __device__ __forceinline__ void start(const AttendArgs& a, int per, int64_t run_, int64_t u0, int64_t u1, int req, int64_t first) {
    run = run_;
    u = u_first = u0;
    u_end = u1;
    r = req;
    base = first;
    t = 0;
    q = read_request(a, r, false);
    x = tile_of<COST>(a, q, per, 0);
    crosses = false;
  }
  __device__ __forceinline__ bool next(const AttendArgs& a, int per) {
    while (u < u_end) {
      // the tile that unit u lies in
      while (true) {
        if (t * per < q.n) {
          const int64_t n = (int64_t)a.H * x.units;
          if (u < base + n) break;
          base += n;
          ++t;
        } else {
          if (++r >= a.R) return false;  // the lengths have changed under the call
          t = 0;
          q = read_request(a, r, false);
        }
        if (t * per < q.n) x = tile_of<COST>(a, q, per, t);
      }
      head = (int)div_small(u - base, x.units);
      const int64_t item0 = base + (int64_t)head * x.units;
      const int ua = max((int)(u - item0) - COST, 0), ub = (int)min((int64_t)x.units, u_end - item0) - COST;
      at_start = u == u_first;
      u = item0 + ub + COST;
      if (ub <= 0) continue;             // none of its keys yet: the item begins in the next CTA
      begins = ua == 0;
      whole = begins && ub == x.units - COST;
      // within the grid, whatever became of the lengths since they were added up
      parts = (int)(min(div_small(item0 + x.units - 1, run), (int64_t)gridDim.x - 1) - (int64_t)blockIdx.x) + 1;
      k_lo = x.kb + ua * kKeys;
      k_hi = min(x.ke, x.kb + ub * kKeys);
      rows = x.toks * a.G;
      return true;
    }
    return false;
  }
  __device__ __forceinline__ int tiles() const { return k_hi > k_lo ? (k_hi - k_lo + kKeys - 1) / kKeys : 0; }
  // The next segment for its workers, and what the join has to know of an item that crosses runs.
  __device__ __forceinline__ void next_into(const AttendArgs& a, int per, Segment& g) {
    if (next(a, per)) {
      g.tiles = tiles();
      g.k_lo = k_lo;
      g.k_hi = k_hi;
      g.k_see = x.see;
      g.rows = rows;
      g.r = r;
      g.lim0 = q.seq - q.n + x.tok0;
      g.head = head;
      g.row0 = q.row0 + x.tok0;
      g.slot = whole ? -1 : 2 * blockIdx.x + (at_start ? 0 : 1);
      crosses = begins && !whole;
      if (crosses) {
        JoinRecord* rec = record_of(a, blockIdx.x);
        rec->parts = parts;
        rec->slot0 = g.slot;
        rec->row0 = q.row0;
        rec->head = head;
        rec->rho0 = x.tok0 * a.G;
        rec->rows = rows;
      }
    } else {
      g.tiles = -1;
      if (!crosses) record_of(a, blockIdx.x)->parts = 0;
    }
  }
};

struct Bars {
  uint64_t q_full, q_empty, done, v_tail;
  uint64_t seg_full[kSegments], seg_empty[kSegments];
  uint64_t kv_full[8], kv_empty[8];
  uint64_t s_full[2], p_full[2][2], o_full[2];   // P in two halves of 64 keys
  uint64_t mask_full[kMaskRing];
};
struct ScaledBars {      // beside them, over a scaled cache
  uint64_t tile_empty[kMaskRing], q_raw;
};

// Bits lo .. hi - 1 of a 32-bit word whose bit 0 is position `at`.
__device__ __forceinline__ uint32_t bits_between(int at, int lo, int hi) {
  const int l = max(lo - at, 0), h = min(hi - at, 32);
  if (h <= l) return 0u;
  return (h - l == 32 ? 0xffffffffu : ((1u << (h - l)) - 1u)) << l;
}

// Eight 8-bit elements as eight fp16 values, exact.
template <bool I8>
__device__ __forceinline__ uint4 widen8(uint32_t lo, uint32_t hi) {
  uint4 r;
  codes_f16x4<I8>(lo, r.x, r.y);
  codes_f16x4<I8>(hi, r.z, r.w);
  return r;
}

// Scaled cache: what eight keys of a block share is K scale, log2 of the V scale
// and 1 / V scale.  A row's factor to their logits stays finite, so that 0 times
// it is 0, and at the smallest normal number or above, so that a hidden logit, -inf,
// times it is -inf (sc > 0; a smaller factor makes every weight 1 in any case).
constexpr int kGroup = 8, kGroups = kKeys / kGroup;
// A tile of keys as its loaders need it.  The tiles of a CTA's run follow one
// another here whatever their segments, so that a tile's codes are on their way
// while those of the tile before it are widened.
struct TileInfo {
  int64_t at[kGroups];   // first K row of the group, in bytes; 0 where no block of it counts
  uint32_t named;        // a bit a group: one does
  int32_t lo, hi;        // its keys that some row may see
  int32_t rows;          // query rows of the segment that it begins, 0: goes on with one; -1: the run has ended
  int32_t row0, head;    // of that segment
};
__device__ __forceinline__ float group_factor(float sc, float ks) { return fminf(fmaxf(sc * ks, FLT_MIN), FLT_MAX); }
__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// 32 bytes to a 32-byte-aligned address.
__device__ __forceinline__ void st_sector(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Where 16-byte chunk c (8 elements) of row `row` lies in a tile.
template <int D>
__device__ __forceinline__ uint32_t at_chunk(int row, int c) {
  return (uint32_t)(row >> 3) * Shape<D, false>::kGroupBytes + (uint32_t)(c >> 3) * 1024u + (uint32_t)(row & 7) * 128u +
         (uint32_t)(((c & 7) ^ (row & 7)) * 16);
}

// A query row, bf16 in a tile, becomes fp16 times a power of two that brings its
// largest element to [2^14, 2^15); *unscale is the inverse.
template <int D>
__device__ __forceinline__ void scale_query_row(uint32_t tile, int row, bool live, float* unscale) {
  constexpr int C = D / 8;
  float down = 1.f;
  if (live) {
    __nv_bfloat162 big(0.f, 0.f);
    auto larger = [&](uint32_t w) {
      w &= 0x7fff7fffu;
      big = __hmax2(big, *reinterpret_cast<const __nv_bfloat162*>(&w));
    };
#pragma unroll 4
    for (int k = 0; k < C; ++k) {
      const uint4 x = ld_shared_v4(tile + at_chunk<D>(row, k));
      larger(x.x);
      larger(x.y);
      larger(x.z);
      larger(x.w);
    }
    const float most = fmaxf(__low2float(big), __high2float(big));
    const int shift = most > 0.f && most < INFINITY ? min(14 - (int)(((__float_as_uint(most) >> 23) & 255u) - 127), 120) : 0;
    const float up = __uint_as_float((uint32_t)(127 + shift) << 23);
    down = __uint_as_float((uint32_t)(127 - shift) << 23);
#pragma unroll 1
    for (int k0 = 0; k0 < C; k0 += 4) {
      uint4 x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = ld_shared_v4(tile + at_chunk<D>(row, k0 + k));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float f[8];
        Vec<__nv_bfloat16>::unpack(x[k], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= up;
        st_shared_v4(tile + at_chunk<D>(row, k0 + k), Vec<__half>::pack(f));
      }
    }
  }
  *unscale = down;
}

// The weights of a tile with rows past kFar: S (logits before their scale) once
// more from tensor memory, weights over it and their sum added to l.  Of 32
// logits S is read before the 16 columns of their weights, which lie before the
// next ones', are written.  A function of its own, since inside the loop it costs
// the other rows registers: the long prompts take 403 us instead of 392.
template <typename W>
__device__ __noinline__ float far_weights(uint32_t s_col, float sc, float m, float l, uint4 named, int key0, int low, int end,
                                          uint32_t p_full, int lane) {
  const float mz = m == -INFINITY ? 0.f : m;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t y[32], p[16];
    tmem_ld32(s_col + 32 * c, y);
    tmem_wait_ld();
    const uint32_t word = c == 0 ? named.x : c == 1 ? named.y : c == 2 ? named.z : named.w;
    const uint32_t see = word & bits_between(key0 + 32 * c, low, end);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float w[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        w[e] = (see >> (2 * i + e)) & 1u ? ex2(__fsub_rn(__fmul_rn(__uint_as_float(y[2 * i + e]), sc), mz)) : 0.f;
      l += w[0] + w[1];
      p[i] = Vec<W>::pack2(w[0], w[1]);
    }
    tmem_st16(s_col + 16 * c, p);
    tmem_wait_st();
    if (c & 1) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full + 8 * (c >> 1));
    }
  }
  return l;
}

// Scaled cache, one tile of a row: S (logits before their scale) becomes weights
// over it.  A weight holds its key's V scale, x = logit + log2 of it, and the sum
// takes that back by groups of GROUP: sixteen where blocks are whole sixteens (606 us
// at the long prompts' sizes, 624 with eight).  S is read twice, for the maximum of x and
// for the weights, in loops of 64 and 32 columns: with all 128 unrolled between one
// read and its use the warps of an SM, each in a part of the code of its own,
// waited for instructions in a quarter of their time.  Of 32 logits S is read
// before the 16 columns of their weights, which lie before the next ones', are
// written.
template <int D, int GROUP>
struct ScaledTile {
  uint32_t s_col;
  float sc;
  const uint32_t* named;
  const float4* groups;
  int key0, low, end;
  bool check;
  uint32_t p_full;
  int lane;

  __device__ __forceinline__ void hide(uint32_t (&y)[32], int c) const {
    if (!check) return;
    const uint32_t see = named[c] & bits_between(key0 + 32 * c, low, end);
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (!((see >> i) & 1u)) y[i] = 0xff800000u;
  }
  __device__ __forceinline__ float top(uint32_t (&y)[32], int c) const {
    hide(y, c);
    float x[32 / GROUP];
#pragma unroll
    for (int g = 0; g < 32 / GROUP; ++g) {
      const float4 k = groups[(c * 32 + g * GROUP) / kGroup];
      const uint32_t* v = y + g * GROUP;
      float x0 = max3(__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]));
      const float x1 = max3(__uint_as_float(v[3]), __uint_as_float(v[4]), __uint_as_float(v[5]));
      x0 = max3(x0, __uint_as_float(v[6]), __uint_as_float(v[7]));
#pragma unroll
      for (int i = 8; i < GROUP; i += 2) x0 = max3(x0, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
      x[g] = fmaf(fmaxf(x0, x1), group_factor(sc, k.x), k.y);   // grows with the logits of a group
    }
    float most = x[0];
#pragma unroll
    for (int g = 1; g < 32 / GROUP; ++g) most = fmaxf(most, x[g]);
    return most;
  }
  // The weights of all columns, the first 32 of which are on their way to y, and their sum on top of l.  FAR: exponents
  // rounded as they were for the maximum (see kFar).
  template <typename W, bool FAR>
  __device__ __forceinline__ float weights(uint32_t (&y)[32], float mz, float l) const {
    unsigned long long sum = pk2(l, 0.f);
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      float4 k[32 / GROUP];
#pragma unroll
      for (int g = 0; g < 32 / GROUP; ++g) k[g] = groups[(c * 32 + g * GROUP) / kGroup];
      tmem_wait_ld32(y);
      hide(y, c);
      float x[32];
#pragma unroll
      for (int g = 0; g < 32 / GROUP; ++g) {
        const float factor = group_factor(sc, k[g].x), off = FAR ? k[g].y : k[g].y - mz;
        const unsigned long long factor2 = pk2(factor, factor), off2 = pk2(off, off);
#pragma unroll
        for (int i = g * GROUP; i < (g + 1) * GROUP; i += 2)
          upk2(fma2_rn(pk2(__uint_as_float(y[i]), __uint_as_float(y[i + 1])), factor2, off2), x[i], x[i + 1]);
      }
      if (c < 3) tmem_ld32(s_col + 32 * (c + 1), y);
      uint32_t p[16];
#pragma unroll
      for (int g = 0; g < 32 / GROUP; ++g) {
        unsigned long long of_group = 0ull;
#pragma unroll
        for (int i = g * GROUP; i < (g + 1) * GROUP; i += 2) {
          const float y0 = ex2(FAR ? __fsub_rn(x[i], mz) : x[i]), y1 = ex2(FAR ? __fsub_rn(x[i + 1], mz) : x[i + 1]);
          of_group = i == g * GROUP ? pk2(y0, y1) : add2_rn(of_group, pk2(y0, y1));
          p[i / 2] = Vec<W>::pack2(y0, y1);
        }
        sum = fma2_rn(of_group, pk2(k[g].z, k[g].z), sum);
      }
      tmem_st16(s_col + 16 * c, p);
      if (c & 1) {                       // half of the keys: their part of O += P V can start
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 8 * (c >> 1));
      }
    }
    float l0, l1;
    upk2(sum, l0, l1);
    return l0 + l1;
  }
  // The tile's weights for maximum m and sum l, both brought up to date with O.
  template <typename W>
  __device__ __forceinline__ float run(uint32_t o_col, bool has_o, float& m, float l) const {
    uint32_t a[32], b[32];
    float most = -INFINITY;
    tmem_ld32(s_col, a);
    tmem_ld32(s_col + 32, b);
#pragma unroll 1
    for (int c = 0; c < 4; c += 2) {
      tmem_wait_ld32(a, b);
      most = fmaxf(most, top(a, c));
      tmem_ld32(s_col + (c ? 0 : 64), a);
      most = fmaxf(most, top(b, c + 1));
      if (c == 0) tmem_ld32(s_col + 96, b);
    }
    // A logit past the bound moves m; far rows come here with every tile.
    if (__any_sync(0xffffffffu, most > (fabsf(m) > kFar ? -INFINITY : lazy_bound<W>(m)))) {
      const float mn = fmaxf(m, most - kRaise<W>);
      const float f = mn == -INFINITY ? 1.f : ex2(m - mn);
      m = mn;
      l *= f;
      if (has_o) {
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t y[16];
          tmem_ld16(o_col + 16 * c, y);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
          tmem_st16(o_col + 16 * c, y);
        }
      }
      if (__any_sync(0xffffffffu, fabsf(m) > kFar && m > -INFINITY)) return weights<W, true>(a, m == -INFINITY ? 0.f : m, l);
    }
    return weights<W, false>(a, m == -INFINITY ? 0.f : m, l);
  }
};

constexpr int threads_of(CacheKind kind) { return kind == kCacheScaledE4m3 || kind == kCacheScaledInt8 ? kScaledThreads : kThreads; }

// LIMITED: the limit of the waits is the call's.  (As a variable in the ordinary form it costs 16 prompts 1.2 us of 53.4.)
template <typename T, CacheKind KIND, int D, bool LIMITED, int GROUP>
__global__ void __launch_bounds__(threads_of(KIND), 1) attend_prompt_kernel(const AttendArgs a, int per, int box,
                                                                           const __grid_constant__ CUtensorMap rows_map) {
  constexpr bool F8 = KIND != kCachePlain, kInt8 = KIND == kCacheScaledInt8;   // F8: 8-bit elements
  constexpr bool kScaled = KIND == kCacheScaledE4m3 || KIND == kCacheScaledInt8;
  using S = Shape<D, F8, kScaled>;
  constexpr int kCost = kScaled ? kScaledItemCost : kItemCost;
  constexpr int kThreads = threads_of(KIND), kMmaWarp = kThreads / 32 - 1;
  const uint64_t limit_ns = LIMITED ? a.wait_ns : kWaitBudgetNs;
  // FP8 keys and values are exact in fp16, and a bf16 query row scaled by a power of two (undone in the logits) loses
  // 2^-39 of its largest element at most: with an FP8 cache both products are taken in fp16.
  using W = typename std::conditional<F8, __half, T>::type;
  constexpr bool kShift = F8 && std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) Bars bars;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ uint32_t s_bulk[8];                       // of both loader warps' `bulk` the larger, after a time-out
  __shared__ __align__(16) uint32_t s_mask[kMaskRing][4];
  __shared__ uint32_t s_raw_mask[S::kRaw][4];
  __shared__ float s_unscale[kShift ? S::kRows : 1];
  __shared__ float4 s_group[kScaled ? kMaskRing : 1][kScaled ? kGroups : 1];
  __shared__ TileInfo s_tile[kScaled ? kMaskRing : 1];
  __shared__ __align__(8) ScaledBars more;             // the plain forms, which fill an SM's shared memory, use none of the three
  __shared__ int64_t scratch[33];
  __shared__ int64_t s_base;
  __shared__ int32_t s_req;
  __shared__ Segment s_seg[kSegments];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &s_abort;
  const uint32_t tiles0 = (smem_addr(smem_raw) + 1023u) & ~1023u;     // Q_A, Q_B, then the ring
  const uint32_t ring0 = tiles0 + S::kQBytes;
  long long* s_off = reinterpret_cast<long long*>(smem_raw + (ring0 - smem_addr(smem_raw)) + S::kRing * S::kTileBytes + S::kRaw * S::kRawBytes);

  if (warp == kMmaWarp) {
    tmem_alloc(smem_addr(&s_tmem), kTmemAll);
    tmem_relinquish();
  }
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < 8; ++i) s_bulk[i] = 0;
    mbar_init(smem_addr(&bars.q_full), kScaled ? kCodeThreads : kLoaders);
    if constexpr (kScaled) {
      mbar_init(smem_addr(&more.q_raw), kCodeThreads);
      for (int i = 0; i < kMaskRing; ++i) mbar_init(smem_addr(&more.tile_empty[i]), 1);
    }
    mbar_init(smem_addr(&bars.q_empty), kShift ? 9 : 1);   // the last logits; eight softmax warps that read s_unscale
    mbar_init(smem_addr(&bars.done), 1);
    mbar_init(smem_addr(&bars.v_tail), 1);
    for (int i = 0; i < S::kRing; ++i) {
      mbar_init(smem_addr(&bars.kv_full[i]), F8 ? kLoaders / 32 : 1);
      mbar_init(smem_addr(&bars.kv_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&bars.s_full[i]), 1);
      mbar_init(smem_addr(&bars.p_full[i][0]), 4);
      mbar_init(smem_addr(&bars.p_full[i][1]), 4);
      mbar_init(smem_addr(&bars.o_full[i]), 1);
    }
    for (int i = 0; i < kMaskRing; ++i) mbar_init(smem_addr(&bars.mask_full[i]), 1);
    for (int i = 0; i < kSegments; ++i) {
      mbar_init(smem_addr(&bars.seg_full[i]), 1);
      mbar_init(smem_addr(&bars.seg_empty[i]), 9);     // eight softmax warps, the MMA warp
    }
    fence_mbar_init();
    if (box > 0) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&rows_map)) : "memory");
  }
  pdl_wait();
  pdl_trigger();

  // This CTA's run of units.
  const int share = (a.R + kThreads - 1) / kThreads;
  const int r0 = min(a.R, tid * share), r1 = min(a.R, r0 + share);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) mine += units_of_request<kCost>(a, read_request(a, r, blockIdx.x == 0), per);
  int64_t total;
  int64_t at = block_exclusive_scan(mine, scratch, &total);
  const int64_t run = max((int64_t)kMinRun, div_small(total + gridDim.x - 1, gridDim.x));
  const int64_t u0 = (int64_t)blockIdx.x * run, u1 = min(total, u0 + run);
  const bool idle = u0 >= u1;
  if (!idle && at <= u0 && u0 < at + mine) {
    for (int r = r0; r < r1; ++r) {
      const int64_t n = units_of_request<kCost>(a, read_request(a, r, false), per);
      if (u0 < at + n || r == r1 - 1) {
        s_req = r;
        s_base = at;
        break;
      }
      at += n;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  if (idle) {
    if (tid == 0) record_of(a, blockIdx.x)->parts = 0;
  } else {
    if constexpr (!kScaled) {
      if (warp < kLoaderWarp)
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
      else
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    }

    if (warp < kLoaderWarp) {
      // ---- softmax ------------------------------------------------------------
      const int side = warp >> 2;                      // 0: tile A, 1: tile B
      const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
      const uint32_t s_col = tmem + lanes + 128u * side, o_col = tmem + lanes + S::kOCol + (uint32_t)(D * side);
      // Never 0: a hidden logit is -inf times it.  (Below the smallest normal number every weight is 1 in any case.)
      const float sc0 = a.scale * kLog2e;
      const int row = side * 128 + (warp & 3) * 32 + lane, tok = row / a.G;
      uint32_t n_s = 0, n_o = 0, n_mask = 0, n_q = 0;  // phases consumed
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = __all_sync(0xffffffffu, ok && wait_or_abort(smem_addr(bar), parity, abort_flag, limit_ns));
        return ok;
      };
      for (uint32_t n_seg = 0;; ++n_seg) {
        if (!wait(&bars.seg_full[n_seg % kSegments], (n_seg / kSegments) & 1u)) break;
        const Segment& g = s_seg[n_seg % kSegments];
        const int n_tiles = g.tiles;
        if (n_tiles < 0) break;
        const bool has = g.rows > 128 * side;          // the side has rows
        const bool live = row < g.rows;
        // The row's last key, and the warp's smallest and largest, for skipping the masks.
        const int lim = live ? g.lim0 + tok : -1;
        const int lim_lo = __reduce_min_sync(0xffffffffu, live ? lim : INT32_MAX);
        const int lim_hi = __reduce_max_sync(0xffffffffu, lim);
        const int low = a.window > 0 ? (int)max((int64_t)lim - a.window + 1, (int64_t)0) : 0;
        const int low_hi = a.window > 0 ? (int)max((int64_t)lim_hi - a.window + 1, (int64_t)0) : 0;
        float m = -INFINITY, l = 0.f, sc = fmaxf(sc0, FLT_MIN);
        if (kShift && n_tiles > 0) {
          if (!wait(&bars.q_full, n_q & 1u)) break;
          ++n_q;
          sc = fmaxf(sc0 * s_unscale[row], FLT_MIN);
          // A segment of one tile may have its logits before these warps, still at the last one's output, come here:
          // the next query rows' factors, and the next phase of q_full, have to wait for them.
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&bars.q_empty));
        }
        if (!has) n_mask += n_tiles;
        for (int j = 0, key0 = g.k_lo; has && j < n_tiles; ++j, ++n_mask, key0 += kKeys) {
          const int slot = n_mask % kMaskRing;
          if (!wait(&bars.mask_full[slot], (n_mask / kMaskRing) & 1u) || !wait(&bars.s_full[side], n_s & 1u)) break;
          ++n_s;
          tc_fence_after();
          if constexpr (kScaled) {
            const uint4 named = *reinterpret_cast<const uint4*>(s_mask[slot]);
            const bool check = (named.x & named.y & named.z & named.w) != 0xffffffffu || key0 + kKeys - 1 > lim_lo || key0 < low_hi;
            const ScaledTile<D, GROUP> tile{s_col, sc, s_mask[slot], s_group[slot], key0, low, lim + 1, check, smem_addr(&bars.p_full[side][0]), lane};
            l = tile.template run<W>(o_col, j > 0, m, l);
            continue;
          }
          uint32_t x[4][32];
          tmem_ld32(s_col, x[0]);
          tmem_ld32(s_col + 32, x[1]);
          const uint4 mw = *reinterpret_cast<const uint4*>(s_mask[slot]);
          const bool check = (mw.x & mw.y & mw.z & mw.w) != 0xffffffffu || key0 + kKeys - 1 > lim_lo || key0 < low_hi;
          auto hide = [&](uint32_t(&y)[32], uint32_t word, int at) {
            const uint32_t see = word & bits_between(at, low, lim + 1);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!((see >> i) & 1u)) y[i] = 0xff800000u;
          };
          auto top = [](const uint32_t(&y)[32]) {
            float t0 = max3(__uint_as_float(y[0]), __uint_as_float(y[1]), __uint_as_float(y[2]));
            float t1 = max3(__uint_as_float(y[3]), __uint_as_float(y[4]), __uint_as_float(y[5]));
#pragma unroll
            for (int i = 6; i + 3 < 32; i += 4) {
              t0 = max3(t0, __uint_as_float(y[i]), __uint_as_float(y[i + 1]));
              t1 = max3(t1, __uint_as_float(y[i + 2]), __uint_as_float(y[i + 3]));
            }
            return max3(max3(t0, t1, __uint_as_float(y[30])), __uint_as_float(y[31]), t0);
          };
          tmem_wait_ld();
          tmem_ld32(s_col + 64, x[2]);
          tmem_ld32(s_col + 96, x[3]);
          if (check) {
            hide(x[0], mw.x, key0);
            hide(x[1], mw.y, key0 + 32);
          }
          float mx = fmaxf(top(x[0]), top(x[1]));
          tmem_wait_ld();
          if (check) {
            hide(x[2], mw.z, key0 + 64);
            hide(x[3], mw.w, key0 + 96);
          }
          mx = __fmul_rn(fmaxf(mx, fmaxf(top(x[2]), top(x[3]))), sc);   // sc > 0
          // A logit past the bound moves m; far rows come here with every tile.
          if (__any_sync(0xffffffffu, mx > (fabsf(m) > kFar ? -INFINITY : lazy_bound<W>(m)))) {
            const float mn = fmaxf(m, mx - kRaise<W>);
            const float f = mn == -INFINITY ? 1.f : ex2(m - mn);
            m = mn;
            l *= f;
            if (j > 0) {
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t y[16];
                tmem_ld16(o_col + 16 * c, y);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * f);
                tmem_st16(o_col + 16 * c, y);
              }
            }
            if (__any_sync(0xffffffffu, fabsf(m) > kFar && m > -INFINITY)) {
              l = far_weights<W>(s_col, sc, m, l, mw, key0, low, lim + 1, smem_addr(&bars.p_full[side][0]), lane);
              continue;
            }
          }
          const float mz = m == -INFINITY ? 0.f : m;
          const unsigned long long sc2 = pk2(sc, sc), mz2 = pk2(-mz, -mz);
          unsigned long long sum = pk2(l, 0.f);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float y0, y1;
              upk2(fma2_rn(pk2(__uint_as_float(x[c][2 * i]), __uint_as_float(x[c][2 * i + 1])), sc2, mz2), y0, y1);
              y0 = ex2(y0);
              y1 = ex2(y1);
              sum = add2_rn(sum, pk2(y0, y1));
              p[i] = Vec<W>::pack2(y0, y1);
            }
            tmem_st16(s_col + 16 * c, p);
            if (c & 1) {                               // half of the keys: their part of O += P V can start
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_addr(&bars.p_full[side][c >> 1]));
            }
          }
          float l0, l1;
          upk2(sum, l0, l1);
          l = l0 + l1;
        }
        if (!ok) break;
        // The segment's output.
        if (has && n_tiles > 0) {
          if (!wait(&bars.o_full[side], n_o & 1u)) break;
          ++n_o;
          tc_fence_after();
        }
        if (has) {
          const int part_slot = g.slot;
          const float inv = l == 0.f ? 0.f : a.v_scale / l;
          // A thread holds a row and writes it in whole 32-byte sectors.  (Exchanging pieces between four lanes so that a
          // store covers 64 bytes of eight rows took four times as long: the shuffles cost more than the sectors.)
          T* dst = reinterpret_cast<T*>(a.out) +
                   ((size_t)(g.row0 + (live ? tok : 0)) * a.Hq + (size_t)g.head * a.G + (live ? row - tok * a.G : 0)) * D;
          auto* part = partial_of<PartialByEights<S::kRows, D>>(a, max(part_slot, 0));
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t y[32];
            if (n_tiles > 0) {
              tmem_ld32(o_col + 32 * c, y);
              tmem_wait_ld();
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] = 0u;
            }
            if (live && part_slot < 0) {
              uint32_t z[16];
#pragma unroll
              for (int i = 0; i < 16; ++i)
                z[i] = l == 0.f ? 0u : Vec<T>::pack2(__uint_as_float(y[2 * i]) * inv, __uint_as_float(y[2 * i + 1]) * inv);
              st_sector(dst + 32 * c, z);
              st_sector(dst + 32 * c + 16, z + 8);
            } else if (live) {
#pragma unroll
              for (int v = 0; v < 4; ++v) st_sector(part->o[4 * c + v][row], y + 8 * v);
            }
            __syncwarp();
          }
          if (live && part_slot < 0) {
            if (a.lse)
              a.lse[(size_t)(g.row0 + tok) * a.Hq + (size_t)g.head * a.G + (row - tok * a.G)] =
                  l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
          } else if (live) {
            part->m[row] = m;
            part->l[row] = l;
          }
        }
        // The next segment's first O += P V follows this side's next p_full, so O has been read by then.
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&bars.seg_empty[n_seg % kSegments]));
      }
      if (!ok) *abort_flag = 1;
    } else if (kScaled && warp == kLoaderWarp) {
      // ---- scaled cache: segments, and the tiles' blocks, masks and scales ---------
      if constexpr (kScaled) {
        Walk<kCost> w;                                 // the first lane's
        bool ok = true;
        if (lane == 0) w.start(a, per, run, u0, u1, s_req, s_base);
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          ok = __all_sync(0xffffffffu, ok && wait_or_abort(smem_addr(bar), parity, abort_flag, limit_ns));
          return ok;
        };
        uint32_t n_tile = 0;
        for (uint32_t n_seg = 0;; ++n_seg) {
          const uint32_t seg = n_seg % kSegments;
          if (!wait(&bars.seg_empty[seg], ((n_seg / kSegments) & 1u) ^ 1u)) break;
          Segment& g = s_seg[seg];
          if (lane == 0) w.next_into(a, per, g);
          __syncwarp();
          const int n_tiles = g.tiles, k_lo = g.k_lo, k_hi = g.k_hi, k_see = g.k_see, rows = g.rows, head = g.head, row_at = g.row0;
          const int32_t* table = a.block_table + (size_t)g.r * a.max_blocks;
          if (lane == 0) mbar_arrive(smem_addr(&bars.seg_full[seg]));
          if (n_tiles < 0) break;
          // Two tiles at a time: half a warp each, a lane to a group.
          const int half = lane >> 4, grp = lane & 15;
          for (int j0 = 0; j0 < n_tiles; j0 += 2) {
            const int j = j0 + half, key0 = k_lo + j * kKeys, p = key0 + grp * kGroup;
            int64_t at = -1;
            float ks = 1.f, vs = 1.f;
            // (of a group of which any key is seen, all eights: the first's scales are the group's)
            if (j < n_tiles && (p & -GROUP) + GROUP > k_see && p < k_hi) {
              const int b = block_of(a, p);
              const int32_t id = table[b];
              if (id >= 0 && id < a.num_blocks) {
                const float* s = a.scales + (int64_t)id * a.H + head;
                ks = s[0];
                vs = s[(int64_t)a.num_blocks * a.H];
                at = (((int64_t)id * a.block_size + (p - b * a.block_size)) * a.H + head) * D;
              } else {
                latch(a.status, IS_ST_BLOCK_ID);
              }
            }
            if (!scale_ok(ks) || !scale_ok(vs)) {      // hidden, as if the table did not name it
              latch(a.status, IS_ST_SCALE);
              at = -1;
              ks = vs = 1.f;
            }
            const uint32_t named = __ballot_sync(0xffffffffu, at >= 0) >> (16 * half);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (j0 + h >= n_tiles) break;
              const uint32_t slot = n_tile % kMaskRing;
              if (!wait(&more.tile_empty[slot], ((n_tile / kMaskRing) & 1u) ^ 1u)) break;
              if (half == h) {
                TileInfo& info = s_tile[slot];
                const int lo = max(0, k_see - key0), hi = min(kKeys, k_hi - key0);
                info.at[grp] = max(at, (int64_t)0);
                s_group[slot][grp] = key_scales(ks, vs);
                if (grp < 4) {                         // a bit a key of 32: four groups' bits to bytes, and the range
                  const uint32_t four = (named >> (4 * grp)) & 15u;
                  s_mask[slot][grp] = ((four * 0x00204081u) & 0x01010101u) * 0xffu & bits_between(32 * grp, lo, hi);
                }
                if (grp == 0) {
                  info.named = named & 0xffffu;
                  info.lo = lo;
                  info.hi = hi;
                  info.rows = j0 + h == 0 ? rows : 0;
                  info.row0 = row_at;
                  info.head = head;
                }
              }
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_addr(&bars.mask_full[slot]));
              ++n_tile;
            }
            if (!ok) break;
          }
          if (!ok) break;
        }
        const uint32_t slot = n_tile % kMaskRing;
        if (ok && wait(&more.tile_empty[slot], ((n_tile / kMaskRing) & 1u) ^ 1u)) {
          if (lane == 0) {
            s_tile[slot].rows = -1;
            mbar_arrive(smem_addr(&bars.mask_full[slot]));
          }
        }
        if (!ok) *abort_flag = 1;
      }
    } else if (kScaled && warp < kMmaWarp) {
      // ---- scaled cache: codes from the cache to fp16 tiles --------------------------
      // Three warps bring K, three V.  A lane has one 16-byte chunk of each of its rows in a place of its own in shared
      // memory; when it has widened and stored four, it asks for the same four of the next tile, which so have a tile's
      // time to arrive.  (In registers they would have no second trip, but would have to be unrolled: see ScaledTile.)
      // Eight lanes of a store (a phase of the shared memory) are four even chunks of a row and of its neighbour, whose
      // swizzle brings them to the odd places: no bank twice.
      if constexpr (kScaled) {
        constexpr int C = D / 16, RW = 32 / C, kUnits = kKeys / RW;   // chunks of a row; a warp's rows
        constexpr int kBatch = 4, kBatches = S::kBatches, kCodeGroup = 32 * kCodeWarps;
        const int kv = warp >= kLoaderWarp + 1 + kCodeWarps, w = (warp - kLoaderWarp - 1) % kCodeWarps;
        const int lt = tid - (kLoaderWarp + 1) * 32;   // 0 .. kCodeThreads - 1
        const int c = (lane & 3) + (C == 8 ? (lane >> 3 & 1) * 4 : 0);
        const int rw = (lane >> 2 & 1) + (C == 8 ? lane >> 4 : lane >> 3) * 2;       // row of the warp's RW
        // Unit u = w + 3 k of RW rows, k = 4 b + i.  With RW 4 two units are a group of 8: units of odd k lie in the other
        // half of one.  Of pair x = i % 2: row in its group, first group (b = i / 2 = 0), bytes from the group to the chunk.
        constexpr int X = RW == 4 ? 2 : 1, kGroupStep = RW == 4 ? 3 : 3;             // groups from i to i + X
        int in_group[X];
        uint32_t put[X], row_off[X];
        int group0[X];
#pragma unroll
        for (int x = 0; x < X; ++x) {
          in_group[x] = RW == 4 ? rw + 4 * ((w + x) & 1) : rw;
          group0[x] = RW == 4 ? (w + 3 * x) >> 1 : w;
          put[x] = group0[x] * S::kGroupBytes + at_chunk<D>(in_group[x], 2 * c);
          row_off[x] = (uint32_t)(in_group[x] * a.H * D) + c * 16;
        }
        const uint8_t* src = a.k_cache + (kv ? a.v_offset : 0);
        // A thread's chunks as they are, 16 bytes for each k.
        const uint32_t raw = ring0 + S::kRing * S::kTileBytes + (kv * kBatches * kBatch * kCodeGroup + lt % kCodeGroup) * 16;
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
          ok = __all_sync(0xffffffffu, ok && wait_or_abort(smem_addr(bar), parity, abort_flag, limit_ns));
          return ok;
        };
        // Asks for batch b of a tile; `named` and `whole` are the tile's.  (A group without a block stands at 0 and is not
        // read; blocks are whole eights, so there are eight rows.)
        auto fetch = [&](const TileInfo& t, uint32_t named, bool whole, int b) {
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int x = i % X, group = group0[x] + (b * (kBatch / X) + i / X) * kGroupStep;
            if (w + kCodeWarps * (kBatch * b + i) >= kUnits) break;
            bool in = (named >> group) & 1u;
            if (!whole) {
              const int row = group * kGroup + in_group[x];
              in = in && row >= t.lo && row < t.hi;
            }
            cp_async16(raw + (kBatch * b + i) * kCodeGroup * 16, src + t.at[group] + row_off[x], in);
          }
        };
        auto load_q = [&](const TileInfo& t, uint32_t n_q) {
          if (!wait(&bars.q_empty, (n_q & 1u) ^ 1u)) return;
          const int rows = t.rows;
          constexpr int QC = D / 8, QP = kCodeThreads / QC;   // chunks of a row; rows of one pass
          const uint32_t g_inv = (65536u + a.G - 1) / a.G;     // row / G = row * g_inv >> 16 for row < 256, G <= 64
          const int qc = lt % QC;
          const uint8_t* q = a.q + (int64_t)t.row0 * a.q_stride + (size_t)t.head * a.G * D * 2 + qc * 16;
#pragma unroll 4
          for (int row = lt / QC; row < S::kRows; row += QP) {
            const int tok = (int)((uint32_t)row * g_inv >> 16);
            cp_async16(tiles0 + (row >> 7) * S::kTileBytes + at_chunk<D>(row & 127, qc),
                       row < rows ? q + tok * a.q_stride + (row - tok * a.G) * (D * 2) : q, row < rows);
          }
          cp_async_commit();
          cp_async_wait<0>();
          if constexpr (kShift) {
            // bf16 to fp16, in place, as over an FP8 cache: a thread scales a row so that its largest element comes to
            // [2^14, 2^15), and leaves the inverse for the softmax.
            mbar_arrive(smem_addr(&more.q_raw));
            if (!wait(&more.q_raw, n_q & 1u)) return;  // the others' chunks have landed
            for (int row = lt; row < S::kRows; row += kCodeThreads) scale_query_row<D>(tiles0 + (row >> 7) * S::kTileBytes, row & 127, row < rows, &s_unscale[row]);
          }
          fence_proxy_async_smem();
          mbar_arrive(smem_addr(&bars.q_full));
        };
        uint32_t n_tile = 0, n_q = 0;
        if (wait(&bars.mask_full[0], 0)) {
          const TileInfo& t = s_tile[0];
#pragma unroll 1
          for (int b = 0; b < kBatches; ++b) {
            if (t.rows >= 0) fetch(t, t.named, false, b);
            cp_async_commit();
          }
          for (;; ++n_tile) {
            const TileInfo& t = s_tile[n_tile % kMaskRing];
            const int rows = t.rows;
            if (rows < 0) break;
            if (kv == 1 && rows > 0) load_q(t, n_q);
            const uint32_t n = 2 * n_tile + kv, next = (n_tile + 1) % kMaskRing;
            if (!ok || !wait(&bars.mask_full[next], ((n_tile + 1) / kMaskRing) & 1u) ||
                !wait(&bars.kv_empty[n % S::kRing], ((n / S::kRing) & 1u) ^ 1u))
              break;
            const TileInfo& ahead = s_tile[next];
            const bool more = ahead.rows >= 0, whole = ahead.lo == 0 && ahead.hi == kKeys;
            const uint32_t named = ahead.named;
            const uint32_t dst = ring0 + (n % S::kRing) * S::kTileBytes;
#pragma unroll 1
            for (int b = 0; b < kBatches; ++b) {
              cp_async_wait<kBatches - 1>();
              uint4 code[kBatch];
#pragma unroll
              for (int i = 0; i < kBatch; ++i) code[i] = ld_shared_v4(raw + (kBatch * b + i) * kCodeGroup * 16);
              uint4 wide[kBatch][2];
#pragma unroll
              for (int i = 0; i < kBatch; ++i) {
                wide[i][0] = widen8<kInt8>(code[i].x, code[i].y);
                wide[i][1] = widen8<kInt8>(code[i].z, code[i].w);
              }
#pragma unroll
              for (int i = 0; i < kBatch; ++i)
                if (w + kCodeWarps * (kBatch * b + i) < kUnits) {
                  const uint32_t to = dst + put[i % X] + (b * (kBatch / X) + i / X) * kGroupStep * S::kGroupBytes;
                  st_shared_v4(to, wide[i][0]);
                  st_shared_v4(to ^ 16u, wide[i][1]);
                }
              if (more) fetch(ahead, named, whole, b);
              cp_async_commit();
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&bars.kv_full[n % S::kRing]));
            if (kv == 0 && rows > 0) load_q(t, n_q);
            n_q += rows > 0;
            if (!ok) break;
          }
        }
        cp_async_wait<0>();
        if (!ok) *abort_flag = 1;
      }
    } else if (!kScaled && warp < kMmaWarp) {
      // ---- loads --------------------------------------------------------------
      const int lt = tid - kLoaderWarp * 32;           // 0 .. kLoaders - 1
      constexpr int EB = F8 ? 1 : 2;
      const int64_t token_bytes = (int64_t)a.H * D * EB;
      uint32_t n_load = 0, n_q = 0, n_tail = 0;        // K and V tiles, query tiles, cleared V tiles
      uint32_t leader;
      asm volatile(
          "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(leader));
      uint32_t bulk = 0;                               // lane i: 1 + this warp's last load into place i if that was a bulk copy
      bool ok = true;                                  // the same in all loaders once they have agreed()
      auto agreed = [&](bool mine_ok) {                // also a barrier of the three warps
        uint32_t r;
        asm volatile(
            "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
            "barrier.cta.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
            : "=r"(r)
            : "r"(mine_ok ? 1u : 0u), "n"(kLoaders)
            : "memory");
        return r != 0;
      };
      auto barrier_loaders = [] { asm volatile("barrier.cta.sync 1, %0;" ::"n"(kLoaders) : "memory"); };
      Walk<kCost> w;                                   // the first thread's
      if (lt == 0) w.start(a, per, run, u0, u1, s_req, s_base);
      for (uint32_t n_seg = 0;; ++n_seg) {
        const uint32_t seg = n_seg % kSegments;
        ok = agreed(wait_or_abort(smem_addr(&bars.seg_empty[seg]), ((n_seg / kSegments) & 1u) ^ 1u, abort_flag, limit_ns));
        if (!ok) break;
        Segment& g = s_seg[seg];
        if (lt == 0) w.next_into(a, per, g);
        barrier_loaders();
        const int n_tiles = g.tiles, k_lo = g.k_lo, k_hi = g.k_hi, k_see = g.k_see, rows = g.rows, head = g.head, row_at = g.row0;
        const int32_t* table = a.block_table + (size_t)g.r * a.max_blocks;
        const uint8_t* kbase = a.k_cache + (size_t)head * D * EB;
        if (lt == 0) mbar_arrive(smem_addr(&bars.seg_full[seg]));
        if (n_tiles < 0) break;
        if (n_tiles == 0) continue;
        // Q once the last segment's logits are done; called after the first tile's loads are on their way.
        auto load_q = [&] {
          ok = agreed(wait_or_abort(smem_addr(&bars.q_empty), (n_q & 1u) ^ 1u, abort_flag, limit_ns));
          ++n_q;
          if (!ok) return;
          constexpr int C = D / 8, RP = kLoaders / C;  // chunks of a row; rows of one pass
          const uint32_t g_inv = (65536u + a.G - 1) / a.G;   // row / G = row * g_inv >> 16 for row < 256, G <= 64
          const int c = lt % C;
          const uint8_t* src = a.q + (int64_t)row_at * a.q_stride + (size_t)head * a.G * D * 2 + c * 16;
          auto from = [&](int row) {
            const int tok = (int)((uint32_t)row * g_inv >> 16);
            return row < rows ? src + tok * a.q_stride + (row - tok * a.G) * (D * 2) : src;
          };
#pragma unroll 8
          for (int row = lt / C; row < S::kRows; row += RP)
            cp_async16(tiles0 + (row >> 7) * S::kTileBytes + at_chunk<D>(row & 127, c), from(row), row < rows);
          cp_async_commit();
          cp_async_wait<0>();
          if constexpr (kShift) {
            // bf16 to fp16, in place: a thread scales a row by a power of two that brings its largest element to
            // [2^14, 2^15), and leaves the inverse for the softmax.  (A row to 16 lanes, with shuffles for the largest:
            // 5 us an item, 82 us for the 16 requests' prompts over FP8 where this takes 72.)
            barrier_loaders();                         // the others' chunks have landed
            for (int row = lt; row < S::kRows; row += kLoaders)
              scale_query_row<D>(tiles0 + (row >> 7) * S::kTileBytes, row & 127, row < rows, &s_unscale[row]);
          }
          fence_proxy_async_smem();
          mbar_arrive(smem_addr(&bars.q_full));
        };
        // Bulk copies: lane g of each warp finds the token of row group g (`box` rows) of a tile, one tile ahead; -1 if
        // it has no key that a row sees (the blocks before a window may be gone from the table) or the table does not
        // name it (the copy then starts behind the cache and reads zeros).
        const int groups = box > 0 ? kKeys / box : 0;
        int64_t token = -1;
        auto look_up_groups = [&](int j) {
          const int key0 = k_lo + j * kKeys, p = key0 + lane * box;
          token = -1;
          if (lane < groups && j < n_tiles && p + box > k_see && p < k_hi) {
            const int b = block_of(a, p);
            const int32_t id = table[b];
            if (id >= 0 && id < a.num_blocks) token = (int64_t)id * a.block_size + (p - b * a.block_size);
            else latch(a.status, IS_ST_BLOCK_ID);
          }
        };
        // Row copies: block ids of this thread's keys of a tile: lt, and lt + 96 for the first warp.
        int32_t id[2];
        auto look_up = [&](int j) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int p = k_lo + j * kKeys + lt + e * kLoaders;
            id[e] = -1;
            if (j < n_tiles && p >= k_see && p < k_hi && lt + e * kLoaders < kKeys) {
              id[e] = table[block_of(a, p)];
              if (id[e] < 0 || id[e] >= a.num_blocks) {
                latch(a.status, IS_ST_BLOCK_ID);
                id[e] = -1;
              }
            }
          }
        };
        if (box > 0) look_up_groups(0);
        else look_up(0);
        // Byte offsets of the tile's keys, for the row copies; -1: no such key.  Returns this thread's keys' mask words.
        auto find_rows = [&](int j, long long* off, uint32_t(&named)[2]) {
          long long at_key[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int p = k_lo + j * kKeys + lt + e * kLoaders;
            at_key[e] = id[e] < 0 ? -1ll : ((long long)id[e] * a.block_size + (p - block_of(a, p) * a.block_size)) * token_bytes;
            named[e] = __ballot_sync(0xffffffffu, at_key[e] >= 0);
          }
          off[lt] = at_key[0];
          if (lt < kKeys - kLoaders) off[lt + kLoaders] = at_key[1];
        };
        bool here = true;                              // this thread's waits
        auto room = [&](uint32_t n) {                  // the ring's place of load n is free
          here = here && wait_or_abort(smem_addr(&bars.kv_empty[n % S::kRing]), ((n / S::kRing) & 1u) ^ 1u, abort_flag,
                                       limit_ns);
          return here;
        };
        if constexpr (F8) {
          // Loads K0, V0, K1, ...: copied as bytes kRaw - 1 loads ahead, then each thread widens the chunks that it copied,
          // so that the three warps meet once a tile only, over the keys' offsets and bits: two tiles' offsets are kept,
          // and a tile's are written when all have passed the tile before it.
          constexpr int C = D / 16, RP = kLoaders / C, N = (kKeys + RP - 1) / RP;   // 16-byte chunks of a row, rows of a pass
          constexpr int kAhead = 6;
          const int c = lt % C, row0 = lt / C, n_loads = 2 * n_tiles;
          const uint32_t raw0 = ring0 + S::kRing * S::kTileBytes + (uint32_t)row0 * D + c * 16;
          auto copy_raw = [&](int i) {
            if (i < n_loads) {
              const int j = i >> 1;
              const long long* off = s_off + (j & 1) * kKeys;
              if ((i & 1) == 0) {
                uint32_t named[2];
                find_rows(j, s_off + (j & 1) * kKeys, named);
                if (lane == 0) s_raw_mask[j % S::kRaw][warp - kLoaderWarp] = named[0];
                if (lt == 0) s_raw_mask[j % S::kRaw][3] = named[1];
                look_up(j + 1);
                ok = agreed(here);
              }
              const uint8_t* src = kbase + ((i & 1) ? a.v_offset : 0) + c * 16;
              const uint32_t dst = raw0 + ((n_load + i) % S::kRaw) * S::kRawBytes;
              long long o[N];
#pragma unroll
              for (int k = 0; k < N; ++k) o[k] = row0 + k * RP < kKeys ? off[row0 + k * RP] : -1ll;
#pragma unroll
              for (int k = 0; k < N; ++k)
                if (row0 + k * RP < kKeys) cp_async16(dst + k * RP * D, src + (o[k] < 0 ? 0 : o[k]), o[k] >= 0);
            }
            cp_async_commit();
          };
#pragma unroll
          for (int i = 0; i < S::kRaw - 1; ++i) copy_raw(i);
          for (int i = 0; i < n_loads; ++i) {
            copy_raw(i + S::kRaw - 1);
            if (!ok) break;
            const uint32_t n = n_load + i, slot = (n >> 1) % kMaskRing;
            here = room(n);
            cp_async_wait<S::kRaw - 1>();
            const uint32_t src = raw0 + (n % S::kRaw) * S::kRawBytes, dst = ring0 + (n % S::kRing) * S::kTileBytes;
            // Some chunks are read before any is written: one at a time, each waits for the one before (the two long
            // prompts over FP8: 669 us, not 611).
#pragma unroll
            for (int k0 = 0; k0 < N; k0 += kAhead) {
              uint4 x[kAhead];
#pragma unroll
              for (int k = k0; k < k0 + kAhead && k < N; ++k)
                if (row0 + k * RP < kKeys) x[k - k0] = ld_shared_v4(src + k * RP * D);
#pragma unroll
              for (int k = k0; k < k0 + kAhead && k < N; ++k) {
                const int row = row0 + k * RP;
                if (row < kKeys) {
                  st_shared_v4(dst + at_chunk<D>(row, 2 * c), widen8<false>(x[k - k0].x, x[k - k0].y));
                  st_shared_v4(dst + at_chunk<D>(row, 2 * c + 1), widen8<false>(x[k - k0].z, x[k - k0].w));
                }
              }
            }
            if ((i & 1) == 0 && lt < 4) s_mask[slot][lt] = s_raw_mask[(i >> 1) % S::kRaw][lt];
            fence_proxy_async_smem();
            __syncwarp();
            if (lt == 0 && (i & 1) == 0) mbar_arrive(smem_addr(&bars.mask_full[slot]));
            if (lane == 0) mbar_arrive(smem_addr(&bars.kv_full[n % S::kRing]));
            if (i == 0) {
              load_q();
              if (!ok) break;
            }
          }
          n_load += n_loads;
          ok = ok && agreed(here);
          if (!ok) break;
          continue;
        }
        for (int j = 0; j < n_tiles; ++j, n_load += 2) {
          const int key0 = k_lo + j * kKeys;
          const uint32_t slot = (n_load >> 1) % kMaskRing;
          if (box > 0) {
            const int64_t from = token;
            look_up_groups(j + 1);
            // The first loader warp brings K, the second V; one elected lane issues.
            const int kv = warp - kLoaderWarp;
            if (kv < 2 && __all_sync(0xffffffffu, room(n_load + kv))) {
              const uint32_t place = (n_load + kv) % S::kRing, full = smem_addr(&bars.kv_full[place]);
              // Before the first key that a row sees and behind the last V has to be zero, whatever its blocks hold
              // there (0 * NaN): those rows are cleared before the tile is handed on.
              const int keys = min(kKeys, k_hi - key0), skip = max(0, k_see - key0);
              const bool clear = kv == 1 && (keys % box != 0 || skip > 0);
              const uint32_t bar = clear ? smem_addr(&bars.v_tail) : full;
              const int64_t rows_of_k = (int64_t)a.num_blocks * a.block_size;
              const int t8 = (int)((from < 0 ? 2 * rows_of_k : from + (kv ? rows_of_k : 0)) >> 3);
              if (kv == 0) {
                const uint32_t named = __ballot_sync(0xffffffffu, lane < groups && from >= 0);
                uint4 bits = make_uint4(~0u, ~0u, ~0u, ~0u);
                if (keys < kKeys || __popc(named) < groups) {
                  auto word = [&](int key) {
                    return __ballot_sync(0xffffffffu, key < keys && ((named >> (key / box)) & 1u));
                  };
                  bits = make_uint4(word(lane), word(32 + lane), word(64 + lane), word(96 + lane));
                }
                if (lane == 0) *reinterpret_cast<uint4*>(s_mask[slot]) = bits;
                if (lane == 0) mbar_arrive(smem_addr(&bars.mask_full[slot]));
              }
              if (leader) mbar_expect_tx(bar, S::kTileBytes);
              __syncwarp();
              const uint32_t step = (uint32_t)(box >> 3) * S::kGroupBytes, dst = ring0 + place * S::kTileBytes;
              for (int g = 0; g < groups; ++g) {
                const int at8 = __shfl_sync(0xffffffffu, t8, g);
                if (leader) tma_load_rows(dst + g * step, &rows_map, head, at8, bar);
              }
              if (lane == (int)place) bulk = n_load + kv + 1;
              if (clear) {
                here = here && __all_sync(0xffffffffu, mbar_wait_bounded(bar, n_tail & 1u, kWaitBudgetNs));
                ++n_tail;
                const int end = (keys + box - 1) / box * box;
                for (int x = lane; x < (end - keys) * (D / 8); x += 32)
                  st_shared_v4(dst + at_chunk<D>(keys + x / (D / 8), x % (D / 8)), make_uint4(0, 0, 0, 0));
                for (int x = lane; x < skip * (D / 8); x += 32)
                  st_shared_v4(dst + at_chunk<D>(x / (D / 8), x % (D / 8)), make_uint4(0, 0, 0, 0));
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(full);
              }
            }
            if (j == 0) {
              load_q();
              if (!ok) break;
            }
            continue;
          }
          // A block size that the bulk copies do not fit.
          ok = agreed(room(n_load));                   // and the last tile's offsets have been read
          if (!ok) break;
          uint32_t named[2];
          find_rows(j, s_off, named);
          if (lane == 0) s_mask[slot][warp - kLoaderWarp] = named[0];
          if (lt == 0) s_mask[slot][3] = named[1];
          look_up(j + 1);
          barrier_loaders();
          if (lt == 0) mbar_arrive(smem_addr(&bars.mask_full[slot]));
          for (int kv = 0; kv < 2; ++kv) {
            if (kv == 1) {
              ok = agreed(room(n_load + 1));
              if (!ok) break;
            }
            const uint32_t place = (n_load + kv) % S::kRing, dst = ring0 + place * S::kTileBytes;
            const uint8_t* src0 = kbase + (kv ? a.v_offset : 0);
            constexpr int C = D / 8, RP = kLoaders / C;   // chunks of a row; rows of one pass of the loaders
            const int c = lt % C;
#pragma unroll 4
            for (int row = lt / C; row < kKeys; row += RP) {
              const long long o = s_off[row];
              cp_async16(dst + at_chunk<D>(row, c), src0 + (o < 0 ? 0 : o) + c * 16, o >= 0);
            }
            cp_async_commit();
            cp_async_wait<0>();
            fence_proxy_async_smem();
            barrier_loaders();
            if (lt == 0) mbar_arrive(smem_addr(&bars.kv_full[place]));
            if (j == 0 && kv == 0) {
              load_q();
              if (!ok) break;
            }
          }
          if (!ok) break;
        }
        ok = ok && agreed(here);
        if (!ok) break;
      }
      // After a time-out bulk copies may be in flight that no MMA waited for:
      // they land before shared memory is let go.  Both warps' copies go into a
      // place of an odd ring in turn: the last one is waited for, as those before
      // it have landed (and their phase's parity comes again two phases later).
      if (!ok) {
        if (bulk > 0) atomicMax(&s_bulk[lane], bulk);
        barrier_loaders();
        const uint32_t last = lane < S::kRing ? s_bulk[lane] : 0u;
        if (last > 0) mbar_wait_bounded(smem_addr(&bars.kv_full[lane]), ((last - 1) / S::kRing) & 1u, kWaitBudgetNs);
      }
      __syncwarp();
      cp_async_wait<0>();
      if (!ok) *abort_flag = 1;
    } else {
      // ---- MMAs ----------------------------------------------------------------
      // One elected lane does it all.  With the branch on elect.sync and
      // descriptors that are sums of uniform values the compiler keeps them in
      // uniform registers: an M128 N128 K16 MMA is issued in the 64 clocks it
      // takes, where a branch on the lane number cost 72 to 97.
      constexpr uint32_t kIdS = idesc_of<W>(128, false), kIdO = idesc_of<W>(D, true);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), q_tile = __shfl_sync(0xffffffffu, tiles0, 0);
      const uint32_t bar0 = __shfl_sync(0xffffffffu, smem_addr(&bars), 0);
      const uint32_t tiles_done = kScaled ? __shfl_sync(0xffffffffu, smem_addr(&more.tile_empty[0]), 0) : 0u;
      uint32_t leader;
      asm volatile(
          "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(leader));
      if (leader) {
        const uint64_t q_desc = tile_desc<D, F8>(q_tile, 1), k_desc = tile_desc<D, F8>(q_tile + S::kQBytes, 1);
        const uint64_t v_desc = tile_desc<D, F8>(q_tile + S::kQBytes, 1024 >> 4);
#define ISK_BAR(member) (bar0 + (uint32_t)offsetof(Bars, member))
        uint32_t n_q = 0, p_turn0 = 0, p_turn1 = 0;
        uint32_t n_tile = 0;
        uint32_t place = 0, turn = 0;                  // of the next load: its place in the ring, and the ring's turn
        bool ok = true;
        auto wait = [&](uint32_t bar, uint32_t parity) {
          if (!mbar_try_wait(bar, parity)) ok = wait_or_abort(bar, parity, abort_flag, limit_ns);
          return ok;
        };
        auto next_place = [&] {
          if (++place == S::kRing) {
            place = 0;
            turn ^= 1u;
          }
        };
        // Each side is code of its own, so that its addresses are constants.
        auto scores = [&](auto side_, uint32_t k_place) {
          constexpr uint32_t side = decltype(side_)::value;
          const uint64_t qd = q_desc + side * (S::kTileBytes >> 4), kd = k_desc + k_place * (S::kTileBytes >> 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t o = ((uint32_t)(k >> 2) * 1024u + 32u * (k & 3)) >> 4;
            mma_ss(tm + 128u * side, qd + o, kd + o, kIdS, k != 0);
          }
          mma_commit(ISK_BAR(s_full) + 8 * side);
        };
        auto values = [&](auto side_, uint64_t vd, uint32_t& p_turn, bool first) {
          constexpr uint32_t side = decltype(side_)::value;
          constexpr uint32_t o_at = S::kOCol + (uint32_t)D * side, p_at = 128u * side;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!wait(ISK_BAR(p_full) + 16 * side + 8 * half, p_turn)) return;
            tc_fence_after();
#pragma unroll
            for (int k = 4 * half; k < 4 * half + 4; ++k)
              mma_ts(tm + o_at, tm + p_at + 8u * k, vd + 2u * k * (S::kGroupBytes >> 4), kIdO, k != 0 || !first);
          }
          p_turn ^= 1u;
        };
        constexpr std::integral_constant<uint32_t, 0> A{};
        constexpr std::integral_constant<uint32_t, 1> B{};
        for (uint32_t n_seg = 0; ok; ++n_seg) {
          const uint32_t seg = n_seg % kSegments;
          if (!wait(ISK_BAR(seg_full) + 8 * seg, (n_seg / kSegments) & 1u)) break;
          const int n_tiles = s_seg[seg].tiles;
          const bool both = s_seg[seg].rows > 128;
          if (n_tiles < 0) break;
          mbar_arrive(ISK_BAR(seg_empty) + 8 * seg);
          if (n_tiles == 0) continue;
          if (!wait(ISK_BAR(q_full), n_q & 1u)) break;
          ++n_q;
          if (!wait(ISK_BAR(kv_full) + 8 * place, turn)) break;
          tc_fence_after();
          scores(A, place);
          if (both) scores(B, place);
          mma_commit(ISK_BAR(kv_empty) + 8 * place);
          for (int j = 0; j < n_tiles; ++j) {
            next_place();                              // V of this tile
            const uint32_t v_place = place;
            if (!wait(ISK_BAR(kv_full) + 8 * v_place, turn)) break;
            next_place();                              // K of the next
            const uint64_t vd = v_desc + v_place * (S::kTileBytes >> 4);
            const bool last = j == n_tiles - 1;
            values(A, vd, p_turn0, j == 0);
            if (!ok) break;
            if (!both) mma_commit(ISK_BAR(kv_empty) + 8 * v_place);
            if (last) {
              mma_commit(ISK_BAR(o_full));
            } else {
              if (!wait(ISK_BAR(kv_full) + 8 * place, turn)) break;
              tc_fence_after();
              scores(A, place);
            }
            if (both) {
              values(B, vd, p_turn1, j == 0);
              if (!ok) break;
              mma_commit(ISK_BAR(kv_empty) + 8 * v_place);
              if (last) mma_commit(ISK_BAR(o_full) + 8);
              else scores(B, place);
            }
            if (!last) mma_commit(ISK_BAR(kv_empty) + 8 * place);
            if constexpr (kScaled) mma_commit(tiles_done + 8 * (n_tile++ % kMaskRing));
          }
          if (ok) mma_commit(ISK_BAR(q_empty));
        }
        if (!ok) *abort_flag = 1;
        // Every MMA issued has ended before tensor and shared memory are let go.
        mma_commit(ISK_BAR(done));
        mbar_wait_bounded(ISK_BAR(done), 0, kWaitBudgetNs);
#undef ISK_BAR
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && s_abort) {
    latch(a.status, IS_ST_TIMEOUT);
    record_of(a, blockIdx.x)->parts = 0;
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemAll);
  }
}

}  // namespace prompt

// Prompts go here when the rows of a request fill a tensor-core tile better
// than the split kernel's 16 rows (see launch_attend).
template <typename T, CacheKind KIND, int D, int GROUP = prompt::kGroup>
static cudaError_t launch_prompt_t(const AttendArgs& a, const LaunchCfg& cfg) {
  constexpr bool F8 = KIND != kCachePlain;
  constexpr bool kScaled = KIND == kCacheScaledE4m3 || KIND == kCacheScaledInt8;
  using S = prompt::Shape<D, F8, kScaled>;
  auto* kern = a.wait_ns < kWaitBudgetNs ? prompt::attend_prompt_kernel<T, KIND, D, true, GROUP>
                                         : prompt::attend_prompt_kernel<T, KIND, D, false, GROUP>;
  static_assert(S::kSmem + (kScaled ? 8192 : F8 ? 2048 : 1024) <= 227 * 1024, "a CTA fits an SM");
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), S::kSmem);
  if (e != cudaSuccess) return e;
  constexpr int kFit = (int)((IS_ATTEND_WORKSPACE_BYTES - partials_offset()) / (2 * sizeof(PartialByEights<S::kRows, D>)));
  const int grid = std::max(1, std::min({cfg.num_sms, kFit, kMaxCtas}));
  const int per = S::kRows / a.G;   // tokens of an item
  // Bulk copies bring `box` rows at once: a block, or 128 rows of a longer one.
  // They need blocks that divide a tile or consist of tiles, 8 rows at least (the
  // swizzle's period), and 16-bit rows; other caches take the row copies.
  int box = 0;
  CUtensorMap map;
  std::memset(&map, 0, sizeof map);
  if (!F8 && a.block_size >= 8 && (prompt::kKeys % a.block_size == 0 || a.block_size % prompt::kKeys == 0)) {
    box = std::min(a.block_size, prompt::kKeys);
    if (!make_rows_map(&map, a.k_cache, a.D, a.H, 2LL * a.num_blocks * a.block_size, box, a.dtype)) box = 0;
  }
  e = launch_ex(kern, dim3(grid), dim3(prompt::threads_of(KIND)), S::kSmem, cfg.stream, cfg.pdl, a, per, box, map);
  if (e != cudaSuccess) return e;
  return launch_ex(attend_join_rows_kernel<T, S::kRows, D, true>, dim3(grid, 32), dim3(kJoinThreads), 0, cfg.stream,
                   cfg.pdl, a);
}

}  // namespace isk
