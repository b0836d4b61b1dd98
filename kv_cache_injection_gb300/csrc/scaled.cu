// Writing a scaled cache (is_append_scaled, is_move_scaled) and reading it back
// (is_read_scaled): 8-bit codes with a scale for each block and KV head, keys
// and values apart.
//
// The rows that a call puts into one block share one scale per head, so the unit
// of work is a group: the tokens of one block, between which others may lie that
// have no slot.  With A the largest finite magnitude of a head's new elements (keys
// rotated in fp32) and qmax 127 or 448,
//   s = A / qmax, in [2^-40, 2^40]; beside earlier rows no smaller than their scale;
//   code = round(y * (1 / s)), and earlier rows' codes round(code * s_old / s) if s grew.
// A CTA takes the groups that begin in its tokens, as many at a time as there is
// room for (a round): their rows come to shared memory by bulk copies while the sines of
// their keys are computed once for all heads; each warp finds the largest elements
// of one head's keys or values at a time, a thread settles each block's scale, and
// the warps go through the rows once more for the codes.  Groups that do not fit
// are brought twice.  The queries are rotated by CTAs of their own, a warp or
// several to a token.
//
// The bytes would take 27 and 40 us in the two large cases below; the steps of a
// round wait for one another and for memory, and what overlaps them is other CTAs
// (the SMs issue in half of their slots).  Of the 62 us of the second case 18 are
// the codes, 7 the search and 38 the way to the rows and the rows themselves.
// Short loops matter more than registers: rows kept in registers and unrolled took
// 56 and 165 us, each CTA running once through code that it has to fetch first.
// Bringing a piece of a CTA's heads while the one before is quantised, 16 KB each,
// took 40 and 68 us: more steps for each byte.
//
// Measured: 8000 tokens, 32 + 8 heads of 128, bf16 to INT8, 183 MB: 36.9 us = 5.0
// TB/s, 73 % of a plain copy (the queries alone 26); 44,000 moved tokens, 8 heads,
// bf16 to E4M3 in blocks of 32, 271 MB: 62 us = 4.4 TB/s, blocks of 16 61 us; 1276
// tokens moved 6.6 us; 1000 requests' single tokens 11.1 us; one token 4.6 us, the
// latency of its steps.  Reading 36,000 tokens back (E4M3 to bf16, 223 MB) 35.6 us
// = 6.3 TB/s, 92 % of a copy; 700 tokens with their keys turned back 3.2 us.
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "scaled_plan.h"

namespace isk {

namespace {

using namespace scaled;

__device__ __forceinline__ float ld_table(const float* p) {   // see ld_param in append.cu
  float x;
  asm("ld.f32 %0, [%1];" : "=f"(x) : "l"(p));
  return x;
}
__device__ __forceinline__ uint32_t ld_table(const uint8_t* p) {
  uint32_t x;
  asm("ld.u8 %0, [%1];" : "=r"(x) : "l"(p));
  return x;
}

// Of a power of two.  (What divides here mostly is one; a division by a variable takes 20 instructions, 64 bits wide 80.)
__device__ __forceinline__ int log2_of(int x) { return 31 - __clz(x); }

__device__ __forceinline__ int64_t block_of_slot(int64_t slot, int32_t size, int32_t shift) {
  return shift >= 0 ? slot >> shift : slot / size;
}

__device__ __forceinline__ float2 turn_of(const AxisTurns& at, int i, float p, float sign) {
  float sn, cs;
  sincospif(2.0f * angle_turns(p, ld_table(&at.t.hi[i]), ld_table(&at.t.lo[i])), &sn, &cs);
  return make_float2(cs, sign * sn);
}

// The sines of a lane's pairs: NeoX vectors f and f + gv of a head rotate element
// e of one with element e of the other, interleaved ones neighbours within each.
// Either way a lane has VE pairs; pair_of(f, e) is the e-th one's number.
template <int VE, int STYLE>
__device__ __forceinline__ int pair_of(int f, int e, int gv) {
  return STYLE == 0 ? f * VE + e : (e < VE / 2 ? f : f + gv) * (VE / 2) + e % (VE / 2);
}
template <int VE>
struct Turn {
  unsigned long long cs[VE / 2], sn[VE / 2];   // two pairs' to a register pair: the paired operations round as the single ones
};
// A row's sines in shared memory: by pieces of four, cosines then sines, a piece of
// all lanes after the other, so that eight lanes' 16 bytes lie in different banks.
template <int VE>
__device__ __forceinline__ int turn_at(int f, int e, int gv) { return ((e / 4) * gv + f) * 4 + e % 4; }
template <int VE>
__device__ __forceinline__ Turn<VE> load_turn(const float* row, int f, int gv) {
  Turn<VE> t;
#pragma unroll
  for (int q = 0; q < VE / 4; ++q) {
    const float4 c = *reinterpret_cast<const float4*>(row + (q * gv + f) * 4);
    const float4 s = *reinterpret_cast<const float4*>(row + ((q + VE / 4) * gv + f) * 4);
    t.cs[2 * q] = pk2(c.x, c.y), t.cs[2 * q + 1] = pk2(c.z, c.w);
    t.sn[2 * q] = pk2(s.x, s.y), t.sn[2 * q + 1] = pk2(s.z, s.w);
  }
  return t;
}
__device__ __forceinline__ unsigned long long neg2(unsigned long long x) { return x ^ 0x8000000080000000ull; }
template <typename T, int STYLE>
__device__ __forceinline__ void rotate_pair(const Turn<Vec<T>::N>& t, float (&x)[Vec<T>::N], float (&z)[Vec<T>::N]) {
  constexpr int VE = Vec<T>::N;
  auto turn = [](float& a0, float& a1, float& b0, float& b1, unsigned long long cs, unsigned long long sn) {
    const unsigned long long a = pk2(a0, a1), b = pk2(b0, b1);
    upk2(fma2_rn(a, cs, mul2_rn(b, neg2(sn))), a0, a1);
    upk2(fma2_rn(b, cs, mul2_rn(a, sn)), b0, b1);
  };
  if constexpr (STYLE == 0) {
#pragma unroll
    for (int e = 0; e < VE / 2; ++e) turn(x[2 * e], x[2 * e + 1], z[2 * e], z[2 * e + 1], t.cs[e], t.sn[e]);
  } else {
#pragma unroll
    for (int e = 0; e < VE / 4; ++e) {           // pairs 2 e and 2 e + 1 of each vector
      turn(x[4 * e], x[4 * e + 2], x[4 * e + 1], x[4 * e + 3], t.cs[e], t.sn[e]);
      turn(z[4 * e], z[4 * e + 2], z[4 * e + 1], z[4 * e + 3], t.cs[VE / 4 + e], t.sn[VE / 4 + e]);
    }
  }
}
// The sines of one token's pairs, computed by a warp and kept by each lane for its f.
template <typename T, int STYLE>
__device__ __forceinline__ Turn<Vec<T>::N> warp_turn(const AxisTurns& at, float* row, int half, int gv, int f, int32_t of_axis, float sign) {
  constexpr int VE = Vec<T>::N;
  const int lane = threadIdx.x & 31;
  for (int i0 = 0; i0 < half; i0 += 32) {        // half may be 8 or 16: then lanes past it repeat pairs
    const int i = (i0 + lane) & (half - 1), g = i / VE, e = i % VE, j = pair_of<VE, STYLE>(g, e, gv);
    const float2 v = turn_of(at, j, (float)__shfl_sync(0xffffffffu, of_axis, ld_table(&at.axis[j])), sign);
    row[turn_at<VE>(g, e, gv)] = v.x;
    row[turn_at<VE>(g, e + VE, gv)] = v.y;
  }
  __syncwarp();
  return load_turn<VE>(row, f, gv);
}

// The magnitudes of a vector's elements as whole numbers, which order as they do
// and put what is not finite on top: the largest so far.
template <typename T>
__device__ __forceinline__ uint32_t larger_bits(uint32_t most, const uint4& v) {
  if constexpr (sizeof(T) == 4)
    return max(max(max(most, v.x & 0x7fffffffu), max(v.y & 0x7fffffffu, v.z & 0x7fffffffu)), v.w & 0x7fffffffu);
  else
    return __vimax3_s16x2(__vimax3_s16x2(most, v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), v.z & 0x7fff7fffu, v.w & 0x7fff7fffu);
}
template <typename T>
__device__ __forceinline__ uint32_t max_bits(uint32_t a, uint32_t b) {
  if constexpr (sizeof(T) == 4) return max(a, b);
  else return __vmaxs2(a, b);
}
// The magnitude itself; inf or NaN if one of the elements was.
template <typename T>
__device__ __forceinline__ float magnitude(uint32_t most) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(most);
  const uint32_t m = max(most & 0xffffu, most >> 16);
  if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(m << 16);
  else return __half2float(__ushort_as_half((unsigned short)m));
}

__device__ __forceinline__ float larger_finite(float most, float x) {
  const float a = fabsf(x);
  return a < INFINITY ? fmaxf(most, a) : most;   // false for NaN
}

// Four INT8 codes of finite elements whose codes are known to be in range: added
// to 1.5 * 2^23 a product is rounded to a whole number, whose low byte is the code.
__device__ __forceinline__ uint32_t int8x4_in_range(const float* y, unsigned long long r2) {
  const unsigned long long magic = pk2(12582912.f, 12582912.f);
  float a, b, c, d;
  upk2(fma2_rn(pk2(y[0], y[1]), r2, magic), a, b);
  upk2(fma2_rn(pk2(y[2], y[3]), r2, magic), c, d);
  return __byte_perm(__byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040),
                     __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040), 0x5410);
}
// N codes (4 or 8) of a vector.  odd: its row has elements that are not finite, or past the largest scale's range.
template <int N, bool I8>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&y)[N], float r, bool odd) {
  uint2 c;
  if (I8 && !odd) {
    const unsigned long long r2 = pk2(r, r);
    c = make_uint2(int8x4_in_range(y, r2), N == 8 ? int8x4_in_range(y + N - 4, r2) : 0u);
  } else {
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = e < N ? y[e % N] : 0.f;
    c = I8 ? to_int8x8(w, r) : to_e4m3x8(w, r);
  }
  if constexpr (N == 8) st_v2(p, c);
  else *reinterpret_cast<uint32_t*>(p) = c.x;
}

// Sixteen codes under a scale that grew.
template <bool I8>
__device__ __forceinline__ uint4 again(const uint4& c, float ratio) {
  const uint32_t in[4] = {c.x, c.y, c.z, c.w};
  uint2 out[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t lo, hi;
      codes_f16x4<I8>(in[2 * h + i], lo, hi);
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
      const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      x[4 * i] = a.x;
      x[4 * i + 1] = a.y;
      x[4 * i + 2] = b.x;
      x[4 * i + 3] = b.y;
    }
    out[h] = I8 ? to_int8x8(x, ratio) : to_e4m3x8(x, ratio);
  }
  return make_uint4(out[0].x, out[0].y, out[1].x, out[1].y);
}

// The queries of a token, one or `share` warps to it; a refused token's row is left as it was.
template <typename T, int STYLE>
__device__ void rotate_queries(const AppendArgs& a, const AxisTurns& at, float* row, int64_t w, int share) {
  constexpr int VE = Vec<T>::N, kBatch = 4;
  const int lane = threadIdx.x & 31, half = a.D / 2, gv = a.D / VE / 2;
  const int64_t t = w >> log2_of(share);
  if (t >= a.T) return;
  const int first = (int)(w - t * share) * 32 + lane, step = share * 32, f = lane & (gv - 1), n = a.Hq * gv;
  const uint8_t* src = a.q + t * a.q_stride;
  auto offset = [&](int i) { return (2 * i - f) * 16; };          // head i / gv, vector f
  uint4 x0[kBatch], x1[kBatch];
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (i0 + u * step < n) {
        const uint8_t* p = src + offset(i0 + u * step);
        x0[u] = *reinterpret_cast<const uint4*>(p);
        x1[u] = *reinterpret_cast<const uint4*>(p + gv * 16);
      }
  };
  const int64_t slot = a.slots[t];
  const int32_t of_axis = lane < a.n_axes ? a.positions[(size_t)lane * a.T + t] : 0;
  load(first);
  if (slot < 0 || slot >= a.n_slots) return;     // padding, or reported by the CTA that looks at the token's block
  if (__any_sync(0xffffffffu, of_axis < 0 || of_axis >= IS_MAX_POSITION)) return;
  const Turn<VE> turn = warp_turn<T, STYLE>(at, row, half, gv, f, of_axis, 1.f);
  uint8_t* dst = a.q_out + (size_t)t * a.Hq * a.D * sizeof(T);
  for (int i0 = first; i0 < n; i0 += kBatch * step) {
    if (i0 != first) load(i0);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * step;
      if (i >= n) continue;
      float x[VE], z[VE];
      Vec<T>::unpack(x0[u], x);
      Vec<T>::unpack(x1[u], z);
      rotate_pair<T, STYLE>(turn, x, z);
      st_v4(dst + offset(i), Vec<T>::pack(x));
      st_v4(dst + offset(i) + gv * 16, Vec<T>::pack(z));
    }
  }
}

// A group of a CTA's round.
struct Group {
  int64_t block, t0, n;
  int32_t row0;          // of its first token among the round's rows
  int32_t low;           // the lowest of its rows in the block: below it the block is held already
  int32_t live;          // some token is not skipped
};

// STYLE -1: no rotation (a move).  (44,000 moved tokens take 62 us with six CTAs an SM, 69 with five.)
template <typename T, int STYLE, bool I8>
__global__ void __launch_bounds__(kThreads, most_per_sm(STYLE >= 0)) scaled_write_kernel(const ScaledWriteArgs p, const __grid_constant__ AxisTurns at,
                                                                  int group_ctas, int turns_of, int window, int heads_of, int cap, int share) {
  constexpr int VE = Vec<T>::N;
  const AppendArgs& a = p.a;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int32_t s_row[kMaxRows];            // row of the block; -1: the token is skipped
  __shared__ int32_t s_token[STYLE >= 0 ? kMaxRows : 1];
  __shared__ uint8_t s_of[kMaxRows];             // group
  __shared__ Group s_group[kMaxGroups];
  __shared__ float s_scale[kMaxGroups * kMaxUnits], s_ratio[kMaxGroups * kMaxUnits];   // 0: no scale; 0: it did not grow
  __shared__ int32_t s_groups;                   // -1: the first warp asks for the nearest token with a slot
  __shared__ int64_t s_from;
  __shared__ int32_t s_way, s_near[kWarps];
  __shared__ uint64_t s_landed;                  // a stage's rows
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, half = a.D / 2;
  // The first 2 turns_of CTAs are a group's and the queries' in turn, then come what is left of the groups' and of the queries'.
  const int at_grid = blockIdx.x, later = at_grid - turns_of;
  const int cta = at_grid >= 2 * turns_of ? (later < group_ctas ? later : at_grid)
                  : at_grid & 1           ? group_ctas + at_grid / 2 : at_grid / 2;
  pdl_wait();
  pdl_trigger();
  if (cta >= group_ctas) {
    if constexpr (STYLE >= 0) {
      rotate_queries<T, STYLE>(a, at, reinterpret_cast<float*>(smem) + warp * a.D,
                               (int64_t)(cta - group_ctas) * kWarps + warp, share);
    }
    return;
  }
  const uint32_t landed = smem_addr(&s_landed);
  uint32_t n_stage = 0;
  if (tid == 0) {
    mbar_init(landed, kThreads);
    fence_mbar_init();
  }
  const int splits = (a.H + heads_of - 1) / heads_of;
  const int of_window = cta / splits;
  const int64_t begin = of_window * (int64_t)window;
  const int head0 = (cta - of_window * splits) * heads_of, heads = min(heads_of, a.H - head0), units = 2 * heads;
  const int gv = a.D / VE / 2, gv_bits = log2_of(gv), f = tid & (gv - 1);
  const int head_bytes = a.D * (int)sizeof(T), part_bytes = heads * head_bytes;   // of a row's keys, or values
  const size_t row_bytes = (size_t)a.H * a.D;    // of the cache
  float* s_turn = reinterpret_cast<float*>(smem + (size_t)2 * cap * heads_of * head_bytes);   // [rows][D]
  float* s_most = s_turn + (STYLE >= 0 ? cap * a.D : 0);                                       // [units][rows]
  // The slot of a token, negative if it has none in the cache, or nothing to move there: a row that is not written does not
  // say what its block holds.  (Loads in any case, so that several are under way at once.)
  auto slot_at = [&](int64_t t) -> int64_t {
    const int64_t u = min(max(t, (int64_t)0), (int64_t)a.T - 1), slot = a.slots[u];
    bool in = t == u && slot < a.n_slots;
    if constexpr (STYLE < 0) {
      const int64_t from = p.from[u];
      in = in && from >= 0 && from < p.n_from;
    }
    return in ? slot : -1;
  };
  auto block_of = [&](int64_t slot) -> int64_t { return slot < 0 ? -1 : block_of_slot(slot, p.block_size, p.block_shift); };
  // The nearest token from `from` on, one way or the other, that has a slot; -1: none.  The whole CTA looks: behind the last
  // token of a padded batch there may be thousands without one (100 tokens of 8192 18.4 us; by a warp, 128 at a time, 64).
  auto nearest = [&](int64_t from, int way) -> int64_t {
    constexpr int kLook = STYLE < 0 ? 8 : 16;    // tokens of a thread at once; of a move's both slots
    for (int64_t d0 = 0; way > 0 ? from + d0 < a.T : from - d0 >= 0; d0 += kThreads * kLook) {
      int64_t slot[kLook];
#pragma unroll
      for (int u = 0; u < kLook; ++u) slot[u] = slot_at(from + way * (d0 + u * kThreads + tid));
      int32_t near = INT32_MAX;
#pragma unroll
      for (int u = kLook - 1; u >= 0; --u) near = slot[u] >= 0 ? u * kThreads + tid : near;
      near = __reduce_min_sync(0xffffffffu, near);
      __syncthreads();                           // the last turn's have been read
      if (lane == 0) s_near[warp] = near;
      __syncthreads();
      for (int w = 0; w < kWarps; ++w) near = min(near, s_near[w]);
      if (near < INT32_MAX) return from + way * (d0 + near);
    }
    return -1;
  };

  // The groups that begin in this CTA's tokens begin .. begin + window - 1: lane i of the first warp looks at token begin -
  // 1 + i and hands them on, so that the CTA agrees on them whatever happens to the caller's slots meanwhile.  A token
  // begins a group if the one before it that has a slot has it in another block.  What precedes the first leader and where
  // the last group ends may lie further off: the 32 tokens on either side are looked at in the same trip to memory.
  int64_t mine = -1, ahead = -1;                 // block of the lane's token; slot of token next + lane
  int32_t mine_row = 0;
  uint32_t present = 0, leaders = 0, starts = 0; // starts: leaders, and first tokens of groups of the next CTA
  int ask = 0;                                   // the whole CTA has to look, backwards (-1) or forwards (1)
  int64_t next = begin + 31, tail = 0;           // the last group, while it is open, goes on from here; its tokens so far
  int32_t tail_low = 0;
  bool open = false;
  if (warp == 0) {
    const int64_t t = begin - 1 + lane, slot = slot_at(t), behind = slot_at(t - 32);
    ahead = slot_at(t + 32);
    mine = block_of(slot);
    mine_row = (int32_t)(slot - mine * p.block_size);
    present = __ballot_sync(0xffffffffu, mine >= 0);
    const uint32_t earlier = present & ((1u << lane) - 1u), of_window = ((2u << window) - 1u) & ~1u;
    const int64_t before = __shfl_sync(0xffffffffu, mine, earlier ? 31 - __clz(earlier) : 0);
    starts = __ballot_sync(0xffffffffu, lane >= 1 && mine >= 0 && (!earlier || mine != before));
    if ((starts & of_window) && !(present & 1u)) {
      const uint32_t some = __ballot_sync(0xffffffffu, behind >= 0);
      const int64_t last = __shfl_sync(0xffffffffu, behind, some ? 31 - __clz(some) : 0);
      if (some && block_of(last) == __shfl_sync(0xffffffffu, mine, __ffs(present) - 1)) starts &= starts - 1u;
      if (!some && begin >= 34) ask = -1;
    }
    leaders = starts & of_window;
    open = next < a.T;
    if (head0 == 0 && ((of_window >> lane) & 1u) && t < a.T && slot < 0) {
      int64_t wrong = a.slots[t];
      if constexpr (STYLE < 0) {
        if (wrong >= 0 && wrong < a.n_slots) wrong = p.from[t];
      }
      if (wrong != -1) latch(a.status, IS_ST_BLOCK_ID);
    }
  }
  if (warp == 1 && lane < window && begin + lane < a.T) {   // what the rows' threads will read next
    if (p.from) prefetch_l1(p.from + begin + lane);
    if constexpr (STYLE >= 0) {
      for (int x = 0; x < a.n_axes; ++x) prefetch_l1(a.positions + (size_t)x * a.T + begin + lane);
    }
  }
  while (true) {
    if (warp == 0 && ask == 0 && open) {         // where the last group ends
      const int first = leaders ? 31 - __clz(leaders) : 0;
      const int64_t block = __shfl_sync(0xffffffffu, mine, first);
      open = leaders && !(starts >> first >> 1);
      if (open && tail == 0) {
        tail = 32 - __clz(present) - first;
        tail_low = lane >= first && mine >= 0 ? mine_row : p.block_size;
      }
      while (open && ask == 0) {
        const int64_t b = block_of(ahead);
        const uint32_t some = __ballot_sync(0xffffffffu, b >= 0), other = __ballot_sync(0xffffffffu, b >= 0 && b != block);
        const uint32_t same = some & ~other & (other ? (other & -other) - 1u : ~0u);
        if (same) tail = next + 32 - __clz(same) - (begin - 1 + first);
        if ((same >> lane) & 1u) tail_low = min(tail_low, (int32_t)(ahead - block * p.block_size));
        next += 32;
        open = !other && next < a.T;
        if (open && !some && a.T - next > 96) ask = 1;   // (for fewer the CTA's look takes as long)
        else if (open) ahead = slot_at(next + lane);
      }
    }
    if (warp == 0 && ask != 0) {
      if (lane == 0) {
        s_groups = -1;
        s_from = ask < 0 ? begin - 34 : next;
        s_way = ask;
      }
    } else if (warp == 0) {                      // as many groups as have room
      int64_t total = 0;
      int ng = 0;
      while (leaders && total < cap && ng < kMaxGroups) {
        const int first = __ffs(leaders) - 1;
        const int64_t block = __shfl_sync(0xffffffffu, mine, first);
        const uint32_t after = starts & ~((2u << first) - 1u);
        const uint32_t in_group = present & ~((1u << first) - 1u) & ((after & -after) - 1u);
        const bool on = !after && tail;          // past this warp's tokens
        const int64_t n = on ? tail : 32 - __clz(in_group) - first;   // to its last token
        int32_t low = on ? tail_low : (in_group >> lane) & 1u ? mine_row : p.block_size;
        if (ng > 0 && total + n > cap) break;
        low = __reduce_min_sync(0xffffffffu, low);
        if (lane == 0) s_group[ng] = {block, begin - 1 + first, n, (int32_t)total, low, 0};
        ++ng;
        total += n;
        leaders &= leaders - 1;
      }
      if (lane == 0) s_groups = ng;
    }
    __syncthreads();
    const int ng = s_groups;
    if (ng == 0) return;
    if (ng < 0) {
      const int64_t found = nearest(s_from, s_way);
      if (warp == 0) {
        const int64_t slot = found < 0 ? -1 : slot_at(found + (ask > 0 ? lane : 0));
        if (ask > 0) {
          open = found >= 0;
          next = found;
          ahead = slot;
        } else if (slot >= 0 && block_of(slot) == __shfl_sync(0xffffffffu, mine, __ffs(present) - 1)) {
          starts &= starts - 1u;
          leaders &= leaders - 1u;
        }
        ask = 0;
      }
      __syncthreads();                           // the question has been read
      continue;
    }
    const int64_t total = s_group[ng - 1].row0 + s_group[ng - 1].n;   // past cap: one long group, which goes through twice

    // Rows i0 .. i0 + cnt - 1 of the round: their places, their elements and their keys' sines.  A row's keys and values are a
    // bulk copy each, and a thread issues one (a warp issues its lanes' one after the other, so neighbours go to other
    // warps: 44,000 moved tokens 63 us, 70 with a warp's lanes side by side, 79 with 16 bytes a thread).  False: the copies
    // did not arrive in time.
    auto stage = [&](int64_t i0, int cnt) {
      for (int x = lane * kWarps + warp; x < 2 * cnt; x += kThreads) {
        const int i = x >> 1, value = x & 1;
        int g = ng - 1;
        while (g > 0 && s_group[g].row0 > i) --g;
        const int64_t t = s_group[g].t0 + (i0 + i - s_group[g].row0);
        const int64_t in_block = a.slots[t] - s_group[g].block * p.block_size;
        int32_t row = in_block >= 0 && in_block < p.block_size ? (int32_t)in_block : -1;
        int64_t from = t;
        if constexpr (STYLE < 0) {
          from = p.from[t];
          if (from < 0 || from >= p.n_from) row = -1;
        }
        if constexpr (STYLE >= 0) {
          for (int x = 0; x < a.n_axes; ++x) {
            const int32_t pos = a.positions[(size_t)x * a.T + t];   // read in any case, beside the slot; of a skipped token it means nothing
            if (row >= 0 && (pos < 0 || pos >= IS_MAX_POSITION)) {
              latch(a.status, IS_ST_POSITION);
              row = -1;
            }
          }
        }
        if (value == 0) {
          s_row[i] = row;
          s_of[i] = (uint8_t)g;
          if (STYLE >= 0) s_token[i] = (int32_t)t;
          if (row >= 0) s_group[g].live = 1;
        }
        if (row >= 0) {
          const uint8_t* src = (value ? a.v + from * a.v_stride : a.k + from * a.k_stride) + (size_t)head0 * head_bytes;
          mbar_add_tx(landed, part_bytes);
          bulk_load(smem_addr(smem) + (uint32_t)(value ? cnt + i : i) * part_bytes, src, part_bytes, landed);
        }
      }
      mbar_arrive(landed);
      if constexpr (STYLE >= 0) {
        __syncthreads();
        for (int x = tid; x < cnt * half; x += kThreads) {
          const int i = x >> log2_of(half), g = (x & (half - 1)) / VE, e = x % VE, j = pair_of<VE, STYLE>(g, e, gv);
          const float2 v = turn_of(at, j, (float)a.positions[(size_t)ld_table(&at.axis[j]) * a.T + s_token[i]], 1.f);
          s_turn[i * a.D + turn_at<VE>(g, e, gv)] = v.x;
          s_turn[i * a.D + turn_at<VE>(g, e + VE, gv)] = v.y;
        }
      }
      const uint32_t parity = n_stage++ & 1u;
      const bool in_time = __syncthreads_and(mbar_wait_bounded(landed, parity, p.wait_ns));
      if (!in_time && tid == 0) {
        latch(a.status, IS_ST_TIMEOUT);
        mbar_wait_bounded(landed, parity, kWaitBudgetNs);   // copies under way land before the shared memory is another CTA's
      }
      return in_time;
    };
    // A warp takes a unit, or two warps where there are two, and gv lanes a row of it: vectors f and f + gv of the head.
    const int sharers = units == 2 ? kWarps / 2 : 1, part = warp & (sharers - 1);
    const int rows_of_warp = 32 >> gv_bits, first_row = part * rows_of_warp + (lane >> gv_bits), step = rows_of_warp * sharers;
    auto unit_rows = [&](int unit, int cnt) {
      return smem + (size_t)(unit < heads ? 0 : cnt) * part_bytes + (unit < heads ? unit : unit - heads) * head_bytes + f * 16;
    };
    auto values = [&](bool key, int i, const uint4& x0, const uint4& z0, float (&x)[VE], float (&z)[VE]) {
      Vec<T>::unpack(x0, x);
      Vec<T>::unpack(z0, z);
      if constexpr (STYLE >= 0) {
        if (key) rotate_pair<T, STYLE>(load_turn<VE>(s_turn + i * a.D, f, gv), x, z);
      }
    };
    auto signed_most = [](float most, bool odd) { return odd ? -most - FLT_MIN : most; };
    // The largest finite magnitude of a unit's rows of one group, or of each of its rows; negative if some element is not
    // finite.
    auto find_most = [&](int cnt, bool by_row) {
      for (int unit = warp / sharers; unit < units; unit += kWarps / sharers) {
        const uint8_t* rows = unit_rows(unit, cnt);
        const bool key = unit < heads;
        const bool turned = STYLE >= 0 && key;
        float most = 0.f;                        // of rotated elements
        uint32_t bits = 0;                       // of elements as they came
        bool odd = false;
        // The largest finite magnitude of the lane's elements since the last time, which are those of rows from, from +
        // step, ... below end: looked at one by one if one of them is not finite (odd).
        auto flush = [&](int from, int end) {
          const float came = magnitude<T>(bits);
          float m = turned ? most : came;
          odd = !(came < INFINITY) || m == INFINITY;
          if (odd) {
            m = 0.f;
#pragma unroll 1
            for (int i = from; i < end; i += step) {
              if (s_row[i] < 0) continue;
              float x[VE], z[VE];
              values(key, i, *reinterpret_cast<const uint4*>(rows + (size_t)i * part_bytes),
                     *reinterpret_cast<const uint4*>(rows + (size_t)i * part_bytes + gv * 16), x, z);
#pragma unroll
              for (int e = 0; e < VE; ++e) m = larger_finite(larger_finite(m, x[e]), z[e]);
            }
          }
          most = 0.f;
          bits = 0;
          return m;
        };
        for (int i0 = 0; i0 < cnt; i0 += step) {
          const int i = i0 + first_row;
          if (i < cnt && s_row[i] >= 0) {
            const uint4 x0 = *reinterpret_cast<const uint4*>(rows + (size_t)i * part_bytes);
            const uint4 z0 = *reinterpret_cast<const uint4*>(rows + (size_t)i * part_bytes + gv * 16);
            bits = larger_bits<T>(larger_bits<T>(bits, x0), z0);
            if (turned) {
              float x[VE], z[VE];
              values(true, i, x0, z0, x, z);
#pragma unroll
              for (int e = 0; e < VE; ++e) most = fmaxf(fmaxf(most, fabsf(x[e])), fabsf(z[e]));
            }
          }
          if (by_row) {
            float m = flush(i, min(cnt, i + 1));
            for (int d = 1; d < gv; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
            if (__any_sync(0xffffffffu, odd)) {
              for (int d = 1; d < gv; d <<= 1) odd |= __shfl_xor_sync(0xffffffffu, (int)odd, d) != 0;
            }
            if (f == 0 && i < cnt) s_most[unit * cap + i] = signed_most(m, odd);
          }
        }
        if (!by_row) {
          const float m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(flush(first_row, cnt))));
          odd = __any_sync(0xffffffffu, odd);
          if (lane == 0) s_most[unit * cap + part] = signed_most(m, odd);
        }
      }
      __syncthreads();
    };
    auto store = [&](int cnt) {
      for (int unit = warp / sharers; unit < units; unit += kWarps / sharers) {
        const uint8_t* rows = unit_rows(unit, cnt);
        const bool key = unit < heads;
        uint8_t* to = a.k_cache + (key ? 0 : a.v_offset) + (size_t)(head0 + (key ? unit : unit - heads)) * a.D + f * VE;
        int group = -1;
        bool odd = false;
        float r = 0.f;
        uint8_t* block = nullptr;
        for (int i = first_row; i < cnt; i += step) {
          const int row = s_row[i], g = s_of[i];
          if (row < 0) continue;
          if (g != group) {
            const float s = s_scale[g * kMaxUnits + unit];
            group = g;
            r = s == 0.f ? 0.f : 1.f / fabsf(s);
            odd = s < 0.f;
            block = to + (size_t)s_group[g].block * p.block_size * row_bytes;
          }
          if (r == 0.f) continue;
          const uint4 x0 = *reinterpret_cast<const uint4*>(rows + (size_t)i * part_bytes);
          const uint4 z0 = *reinterpret_cast<const uint4*>(rows + (size_t)i * part_bytes + gv * 16);
          float x[VE], z[VE];
          values(key, i, x0, z0, x, z);
          uint8_t* c = block + row * row_bytes;
          store_codes<VE, I8>(c, x, r, odd);
          store_codes<VE, I8>(c + gv * VE, z, r, odd);
        }
      }
    };
    // Thread x settles unit x % kMaxUnits of group x / kMaxUnits: its block's scale there.
    static_assert(kMaxGroups * kMaxUnits == kThreads, "a thread to each");
    const int my_group = tid / kMaxUnits, my_unit = tid % kMaxUnits;
    const bool settles = my_group < ng && my_unit < units;
    const int64_t my_scale = settles ? (my_unit < heads ? 0 : p.v_scales) + s_group[my_group].block * a.H + head0 +
                                           (my_unit < heads ? my_unit : my_unit - heads) : 0;
    const float old = settles ? p.scales[my_scale] : 0.f;
    float most = 0.f;
    bool odd = false;
    auto gather = [&](bool by_row) {
      if (!settles) return;
      const int first = by_row ? s_group[my_group].row0 : 0, n = by_row ? (int)s_group[my_group].n : sharers;
      for (int i = first; i < first + n; ++i) {
        const float x = s_most[my_unit * cap + i];
        most = fmaxf(most, fabsf(x));
        odd |= x < 0.f;
      }
    };
    auto settle = [&] {
      float s = 0.f, ratio = 0.f;
      if (settles && s_group[my_group].live) {
        s = fminf(fmaxf(most / (I8 ? 127.f : 448.f), kSmallestScale), kLargestScale);
        if (s_group[my_group].low > 0) {
          if (!scale_ok(old)) {
            latch(a.status, IS_ST_SCALE);
            s = 0.f;
          } else if (s > old) {
            ratio = old / s;
          } else {
            s = old;
          }
        }
        if (s > 0.f) p.scales[my_scale] = s;
      }
      s_scale[tid] = odd || s == kLargestScale ? -s : s;   // negative: elements past the codes' range, or none of it
      s_ratio[tid] = ratio;
      __syncthreads();
      for (int x = warp; x < ng * kMaxUnits; x += kWarps) {   // what blocks held already, rounded anew
        const float r = s_ratio[x];
        if (r == 0.f) continue;
        const int g = x / kMaxUnits, unit = x % kMaxUnits, chunks = a.D / 16;
        uint8_t* codes = a.k_cache + (unit < heads ? 0 : a.v_offset) + (size_t)s_group[g].block * p.block_size * row_bytes +
                         (size_t)(head0 + (unit < heads ? unit : unit - heads)) * a.D;
        for (int64_t y = lane; y < (int64_t)s_group[g].low * chunks; y += 32) {
          uint4* c = reinterpret_cast<uint4*>(codes + y / chunks * row_bytes + y % chunks * 16);
          *c = again<I8>(*c, r);
        }
      }
    };
    if (total <= cap) {
      if (!stage(0, (int)total)) return;
      find_most((int)total, ng > 1);
      gather(ng > 1);
      settle();
      store((int)total);
    } else {
      auto rows_from = [&](int64_t i0) { return (int)min((int64_t)cap, total - i0); };
      for (int64_t i0 = 0; i0 < total; i0 += cap) {
        if (!stage(i0, rows_from(i0))) return;
        find_most(rows_from(i0), false);
        gather(false);
        __syncthreads();                         // before the next rows are staged
      }
      settle();
      for (int64_t i0 = 0; i0 < total; i0 += cap) {
        if (!stage(i0, rows_from(i0))) return;
        store(rows_from(i0));
        __syncthreads();
      }
    }
    __syncthreads();                             // the round's rows and groups have been read
  }
}

// ---- reading back -----------------------------------------------------------------------

// Pairs of vectors that a lane has on their way at once, and small CTAs: more of them leave room for other warps' instead
// (36,000 tokens 35.7 us; pairs by four 37.5, with 256 threads 38.7, by eight 46).
constexpr int kReadThreads = 64;
constexpr int kReadBatch = 2;

// A warp to a token: items are pairs of vectors, keys' then values'.
template <typename T, int STYLE, bool I8>
__global__ void __launch_bounds__(kReadThreads) scaled_read_kernel(const ScaledReadArgs a, const __grid_constant__ AxisTurns at,
                                                                   int share) {
  constexpr int VE = Vec<T>::N;
  extern __shared__ __align__(16) float s_turn[];   // [warps][D]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = a.D / 2, gv = a.D / VE / 2, gv_bits = log2_of(gv), f = lane & (gv - 1);
  const int64_t w = (int64_t)blockIdx.x * (kReadThreads / 32) + warp, t = w >> log2_of(share);
  pdl_wait();
  pdl_trigger();
  if (t >= a.T) return;
  const int64_t slot = a.slots[t];
  if (slot == -1) return;                        // padding
  const int32_t of_axis = STYLE >= 0 && lane < a.n_axes ? a.positions[(size_t)lane * a.T + t] : 0;
  uint32_t bad = slot < 0 || slot >= a.n_slots ? IS_ST_BLOCK_ID : 0u;
  if (of_axis < 0 || of_axis >= IS_MAX_POSITION) bad |= IS_ST_POSITION;
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (bad) {
    if (lane == 0) latch(a.status, bad);
    return;
  }
  const int64_t block = block_of_slot(slot, a.block_size, a.block_shift);
  Turn<VE> turn;
  if constexpr (STYLE >= 0) {
    turn = warp_turn<T, STYLE>(at, s_turn + warp * a.D, half, gv, f, of_axis, -1.f);
  }
  const int n = a.H * gv;
  const uint8_t* krow = a.k_cache + (size_t)slot * a.H * a.D;
  auto load_codes = [&](const uint8_t* p) {
    if constexpr (VE == 8) return *reinterpret_cast<const uint2*>(p);
    else return make_uint2(*reinterpret_cast<const uint32_t*>(p), 0u);
  };
  auto widen = [&](const uint2& c, float s, float (&x)[VE]) {
    const uint32_t in[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < VE / 4; ++i) {
      uint32_t lo, hi;
      codes_f16x4<I8>(in[i], lo, hi);
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&lo));
      const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&hi));
      x[4 * i] = __fmul_rn(p.x, s);
      x[4 * i + 1] = __fmul_rn(p.y, s);
      x[4 * i + 2] = __fmul_rn(q.x, s);
      x[4 * i + 3] = __fmul_rn(q.y, s);
    }
  };
  const int first = (int)(w - t * share) * 32 + lane, step = share * 32;
  for (int kv = 0; kv < 2; ++kv) {
    uint8_t* out = kv ? a.v_out : a.k_out;
    if (!out) continue;
    out += (size_t)t * a.H * a.D * sizeof(T);
    const uint8_t* codes = krow + (kv ? a.v_offset : 0);
    const float* scales = a.scales + (kv ? a.v_scales : 0) + block * a.H;
    for (int i0 = first; i0 < n; i0 += kReadBatch * step) {
      uint2 c0[kReadBatch], c1[kReadBatch];
      float s[kReadBatch];
#pragma unroll
      for (int u = 0; u < kReadBatch; ++u) {
        const int i = i0 + u * step;
        if (i < n) {
          c0[u] = load_codes(codes + (2 * i - f) * VE);
          c1[u] = load_codes(codes + (2 * i - f) * VE + gv * VE);
          s[u] = scales[i >> gv_bits];
        }
      }
#pragma unroll
      for (int u = 0; u < kReadBatch; ++u) {
        const int i = i0 + u * step;
        if (i >= n) continue;
        if (!scale_ok(s[u])) {
          latch(a.status, IS_ST_SCALE);
          continue;
        }
        float x[VE], z[VE];
        widen(c0[u], s[u], x);
        widen(c1[u], s[u], z);
        if constexpr (STYLE >= 0) {
          if (kv == 0) rotate_pair<T, STYLE>(turn, x, z);
        }
        st_v4(out + (2 * i - f) * 16, Vec<T>::pack(x));
        st_v4(out + (2 * i - f) * 16 + gv * 16, Vec<T>::pack(z));
      }
    }
  }
}

template <typename T, int STYLE, bool I8>
cudaError_t launch_write_t(const ScaledWriteArgs& p, const AxisTurns& turns, const LaunchCfg& cfg) {
  const AppendArgs& a = p.a;
  const WritePlan w = plan_write(a.T, a.Hq, a.H, a.D, (int)sizeof(T), p.block_size, cfg.num_sms, STYLE >= 0);
  if (w.group_ctas + w.query_ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(&scaled_write_kernel<T, STYLE, I8>), w.smem);
  if (e != cudaSuccess) return e;
  return launch_ex(scaled_write_kernel<T, STYLE, I8>, dim3((unsigned)(w.group_ctas + w.query_ctas)), dim3(kThreads), w.smem,
                   cfg.stream, cfg.pdl, p, turns, (int)w.group_ctas, (int)w.turns, w.window, w.heads_of, w.rows, w.share);
}

template <typename T, bool I8>
cudaError_t launch_write_i(const ScaledWriteArgs& p, const AxisTurns& turns, const LaunchCfg& cfg) {
  if (!p.rotate) return launch_write_t<T, -1, I8>(p, turns, cfg);
  return p.a.style == 0 ? launch_write_t<T, 0, I8>(p, turns, cfg) : launch_write_t<T, 1, I8>(p, turns, cfg);
}

template <typename T>
cudaError_t launch_write(const ScaledWriteArgs& p, const AxisTurns& turns, const LaunchCfg& cfg) {
  return p.int8 ? launch_write_i<T, true>(p, turns, cfg) : launch_write_i<T, false>(p, turns, cfg);
}

template <typename T, int STYLE, bool I8>
cudaError_t launch_read_t(const ScaledReadArgs& a, const AxisTurns& turns, const LaunchCfg& cfg) {
  const int64_t items = (int64_t)a.H * (a.D / Vec<T>::N / 2);
  int share = 1;
  while (share < 16 && (int64_t)a.T * share < 32LL * cfg.num_sms && (int64_t)share * 32 < items) share *= 2;
  const int64_t ctas = ((int64_t)a.T * share + kReadThreads / 32 - 1) / (kReadThreads / 32);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  const size_t smem = STYLE >= 0 ? (size_t)(kReadThreads / 32) * a.D / 2 * sizeof(float2) : 0;
  return launch_ex(scaled_read_kernel<T, STYLE, I8>, dim3((unsigned)ctas), dim3(kReadThreads), smem, cfg.stream, cfg.pdl, a,
                   turns, share);
}

template <typename T, bool I8>
cudaError_t launch_read_i(const ScaledReadArgs& a, const AxisTurns& turns, const LaunchCfg& cfg) {
  if (!a.positions) return launch_read_t<T, -1, I8>(a, turns, cfg);
  return a.style == 0 ? launch_read_t<T, 0, I8>(a, turns, cfg) : launch_read_t<T, 1, I8>(a, turns, cfg);
}

template <typename T>
cudaError_t launch_read(const ScaledReadArgs& a, const AxisTurns& turns, const LaunchCfg& cfg) {
  return a.int8 ? launch_read_i<T, true>(a, turns, cfg) : launch_read_i<T, false>(a, turns, cfg);
}

}  // namespace

cudaError_t launch_scaled_write(const ScaledWriteArgs& p, const AxisTurns& turns, const LaunchCfg& cfg) {
  if (p.a.dtype == IS_F32) return launch_write<float>(p, turns, cfg);
  return p.a.dtype == IS_BF16 ? launch_write<__nv_bfloat16>(p, turns, cfg) : launch_write<__half>(p, turns, cfg);
}

cudaError_t launch_scaled_read(const ScaledReadArgs& a, const AxisTurns& turns, const LaunchCfg& cfg) {
  if (a.dtype == IS_F32) return launch_read<float>(a, turns, cfg);
  return a.dtype == IS_BF16 ? launch_read<__nv_bfloat16>(a, turns, cfg) : launch_read<__half>(a, turns, cfg);
}

}  // namespace isk
