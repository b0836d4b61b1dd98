// Writing a scaled cache (is_append_scaled, is_move_scaled) and reading it back
// (is_read_scaled): 8-bit codes with a scale for each block and KV head, keys
// and values apart.
//
// The rows that a call puts into one block share one scale per head, so the unit
// of work is a group: the adjacent tokens of one block.  With A the largest
// finite magnitude of a head's new elements (keys rotated in fp32) and qmax 127
// or 448,
//   s = A / qmax, in [2^-40, 2^40]; beside earlier rows no smaller than their scale;
//   code = round(y * (1 / s)), and earlier rows' codes round(code * s_old / s) if s grew.
// A CTA whose token begins a group takes it for up to 8 heads (other CTAs look
// at two slots and end): it computes the sines of the group's keys once, then
// each warp takes one head's keys or values.  A warp holds up to 128 pairs of
// 16-byte vectors, which is a block of 16 rows at head_dim 128 in 16 bits: loaded
// once, the largest found by shuffles, quantised and stored from registers.
// Longer groups go through twice, once for the scale and once for the codes.
// The queries are rotated by CTAs of their own, a warp or several to a token.
// Bound by memory; each input is read once and each code written once.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace isk {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHeadsPerCta = 8;
constexpr int kPairs = 4;                        // pairs of vectors a lane holds
constexpr int kRowsOfTile = 32 * kPairs;         // rows of a warp's tile with one pair a row

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
  float cs[VE], sn[VE];
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
    t.cs[4 * q] = c.x, t.cs[4 * q + 1] = c.y, t.cs[4 * q + 2] = c.z, t.cs[4 * q + 3] = c.w;
    t.sn[4 * q] = s.x, t.sn[4 * q + 1] = s.y, t.sn[4 * q + 2] = s.z, t.sn[4 * q + 3] = s.w;
  }
  return t;
}
template <typename T, int STYLE>
__device__ __forceinline__ void rotate_pair(const Turn<Vec<T>::N>& t, float (&x)[Vec<T>::N], float (&z)[Vec<T>::N]) {
  constexpr int VE = Vec<T>::N;
  if constexpr (STYLE == 0) {
#pragma unroll
    for (int e = 0; e < VE; ++e) {
      const float a = x[e], b = z[e];
      x[e] = fmaf(a, t.cs[e], -__fmul_rn(b, t.sn[e]));
      z[e] = fmaf(b, t.cs[e], __fmul_rn(a, t.sn[e]));
    }
  } else {
#pragma unroll
    for (int e = 0; e < VE / 2; ++e) {
      const float a = x[2 * e], b = x[2 * e + 1], c = z[2 * e], d = z[2 * e + 1];
      x[2 * e] = fmaf(a, t.cs[e], -__fmul_rn(b, t.sn[e]));
      x[2 * e + 1] = fmaf(b, t.cs[e], __fmul_rn(a, t.sn[e]));
      z[2 * e] = fmaf(c, t.cs[VE / 2 + e], -__fmul_rn(d, t.sn[VE / 2 + e]));
      z[2 * e + 1] = fmaf(d, t.cs[VE / 2 + e], __fmul_rn(c, t.sn[VE / 2 + e]));
    }
  }
}
// The sines of one token's pairs, computed by a warp and kept by each lane for its f.
template <typename T, int STYLE>
__device__ __forceinline__ Turn<Vec<T>::N> warp_turn(const AxisTurns& at, float* row, int half, int gv, int f, int32_t of_axis, float sign) {
  constexpr int VE = Vec<T>::N;
  const int lane = threadIdx.x & 31;
  for (int i0 = 0; i0 < half; i0 += 32) {        // half may be 8 or 16: then lanes past it repeat pairs
    const int i = (i0 + lane) % half, g = i / VE, e = i % VE, j = pair_of<VE, STYLE>(g, e, gv);
    const float2 v = turn_of(at, j, (float)__shfl_sync(0xffffffffu, of_axis, ld_table(&at.axis[j])), sign);
    row[turn_at<VE>(g, e, gv)] = v.x;
    row[turn_at<VE>(g, e + VE, gv)] = v.y;
  }
  __syncwarp();
  return load_turn<VE>(row, f, gv);
}

__device__ __forceinline__ float larger_finite(float most, float x) {
  const float a = fabsf(x);
  return a < INFINITY ? fmaxf(most, a) : most;   // false for NaN
}

// N codes (4 or 8) of a vector.
template <int N, bool I8>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&y)[N], float r) {
  float w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = e < N ? y[e % N] : 0.f;
  const uint2 c = I8 ? to_int8x8(w, r) : to_e4m3x8(w, r);
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
  const int64_t t = w / share;
  if (t >= a.T) return;
  const int first = (int)(w - t * share) * 32 + lane, step = share * 32, f = lane % gv, n = a.Hq * gv;
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

// STYLE -1: no rotation (a move).
template <typename T, int STYLE, bool I8>
__global__ void __launch_bounds__(kThreads, 2) scaled_write_kernel(const ScaledWriteArgs p, const __grid_constant__ AxisTurns at,
                                                                  int64_t group_ctas, int window, int splits, int share) {
  constexpr int VE = Vec<T>::N;
  const AppendArgs& a = p.a;
  extern __shared__ __align__(16) float s_turn[];   // the group's tile [rows][D], or a query warp's [D] each
  __shared__ int32_t s_row[kRowsOfTile];         // row of the block; -1: the token is skipped
  __shared__ int64_t s_from[kRowsOfTile];
  __shared__ uint32_t s_leaders;
  __shared__ struct { int64_t block, n; int32_t low; } s_group;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, half = a.D / 2;
  pdl_wait();
  pdl_trigger();
  if ((int64_t)blockIdx.x >= group_ctas) {
    if constexpr (STYLE >= 0) {
      rotate_queries<T, STYLE>(a, at, s_turn + warp * a.D, ((int64_t)blockIdx.x - group_ctas) * kWarps + warp, share);
    }
    return;
  }
  const int64_t begin = blockIdx.x / splits * (int64_t)window;
  const int head0 = (int)(blockIdx.x % splits) * kHeadsPerCta, heads = min(kHeadsPerCta, a.H - head0);
  auto block_at = [&](int64_t t) -> int64_t {
    if (t < 0 || t >= a.T) return -1;
    const int64_t slot = a.slots[t];
    return slot < 0 || slot >= a.n_slots ? -1 : block_of_slot(slot, p.block_size, p.block_shift);
  };
  // The groups that begin in this CTA's tokens begin .. begin + window - 1 (window <= 16): lane i looks at token begin - 1 + i.
  // One warp looks, so that the CTA agrees on its groups whatever happens to the caller's slots meanwhile.
  int64_t mine = -1;
  if (warp == 0) {
    mine = block_at(begin - 1 + lane);
    const int64_t before = __shfl_up_sync(0xffffffffu, mine, 1);
    const bool ours = lane >= 1 && lane <= window && begin - 1 + lane < a.T;
    const uint32_t found = __ballot_sync(0xffffffffu, ours && mine >= 0 && mine != before);
    if (head0 == 0 && ours && mine < 0 && a.slots[begin - 1 + lane] != -1) latch(a.status, IS_ST_BLOCK_ID);
    if (lane == 0) s_leaders = found;
  }
  __syncthreads();
  for (uint32_t leaders = s_leaders; leaders; leaders &= leaders - 1) {
  const int first = __ffs(leaders) - 1;
  const int64_t t0 = begin - 1 + first;
  if (warp == 0) {
    const int64_t block = __shfl_sync(0xffffffffu, mine, first);
    int64_t n = 0;                               // its tokens, 31 at a time
    int32_t low = p.block_size;                  // the lowest of their rows: below it the block is held already
    for (uint32_t more = ~0u; n % 31 == 0 && more != 0;) {
      const int64_t t = t0 + n + lane;
      const bool in = lane < 31 && block_at(t) == block;
      if (in) low = min(low, (int32_t)max(a.slots[t] - block * p.block_size, (int64_t)0));
      more = __ballot_sync(0xffffffffu, in);
      n += __ffs(~more) - 1;             // bit 31 is 0
    }
    low = __reduce_min_sync(0xffffffffu, low);
    if (lane == 0) {
      s_group.block = block;
      s_group.n = max(n, (int64_t)1);
      s_group.low = low;
    }
  }
  __syncthreads();
  const int64_t block = s_group.block, n = s_group.n;
  const int32_t low = s_group.low;
  const int gv = a.D / VE / 2, f = lane % gv, tile_rows = kRowsOfTile / gv, row_step = 32 / gv;
  const int units = 2 * heads;                   // keys of each head, then values
  // Tokens t0 + i0 .. of the group: their rows and sources, and their keys' sines.
  bool any = false;                              // some token is not skipped
  auto stage = [&](int64_t i0) {
    const int cnt = (int)min((int64_t)tile_rows, n - i0);
    bool put = false;
    __syncthreads();
    for (int i = tid; i < cnt; i += kThreads) {
      const int64_t t = t0 + i0 + i;
      const int64_t in_block = a.slots[t] - block * p.block_size;
      int32_t row = in_block >= 0 && in_block < p.block_size ? (int32_t)in_block : -1;
      int64_t from = t;
      if (p.from) {
        from = p.from[t];
        if (from < 0 || from >= p.n_from) {
          if (from != -1) latch(a.status, IS_ST_BLOCK_ID);
          row = -1;
        }
      }
      if constexpr (STYLE >= 0) {
        for (int x = 0; x < a.n_axes; ++x) {
          const int32_t pos = a.positions[(size_t)x * a.T + t];
          if (pos < 0 || pos >= IS_MAX_POSITION) {
            latch(a.status, IS_ST_POSITION);
            row = -1;
          }
        }
      }
      s_row[i] = row;
      s_from[i] = from;
      put |= row >= 0;
    }
    any |= __syncthreads_or(put) != 0;
    return cnt;
  };
  auto stage_turns = [&](int64_t i0, int cnt) {
    if constexpr (STYLE >= 0) {
      for (int x = tid; x < cnt * half; x += kThreads) {
        const int i = x / half, g = (x - i * half) / VE, e = x % VE, j = pair_of<VE, STYLE>(g, e, gv);
        const float2 v = turn_of(at, j, (float)a.positions[(size_t)ld_table(&at.axis[j]) * a.T + t0 + i0 + i], 1.f);
        s_turn[i * a.D + turn_at<VE>(g, e, gv)] = v.x;
        s_turn[i * a.D + turn_at<VE>(g, e + VE, gv)] = v.y;
      }
      __syncthreads();
    }
  };
  constexpr int kMine = 2 * kHeadsPerCta / kWarps;   // units of a warp, at most
  uint4 x0[kMine][kPairs], x1[kMine][kPairs];
  auto load = [&](int m, int cnt) {
    const int unit = warp + m * kWarps;
    if (unit >= units) return;
    const int head = head0 + unit % heads;
    const uint8_t* src = (unit < heads ? a.k : a.v) + ((size_t)head * a.D) * sizeof(T) + f * 16;
    const int64_t stride = unit < heads ? a.k_stride : a.v_stride;
#pragma unroll
    for (int u = 0; u < kPairs; ++u) {
      const int i = lane / gv + u * row_step;
      x0[m][u] = x1[m][u] = make_uint4(0, 0, 0, 0);
      if (i < cnt && s_row[i] >= 0) {
        const uint8_t* r = src + s_from[i] * stride;
        x0[m][u] = *reinterpret_cast<const uint4*>(r);
        x1[m][u] = *reinterpret_cast<const uint4*>(r + gv * 16);
      }
    }
  };
  auto values = [&](int m, int u, float (&x)[VE], float (&z)[VE]) {
    Vec<T>::unpack(x0[m][u], x);
    Vec<T>::unpack(x1[m][u], z);
    if constexpr (STYLE >= 0) {
      if (warp + m * kWarps < heads)
        rotate_pair<T, STYLE>(load_turn<VE>(s_turn + (lane / gv + u * row_step) * a.D, f, gv), x, z);
    }
  };
  auto largest = [&](int m, int cnt, float most) {
#pragma unroll
    for (int u = 0; u < kPairs; ++u) {
      const int i = lane / gv + u * row_step;
      if (i < cnt && s_row[i] >= 0) {
        float x[VE], z[VE];
        values(m, u, x, z);
#pragma unroll
        for (int e = 0; e < VE; ++e) most = larger_finite(larger_finite(most, x[e]), z[e]);
      }
    }
    return most;
  };
  auto codes_of = [&](int unit) {                // row 0 of the block, this head
    return a.k_cache + (unit < heads ? 0 : a.v_offset) + ((size_t)block * p.block_size * a.H + head0 + unit % heads) * a.D;
  };
  const size_t row_bytes = (size_t)a.H * a.D;
  // The block's scale, and what it holds already rounded anew; 0: the block's scale is none.
  auto settle = [&](int unit, float most) -> float {
    most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
    float* at_scale = p.scales + (unit < heads ? 0 : p.v_scales) + block * a.H + head0 + unit % heads;
    float s = fminf(fmaxf(most / (I8 ? 127.f : 448.f), kSmallestScale), kLargestScale);
    if (low > 0) {
      const float old = *at_scale;
      if (!scale_ok(old)) {
        if (lane == 0) latch(a.status, IS_ST_SCALE);
        return 0.f;
      }
      if (s > old) {
        const float ratio = old / s;
        uint8_t* codes = codes_of(unit);
        const int chunks = a.D / 16;
        for (int64_t x = lane; x < (int64_t)low * chunks; x += 32) {
          uint4* c = reinterpret_cast<uint4*>(codes + x / chunks * row_bytes + x % chunks * 16);
          *c = again<I8>(*c, ratio);
        }
      } else {
        s = old;
      }
    }
    __syncwarp();
    if (lane == 0) *at_scale = s;
    return s;
  };
  auto put = [&](int m, int cnt, float s) {
    const int unit = warp + m * kWarps;
    const float r = 1.f / s;
    uint8_t* codes = codes_of(unit) + f * VE;
#pragma unroll
    for (int u = 0; u < kPairs; ++u) {
      const int i = lane / gv + u * row_step;
      if (i < cnt && s_row[i] >= 0) {
        float x[VE], z[VE];
        values(m, u, x, z);
        uint8_t* c = codes + s_row[i] * row_bytes;
        store_codes<VE, I8>(c, x, r);
        store_codes<VE, I8>(c + gv * VE, z, r);
      }
    }
  };
  if (n <= tile_rows) {
    const int cnt = stage(0);
    if (!any) continue;
#pragma unroll
    for (int m = 0; m < kMine; ++m) load(m, cnt);    // under way while the sines are computed
    stage_turns(0, cnt);
#pragma unroll
    for (int m = 0; m < kMine; ++m)
      if (warp + m * kWarps < units) {
        const float s = settle(warp + m * kWarps, largest(m, cnt, 0.f));
        if (s > 0.f) put(m, cnt, s);
      }
    continue;
  }
  float most[kMine], scale[kMine];
#pragma unroll
  for (int m = 0; m < kMine; ++m) most[m] = 0.f;
  for (int64_t i0 = 0; i0 < n; i0 += tile_rows) {
    const int cnt = stage(i0);
    stage_turns(i0, cnt);
#pragma unroll
    for (int m = 0; m < kMine; ++m)
      if (warp + m * kWarps < units) {
        load(m, cnt);
        most[m] = largest(m, cnt, most[m]);
      }
  }
  if (!any) continue;
#pragma unroll
  for (int m = 0; m < kMine; ++m) scale[m] = warp + m * kWarps < units ? settle(warp + m * kWarps, most[m]) : 0.f;
  for (int64_t i0 = 0; i0 < n; i0 += tile_rows) {
    const int cnt = stage(i0);
    stage_turns(i0, cnt);
#pragma unroll
    for (int m = 0; m < kMine; ++m)
      if (scale[m] > 0.f) {
        load(m, cnt);
        put(m, cnt, scale[m]);
      }
  }
  }
}

// ---- reading back -----------------------------------------------------------------------

constexpr int kReadThreads = 256;
constexpr int kReadBatch = 4;

// A warp to a token: items are pairs of vectors, keys' then values'.
template <typename T, int STYLE, bool I8>
__global__ void __launch_bounds__(kReadThreads) scaled_read_kernel(const ScaledReadArgs a, const __grid_constant__ AxisTurns at,
                                                                   int share) {
  constexpr int VE = Vec<T>::N;
  extern __shared__ __align__(16) float s_turn[];   // [warps][D]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = a.D / 2, gv = a.D / VE / 2, f = lane % gv;
  const int64_t w = (int64_t)blockIdx.x * (kReadThreads / 32) + warp, t = w / share;
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
          s[u] = scales[i / gv];
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
  constexpr int VE = Vec<T>::N;
  const AppendArgs& a = p.a;
  const int splits = (a.H + kHeadsPerCta - 1) / kHeadsPerCta;
  // One token a CTA up to 16 CTAs an SM, then several: most tokens of a prompt begin no group, and their CTAs, though they
  // end at once, hold up the others (8000 tokens: 74.6 us with one token a CTA).
  const int window = (int)std::min<int64_t>(16, (a.T + 16LL * cfg.num_sms - 1) / (16LL * cfg.num_sms));
  const int64_t group_ctas = ((int64_t)a.T + window - 1) / window * splits;
  // Warps to a token's queries: as many as keep a lane one batch busy while the SMs have room for 32 warps each.
  const int64_t items = (int64_t)a.Hq * (a.D / VE / 2);
  int share = 1;
  while (share < 16 && (int64_t)a.T * share < 32LL * cfg.num_sms && (int64_t)share * 32 < items) share *= 2;
  const int64_t q_ctas = a.Hq > 0 ? ((int64_t)a.T * share + kWarps - 1) / kWarps : 0;
  if (group_ctas + q_ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  const size_t tile = STYLE >= 0 ? (size_t)kRowsOfTile * VE * sizeof(float2) : 0;   // kRowsOfTile / gv rows of D floats
  const size_t queries = STYLE >= 0 ? (size_t)kWarps * a.D / 2 * sizeof(float2) : 0;
  return launch_ex(scaled_write_kernel<T, STYLE, I8>, dim3((unsigned)(group_ctas + q_ctas)), dim3(kThreads),
                   tile > queries ? tile : queries, cfg.stream, cfg.pdl, p, turns, group_ctas, window, splits, share);
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
