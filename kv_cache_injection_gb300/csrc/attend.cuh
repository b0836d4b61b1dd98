// What the kernels of is_attend share: the batch as they see it, the workspace
// and the join of an item's parts.
#pragma once

#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace isk {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// The reference m of a row, in the base-2 exponent: a weight is 2^(x - m), and m
// moves only when a logit passes it by more than kLazy + kRaise, to kRaise
// below that logit.  So the largest weight is at least 2^kRaise and none passes
// 2^(kLazy + kRaise).  fp16 weights are raised by 7, to 2^15 at most (fp16 ends
// at 65504): the faintest steps, 2^-24, are then 2^-31 of the largest weight, and
// weights keep 11 bits down to 2^-21 of it.  (Unraised, of what 2999 keys at
// 2^-26 add beside a strong one, such as a prompt's first token, a seventh to
// a fifth was lost.)  bf16 and fp32 have the exponents.
constexpr float kLazy = 8.f;
template <typename M>
constexpr float kRaise = std::is_same<M, __half>::value ? 7.f : 0.f;
// What a logit has to pass to move m; rounded down, so that it holds where a
// step of m is larger than the bound.
template <typename M>
__device__ __forceinline__ float lazy_bound(float m) {
  return __fadd_rd(m, kLazy + kRaise<M>);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// What the attention takes of the scales of a key (scaled cache): K scale, log2 of
// the V scale and its reciprocal.  The hardware's log2 is off by 2^-22 near 1, so
// the exponent is taken off first; the reciprocal is off by one step.
__device__ __forceinline__ float4 key_scales(float ks, float vs) {
  const int e = (__float_as_int(vs) - 0x3f400000) >> 23;   // vs = 2^e f, f in [0.75, 1.5)
  float l, r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(l) : "f"(__int_as_float(__float_as_int(vs) - (e << 23))));
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(vs));
  return make_float4(ks, (float)e + l, r, 0.f);
}

// Block of position p: a shift where the block size is a power of two.
__device__ __forceinline__ int32_t block_of(const AttendArgs& a, int32_t p) {
  return a.block_shift >= 0 ? p >> a.block_shift : p / a.block_size;
}

// ---- the batch ------------------------------------------------------------------

// One request as the kernel sees it.
struct Req {
  int32_t row0, n;       // first query row, query rows
  int32_t seq;           // tokens in the cache
  int32_t kb, ke;        // positions some row may see
};

// Requests whose rows or length make no sense have no rows.
__device__ __forceinline__ Req read_request(const AttendArgs& a, int r, bool report) {
  Req q;
  const int32_t s0 = a.q_start ? a.q_start[r] : r, s1 = a.q_start ? a.q_start[r + 1] : r + 1;
  const int32_t seq = a.seq_len[r];
  const int64_t n = (int64_t)s1 - s0;
  if (n < 0 || n > a.max_q || s0 < 0 || s1 > a.T || seq < 0 || seq > IS_MAX_POSITION) {
    if (report) latch(a.status, IS_ST_COUNT);
    q.row0 = q.n = q.seq = q.kb = q.ke = 0;
    return q;
  }
  q.row0 = s0;
  q.n = (int32_t)n;
  q.seq = seq;
  const int64_t cap = (int64_t)a.max_blocks * a.block_size;
  q.ke = (int32_t)min((int64_t)seq, cap);
  if (report && n > 0 && q.ke < seq) latch(a.status, IS_ST_BLOCK_TABLE);
  q.kb = a.window > 0 ? max(0, (int32_t)max((int64_t)seq - n - a.window + 1, (int64_t)0)) : 0;
  if (q.kb > q.ke) q.kb = q.ke;
  return q;
}

// x / d for non-negative operands, in 32-bit arithmetic when both fit.
__device__ __forceinline__ int64_t div_small(int64_t x, int64_t d) {
  return ((x | d) >> 31) == 0 ? (int64_t)((uint32_t)x / (uint32_t)d) : x / d;
}

// ---- workspace -------------------------------------------------------------------
// [ctas] join records, then two partials per CTA: of the item its run begins
// in (slot 2 c) and of the one it ends in (2 c + 1), when those cross its ends.
struct JoinRecord {
  int32_t parts;         // 0: nothing to join
  int32_t slot0;         // the first part; part i > 0 is slot 2 * (cta + i)
  int32_t row0;          // first query row of the request
  int32_t head;          // KV head
  int32_t rho0, rows;    // the item's first query row (token * G + head of the group) and their number
};
constexpr size_t kRecordBytes = 32;
constexpr int kMaxCtas = 1024;
constexpr size_t partials_offset() { return kMaxCtas * kRecordBytes; }
template <int ROWS, int D>
struct Partial {
  float o[ROWS][D];
  float m[ROWS], l[ROWS];
};
// The same where a thread writes whole rows (the prompt kernel): by columns of
// eight, so that the 32 lanes' rows of a store lie behind one another.
template <int ROWS, int D>
struct PartialByEights {
  float o[D / 8][ROWS][8];
  float m[ROWS], l[ROWS];
};

__device__ __forceinline__ JoinRecord* record_of(const AttendArgs& a, int cta) {
  return reinterpret_cast<JoinRecord*>(a.workspace + (size_t)cta * kRecordBytes);
}
template <typename P>
__device__ __forceinline__ P* partial_of(const AttendArgs& a, int slot) {
  return reinterpret_cast<P*>(a.workspace + partials_offset()) + slot;
}

template <typename T>
__device__ __forceinline__ void store_out(const AttendArgs& a, const Req& q, int head, int rho, int d, float x, float y) {
  const int tok = rho / a.G;
  T* p = reinterpret_cast<T*>(a.out) + ((size_t)(q.row0 + tok) * a.Hq + (size_t)head * a.G + (rho - tok * a.G)) * a.D + d;
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float2*>(p) = make_float2(x, y);
  else
    *reinterpret_cast<uint32_t*>(p) = Vec<T>::pack2(x, y);
}
__device__ __forceinline__ void store_lse(const AttendArgs& a, const Req& q, int head, int rho, float m, float l) {
  if (!a.lse) return;
  const int tok = rho / a.G;
  a.lse[(size_t)(q.row0 + tok) * a.Hq + (size_t)head * a.G + (rho - tok * a.G)] =
      l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Parts first, first + stride, ... of four columns of a row, added to m, l and
// o; read N at a time so that their latencies overlap.  (One at a time: one
// request of 1313 tokens 8.6 us, 8.2 with four; where a row has two or three
// parts two at a time are best, 16 requests' prompts 53.7 us, 55.0 with four.)
template <int N, typename P, typename At>
__device__ __forceinline__ void add_parts(const AttendArgs& a, const JoinRecord& rec, int first, int stride, int row, At at,
                                          float& m, float& l, float4& o) {
  for (int i0 = first; i0 < rec.parts; i0 += N * stride) {
    float pm[N], pl[N];
    float4 v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int i = i0 + k * stride;
      pm[k] = -INFINITY;
      pl[k] = 0.f;
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i < rec.parts) {
        const P* p = partial_of<P>(a, i == 0 ? rec.slot0 : 2 * ((int)blockIdx.x + i));
        pm[k] = p->m[row];
        pl[k] = p->l[row];
        v[k] = *reinterpret_cast<const float4*>(at(p));
      }
    }
    float mn = m;
#pragma unroll
    for (int k = 0; k < N; ++k) mn = fmaxf(mn, pm[k]);
    const float mz = mn == -INFINITY ? 0.f : mn, f = ex2(m - mz);
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
    l *= f;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const float g = ex2(pm[k] - mz);
      o = make_float4(fmaf(g, v[k].x, o.x), fmaf(g, v[k].y, o.y), fmaf(g, v[k].z, o.z), fmaf(g, v[k].w, o.w));
      l = fmaf(g, pl[k], l);
    }
    m = mn;
  }
}

// Adds up the parts of an item that several CTAs worked on: one CTA per
// (record, row) or several rows of a record, the threads splitting the parts
// and the head dimension.
constexpr int kJoinThreads = 256;

template <typename T, int ROWS, int D>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const AttendArgs a) {
  constexpr int LANES = D / 4, GROUPS = kJoinThreads / LANES;
  __shared__ float4 s_o[GROUPS][LANES];
  __shared__ float s_m[GROUPS], s_l[GROUPS];
  pdl_wait();
  pdl_trigger();
  const int cta = blockIdx.x;
  const JoinRecord rec = *record_of(a, cta);
  if (rec.parts == 0) return;
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  for (int row = blockIdx.y; row < rec.rows; row += gridDim.y) {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    using P = Partial<ROWS, D>;
    add_parts<4, P>(a, rec, group, GROUPS, row, [&](const P* p) { return &p->o[row][lane * 4]; }, m, l, o);
    s_o[group][lane] = o;
    if (lane == 0) {
      s_m[group] = m;
      s_l[group] = l;
    }
    __syncthreads();
    if (group == 0) {
      float mx = -INFINITY;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) mx = fmaxf(mx, s_m[g]);
      const float mz = mx == -INFINITY ? 0.f : mx;
      o = make_float4(0.f, 0.f, 0.f, 0.f);
      l = 0.f;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        const float f = ex2(s_m[g] - mz);
        const float4 v = s_o[g][lane];
        o = make_float4(fmaf(f, v.x, o.x), fmaf(f, v.y, o.y), fmaf(f, v.z, o.z), fmaf(f, v.w, o.w));
        l = fmaf(f, s_l[g], l);
      }
      Req q;
      q.row0 = rec.row0;
      const float inv = l == 0.f ? 0.f : a.v_scale / l;
      if (l == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
      const int rho = rec.rho0 + row;
      store_out<T>(a, q, rec.head, rho, lane * 4, o.x * inv, o.y * inv);
      store_out<T>(a, q, rec.head, rho, lane * 4 + 2, o.z * inv, o.w * inv);
      if (lane == 0) store_lse(a, q, rec.head, rho, mx, l);
    }
    __syncthreads();                     // s_o is read before the next row's is written
  }
}

// The same for items of many rows and few parts: D / 4 lanes take a row, all
// parts of it.  By eights a warp takes 32 columns of four rows, so that it reads
// 128 bytes at a time.
template <typename T, int ROWS, int D, bool EIGHTS>
__global__ void __launch_bounds__(kJoinThreads) attend_join_rows_kernel(const AttendArgs a) {
  constexpr int LANES = D / 4, AT_ONCE = kJoinThreads / LANES;
  pdl_wait();
  pdl_trigger();
  const int cta = blockIdx.x;
  const JoinRecord rec = *record_of(a, cta);
  if (rec.parts == 0) return;
  using P = std::conditional_t<EIGHTS, PartialByEights<ROWS, D>, Partial<ROWS, D>>;
  const int warp = threadIdx.x / 32, in_warp = threadIdx.x % 32;
  const int lane = EIGHTS ? warp % (D / 32) * 8 + in_warp / 8 * 2 + in_warp % 2 : threadIdx.x % LANES;
  const int first = EIGHTS ? warp / (D / 32) * 4 + in_warp / 2 % 4 : threadIdx.x / LANES;
  for (int row = blockIdx.y * AT_ONCE + first; row < rec.rows; row += gridDim.y * AT_ONCE) {
    float m = -INFINITY, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto at = [&](const P* p) {
      if constexpr (EIGHTS)
        return &p->o[lane / 2][row][lane % 2 * 4];
      else
        return &p->o[row][lane * 4];
    };
    add_parts<2, P>(a, rec, 0, 1, row, at, m, l, o);
    Req q;
    q.row0 = rec.row0;
    const float inv = l == 0.f ? 0.f : a.v_scale / l;
    if (l == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
    const int rho = rec.rho0 + row;
    store_out<T>(a, q, rec.head, rho, lane * 4, o.x * inv, o.y * inv);
    store_out<T>(a, q, rec.head, rho, lane * 4 + 2, o.z * inv, o.w * inv);
    if (lane == 0) store_lse(a, q, rec.head, rho, m, l);
  }
}

}  // namespace isk
