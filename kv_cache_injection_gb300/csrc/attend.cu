// Softmax attention of each request's last tokens over its paged cache
// (is_attend), for few query rows per request: one new token, or a handful.
//
// With one new token every key and value is used once per query head of its
// group, so the time is that of reading the cache: 2 * keys * H * D elements.
// What the kernel is built around:
//
// - One item is a (request, KV head, tile of up to 8 * NT query rows), its
//   rows being the query heads of the group for each new token; the keys and
//   values are read once for all of them.
// - The items' keys are numbered in units of kWarps * KT keys over the whole
//   call and each CTA of a persistent grid takes one contiguous run of units,
//   found from the lengths on the device: a long request is spread over many
//   CTAs, short ones share one, whatever the batch looks like.  An item that
//   crosses CTAs leaves an unnormalised partial (m, l, O) per CTA in the
//   workspace and a second kernel adds them up in CTA order, so results do not
//   depend on timing.  (Joining in the CTA that finishes last instead, counted
//   with atomics, measured the same at 100 requests and 17 us instead of 9 at
//   one, where a dozen CTAs meet on one counter.)
// - Inside a CTA every warp runs alone on its own tiles of KT keys, with its
//   own cp.async ring in shared memory (no block barrier in the loop) and its
//   own running maximum m, sum l and output O, joined once at the end, under
//   the first loads of the CTA's next item.  Three CTAs of 64 KB rings fit an SM:
//   12 warps with a tile of 8 KB on its way each.  (Two CTAs with three tiles a
//   warp: 100 requests 51.5 us, 48.5 with three CTAs of two; a ring with K and V
//   released separately, so that half a tile more is in flight: 4 % slower, for
//   the second pass over the rows' addresses.)
// - The tensor cores take the transposed products S^T = K Q^T and
//   O^T = V^T P^T (mma.m16n8k16): the keys and the head dimension fill the
//   16-row side and the query rows the 8-column side, so a group of 4 to 8
//   query heads wastes little.  tcgen05 wants 128 (or 64) rows and gains
//   nothing here: the SMs issue in 28 % of their slots (bf16) while the memory
//   is the limit.
// - The maximum moves only when a logit passes it by more than 2^8 (in the
//   base-2 exponent), so the usual tile costs one vote instead of a reduction;
//   fp16 weights are raised by 2^7 (see kRaise).
//
// Sums, maxima and O are fp32; the weights are rounded to 16 bits for the
// second product, which takes nothing else.  Up to 8 rows a request what the
// rounding took off is multiplied too (kRest), so that a weight keeps 2^-16 or
// 2^-22; with more rows it is off by 2^-8 or 2^-11, like the output.  FP8 keys and
// values are exact in fp16, so that path computes in fp16, a bf16 query row
// being scaled by a power of two that brings its largest element to [2^14,
// 2^15) (undone in fp32).  That is exact for elements down to 2^-31 of the
// largest; fainter ones are rounded by 2^-39 of the largest at most.
// fp32 caches use fp32 fused multiply-adds throughout.
//
// Measured (H = 8, D = 128, bf16 unless said): 4 requests of 60,000-131,000
// tokens 260 us on one GPU and 268 on another, 6.7 to 6.9 TB/s, the rate of a
// plain copy; 64 requests of 500-8000 tokens 173 us (6.2 TB/s), with an FP8 cache
// 92 and 101 us (5.9 and 5.3 TB/s, the SMs issuing in 34 % of their slots); 100
// requests of 300-2048 tokens (H = 4) 46.2 and 46.8 us against 34.3 for their
// bytes, the rest being the start (2 us to find the runs, 3 more until the first
// tile has landed), the last tiles and the join.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "attend.cuh"
#include "block_scan.cuh"

namespace isk {

constexpr int kWarps = 4;
constexpr int kAttendThreads = kWarps * 32;
// ---- primitives ---------------------------------------------------------------

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// The two 16-bit values of a register.
template <typename M>
__device__ __forceinline__ float2 unpack2(uint32_t x) {
  if constexpr (std::is_same<M, __half>::value) return __half22float2(*reinterpret_cast<const __half2*>(&x));
  else return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}
template <typename M>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (sizeof(M) == 2 && std::is_same<M, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Item tables of a request: tiles of `rows` query rows, units of `unit` keys.
__device__ __forceinline__ int32_t tiles_of(const AttendArgs& a, const Req& q, int rows) {
  return (q.n * a.G + rows - 1) / rows;
}
__device__ __forceinline__ int32_t units_of(const Req& q, int unit) { return max(1, (q.ke - q.kb + unit - 1) / unit); }

// ---- tile engines -------------------------------------------------------------------
// An engine holds one warp's share of an item: the query rows, m, l and O.
//   kRows rows, kKeys keys a tile, kRowBytes bytes of a K or V row in shared memory
//   begin   loads the query rows
//   step    adds one tile (K rows at ks, V rows at vs, swizzled 16-byte chunks)
//   finish  writes O to so[kRows][kPitch] and (m, l) to sm[2 kRows]

// Which keys of a tile which rows see.
struct TileMask {
  int key0;              // position of the tile's first key
  uint32_t valid;        // keys that are read (in range and named by the table)
  bool check;            // some row does not see some valid key, or a key is not valid
};

// 16-byte chunk c of row `row`: rows of 128 bytes or more rotate their chunks
// by the row so that eight rows' chunks of one column lie in different banks;
// rows of 64 bytes, two to a line, by half the row.
template <int ROWB>
__device__ __forceinline__ uint32_t chunk_at(int row, int c) {
  return (uint32_t)row * ROWB + (uint32_t)((ROWB >= 128 ? c ^ (row & 7) : c ^ ((row >> 1) & 3)) * 16);
}

template <typename T, bool F8, int D_, int NT>
struct MmaEngine {
  static constexpr int D = D_;
  static constexpr int kRows = 8 * NT;
  static constexpr int kRowBytes = F8 ? D : 2 * D;
  static constexpr int kKeys = kRowBytes >= 256 ? 16 : 32;
  static constexpr int kMt = kKeys / 16;
  static constexpr int kPitch = kRows * (D + 4) * 4 <= 2 * kKeys * kRowBytes ? D + 4 : D;   // fits a tile
  static constexpr int kSharedQ = 0;
  static constexpr int kMostPerSm = D * NT >= 256 ? 2 : 3;   // what the registers allow
  using M = typename std::conditional<F8, __half, T>::type;   // type of the products' operands
  // Whether what a weight's rounding to M takes off is multiplied too: where M is no finer than the output, and the
  // memory hides it.  100 requests of 300-2048 tokens: 45.9 us without, 46.2 with, error against 64 bits 2.29e-3 and
  // 1.66e-3, the output's own rounding.  With two column tiles it costs 1.3 % at head_dim 128, 4.5 % at 64.
  static constexpr bool kRest = NT == 1 && !(F8 && !std::is_same<T, __half>::value);

  uint32_t q[D / 16][NT][2];
  float o[D / 16][NT][4];
  float m[NT][2], l[NT][2], sc[NT][2];
  int lim[NT][2];        // last position the row sees; -1 and below: none

  __device__ __forceinline__ void begin(const AttendArgs& a, const Req& rq, int head, int tile, float*) {
    const int lane = threadIdx.x & 31, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int rho = tile * kRows + nt * 8 + (lane >> 2), tok = rho / a.G;
      const bool in = tok < rq.n;
      const T* src = reinterpret_cast<const T*>(a.q + (int64_t)(rq.row0 + (in ? tok : 0)) * a.q_stride) +
                     ((size_t)head * a.G + (in ? rho - tok * a.G : 0)) * D;
      int shift = 0;
      if (F8 && !std::is_same<T, __half>::value) {
        // bf16 to fp16: scale the row by a power of two that brings its largest element to [2^14, 2^15)
        float big = 0.f;
        uint32_t raw[D / 16][2];
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint2 w = in ? *reinterpret_cast<const uint2*>(src + 16 * c + 4 * t) : make_uint2(0, 0);
          raw[c][0] = w.x;
          raw[c][1] = w.y;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            big = fmaxf(big, fmaxf(fabsf(__uint_as_float(raw[c][i] << 16)), fabsf(__uint_as_float(raw[c][i] & 0xffff0000u))));
        }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        if (big > 0.f && big < INFINITY) shift = min(14 - (int)(((__float_as_uint(big) >> 23) & 255u) - 127), 120);
        const float f = __uint_as_float((uint32_t)(shift + 127) << 23);
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            q[c][nt][i] = Vec<__half>::pack2(__uint_as_float(raw[c][i] << 16) * f, __uint_as_float(raw[c][i] & 0xffff0000u) * f);
      } else {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          if (F8) {        // four consecutive elements: see the key fragments in step()
            const uint2 w = in ? *reinterpret_cast<const uint2*>(src + 16 * c + 4 * t) : make_uint2(0, 0);
            q[c][nt][0] = w.x;
            q[c][nt][1] = w.y;
          } else {
            q[c][nt][0] = in ? *reinterpret_cast<const uint32_t*>(src + 16 * c + 2 * t) : 0u;
            q[c][nt][1] = in ? *reinterpret_cast<const uint32_t*>(src + 16 * c + 2 * t + 8) : 0u;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {      // the columns of S^T this lane holds: rows 2 t and 2 t + 1
        const int col = nt * 8 + 2 * t + i, ctok = (tile * kRows + col) / a.G;
        lim[nt][i] = ctok < rq.n ? rq.seq - rq.n + ctok : -1;
        m[nt][i] = -INFINITY;
        l[nt][i] = 0.f;
        const int sh = F8 ? __shfl_sync(0xffffffffu, shift, (2 * t + i) * 4) : 0;
        sc[nt][i] = a.scale * kLog2e * (F8 ? __uint_as_float((uint32_t)(127 - sh) << 23) : 1.f);
      }
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[c][nt][e] = 0.f;
    }
  }

  __device__ __forceinline__ void step(const AttendArgs& a, uint32_t ks, uint32_t vs, const TileMask& tm, float*) {
    const int lane = threadIdx.x & 31;
    float s[kMt][NT][4];
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
    // S^T.  ldmatrix lane i addresses row (i & 7) of 8x8 matrix i >> 3.
    const int mrow = lane & 7, mat = lane >> 3;
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt) {
      const int row = mt * 16 + (mat & 1) * 8 + mrow;
      if constexpr (!F8) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t k[4];
          ldmatrix4(ks + chunk_at<kRowBytes>(row, 2 * c + (mat >> 1)), k);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816<M>(s[mt][nt], k, q[c][nt][0], q[c][nt][1]);
        }
      } else {
        // A chunk holds 16 elements; lane t of a row gets elements 4 t .. 4 t + 3, which stand in for the
        // product's k = 2 t, 2 t + 1, 2 t + 8, 2 t + 9 (the query fragment uses the same order).
#pragma unroll
        for (int c = 0; c < D / 16; c += 2) {
          uint32_t b[4];
          ldmatrix4(ks + chunk_at<kRowBytes>(row, c + (mat >> 1)), b);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t k[4];
            e4m3x4_f16x4(b[2 * u], k[0], k[2]);
            e4m3x4_f16x4(b[2 * u + 1], k[1], k[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<M>(s[mt][nt], k, q[c + u][nt][0], q[c + u][nt][1]);
          }
        }
      }
    }
    // Scaled logits (base 2), hidden keys at -inf.
    bool over = false;
    float bound[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) bound[nt][i] = lazy_bound<M>(m[nt][i]);
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = __fmul_rn(s[mt][nt][e], sc[nt][e & 1]);   // not fused with - m: far logits
          if (tm.check) {
            const int key = mt * 16 + (lane >> 2) + (e >> 1) * 8, j = tm.key0 + key;
            const bool see = ((tm.valid >> key) & 1u) && j <= lim[nt][e & 1] &&
                             (a.window == 0 || j > lim[nt][e & 1] - a.window);
            if (!see) x = -INFINITY;
          }
          s[mt][nt][e] = x;
          over |= x > bound[nt][e & 1];
        }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float x = -INFINITY;
#pragma unroll
          for (int mt = 0; mt < kMt; ++mt) x = fmaxf(x, fmaxf(s[mt][nt][i], s[mt][nt][i + 2]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          const float mn = fmaxf(m[nt][i], x - kRaise<M>);
          const float f = mn == -INFINITY ? 1.f : ex2(m[nt][i] - mn);
          m[nt][i] = mn;
          l[nt][i] *= f;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) {
            o[c][nt][i] *= f;
            o[c][nt][i + 2] *= f;
          }
        }
    }
    uint32_t p[kMt][NT][2], rest[kMt][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0], m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
      for (int mt = 0; mt < kMt; ++mt) {
        const float p0 = ex2(s[mt][nt][0] - m0), p1 = ex2(s[mt][nt][1] - m1);
        const float p2 = ex2(s[mt][nt][2] - m0), p3 = ex2(s[mt][nt][3] - m1);
        l[nt][0] += p0 + p2;
        l[nt][1] += p1 + p3;
        // [key][row] pairs to the product's [row][key] pairs
        const uint32_t h0 = Vec<M>::pack2(p0, p1), h1 = Vec<M>::pack2(p2, p3);
        p[mt][nt][0] = movmatrix_t(h0);
        p[mt][nt][1] = movmatrix_t(h1);
        if constexpr (kRest) {
          const float2 w0 = unpack2<M>(h0), w1 = unpack2<M>(h1);
          rest[mt][nt][0] = movmatrix_t(Vec<M>::pack2(p0 - w0.x, p1 - w0.y));
          rest[mt][nt][1] = movmatrix_t(Vec<M>::pack2(p2 - w1.x, p3 - w1.y));
        }
      }
    }
    // O^T += V^T P^T
#pragma unroll
    for (int mt = 0; mt < kMt; ++mt) {
      if constexpr (!F8) {
        const int row = mt * 16 + (mat >> 1) * 8 + mrow;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t v[4];
          ldmatrix4_t(vs + chunk_at<kRowBytes>(row, 2 * c + (mat & 1)), v);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma16816<M>(o[c][nt], v, p[mt][nt][0], p[mt][nt][1]);
            if constexpr (kRest) mma16816<M>(o[c][nt], v, rest[mt][nt][0], rest[mt][nt][1]);
          }
        }
      } else {
        // A transposed 16-bit unit is a pair of elements (2 i, 2 i + 1) of one key; two keys' pairs are
        // regrouped by element: output rows 0-7 are the chunk's even elements, rows 8-15 the odd ones.
        const int row = mt * 16 + (mat & 1) * 8 + mrow;
#pragma unroll
        for (int c = 0; c < D / 16; c += 2) {
          uint32_t b[4];
          ldmatrix4_t(vs + chunk_at<kRowBytes>(row, c + (mat >> 1)), b);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t v[4];
            e4m3x4_f16x4(__byte_perm(b[2 * u], 0, 0x3120), v[0], v[1]);
            e4m3x4_f16x4(__byte_perm(b[2 * u + 1], 0, 0x3120), v[2], v[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816<M>(o[c + u][nt], v, p[mt][nt][0], p[mt][nt][1]);
              if constexpr (kRest) mma16816<M>(o[c + u][nt], v, rest[mt][nt][0], rest[mt][nt][1]);
            }
          }
        }
      }
    }
  }

  __device__ __forceinline__ void finish(float* so, float* sm) {
    const int lane = threadIdx.x & 31, t = lane & 3, g = lane >> 2;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = l[nt][i];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        const int row = nt * 8 + 2 * t + i;
        if (g == 0) {
          sm[row] = m[nt][i];
          sm[kRows + row] = x;
        }
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          so[row * kPitch + 16 * c + (F8 ? 2 * g : g)] = o[c][nt][i];
          so[row * kPitch + 16 * c + (F8 ? 2 * g + 1 : g + 8)] = o[c][nt][i + 2];
        }
      }
  }
};

// fp32: for the logits a lane has one key and kPer of the 8 rows, for the
// output a 16-byte chunk of the head; the weights change hands through shared
// memory.
template <int D_>
struct FmaEngine {
  static constexpr int D = D_;
  static constexpr int kRows = 8;
  static constexpr int kRowBytes = 4 * D;
  static constexpr int kKeys = D >= 128 ? 8 : 16;
  static constexpr int kPitch = D + 4;
  static constexpr int kSharedQ = kRows * D + kWarps * (kKeys * kRows + kRows);   // floats: q, then each warp's weights and factors
  static constexpr int kPer = kRows * kKeys / 32;
  static constexpr int kMostPerSm = 3;
  static constexpr int kLaneChunks = D / 4 >= 32 ? D / 128 : 1;
  static constexpr int kGroups = D / 4 >= 32 ? 1 : 32 / (D / 4);   // lanes sharing a chunk, each with its keys

  float o[kRows][kLaneChunks * 4];
  float m[kPer], l[kPer], sc;
  int lim[kPer];

  __device__ __forceinline__ void begin(const AttendArgs& a, const Req& rq, int head, int tile, float* sq) {
    for (int i = threadIdx.x; i < kRows * D / 4; i += kAttendThreads) {
      const int rho = tile * kRows + i / (D / 4), tok = rho / a.G;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (tok < rq.n)
        x = *reinterpret_cast<const float4*>(a.q + (int64_t)(rq.row0 + tok) * a.q_stride +
                                             (((size_t)head * a.G + (rho - tok * a.G)) * D + (i % (D / 4)) * 4) * 4);
      reinterpret_cast<float4*>(sq)[i] = x;
    }
    __syncthreads();
    const int part = (threadIdx.x & 31) / kKeys;
    sc = a.scale * kLog2e;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int tok = (tile * kRows + part * kPer + i) / a.G;
      lim[i] = tok < rq.n ? rq.seq - rq.n + tok : -1;
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int e = 0; e < kLaneChunks * 4; ++e) o[r][e] = 0.f;
  }

  __device__ __forceinline__ void step(const AttendArgs& a, uint32_t ks, uint32_t vs, const TileMask& tm, float* sq) {
    const int lane = threadIdx.x & 31, key = lane % kKeys, part = lane / kKeys;
    float* sp = sq + kRows * D + (threadIdx.x >> 5) * (kKeys * kRows + kRows);   // [key][row]
    float* sf = sp + kKeys * kRows;
    float s[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) s[i] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D / 4; ++c) {
      float k[4];
      Vec<float>::unpack(ld_shared_v4(ks + chunk_at<kRowBytes>(key, c)), k);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float4 q = reinterpret_cast<const float4*>(sq)[(part * kPer + i) * (D / 4) + c];
        s[i] = fmaf(q.x, k[0], fmaf(q.y, k[1], fmaf(q.z, k[2], fmaf(q.w, k[3], s[i]))));
      }
    }
    bool over = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      s[i] = __fmul_rn(s[i], sc);         // not fused with - m: far logits
      const int j = tm.key0 + key;
      if (tm.check && !(((tm.valid >> key) & 1u) && j <= lim[i] && (a.window == 0 || j > lim[i] - a.window))) s[i] = -INFINITY;
      over |= s[i] > lazy_bound<float>(m[i]);
    }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        float x = s[i];
#pragma unroll
        for (int d = kKeys / 2; d > 0; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
        const float mn = fmaxf(m[i], x);
        const float f = mn == -INFINITY ? 1.f : ex2(m[i] - mn);
        m[i] = mn;
        l[i] *= f;
        if (key == 0) sf[part * kPer + i] = f;
      }
      __syncwarp();
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float f = sf[r];
#pragma unroll
        for (int e = 0; e < kLaneChunks * 4; ++e) o[r][e] *= f;
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float p = ex2(s[i] - (m[i] == -INFINITY ? 0.f : m[i]));
      l[i] += p;
      sp[key * kRows + part * kPer + i] = p;
    }
    __syncwarp();
    const int chunk = kGroups > 1 ? lane % (D / 4) : lane, group = kGroups > 1 ? lane / (D / 4) : 0;
#pragma unroll 4
    for (int kk = 0; kk < kKeys / kGroups; ++kk) {
      const int row = group * (kKeys / kGroups) + kk;
      const float4 w0 = *reinterpret_cast<const float4*>(sp + row * kRows), w1 = *reinterpret_cast<const float4*>(sp + row * kRows + 4);
      const float w[kRows] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
      for (int u = 0; u < kLaneChunks; ++u) {
        float v[4];
        Vec<float>::unpack(ld_shared_v4(vs + chunk_at<kRowBytes>(row, chunk + 32 * u)), v);
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[r][u * 4 + e] = fmaf(w[r], v[e], o[r][u * 4 + e]);
      }
    }
    __syncwarp();                        // the weights are read before the next tile's are written
  }

  __device__ __forceinline__ void finish(float* so, float* sm) {
    const int lane = threadIdx.x & 31, part = lane / kKeys;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      float x = l[i];
#pragma unroll
      for (int d = kKeys / 2; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      if (lane % kKeys == 0) {
        sm[part * kPer + i] = m[i];
        sm[kRows + part * kPer + i] = x;
      }
    }
    const int chunk = kGroups > 1 ? lane % (D / 4) : lane;
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int e = 0; e < kLaneChunks * 4; ++e) {
        float x = o[r][e];
#pragma unroll
        for (int d = D / 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        if (lane < D / 4 || kGroups == 1) so[r * kPitch + (chunk + 32 * (e / 4)) * 4 + (e & 3)] = x;
      }
  }
};

// ---- the split kernel ----------------------------------------------------------------

constexpr int kRingBytes = 16384;        // of a warp's ring
template <class E>
struct SplitShape {
  static constexpr int kUnit = kWarps * E::kKeys;                     // keys of a unit
  static constexpr int kTileBytes = 2 * E::kKeys * E::kRowBytes;      // K and V of a tile
  static constexpr int kStages = kRingBytes / kTileBytes >= 2 ? kRingBytes / kTileBytes : 2;
  static constexpr int kWarpBytes = kStages * kTileBytes;
  // A warp's output waits for the join in the last tile of its ring: the next
  // segment's first loads take the others.
  static constexpr int kJoinAt = (kStages - 1) * kTileBytes;
  static_assert(E::kRows * E::kPitch * 4 <= kTileBytes, "the output fits a tile");
  static constexpr size_t kSmem = (size_t)kWarps * kWarpBytes + (size_t)E::kSharedQ * 4;
  static constexpr int kFit = 227 * 1024 / (int)(kSmem + 2048);
  static constexpr int kPerSm = kFit < E::kMostPerSm ? kFit : E::kMostPerSm;
  static_assert(kPerSm >= 1, "a CTA fits an SM");
};
constexpr int kMinUnits = 1;             // units of a CTA's run, at least

// A segment: a CTA's share of one item.
struct SplitSeg {
  int32_t r;                             // request; -1: the run has ended
  int32_t row0, n, seq;
  int32_t head, tile;
  int32_t k_lo, k_hi;                    // keys
  int32_t slot;                          // of the partial result; -1: the item is whole
  int32_t parts;                         // of an item that begins here and goes on in other CTAs; else 0
};

// One thread's walk over the segments of its CTA's run.  What it reads of a
// request is handed to the CTA through shared memory, so that the CTA agrees
// on its segments whatever happens to the caller's arrays meanwhile; the next
// request is read one step ahead.
struct SplitWalk {
  int64_t u, u_end, u_first, run, base;  // base: first unit of request r
  int r;
  Req q, ahead;

  __device__ __forceinline__ void start(const AttendArgs& a, int r_, const Req& q_, int64_t base_, int64_t u_, int64_t u_end_,
                                        int64_t run_) {
    r = r_;
    q = q_;
    base = base_;
    u = u_first = u_;
    u_end = u_end_;
    run = run_;
    look_ahead(a);
  }
  __device__ __forceinline__ void look_ahead(const AttendArgs& a) {
    if (r + 1 < a.R) ahead = read_request(a, r + 1, false);
    else ahead.n = 0;
  }
  template <int ROWS, int UNIT>
  __device__ __forceinline__ void next(const AttendArgs& a, SplitSeg* out) {
    out->r = -1;
    if (u >= u_end) return;
    while (true) {
      const int tiles = tiles_of(a, q, ROWS), units = units_of(q, UNIT);
      if (u >= base + (int64_t)a.H * tiles * units) {
        base += (int64_t)a.H * tiles * units;
        if (++r >= a.R) return;          // the arrays have changed under the call
        q = ahead;
        look_ahead(a);
        continue;
      }
      const int item = (int)div_small(u - base, units);
      const int64_t item0 = base + (int64_t)item * units;
      const int ua = (int)(u - item0), ub = (int)min((int64_t)units, u_end - item0);
      const int head = item / tiles, tile = item - head * tiles;
      const int last_tok = min(q.n - 1, (tile * ROWS + ROWS - 1) / a.G);
      out->row0 = q.row0;
      out->n = q.n;
      out->seq = q.seq;
      out->head = head;
      out->tile = tile;
      out->k_lo = q.kb + ua * UNIT;
      out->k_hi = min(min(q.ke, q.seq - q.n + last_tok + 1), q.kb + ub * UNIT);
      out->slot = ua == 0 && ub == units ? -1 : 2 * (int)blockIdx.x + (u == u_first ? 0 : 1);
      // Within the grid, whatever became of the lengths since they were added up.
      out->parts = ua == 0 && ub < units
                       ? (int)(min(div_small(item0 + units - 1, run), (int64_t)gridDim.x - 1) - (int64_t)blockIdx.x) + 1
                       : 0;
      out->r = r;
      u = item0 + ub;
      return;
    }
  }
};

template <typename T, class E>
__global__ void __launch_bounds__(kAttendThreads, SplitShape<E>::kPerSm) attend_split_kernel(const AttendArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  using S = SplitShape<E>;
  constexpr int ROWS = E::kRows, D = E::D, KT = E::kKeys, PITCH = E::kPitch;
  __shared__ int64_t scratch[kWarps];
  __shared__ SplitSeg s_seg[2];
  __shared__ float s_ml[kWarps][2 * ROWS];
  __shared__ uint32_t s_valid[kWarps][S::kStages];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float* outs = reinterpret_cast<const float*>(smem + S::kJoinAt);
  float* so = reinterpret_cast<float*>(smem + warp * S::kWarpBytes + S::kJoinAt);
  float* sq = reinterpret_cast<float*>(smem + kWarps * S::kWarpBytes);
  pdl_wait();
  pdl_trigger();

  // This CTA's run of units.
  const int per = (a.R + kAttendThreads - 1) / kAttendThreads;
  const int r0 = min(a.R, tid * per), r1 = min(a.R, r0 + per);
  int64_t mine = 0;
  for (int r = r0; r < r1; ++r) {
    const Req q = read_request(a, r, blockIdx.x == 0);
    mine += (int64_t)a.H * tiles_of(a, q, ROWS) * units_of(q, S::kUnit);
  }
  int64_t total;
  int64_t at = block_exclusive_scan_1bar<kWarps>(mine, scratch, &total);
  const int64_t run = max((int64_t)kMinUnits, div_small(total + gridDim.x - 1, gridDim.x));
  const int64_t u = (int64_t)blockIdx.x * run, u_end = min(total, u + run);
  if (u >= u_end) {
    if (tid == 0) record_of(a, blockIdx.x)->parts = 0;
    return;
  }
  // The thread whose requests the run begins in walks along it.
  SplitWalk walk;
  const bool walker = at <= u && u < at + mine;
  if (walker) {
    for (int r = r0; r < r1; ++r) {
      const Req q = read_request(a, r, false);
      const int64_t n = (int64_t)a.H * tiles_of(a, q, ROWS) * units_of(q, S::kUnit);
      if (u < at + n || r == r1 - 1) {
        walk.start(a, r, q, at, u, u_end, run);
        break;
      }
      at += n;
    }
    walk.template next<ROWS, S::kUnit>(a, &s_seg[0]);
  }
  __syncthreads();

  const uint32_t ring = smem_addr(smem) + warp * S::kWarpBytes;
  const int64_t token_bytes = (int64_t)a.H * E::kRowBytes;

  // Loads of the current segment's tiles of this warp: tile warp + i * kWarps.  Lane i < KT looks up key i of a tile,
  // one tile ahead of its loads.
  int k_lo = 0, k_hi = 0, n_mine = 0;
  const int32_t* table = nullptr;
  const uint8_t* kbase = nullptr;
  int32_t id_next = -1, off_next = 0;
  auto look_up = [&](int i) {
    const int j = k_lo + (warp + i * kWarps) * KT + lane;
    id_next = -1;
    if (i < n_mine && lane < KT && j < k_hi) {
      const int b = block_of(a, j);
      off_next = j - b * a.block_size;
      id_next = table[b];
      if (id_next < 0 || id_next >= a.num_blocks) {
        latch(a.status, IS_ST_BLOCK_ID);
        id_next = -1;
      }
    }
  };
  auto issue = [&](int i, int stage) {
    if (i < n_mine) {
      const long long off = id_next < 0 ? -1ll : ((long long)id_next * a.block_size + off_next) * token_bytes;
      const uint32_t valid = __ballot_sync(0xffffffffu, off >= 0);
      if (lane == 0) s_valid[warp][stage] = valid;
      look_up(i + 1);
      constexpr int CPR = E::kRowBytes / 16;             // chunks of a row
      constexpr int RPI = CPR >= 32 ? 1 : 32 / CPR;      // rows of one pass of the warp
      constexpr int PASS = CPR >= 32 ? CPR / 32 : 1;     // passes of one row
      const uint32_t kd = ring + stage * S::kTileBytes, vd = kd + KT * E::kRowBytes;
#pragma unroll
      for (int x = 0; x < KT; x += RPI) {
        const int row = x + (RPI > 1 ? lane / CPR : 0);
        const long long o = __shfl_sync(0xffffffffu, off, row);
        const bool in = o >= 0;
#pragma unroll
        for (int y = 0; y < PASS; ++y) {
          const int c = (RPI > 1 ? lane % CPR : lane) + 32 * y;
          const uint8_t* src = kbase + (in ? o : 0) + c * 16;
          const uint32_t dst = chunk_at<E::kRowBytes>(row, c);
          cp_async16(kd + dst, src, in);
          cp_async16(vd + dst, src + a.v_offset, in);
        }
      }
    }
    cp_async_commit();
  };
  auto open = [&](const SplitSeg& g) {
    k_lo = g.k_lo;
    k_hi = g.k_hi;
    table = a.block_table + (size_t)g.r * a.max_blocks;
    kbase = a.k_cache + (size_t)g.head * E::kRowBytes;
    const int n_tiles = k_hi > k_lo ? (k_hi - k_lo + KT - 1) / KT : 0;
    n_mine = n_tiles > warp ? (n_tiles - warp + kWarps - 1) / kWarps : 0;
    look_up(0);
#pragma unroll
    for (int s = 0; s < S::kStages - 1; ++s) issue(s, s);
  };

  bool crossed = false;                  // the run's last item began here and goes on in the next CTA
  if (s_seg[0].r >= 0) open(s_seg[0]);
  for (int k = 0; s_seg[k & 1].r >= 0; ++k) {
    const SplitSeg& g = s_seg[k & 1];
    if (walker) walk.template next<ROWS, S::kUnit>(a, &s_seg[(k + 1) & 1]);
    Req q;
    q.row0 = g.row0;
    q.n = g.n;
    q.seq = g.seq;
    const int head = g.head, tile = g.tile;
    const int p_first = q.seq - q.n + tile * ROWS / a.G;
    const int p_last = q.seq - q.n + min(q.n - 1, (tile * ROWS + ROWS - 1) / a.G);

    E e;
    e.begin(a, q, head, tile, sq);
    for (int i0 = 0; i0 < n_mine; i0 += S::kStages) {
#pragma unroll
      for (int s = 0; s < S::kStages; ++s) {
        const int i = i0 + s;
        if (i < n_mine) {
          cp_async_wait<S::kStages - 2>();
          __syncwarp();                  // every lane's part of tile i has landed, and all are done with tile i - 1
          TileMask tm;
          tm.valid = s_valid[warp][s];
          issue(i + S::kStages - 1, (s + S::kStages - 1) % S::kStages);
          tm.key0 = k_lo + (warp + i * kWarps) * KT;
          constexpr uint32_t kFull = KT == 32 ? 0xffffffffu : (1u << KT) - 1u;
          tm.check = tm.valid != kFull || tm.key0 + KT - 1 > p_first || (a.window > 0 && tm.key0 <= p_last - a.window);
          const uint32_t kd = ring + s * S::kTileBytes;
          e.step(a, kd, kd + KT * E::kRowBytes, tm, sq);
        }
      }
    }
    cp_async_wait<0>();
    __syncwarp();                        // every lane is done with the ring
    e.finish(so, s_ml[warp]);
    __syncthreads();
    // The next segment's first tiles are on their way while this one's output is joined.
    if (s_seg[(k + 1) & 1].r >= 0) open(s_seg[(k + 1) & 1]);

    // Join the warps.  Every thread takes pairs of elements.
    const int rho0 = tile * ROWS, rows = min(ROWS, q.n * a.G - rho0);
    const int slot = g.slot;
    Partial<ROWS, D>* part = partial_of<Partial<ROWS, D>>(a, max(slot, 0));
    for (int x = tid; x < rows * (D / 2); x += kAttendThreads) {
      const int row = x / (D / 2), d = (x % (D / 2)) * 2;
      float mx = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_ml[w][row]);
      const float m0 = mx == -INFINITY ? 0.f : mx;
      float ox = 0.f, oy = 0.f, l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(s_ml[w][row] - m0);
        const float2 v = *reinterpret_cast<const float2*>(outs + (size_t)w * (S::kWarpBytes / 4) + row * PITCH + d);
        ox = fmaf(f, v.x, ox);
        oy = fmaf(f, v.y, oy);
        l = fmaf(f, s_ml[w][ROWS + row], l);
      }
      if (slot < 0) {
        const float inv = l == 0.f ? 0.f : a.v_scale / l;
        store_out<T>(a, q, head, rho0 + row, d, l == 0.f ? 0.f : ox * inv, l == 0.f ? 0.f : oy * inv);
        if (d == 0) store_lse(a, q, head, rho0 + row, mx, l);
      } else {
        *reinterpret_cast<float2*>(&part->o[row][d]) = make_float2(ox, oy);
        if (d == 0) {
          part->m[row] = mx;
          part->l[row] = l;
        }
      }
    }
    if (slot >= 0 && g.parts > 0 && tid == 0) {
      // The item begins here and goes on in other CTAs: this CTA's record names its parts.
      JoinRecord* rec = record_of(a, blockIdx.x);
      rec->parts = g.parts;
      rec->slot0 = slot;
      rec->row0 = q.row0;
      rec->head = head;
      rec->rho0 = rho0;
      rec->rows = rows;
    }
    crossed = slot >= 0 && g.parts > 0;
    __syncthreads();                     // s_ml and the warps' outputs are free again
  }
  if (!crossed && tid == 0) record_of(a, blockIdx.x)->parts = 0;
}

// ---- host side -----------------------------------------------------------------------

template <typename T, class E>
static cudaError_t launch_split(const AttendArgs& a, const LaunchCfg& cfg) {
  using S = SplitShape<E>;
  auto* kern = attend_split_kernel<T, E>;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), S::kSmem);
  if (e != cudaSuccess) return e;
  static_assert(partials_offset() + kMaxCtas * 2 * sizeof(Partial<E::kRows, E::D>) <= IS_ATTEND_WORKSPACE_BYTES,
                "the workspace holds every partial");
  // As many CTAs as the SMs hold; fewer when the table's reach shows that there are fewer runs.
  const int64_t keys = (int64_t)a.max_blocks * a.block_size;
  const int64_t units = std::max<int64_t>(1, (std::min<int64_t>(keys, IS_MAX_POSITION) + S::kUnit - 1) / S::kUnit);
  const int64_t items = (int64_t)a.R * a.H * ((a.max_q * (int64_t)a.G + E::kRows - 1) / E::kRows);
  const int64_t runs = (items * units + kMinUnits - 1) / kMinUnits;
  const int grid = (int)std::min<int64_t>(std::min<int64_t>(runs, (int64_t)S::kPerSm * cfg.num_sms), kMaxCtas);
  e = launch_ex(kern, dim3(grid), dim3(kAttendThreads), S::kSmem, cfg.stream, cfg.pdl, a);
  if (e != cudaSuccess) return e;
  // Few parts an item: a CTA joins all rows of a record; else four CTAs, each splitting the parts of a row at a time.
  if (items * 4 >= grid)
    return launch_ex(attend_join_rows_kernel<T, E::kRows, E::D, false>, dim3(grid, 1), dim3(kJoinThreads), 0, cfg.stream, cfg.pdl, a);
  return launch_ex(attend_join_kernel<T, E::kRows, E::D>, dim3(grid, 4), dim3(kJoinThreads), 0, cfg.stream,
                   cfg.pdl, a);
}

template <typename T, bool F8>
static cudaError_t launch_mma(const AttendArgs& a, const LaunchCfg& cfg) {
  // Two column tiles when a request has more than 8 rows: the keys are then
  // read once for 16 rows.  At head_dim 256 their output would not fit the registers.
  const bool two = (int64_t)a.max_q * a.G > 8;
  if (a.D == 64)
    return two ? launch_split<T, MmaEngine<T, F8, 64, 2>>(a, cfg) : launch_split<T, MmaEngine<T, F8, 64, 1>>(a, cfg);
  if (a.D == 128)
    return two ? launch_split<T, MmaEngine<T, F8, 128, 2>>(a, cfg) : launch_split<T, MmaEngine<T, F8, 128, 1>>(a, cfg);
  return launch_split<T, MmaEngine<T, F8, 256, 1>>(a, cfg);
}

cudaError_t launch_attend(const AttendArgs& a, const LaunchCfg& cfg) {
  // Many rows go to the kernel of attend_prompt.cu, which reads the keys once
  // for 256 rows (128 at head_dim 256), from the number of rows on at which the
  // kernel here would read them more than once.  100 requests of 300-2048 tokens
  // with 4 new ones, 28 rows: 98 us here, 68 there; at head_dim 256, 16 rows: 178
  // and 98; 4 requests of up to 131,000 tokens, 32 rows: 542 and 278; a single
  // one of 1313: 18.1 and 17.3.  FP8 rows are widened faster here, so there they go
  // from 33 on (32 rows, 64 requests of 500-8000 tokens: 259 and 293 us), and not
  // at all at head_dim 256, where the other kernel's shared memory has no room for
  // them: 64 KB of Q and two widened tiles of 64 KB leave 35 KB, one tile of raw
  // rows and none ahead of it.  (Two prompts of 2000-2500 tokens behind up to 8192,
  // H = 4, G = 2: 2100 us here over FP8, 255 there over bf16.)
  // Maxima there are of unscaled logits, so the scale has to be positive.
  const int most = a.fp8 ? 32 : a.D == 256 ? 8 : 16;
  if (a.dtype != IS_F32 && (a.D <= 128 || !a.fp8) && a.G <= 64 && (int64_t)a.max_q * a.G > most && a.scale > 0.f)
    return launch_attend_prompt(a, cfg);
  if (a.dtype == IS_BF16)
    return a.fp8 ? launch_mma<__nv_bfloat16, true>(a, cfg) : launch_mma<__nv_bfloat16, false>(a, cfg);
  if (a.dtype == IS_F16) return a.fp8 ? launch_mma<__half, true>(a, cfg) : launch_mma<__half, false>(a, cfg);
  if (a.D == 64) return launch_split<float, FmaEngine<64>>(a, cfg);
  if (a.D == 128) return launch_split<float, FmaEngine<128>>(a, cfg);
  return launch_split<float, FmaEngine<256>>(a, cfg);
}

}  // namespace isk
