// Softmax attention of each request's last tokens over its paged cache (is_attend).
//
// One warp per (query row, query head): the lanes split the head, the running
// maximum m and sum l of the softmax rescale the output as keys come by.
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace isk {

template <typename T> __device__ __forceinline__ float to_f(T x) { return (float)x; }
__device__ __forceinline__ float e4m3_f(uint8_t x) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(x, __NV_E4M3)));
}

template <typename T, bool F8>
__global__ void __launch_bounds__(256) attend_rows_kernel(const AttendArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int h = (int)(w % a.Hq);
  w /= a.Hq;
  const int i = (int)(w % a.max_q), r = (int)(w / a.max_q);
  if (r >= a.R) return;
  const int64_t s0 = a.q_start ? a.q_start[r] : r, s1 = a.q_start ? a.q_start[r + 1] : r + 1;
  const int seq = a.seq_len[r];
  const int64_t n = s1 - s0;
  if (n < 0 || n > a.max_q || s0 < 0 || s1 > a.T || seq < 0 || seq > IS_MAX_POSITION) {
    if (lane == 0) latch(a.status, IS_ST_COUNT);
    return;
  }
  if (i >= n) return;
  const int64_t row = s0 + i;
  const int p = seq - (int)n + i;
  const int first = a.window > 0 ? max(0, p - a.window + 1) : 0;
  const int epl = a.D / 32;
  float q[8], o[8];
  const T* qp = reinterpret_cast<const T*>(a.q + row * a.q_stride) + (size_t)h * a.D;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    q[e] = e < epl ? to_f(qp[lane * epl + e]) : 0.f;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const float c = a.scale * 1.4426950408889634f;
  for (int j = first; j <= p; ++j) {
    const int b = j / a.block_size;
    if (b >= a.max_blocks) {
      if (lane == 0) latch(a.status, IS_ST_BLOCK_TABLE);
      break;
    }
    const int id = a.block_table[(size_t)r * a.max_blocks + b];
    if (id < 0 || id >= a.num_blocks) {
      if (lane == 0) latch(a.status, IS_ST_BLOCK_ID);
      continue;
    }
    const size_t at = (((size_t)id * a.block_size + (j - b * a.block_size)) * a.H + h / a.G) * a.D + lane * epl;
    float k[8], v[8], s = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (e < epl) {
        if (F8) {
          k[e] = e4m3_f(a.k_cache[at + e]);
          v[e] = e4m3_f(a.k_cache[a.v_offset + at + e]);
        } else {
          k[e] = to_f(reinterpret_cast<const T*>(a.k_cache)[at + e]);
          v[e] = to_f(reinterpret_cast<const T*>(a.k_cache + a.v_offset)[at + e]);
        }
        s = fmaf(q[e], k[e], s);
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= c;
    const float m1 = fmaxf(m, s);
    const float base = m1 == -INFINITY ? 0.f : m1;
    const float f = exp2f(m - base), w1 = exp2f(s - base);
    l = l * f + w1;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < epl) o[e] = o[e] * f + w1 * v[e];
    m = m1;
  }
  T* out = reinterpret_cast<T*>(a.out) + ((size_t)row * a.Hq + h) * a.D + lane * epl;
  const float inv = l == 0.f ? 0.f : a.v_scale / l;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < epl) out[e] = T(l == 0.f ? 0.f : o[e] * inv);
  if (a.lse && lane == 0)
    a.lse[(size_t)row * a.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

cudaError_t launch_attend(const AttendArgs& a, const LaunchCfg& cfg) {
  const int64_t warps = (int64_t)a.R * a.max_q * a.Hq;
  const int64_t blocks = (warps + 7) / 8;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  auto* kern = a.dtype == IS_F32 ? attend_rows_kernel<float, false>
             : a.dtype == IS_BF16 ? (a.fp8 ? attend_rows_kernel<__nv_bfloat16, true> : attend_rows_kernel<__nv_bfloat16, false>)
                                  : (a.fp8 ? attend_rows_kernel<__half, true> : attend_rows_kernel<__half, false>);
  return launch_ex(kern, dim3((unsigned)blocks), dim3(256), 0, cfg.stream, cfg.pdl, a);
}

}  // namespace isk
