// Rotary positions of one or several axes, and the paged K/V write (is_append).
//
// Pair i of a head turns by the angle p_axis(i) * w_i (the turns are reduced
// in fp32 as for the injected facts, see angle_turns): (a, b) becomes
// (a cos - b sin, b cos + a sin), in fp32, rounded once to the output type.
// The sines of a token depend on its positions alone, so a CTA takes one
// token: half a head's worth of threads compute them once into shared memory,
// and all heads use them.  A thread's 16-byte vectors of different heads share
// one frequency group, whose sines it keeps in registers.  Bound by memory:
// every input is read once and every output written once.
#include "common.cuh"
#include "internal.h"

namespace isk {

constexpr int kAppendThreads = 128;

template <typename T, int STYLE, bool F8>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a, const AxisTurns at) {
  constexpr int VE = Vec<T>::N;
  constexpr int NF = STYLE == 0 ? VE : VE / 2;   // frequencies of one vector
  __shared__ float s_cos[kMaxHalfDim], s_sin[kMaxHalfDim];
  __shared__ uint32_t s_bad;
  const int tid = threadIdx.x, half = a.D / 2;
  const int64_t t = blockIdx.x;
  if (tid == 0) s_bad = 0;
  pdl_wait();
  pdl_trigger();
  const int64_t slot = a.slots[t];
  if (slot == -1) return;                        // padding
  __syncthreads();
  uint32_t bad = slot < 0 || slot >= a.n_slots ? IS_ST_BLOCK_ID : 0u;
  if (tid < a.n_axes) {
    const int32_t p = a.positions[(size_t)tid * a.T + t];
    if (p < 0 || p >= IS_MAX_POSITION) bad |= IS_ST_POSITION;
  }
  if (bad) atomicOr(&s_bad, bad);
  for (int i = tid; i < half; i += kAppendThreads) {
    const float p = (float)a.positions[(size_t)at.axis[i] * a.T + t];
    float sn, cs;
    sincospif(2.0f * angle_turns(p, at.t.hi[i], at.t.lo[i]), &sn, &cs);
    s_cos[i] = cs;
    s_sin[i] = sn;
  }
  __syncthreads();
  if (s_bad) {
    if (tid == 0) latch(a.status, s_bad);
    return;
  }
  const int hv = a.D / VE;                       // vectors per head
  const int gv = STYLE == 0 ? hv / 2 : hv;       // rotated items per head: a pair of vectors, or one
  const int f = tid % gv;
  float cs[NF], sn[NF];
#pragma unroll
  for (int e = 0; e < NF; ++e) {
    cs[e] = s_cos[f * NF + e];
    sn[e] = s_sin[f * NF + e];
  }
  const uint8_t* qrow = a.q + t * a.q_stride;
  const uint8_t* krow = a.k + t * a.k_stride;
  const uint8_t* vrow = a.v + t * a.v_stride;
  uint8_t* qout = a.q_out + (size_t)t * a.Hq * a.D * sizeof(T);
  constexpr int CB = F8 ? 1 : (int)sizeof(T);    // cache bytes per element
  uint8_t* kout = a.k_cache + (size_t)slot * a.H * a.D * CB;
  uint8_t* vout = kout + a.v_offset;
  auto put_k = [&](int v, const float* y) {
    if (F8) st_v2(kout + (size_t)v * 8, to_e4m3x8(y, a.k_inv));
    else st_v4(kout + (size_t)v * 16, Vec<T>::pack(y));
  };
  for (int h = tid / gv; h < a.Hq + a.H; h += kAppendThreads / gv) {
    const bool is_q = h < a.Hq;
    const int head = is_q ? h : h - a.Hq;
    const uint8_t* src = (is_q ? qrow : krow);
    const int v0 = head * hv + f;
    float x[VE], y[VE];
    Vec<T>::unpack(*reinterpret_cast<const uint4*>(src + (size_t)v0 * 16), x);
    if (STYLE == 0) {
      const int v1 = v0 + gv;
      float z[VE], w[VE];
      Vec<T>::unpack(*reinterpret_cast<const uint4*>(src + (size_t)v1 * 16), z);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        y[e] = fmaf(x[e], cs[e], -z[e] * sn[e]);
        w[e] = fmaf(z[e], cs[e], x[e] * sn[e]);
      }
      if (is_q) {
        st_v4(qout + (size_t)v0 * 16, Vec<T>::pack(y));
        st_v4(qout + (size_t)v1 * 16, Vec<T>::pack(w));
      } else {
        put_k(v0, y);
        put_k(v1, w);
      }
    } else {
#pragma unroll
      for (int e = 0; e < VE / 2; ++e) {
        y[2 * e] = fmaf(x[2 * e], cs[e], -x[2 * e + 1] * sn[e]);
        y[2 * e + 1] = fmaf(x[2 * e + 1], cs[e], x[2 * e] * sn[e]);
      }
      if (is_q) st_v4(qout + (size_t)v0 * 16, Vec<T>::pack(y));
      else put_k(v0, y);
    }
  }
  for (int v = tid; v < a.H * hv; v += kAppendThreads) {
    const uint4 x = *reinterpret_cast<const uint4*>(vrow + (size_t)v * 16);
    if (F8) {
      float y[VE];
      Vec<T>::unpack(x, y);
      st_v2(vout + (size_t)v * 8, to_e4m3x8(y, a.v_inv));
    } else {
      st_v4(vout + (size_t)v * 16, x);
    }
  }
}

template <typename T, bool F8>
static cudaError_t launch_append_t(const AppendArgs& a, const AxisTurns& turns, const LaunchCfg& cfg) {
  auto* kern = a.style == 0 ? append_kernel<T, 0, F8> : append_kernel<T, 1, F8>;
  return launch_ex(kern, dim3((unsigned)a.T), dim3(kAppendThreads), 0, cfg.stream, cfg.pdl, a, turns);
}

cudaError_t launch_append(const AppendArgs& a, const AxisTurns& turns, const LaunchCfg& cfg) {
  if (a.dtype == IS_F32) return launch_append_t<float, false>(a, turns, cfg);
  if (a.dtype == IS_BF16)
    return a.fp8 ? launch_append_t<__nv_bfloat16, true>(a, turns, cfg)
                 : launch_append_t<__nv_bfloat16, false>(a, turns, cfg);
  return a.fp8 ? launch_append_t<__half, true>(a, turns, cfg) : launch_append_t<__half, false>(a, turns, cfg);
}

}  // namespace isk
