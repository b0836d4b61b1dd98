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

// Vectors a thread loads before the token's sines are known: as many rotated
// items (a pair of vectors for half-split heads, else one) and plain ones.
constexpr int kAppendAhead = 3;

template <typename T, int STYLE, bool F8>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a, const __grid_constant__ AxisTurns at) {
  constexpr int VE = Vec<T>::N;
  constexpr int NF = STYLE == 0 ? VE : VE / 2;   // frequencies of one vector
  constexpr int CB = F8 ? 1 : (int)sizeof(T);    // cache bytes per element
  __shared__ float s_cos[kMaxHalfDim], s_sin[kMaxHalfDim];
  __shared__ uint32_t s_bad;
  const int tid = threadIdx.x, half = a.D / 2;
  const int64_t t = blockIdx.x;
  const int hv = a.D / VE;                       // vectors per head
  const int gv = STYLE == 0 ? hv / 2 : hv;       // rotated items per head
  const int f = tid % gv;                        // this thread's frequency group
  const int h0 = tid / gv, hs = kAppendThreads / gv, heads = a.Hq + a.H;
  const uint8_t* qrow = a.q + t * a.q_stride;
  const uint8_t* krow = a.k + t * a.k_stride;
  const uint8_t* vrow = a.v + t * a.v_stride;
  if (tid == 0) s_bad = 0;
  pdl_wait();
  pdl_trigger();

  // Everything that does not need the token's slot is under way before it is read.
  const int64_t slot = a.slots[t];
  auto item = [&](int h, bool second) -> const uint8_t* {
    const uint8_t* row = h < a.Hq ? qrow + (size_t)h * hv * 16 : krow + (size_t)(h - a.Hq) * hv * 16;
    return row + (size_t)(f + (second ? gv : 0)) * 16;
  };
  uint4 x0[kAppendAhead], x1[kAppendAhead], xv[kAppendAhead];
#pragma unroll
  for (int i = 0; i < kAppendAhead; ++i) {
    const int h = h0 + i * hs, v = tid + i * kAppendThreads;
    if (h < heads) {
      x0[i] = *reinterpret_cast<const uint4*>(item(h, false));
      if (STYLE == 0) x1[i] = *reinterpret_cast<const uint4*>(item(h, true));
    }
    if (v < a.H * hv) xv[i] = *reinterpret_cast<const uint4*>(vrow + (size_t)v * 16);
  }
  if (slot == -1) return;                        // padding: the whole CTA
  __syncthreads();                               // s_bad is zero
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
  float cs[NF], sn[NF];
#pragma unroll
  for (int e = 0; e < NF; ++e) {
    cs[e] = s_cos[f * NF + e];
    sn[e] = s_sin[f * NF + e];
  }
  uint8_t* qout = a.q_out + (size_t)t * a.Hq * a.D * sizeof(T);
  uint8_t* kout = a.k_cache + (size_t)slot * a.H * a.D * CB;
  uint8_t* vout = kout + a.v_offset;
  auto put = [&](int h, int v, const float* y) {
    if (h < a.Hq) st_v4(qout + ((size_t)h * hv + v) * 16, Vec<T>::pack(y));
    else if (F8) st_v2(kout + ((size_t)(h - a.Hq) * hv + v) * 8, to_e4m3x8(y, a.k_inv));
    else st_v4(kout + ((size_t)(h - a.Hq) * hv + v) * 16, Vec<T>::pack(y));
  };
  auto rotate = [&](int h, const uint4& u, const uint4& w) {
    float x[VE], y[VE];
    Vec<T>::unpack(u, x);
    if (STYLE == 0) {
      float z[VE], r[VE];
      Vec<T>::unpack(w, z);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        y[e] = fmaf(x[e], cs[e], -z[e] * sn[e]);
        r[e] = fmaf(z[e], cs[e], x[e] * sn[e]);
      }
      put(h, f, y);
      put(h, f + gv, r);
    } else {
#pragma unroll
      for (int e = 0; e < VE / 2; ++e) {
        y[2 * e] = fmaf(x[2 * e], cs[e], -x[2 * e + 1] * sn[e]);
        y[2 * e + 1] = fmaf(x[2 * e + 1], cs[e], x[2 * e] * sn[e]);
      }
      put(h, f, y);
    }
  };
  auto copy = [&](int v, const uint4& x) {
    if (F8) {
      float y[VE];
      Vec<T>::unpack(x, y);
      st_v2(vout + (size_t)v * 8, to_e4m3x8(y, a.v_inv));
    } else {
      st_v4(vout + (size_t)v * 16, x);
    }
  };
#pragma unroll
  for (int i = 0; i < kAppendAhead; ++i) {
    const int h = h0 + i * hs, v = tid + i * kAppendThreads;
    if (h < heads) rotate(h, x0[i], x1[i]);
    if (v < a.H * hv) copy(v, xv[i]);
  }
  // Wider models' remaining heads.
  for (int h = h0 + kAppendAhead * hs; h < heads; h += hs) {
    const uint4 u = *reinterpret_cast<const uint4*>(item(h, false));
    rotate(h, u, STYLE == 0 ? *reinterpret_cast<const uint4*>(item(h, true)) : u);
  }
  for (int v = tid + kAppendAhead * kAppendThreads; v < a.H * hv; v += kAppendThreads)
    copy(v, *reinterpret_cast<const uint4*>(vrow + (size_t)v * 16));
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
