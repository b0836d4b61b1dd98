// Rotary positions of one or several axes, and the paged K/V write (is_append).
//
// Pair i of a head turns by the angle p_axis(i) * w_i (the turns are reduced
// in fp32 as for the injected facts, see angle_turns): (a, b) becomes
// (a cos - b sin, b cos + a sin), in fp32, rounded once to the output type.
// The sines of a token depend on its positions alone.  A warp works on one
// token: its lanes compute the sines of all D / 2 pairs between them, exchange
// them through the warp's shared memory, and go through the token's heads; a
// lane's 16-byte vectors of different heads share one frequency group, whose
// sines it keeps in registers.  With few tokens several warps share one, each
// with its own heads (and its own copy of the sines: 2 a lane, less than a
// block barrier costs), so that a single token is still one round of loads.
// Bound by memory: every input is read once and every output written once.
//
// Measured: 8192 tokens, 32 + 8 heads of 128, bf16, three axes, 201 MB: 38 us =
// 5.3 TB/s, 78 % of a plain copy.  A CTA per token with block barriers took 44.7
// us, rows loaded before the slot was known 40.5; a division per vector and the
// table read through the constant path (one address at a time) cost 10 us of a
// first warp-per-token form.  Batches of 3 to 10 vectors and smaller register
// budgets measured the same or worse.  One token: 3 us, the launch.
#include "common.cuh"
#include "internal.h"

namespace isk {

constexpr int kAppendThreads = 128;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kAppendBatch = 4;                  // vectors (or pairs) a lane loads before it uses any

// One element of a parameter table, another one in each lane: through the
// memory path, which serves a warp's 32 addresses together (the constant path
// takes them one by one).
__device__ __forceinline__ float ld_param(const float* p) {
  float x;
  asm("ld.f32 %0, [%1];" : "=f"(x) : "l"(p));
  return x;
}
__device__ __forceinline__ uint32_t ld_param(const uint8_t* p) {
  uint32_t x;
  asm("ld.u8 %0, [%1];" : "=r"(x) : "l"(p));
  return x;
}

template <typename T, int STYLE, bool F8>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const AppendArgs a, const __grid_constant__ AxisTurns at,
                                                                int share) {
  constexpr int VE = Vec<T>::N;
  constexpr int NF = STYLE == 0 ? VE : VE / 2;   // frequencies of one vector
  constexpr int CB = F8 ? 1 : (int)sizeof(T);    // cache bytes per element
  extern __shared__ float2 s_turn[];             // [warps][D / 2] (cos, sin)
  const int lane = threadIdx.x & 31, half = a.D / 2;
  const int64_t w = (int64_t)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  const int64_t t = w / share;                   // `share` warps to a token
  const int first = (int)(w - t * share) * 32 + lane, step = share * 32;
  float2* turn = s_turn + (threadIdx.x >> 5) * half;
  const int hv = a.D / VE;                       // vectors per head
  const int gv = STYLE == 0 ? hv / 2 : hv;       // rotated items per head (a power of two, at most 32)
  const int f = lane % gv;                       // this lane's frequency group
  const int nr = (a.Hq + a.H) * gv, nv = a.H * hv;
  pdl_wait();
  pdl_trigger();
  if (t >= a.T) return;
  const uint8_t* qrow = a.q + t * a.q_stride;
  const uint8_t* krow = a.k + t * a.k_stride;
  const uint8_t* vrow = a.v + t * a.v_stride;

  // Item i is head i / gv's vector (or pair of vectors) f = i % gv; byte offsets from the head 0 of q or k need no
  // division.  The first batch is under way before the slot and the positions are read.
  const int nq = a.Hq * gv;
  const uint8_t* kbase = krow - (size_t)a.Hq * hv * 16;
  auto offset = [&](int i) { return STYLE == 0 ? (2 * i - f) * 16 : i * 16; };
  uint4 x0[kAppendBatch], x1[kAppendBatch];
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kAppendBatch; ++u) {
      const int i = i0 + u * step;
      if (i < nr) {
        const uint8_t* src = (i < nq ? qrow : kbase) + offset(i);
        x0[u] = *reinterpret_cast<const uint4*>(src);
        if (STYLE == 0) x1[u] = *reinterpret_cast<const uint4*>(src + gv * 16);
      }
    }
  };
  const int64_t slot = a.slots[t];
  const int32_t of_axis = lane < a.n_axes ? a.positions[(size_t)lane * a.T + t] : 0;
  load(first);
  if (slot == -1) return;                        // padding
  uint32_t bad = slot < 0 || slot >= a.n_slots ? IS_ST_BLOCK_ID : 0u;
  if (of_axis < 0 || of_axis >= IS_MAX_POSITION) bad |= IS_ST_POSITION;
  bad = __reduce_or_sync(0xffffffffu, bad);
  if (bad) {
    if (lane == 0) latch(a.status, bad);
    return;
  }
  for (int i0 = 0; i0 < half; i0 += 32) {        // half may be 8 or 16: then lanes past it repeat pairs
    const int i = (i0 + lane) % half;
    const float p = (float)__shfl_sync(0xffffffffu, of_axis, ld_param(&at.axis[i]));
    float sn, cs;
    sincospif(2.0f * angle_turns(p, ld_param(&at.t.hi[i]), ld_param(&at.t.lo[i])), &sn, &cs);
    turn[i] = make_float2(cs, sn);
  }
  __syncwarp();
  // Two frequencies to a register pair: the paired multiply and fused
  // multiply-add round each lane as the scalar forms do.
  unsigned long long cs[NF / 2], sn[NF / 2], ns[NF / 2];
#pragma unroll
  for (int e = 0; e < NF / 2; ++e) {
    const float2 c0 = turn[f * NF + 2 * e], c1 = turn[f * NF + 2 * e + 1];
    cs[e] = pk2(c0.x, c1.x);
    sn[e] = pk2(c0.y, c1.y);
    ns[e] = pk2(-c0.y, -c1.y);
  }
  uint8_t* qout = a.q_out + (size_t)t * a.Hq * a.D * sizeof(T);
  uint8_t* kout = a.k_cache + (size_t)slot * a.H * a.D * CB;
  uint8_t* vout = kout + a.v_offset;
  uint8_t* kput = kout - (size_t)a.Hq * a.D * CB;
  auto put = [&](int i, int o, const float* y) {   // o: byte offset in 16-byte vectors' terms
    if (i < nq) st_v4(qout + o, Vec<T>::pack(y));
    else if (F8) st_v2(kput + o / 2, to_e4m3x8(y, a.k_inv));
    else st_v4(kput + o, Vec<T>::pack(y));
  };
  for (int i0 = first; i0 < nr; i0 += kAppendBatch * step) {
    if (i0 != first) load(i0);
#pragma unroll
    for (int u = 0; u < kAppendBatch; ++u) {
      const int i = i0 + u * step;
      if (i >= nr) continue;
      float x[VE], y[VE];
      Vec<T>::unpack(x0[u], x);
      if (STYLE == 0) {
        float z[VE], r[VE];
        Vec<T>::unpack(x1[u], z);
#pragma unroll
        for (int e = 0; e < VE / 2; ++e) {
          const unsigned long long p = pk2(x[2 * e], x[2 * e + 1]), q = pk2(z[2 * e], z[2 * e + 1]);
          upk2(fma2_rn(p, cs[e], mul2_rn(q, ns[e])), y[2 * e], y[2 * e + 1]);
          upk2(fma2_rn(q, cs[e], mul2_rn(p, sn[e])), r[2 * e], r[2 * e + 1]);
        }
        put(i, offset(i), y);
        put(i, offset(i) + gv * 16, r);
      } else {
#pragma unroll
        for (int e = 0; e < VE / 4; ++e) {         // pairs 2 e and 2 e + 1
          const unsigned long long p = pk2(x[4 * e], x[4 * e + 2]), q = pk2(x[4 * e + 1], x[4 * e + 3]);
          upk2(fma2_rn(p, cs[e], mul2_rn(q, ns[e])), y[4 * e], y[4 * e + 2]);
          upk2(fma2_rn(q, cs[e], mul2_rn(p, sn[e])), y[4 * e + 1], y[4 * e + 3]);
        }
        put(i, offset(i), y);
      }
    }
  }
  for (int i0 = first; i0 < nv; i0 += kAppendBatch * step) {
#pragma unroll
    for (int u = 0; u < kAppendBatch; ++u)
      if (i0 + u * step < nv) x0[u] = *reinterpret_cast<const uint4*>(vrow + (size_t)(i0 + u * step) * 16);
#pragma unroll
    for (int u = 0; u < kAppendBatch; ++u) {
      const int v = i0 + u * step;
      if (v >= nv) continue;
      if (F8) {
        float y[VE];
        Vec<T>::unpack(x0[u], y);
        st_v2(vout + (size_t)v * 8, to_e4m3x8(y, a.v_inv));
      } else {
        st_v4(vout + (size_t)v * 16, x0[u]);
      }
    }
  }
}

template <typename T, bool F8>
static cudaError_t launch_append_t(const AppendArgs& a, const AxisTurns& turns, const LaunchCfg& cfg) {
  auto* kern = a.style == 0 ? append_kernel<T, 0, F8> : append_kernel<T, 1, F8>;
  // Warps to a token: as many as keep a lane one batch busy while the SMs have room for 32 warps each.
  const int gv = a.D * (int)sizeof(T) / 16 / (a.style == 0 ? 2 : 1);
  const int64_t items = (int64_t)(a.Hq + a.H) * gv;
  int share = 1;
  while (share < 16 && (int64_t)a.T * share < 32LL * cfg.num_sms && (int64_t)share * 32 < items) share *= 2;
  const int64_t ctas = ((int64_t)a.T * share + kAppendWarps - 1) / kAppendWarps;
  return launch_ex(kern, dim3((unsigned)ctas), dim3(kAppendThreads), (size_t)kAppendWarps * a.D / 2 * sizeof(float2),
                   cfg.stream, cfg.pdl, a, turns, share);
}

cudaError_t launch_append(const AppendArgs& a, const AxisTurns& turns, const LaunchCfg& cfg) {
  if (a.dtype == IS_F32) return launch_append_t<float, false>(a, turns, cfg);
  if (a.dtype == IS_BF16)
    return a.fp8 ? launch_append_t<__nv_bfloat16, true>(a, turns, cfg)
                 : launch_append_t<__nv_bfloat16, false>(a, turns, cfg);
  return a.fp8 ? launch_append_t<__half, true>(a, turns, cfg) : launch_append_t<__half, false>(a, turns, cfg);
}

}  // namespace isk
