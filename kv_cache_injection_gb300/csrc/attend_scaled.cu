// is_attend_scaled: softmax attention over a cache of 8-bit codes c, d (keys,
// values) with a scale for each block and KV head, ks and vs.  With y_j = scale *
// (q . c_j) * ks_j + ln vs_j,
//   out = sum_j exp(y_j) d_j / sum_j exp(y_j) / vs_j,   lse = log of that sum:
// the V scale goes into the exponent, so that the second product takes the codes
// as they are, one maximum (of y) and one exponential a logit serve both sums,
// and no weight leaves the range of its 16 bits whatever the blocks' scales are
// to one another (a weight times a scale of its own would, for blocks 2^15 apart).
//
// Measured (bf16 queries): 4 requests of 60,000-131,000 tokens over INT8 (H = 8, D =
// 128, 904 MB) 159 us = 5.7 TB/s, 84 % of a plain copy; 100 requests of 300-2048 tokens
// (H = 4, 117 MB) 38 us over INT8 and 35 over E4M3, 17 for their bytes: a tile of 32 keys
// is about 1000 instructions of a warp, a third of them the widening, 12 warps an SM;
// one request of 1313 tokens 9.1 us, the latency of two kernels.
#include "attend_split.cuh"

namespace isk {

cudaError_t launch_attend_scaled(const AttendArgs& a, bool int8, const LaunchCfg& cfg) {
  // As over an FP8 cache (launch_attend): more than 32 rows go to the prompt
  // kernel where its shared memory has room and the scale is positive.  It takes
  // a block's scales once for eight keys, so blocks have to be whole eights.
  if (a.D <= 128 && a.block_size % 8 == 0 && a.G <= 64 && (int64_t)a.max_q * a.G > 32 && a.scale > 0.f)
    return a.dtype == IS_BF16 ? launch_attend_prompt_scaled_bf16(a, int8, cfg) : launch_attend_prompt_scaled_f16(a, int8, cfg);
  if (a.dtype == IS_BF16)
    return int8 ? launch_mma<__nv_bfloat16, kCacheScaledInt8>(a, cfg) : launch_mma<__nv_bfloat16, kCacheScaledE4m3>(a, cfg);
  return int8 ? launch_mma<__half, kCacheScaledInt8>(a, cfg) : launch_mma<__half, kCacheScaledE4m3>(a, cfg);
}

}  // namespace isk
