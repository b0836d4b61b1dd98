// is_attend_scaled: softmax attention over a cache of 8-bit codes c, d (keys,
// values) with a scale for each block and KV head, ks and vs.  With y_j = scale *
// (q . c_j) * ks_j + ln vs_j,
//   out = sum_j exp(y_j) d_j / sum_j exp(y_j) / vs_j,   lse = log of that sum:
// the V scale goes into the exponent, so that the second product takes the codes
// as they are, one maximum (of y) and one exponential a logit serve both sums,
// and no weight leaves the range of its 16 bits whatever the blocks' scales are
// to one another (a weight times a scale of its own would, for blocks 2^15 apart).
#include "attend_split.cuh"

namespace isk {

cudaError_t launch_attend_scaled(const AttendArgs& a, bool int8, const LaunchCfg& cfg) {
  if (a.dtype == IS_BF16)
    return int8 ? launch_mma<__nv_bfloat16, kCacheScaledInt8>(a, cfg) : launch_mma<__nv_bfloat16, kCacheScaledE4m3>(a, cfg);
  return int8 ? launch_mma<__half, kCacheScaledInt8>(a, cfg) : launch_mma<__half, kCacheScaledE4m3>(a, cfg);
}

}  // namespace isk
