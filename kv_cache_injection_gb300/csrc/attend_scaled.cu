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
  // More than 32 rows go to the prompt kernel where its shared memory has room
  // and the scale is positive.  It takes a block's scales once for eight keys, so
  // blocks have to be whole eights.  Its time hardly depends on the rows, this
  // kernel's grows with every 16 of them, and where they meet depends on the
  // requests.  Here and there, INT8, 32 + 8 heads: 4 requests of up to 131,000
  // tokens, 32 rows 397 and 408 us, 36 rows 577 and 409; 16 of 900-2000, 32 rows 42
  // and 45, 36 rows 57 and 45.  Of more requests the prompt kernel is ahead from 17
  // rows on (100 of 300-2048, 16 rows 115 and 150 us, 32 rows 217 and 150; 64 of
  // 500-8000, 32 rows 319 and 269), of a single short one not yet at 48 (1313
  // tokens, 16 and 20): 32 rows lie between them.  Prompts that have to stay here:
  // two of 2000-2500 tokens behind up to 8192, 4135 us over blocks of 7 where those
  // of 8 take 622 there; with 8 + 4 heads of 256 3014.
  if (a.D <= 128 && a.block_size % 8 == 0 && a.G <= 64 && (int64_t)a.max_q * a.G > 32 && a.scale > 0.f)
    return a.dtype == IS_BF16 ? launch_attend_prompt_scaled_bf16(a, int8, cfg) : launch_attend_prompt_scaled_f16(a, int8, cfg);
  if (a.dtype == IS_BF16)
    return int8 ? launch_mma<__nv_bfloat16, kCacheScaledInt8>(a, cfg) : launch_mma<__nv_bfloat16, kCacheScaledE4m3>(a, cfg);
  return int8 ? launch_mma<__half, kCacheScaledInt8>(a, cfg) : launch_mma<__half, kCacheScaledE4m3>(a, cfg);
}

}  // namespace isk
