// Which kernel of is_attend takes a call: the split kernel (attend_split.cuh) for
// few query rows per request, the prompt kernel (attend_prompt.cuh) for many.
#include "attend_split.cuh"

namespace isk {

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
    return a.fp8 ? launch_mma<__nv_bfloat16, kCacheE4m3>(a, cfg) : launch_mma<__nv_bfloat16, kCachePlain>(a, cfg);
  if (a.dtype == IS_F16) return a.fp8 ? launch_mma<__half, kCacheE4m3>(a, cfg) : launch_mma<__half, kCachePlain>(a, cfg);
  if (a.D == 64) return launch_split<float, FmaEngine<64>>(a, cfg);
  if (a.D == 128) return launch_split<float, FmaEngine<128>>(a, cfg);
  return launch_split<float, FmaEngine<256>>(a, cfg);
}

}  // namespace isk
