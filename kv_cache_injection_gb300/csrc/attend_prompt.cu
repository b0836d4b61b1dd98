// is_attend with prompts: the forms of the prompt kernel (attend_prompt.cuh).
#include "attend_prompt.cuh"

namespace isk {

cudaError_t launch_attend_prompt(const AttendArgs& a, const LaunchCfg& cfg) {
  if (a.D == 256) return a.dtype == IS_BF16 ? launch_prompt_t<__nv_bfloat16, kCachePlain, 256>(a, cfg) : launch_prompt_t<__half, kCachePlain, 256>(a, cfg);
  if (a.dtype == IS_BF16) {
    if (a.D == 64)
      return a.fp8 ? launch_prompt_t<__nv_bfloat16, kCacheE4m3, 64>(a, cfg) : launch_prompt_t<__nv_bfloat16, kCachePlain, 64>(a, cfg);
    return a.fp8 ? launch_prompt_t<__nv_bfloat16, kCacheE4m3, 128>(a, cfg) : launch_prompt_t<__nv_bfloat16, kCachePlain, 128>(a, cfg);
  }
  if (a.D == 64) return a.fp8 ? launch_prompt_t<__half, kCacheE4m3, 64>(a, cfg) : launch_prompt_t<__half, kCachePlain, 64>(a, cfg);
  return a.fp8 ? launch_prompt_t<__half, kCacheE4m3, 128>(a, cfg) : launch_prompt_t<__half, kCachePlain, 128>(a, cfg);
}

}  // namespace isk
