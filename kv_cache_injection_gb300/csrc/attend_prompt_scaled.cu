// is_attend_scaled with prompts: the forms of the prompt kernel (attend_prompt.cuh)
// over codes.
#include "attend_prompt.cuh"

namespace isk {

template <typename T, CacheKind KIND>
static cudaError_t launch_prompt_scaled(const AttendArgs& a, const LaunchCfg& cfg) {
  return a.D == 64 ? launch_prompt_t<T, KIND, 64>(a, cfg) : launch_prompt_t<T, KIND, 128>(a, cfg);
}

cudaError_t launch_attend_prompt_scaled(const AttendArgs& a, bool int8, const LaunchCfg& cfg) {
  if (a.dtype == IS_BF16)
    return int8 ? launch_prompt_scaled<__nv_bfloat16, kCacheScaledInt8>(a, cfg) : launch_prompt_scaled<__nv_bfloat16, kCacheScaledE4m3>(a, cfg);
  return int8 ? launch_prompt_scaled<__half, kCacheScaledInt8>(a, cfg) : launch_prompt_scaled<__half, kCacheScaledE4m3>(a, cfg);
}

}  // namespace isk
