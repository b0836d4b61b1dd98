// is_attend_scaled with prompts: the forms of the prompt kernel (attend_prompt.cuh)
// over codes, for queries of type T.
#pragma once

#include "attend_prompt.cuh"

namespace isk {

template <typename T, CacheKind KIND>
static cudaError_t launch_prompt_scaled(const AttendArgs& a, const LaunchCfg& cfg) {
  // What eight keys share is shared by sixteen where blocks are whole sixteens.
  if (a.block_size % 16 == 0)
    return a.D == 64 ? launch_prompt_t<T, KIND, 64, 16>(a, cfg) : launch_prompt_t<T, KIND, 128, 16>(a, cfg);
  return a.D == 64 ? launch_prompt_t<T, KIND, 64, 8>(a, cfg) : launch_prompt_t<T, KIND, 128, 8>(a, cfg);
}
template <typename T>
static cudaError_t launch_prompt_scaled(const AttendArgs& a, bool int8, const LaunchCfg& cfg) {
  return int8 ? launch_prompt_scaled<T, kCacheScaledInt8>(a, cfg) : launch_prompt_scaled<T, kCacheScaledE4m3>(a, cfg);
}

}  // namespace isk
