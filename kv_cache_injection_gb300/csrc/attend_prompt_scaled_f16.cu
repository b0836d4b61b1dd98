// is_attend_scaled with prompts, fp16 queries.
#include "attend_prompt_scaled.cuh"

namespace isk {

cudaError_t launch_attend_prompt_scaled_f16(const AttendArgs& a, bool int8, const LaunchCfg& cfg) {
  return launch_prompt_scaled<__half>(a, int8, cfg);
}

}  // namespace isk
