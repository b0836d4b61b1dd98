// is_attend_scaled with prompts, bf16 queries.
#include "attend_prompt_scaled.cuh"

namespace isk {

cudaError_t launch_attend_prompt_scaled_bf16(const AttendArgs& a, bool int8, const LaunchCfg& cfg) {
  return launch_prompt_scaled<__nv_bfloat16>(a, int8, cfg);
}

}  // namespace isk
