// ss_attend_prompt for bf16.
#include "ss_kv_prompt.cuh"

namespace ss {
PromptKernel kv_prompt_bf16(int head_dim, int tiles) { return kv::prompt::pick<__nv_bfloat16>(head_dim, tiles); }
}  // namespace ss
