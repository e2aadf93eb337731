// ss_attend_prompt for f16.
#include "ss_kv_prompt.cuh"

namespace ss {
PromptKernel kv_prompt_f16(int head_dim, int tiles) { return kv::prompt::pick<__half>(head_dim, tiles); }
}  // namespace ss
