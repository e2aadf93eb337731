// ss_attend_blocks for bf16 activations.
#include "ss_kv_attend.cuh"
#include "ss_kv_attend8.cuh"

namespace ss {
// As without factors of blocks (ss_kv_attend_bf16_e4m3.cu).
AttendKernel kv_attend_bf16_blocks(int head_dim, int row_tile) {
  return head_dim <= 128 && row_tile <= 16 ? kv8::pick<__nv_bfloat16, true>(head_dim) : kv::pick<__nv_bfloat16, true, true>(head_dim, row_tile);
}
}  // namespace ss
