// ss_attend_blocks for bf16 activations.
#include "ss_kv_attend.cuh"
#include "ss_kv_attend8.cuh"

namespace ss {
// As without factors of blocks (ss_kv_attend_bf16_e4m3.cu).  Measured (us, with factors of blocks / of heads): 80 rows of up to
// 12000 tokens, 16 query rows, 158 / 155; 32 x 4 of 8000 with 32 query rows 82 / 76; 32 x 8 with 64 88 / 86; 26 x 5 of 256
// columns 84 / 80.
AttendKernel kv_attend_bf16_blocks(int head_dim, int row_tile) {
  return head_dim <= 128 && row_tile <= 16 ? kv8::pick<__nv_bfloat16, true>(head_dim) : kv::pick<__nv_bfloat16, true, true>(head_dim, row_tile);
}
}  // namespace ss
