// ss_attend_blocks for f16 activations.
#include "ss_kv_attend.cuh"
#include "ss_kv_attend8.cuh"

namespace ss {
// As without factors of blocks (ss_kv_attend_f16_e4m3.cu).  Measured (us, with factors of blocks / of heads): 40 x 5 of up to
// 16000 tokens, 64 query rows, 155 / 148.
AttendKernel kv_attend_f16_blocks(int head_dim, int row_tile) {
  return head_dim <= 128 && row_tile <= 16 ? kv8::pick<__half, true>(head_dim) : kv::pick<__half, true, true>(head_dim, row_tile);
}
}  // namespace ss
