// ss_attend for bf16 activations and an e4m3 cache.
#include "ss_kv_attend.cuh"
#include "ss_kv_attend8.cuh"

namespace ss {
// Few query rows: keys and values converted in registers, each by the one warp that has it.  More: converted once into
// shared memory for all rows.  Measured (us, registers / shared memory): 32 rows x 4 tokens x 4 query heads to a key
// head (16 query rows) 155 / 202, 32 x 4 x 8 (32 query rows) 127 / 76, 32 x 8 x 8 (64) 199 / 98; 256 columns, 26 x 5 x 2
// (10 query rows) 94 / 77.
AttendKernel kv_attend_bf16_e4m3(int head_dim, int row_tile) {
  return head_dim <= 128 && row_tile <= 16 ? kv8::pick<__nv_bfloat16>(head_dim) : kv::pick<__nv_bfloat16, true>(head_dim, row_tile);
}
}  // namespace ss
