// ss_attend for bf16 activations and an e4m3 cache.
#include "ss_kv_attend.cuh"
#include "ss_kv_attend8.cuh"

namespace ss {
constexpr int kFew = 16;
AttendKernel kv_attend_bf16_e4m3(int head_dim, int row_tile) {
  return head_dim <= 128 && row_tile <= kFew ? kv8::pick<__nv_bfloat16>(head_dim, row_tile) : kv::pick<__nv_bfloat16, true>(head_dim, row_tile);
}
}  // namespace ss
