// ss_attend for bf16 activations and a bf16 cache.
#include "ss_kv_attend.cuh"

namespace ss {
AttendKernel kv_attend_bf16(int head_dim, int row_tile) { return kv::pick<__nv_bfloat16, false>(head_dim, row_tile); }
}  // namespace ss
