// ss_attend for f16 activations and an f16 cache.
#include "ss_kv_attend.cuh"

namespace ss {
AttendKernel kv_attend_f16(int head_dim, int row_tile) { return kv::pick<__half, false>(head_dim, row_tile); }
}  // namespace ss
