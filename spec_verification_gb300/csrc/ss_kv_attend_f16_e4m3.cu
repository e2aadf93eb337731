// ss_attend for f16 activations and an e4m3 cache.
#include "ss_kv_attend8.cuh"

namespace ss {
AttendKernel kv_attend_f16_e4m3(int head_dim, int row_tile) { return kv8::pick<__half>(head_dim, row_tile); }
}  // namespace ss
