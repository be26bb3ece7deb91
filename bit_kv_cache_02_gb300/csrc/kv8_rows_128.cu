// The few-rows attention kernels of the 8-bit cache for head_dim 128.
#include "kv8_rows.cuh"

namespace kv8 {
cudaError_t launch_rows_128(const AttnArgs &a, cudaStream_t stream) { return rows::launch_dim<128, false>(a, stream); }
}  // namespace kv8
