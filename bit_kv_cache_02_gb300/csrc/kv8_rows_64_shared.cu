// The few-rows kernels of cross attention and shared blocks for head_dim 64.
#include "kv8_rows.cuh"

namespace kv8 {
cudaError_t launch_rows_64_shared(const AttnArgs &a, cudaStream_t stream) { return rows::launch_dim<64, true>(a, stream); }
}  // namespace kv8
