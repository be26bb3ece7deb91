// The few-rows kernels of cross attention and shared blocks for head_dim 128.
#include "kv8_rows.cuh"

namespace kv8 {
cudaError_t launch_rows_128_shared(const AttnArgs &a, cudaStream_t stream) { return rows::launch_dim<128, true>(a, stream); }
}  // namespace kv8
