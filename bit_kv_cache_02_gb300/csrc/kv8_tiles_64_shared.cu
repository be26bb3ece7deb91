// The many-rows kernels of cross attention and shared blocks for head_dim 64.
#include "kv8_tiles.cuh"

namespace kv8 {
cudaError_t launch_tiles_64_shared(const AttnArgs &a, cudaStream_t stream) { return tiles::launch_dim<64, true>(a, stream); }
}  // namespace kv8
