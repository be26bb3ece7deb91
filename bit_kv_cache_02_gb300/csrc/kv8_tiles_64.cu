// The many-rows attention kernels of the 8-bit cache for head_dim 64.
#include "kv8_tiles.cuh"

namespace kv8 {
cudaError_t launch_tiles_64(const AttnArgs &a, cudaStream_t stream) { return tiles::launch_dim<64, false>(a, stream); }
}  // namespace kv8
