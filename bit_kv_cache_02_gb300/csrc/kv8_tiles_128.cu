// The many-rows attention kernels of the 8-bit cache for head_dim 128.
#include "kv8_tiles.cuh"

namespace kv8 {
cudaError_t launch_tiles_128(const AttnArgs &a, cudaStream_t stream) { return tiles::launch_dim<128, false>(a, stream); }
}  // namespace kv8
