#include "kv8_append.cuh"

namespace kv8 {
cudaError_t launch_append_axes(const Geo &geo, const Rows &k, const Rows &v, const Rows &q, const Rows &q_out, int Hq,
                               const int *row_start, int rows, int max_new, const float *rope, int rot_dim,
                               int interleaved, const Axes &axes, cudaStream_t stream, uint64_t *launches) {
  return append::launch<true>(geo, k, v, q, q_out, Hq, row_start, rows, max_new, rope, rot_dim, interleaved, axes,
                              stream, launches);
}
}  // namespace kv8
