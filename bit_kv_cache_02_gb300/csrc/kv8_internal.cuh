// Internal definitions shared by the kernels of the 8-bit paged KV cache
// (include/kv8.h).
#pragma once

#include <cuda_bf16.h>

#include "../../include/kv8.h"
#include "kvq_internal.cuh"

namespace kv8 {

using kvq::set_status;

// Cache geometry and buffers as the kernels see them.
struct Geo {
  int S, H, D, B, fmt, bf16, capacity, max_blocks, num_blocks;
  uint8_t *codes;
  float *scales;
  uint16_t *k_win, *v_win;
  const int *seq_len;
  const int *table;
  int *status;
};

// A 16-bit tensor [rows][heads][D] (strides in elements).
struct Rows {
  uint16_t *p;
  long long row, head;
};

// The new rows of sequence s and its length; ok: the row range is usable.
struct Seq {
  int L, n, row0;
  bool ok;
};

__device__ __forceinline__ Seq load_seq(const Geo &geo, const int *row_start, int rows, int max_new, int s) {
  Seq q;
  q.L = geo.seq_len[s];
  long long r0 = s, r1 = s + 1;
  if (row_start) {
    r0 = row_start[s];
    r1 = row_start[s + 1];
  }
  q.ok = r0 >= 0 && r1 >= r0 && r1 <= rows && r1 - r0 <= max_new;
  q.row0 = static_cast<int>(r0);
  q.n = q.ok ? static_cast<int>(r1 - r0) : 0;
  return q;
}

// x / y for x >= 0, y > 0.  32 bits are enough but for the longest lines, and a
// 64-bit division costs hundreds of clocks, which a short call would wait for.
__device__ __forceinline__ long long divide(long long x, long long y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}

// Largest s with key(s) <= x, where key rises with s (0 if there is none).
template <typename F>
__device__ __forceinline__ int last_at_or_below(int S, int x, F key) {
  int lo = 0, hi = S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (key(mid) <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// 2^e as fp32 for -126 <= e <= 127.
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

// The two 16-bit floats of a word as fp32.
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// Two fp32 values rounded to a word of 16-bit floats (x0 in the low half).
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float x0, float x1) {
  if (BF16) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x0, x1);
    return *reinterpret_cast<const uint32_t *>(&b);
  }
  return kvq::h2_as_u32(__floats2half2_rn(x0, x1));
}

// Magnitude bits from which a 16-bit float is an infinity or a NaN.
template <bool BF16>
__host__ __device__ constexpr uint32_t nonfinite_bits() {
  return BF16 ? 0x7f80u : 0x7c00u;
}

// ------------------------------------------------------- host-side launchers

cudaError_t launch_append(const Geo &geo, const Rows &k, const Rows &v, const Rows &q, const Rows &q_out, int Hq,
                          const int *row_start, int rows, int max_new, const float *rope, int rot_dim,
                          int interleaved, cudaStream_t stream, uint64_t *launches);

// Attention counts the values of a block whose scale is smaller (2^-80) as
// zeros: 1 / scale times the weights of 2^31 tokens stays finite.  Weights are
// formed relative to the largest score times scale that a row has met; blocks
// of zeros enter that maximum with this scale, below all others, so that small
// values beside them keep their weights' bits.
constexpr float kZeroScale = 8.27180613e-25f;
constexpr float kZeroLog = -80.f;

// What a row's weighted sum is multiplied by, `last` being the last position that
// the row sees: 0 where it sees no token.  Where it sees some the weights' sum is
// above 0, but for scores that are all -infinity, as an infinite query can make
// them: NaN.
__device__ __forceinline__ float inverse_sum(float sum, int last) {
  return sum != 0.f ? 1.f / sum : last < 0 ? 0.f : __int_as_float(0x7fc00000);
}

// CTAs of one attention launch at most (sizes the workspace's partial slots).
constexpr int kMaxCtas = 640;
constexpr int kRowTile = 16;  // (token, query head) rows that share one pass over the keys

// Sequences with more rows per KV head than this go to the tile kernel.  The
// rows kernel reads the keys once for 16 rows, the tile kernel once for 256
// after a longer start.  Rows against tile kernel, int8, D 128, 16 sequences x 8
// KV heads x 4000 tokens: 54 and 89 us at 32 rows, 95 and 90 at 64, 177 and 86
// at 128; 32 x 32 x 2000 tokens at 48 rows: 284 and 267.  Rows alone do not
// decide: with one sequence of 30,000 tokens x 8 heads, which gives the tile
// kernel few items to fill the SMs with, the border lies higher (34 and 70 us at
// 32 rows, 49 and 66 at 64, 91 and 69 at 128).
constexpr int kRowsMax = 48;
constexpr int kTileRows = 256;      // rows of an item of the tile kernel
constexpr int kMaxTileCtas = 160;

// Byte offsets of the workspace regions.  One merge counter per CTA of either
// kernel comes first, at places that do not depend on the call: what a call of
// one shape leaves of its partial results is never another's counter.  Rows
// kernel: partial outputs [2 kMaxCtas][16][D] and their (max, sum).  Tile
// kernel, where a sequence can bring enough rows: the same for
// [2 kMaxTileCtas][256].
struct AttnPlan {
  size_t off_cnt, off_tile_cnt, off_o, off_ml, off_tile_o, off_tile_ml, bytes;
  bool tiles;
};
AttnPlan plan_attn(int D, long long rows_per_head);

struct AttnArgs {
  Geo geo;
  int Hq, group;
  Rows q, out;
  const int *row_start;
  int rows, max_new, max_len;
  float zscale;       // softmax scale * log2(e)
  float *part_o;      // [2 kMaxCtas][16][D] unnormalized partial outputs
  float2 *part_ml;    // [2 kMaxCtas][16] (max, sum) in log2 units
  int *counters;      // [kMaxCtas], zero on entry, left zero on exit
  float *tile_o;      // [2 kMaxTileCtas][D / 4][256][4] unnormalized partial outputs
  float2 *tile_ml;    // [2 kMaxTileCtas][256] (reference, sum)
  int *tile_counters; // [kMaxTileCtas], zero on entry, left zero on exit
  int rows_max;       // rows per KV head up to which the rows kernel takes a sequence
  long long wait_limit;  // SM cycles that a wait of the tile kernel may last before it gives up
  int wait_test;         // test aid: a wait of the tile kernel that nothing completes
};

// Debug builds: the tensors' row and head of a KV head's row are in range.
__device__ __forceinline__ bool row_in_bounds(const AttnArgs &a, const Seq &q, int h, int row) {
  return KVQ_IN_BOUNDS(a.geo.status, static_cast<long long>(q.row0) + row / a.group, a.rows) &&
         KVQ_IN_BOUNDS(a.geo.status, static_cast<long long>(h) * a.group + row % a.group, a.Hq);
}

cudaError_t launch_attn(const AttnArgs &a, bool tiles, cudaStream_t stream, uint64_t *launches);
// the kernels for one head dimension (one translation unit each)
cudaError_t launch_rows_128(const AttnArgs &a, cudaStream_t stream);
cudaError_t launch_rows_64(const AttnArgs &a, cudaStream_t stream);
cudaError_t launch_tiles_128(const AttnArgs &a, cudaStream_t stream);
cudaError_t launch_tiles_64(const AttnArgs &a, cudaStream_t stream);

}  // namespace kv8
