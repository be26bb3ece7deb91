// What cross attention and attention with shared blocks need besides the rows and
// the tile kernel: the segments, looked up once for all CTAs, and the join of the
// tile kernel's parts over shared blocks.  Both are bound by latency: 3 us for 65
// segments, of which a launch is two, and 8 us for 8 items of 19 parts of 256 rows
// (18 MB).
#include "kv8_rows.cuh"
#include "kv8_tiles.cuh"

namespace kv8 {
namespace shared {

// A thread per group, if there are any, then per sequence.
__global__ void __launch_bounds__(kSegThreads) segments_kernel(const AttnArgs a) {
  asm volatile("griddepcontrol.launch_dependents;");
  const int i = blockIdx.x * kSegThreads + threadIdx.x;
  if (a.groups)  // nothing to join so far
    for (int k = i; k < kMaxTileCtas; k += gridDim.x * kSegThreads) a.items[2 * k] = make_int4(0, 0, 0, 0);
  const int s = i - a.groups;
  bool shut = false, falls = false;
  if (i < a.groups + a.geo.S) {
    if (i < a.groups)
      falls = a.group_start[i + 1] < a.group_start[i];
    else if (a.row_start)
      falls = a.row_start[s + 1] < a.row_start[s];
    const Seg x = i < a.groups ? group_seg(a, i) : a.groups ? own_seg(a, s, shut) : load_seg<false>(a, i);
    store_plan(a, i, x, rows::plan_of(a, x, i < a.groups ? a.group_rows_max : a.rows_max));
  }
  falls = __any_sync(0xffffffffu, falls);
  if ((i & 31) == 0) a.falls[i >> 5] = falls;
  // Rows that the launch over their group's blocks is not to write, a sequence after
  // the other by the whole warp: all later kernels wait for this one (2000 rows x
  // 32 query heads: 25 us; by the sequence's thread alone 330).
  for (unsigned m = __ballot_sync(0xffffffffu, shut); m; m &= m - 1) {
    const int j = __shfl_sync(0xffffffffu, s, __ffs(m) - 1);
    const long long from = max(a.row_start ? a.row_start[j] : j, 0);
    const long long to = min(a.row_start ? a.row_start[j + 1] : j + 1, a.rows);
    for (int h = 0; h < a.geo.H; ++h)
      for (long long r = from * a.group + (threadIdx.x & 31); r < to * a.group; r += 32)
        a.carry_ml[h * a.carry_blocks * 32 + r] = make_float2(0.f, -1.f);
  }
}

// The parts of an item, a (group, 256 rows, KV head), over its keys, and what the
// launches behind the shared blocks have left: the CTAs of the tile kernel leave
// them, and here a CTA joins 32 rows, 64 channels.  (The last CTA that finishes
// would read them alone: a group of 256 rows, 8 KV heads, has 19 for each head.)
// A thread takes eight channels of a row, from the parts with 32 rows side by
// side, eight parts at a time; shared memory turns them into whole rows.  An item
// of so many parts ends four CTAs behind its first: there are kMaxTileCtas / 4 at
// most, found by a look at all.
constexpr int kJoinRows = 32, kJoinThreads = 256, kAtOnce = 8;
template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const AttnArgs a) {
  constexpr int PIECES = D / 64, SUBS = tiles::kRows / kJoinRows;
  const int piece = blockIdx.x % PIECES, sub = blockIdx.x / PIECES % SUBS, nth = blockIdx.x / (PIECES * SUBS);
  __shared__ int counts[kJoinThreads / 32], found;
  wait_before();
  const bool has = threadIdx.x < kMaxTileCtas && a.items[2 * threadIdx.x].y > 0;
  const unsigned mask = __ballot_sync(0xffffffffu, has);
  if (threadIdx.x == 0) found = -1;
  if ((threadIdx.x & 31) == 0) counts[threadIdx.x >> 5] = __popc(mask);
  __syncthreads();
  int before = __popc(mask & ((1u << (threadIdx.x & 31)) - 1u));
  for (int w = 0; w < static_cast<int>(threadIdx.x >> 5); ++w) before += counts[w];
  if (has && before == nth) found = threadIdx.x;
  __syncthreads();
  const int c0 = found;
  if (c0 < 0) return;
  const int4 item = a.items[2 * c0];
  const int first = item.x, n = item.y, h = item.z, row0 = item.w + sub * kJoinRows;
  const int4 rows = a.items[2 * c0 + 1];
  const int t0 = rows.x, n_rows = rows.y;  // the group's first tensor row, its rows of a KV head
  if (row0 >= n_rows || !KVQ_IN_BOUNDS(a.geo.status, first, 2 * kMaxTileCtas) ||
      !KVQ_IN_BOUNDS(a.geo.status, c0 + n - 1, kMaxTileCtas) || c0 + n > kMaxTileCtas)
    return;
  __shared__ float4 turned[kJoinRows][17];
  __shared__ float2 sums[kJoinRows];
  const float ninf = __int_as_float(0xff800000);
  {
    const int r = threadIdx.x & 31, q = threadIdx.x >> 5;  // row, and two of its float4
    float4 o[2] = {};
    float2 ml = make_float2(ninf, 0.f);
    const size_t at = static_cast<size_t>(sub) * kJoinRows + r;
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += kAtOnce) {
      float2 e[kAtOnce];
      float4 x[kAtOnce][2];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int sl = i0 + i == 0 ? first : 2 * (c0 + min(i0 + i, n - 1));
        e[i] = __ldcg(a.tile_ml + static_cast<size_t>(sl) * tiles::kRows + at);
        const float4 *src = reinterpret_cast<const float4 *>(a.tile_o) +
                            (static_cast<size_t>(sl) * (D / 4) + 16 * piece + 2 * q) * tiles::kRows + at;
        x[i][0] = __ldcg(src);
        x[i][1] = __ldcg(src + tiles::kRows);
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (i0 + i >= n) break;  // (the last part again)
        const Join j = join(ml, e[i]);
        ml = make_float2(fmaxf(ml.x, e[i].x), j.sum);
#pragma unroll
        for (int k = 0; k < 2; ++k)
          o[k] = make_float4(fmaf(o[k].x, j.x, x[i][k].x * j.y), fmaf(o[k].y, j.x, x[i][k].y * j.y),
                             fmaf(o[k].z, j.x, x[i][k].z * j.y), fmaf(o[k].w, j.x, x[i][k].w * j.y));
      }
    }
    turned[r][2 * q] = o[0];
    turned[r][2 * q + 1] = o[1];
    if (q == 0) sums[r] = make_float2(ml.x == ninf ? ninf : ml.x - tiles::kShift, ml.y);
  }
  __syncthreads();
  const int r = threadIdx.x >> 3, q = threadIdx.x & 7, row = row0 + r;
  if (row >= n_rows || !row_in_bounds(a, t0, h, row)) return;
  const int tok = row / a.group, head = h * a.group + row - tok * a.group;
  const CarryRow carry = carry_row<D>(a, h, t0, row);
  const float2 own = *carry.ml;
  if (own.y < 0.f) return;
  const Join j = join(sums[r], own);
  const float f = inverse_sum(j.sum, 0);
  uint32_t e[4];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float4 x = turned[r][2 * q + k];
    const float4 y = carry.at(16 * piece + 2 * q + k);
    e[2 * k] = pack2<BF16>(fmaf(x.x, j.x, y.x * j.y) * f, fmaf(x.y, j.x, y.y * j.y) * f);
    e[2 * k + 1] = pack2<BF16>(fmaf(x.z, j.x, y.z * j.y) * f, fmaf(x.w, j.x, y.w * j.y) * f);
  }
  *reinterpret_cast<uint4 *>(a.out.p + (static_cast<long long>(t0) + tok) * a.out.row + head * a.out.head +
                             64 * piece + 8 * q) = make_uint4(e[0], e[1], e[2], e[3]);
}

}  // namespace shared

cudaError_t launch_segments(const AttnArgs &a, cudaStream_t stream) {
  shared::segments_kernel<<<seg_ctas(a.groups, a.geo.S), kSegThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_join(const AttnArgs &a, cudaStream_t stream) {
  static_assert(kMaxTileCtas <= shared::kJoinThreads, "a thread per CTA of the tile kernel");
  const unsigned grid = kMaxTileCtas / 4 * (a.geo.D / 64) * (kTileRows / shared::kJoinRows);
  auto kernel = a.geo.D == 128 ? (a.geo.bf16 ? shared::join_kernel<128, true> : shared::join_kernel<128, false>)
                               : (a.geo.bf16 ? shared::join_kernel<64, true> : shared::join_kernel<64, false>);
  return launch_after(kernel, grid, shared::kJoinThreads, 0, stream, a);
}

}  // namespace kv8
