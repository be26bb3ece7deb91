// What attention behind shared blocks needs besides the kernels of the two
// attentions: the segments, looked up once for all CTAs, and the join of the
// tile kernel's parts.
#include "kv8_tiles.cuh"

namespace kv8 {
namespace shared {

constexpr int kSegThreads = 128;
constexpr int kQuads = 4;  // float4 of a row that a thread of the join takes

// A thread per group, then per sequence.
__global__ void __launch_bounds__(kSegThreads) segments_kernel(const AttnArgs a) {
  asm volatile("griddepcontrol.launch_dependents;");
  const int i = blockIdx.x * kSegThreads + threadIdx.x;
  if (i >= a.groups + a.geo.S) return;
  const Seg x = i < a.groups ? group_seg(a, i) : own_seg(a, i - a.groups);
  a.plan[2 * i] = make_int4(x.L, x.n, x.row0, x.base);
  a.plan[2 * i + 1] = make_int4(x.entry, x.ok, 0, 0);
}

// The parts of an item, a (group, 256 rows, KV head), over its keys: the CTAs of
// the tile kernel leave them, and here a thread per row and 16 channels joins
// them, all SMs together.  (The last CTA that finishes would read them alone: a
// group of 256 rows, 8 KV heads, has 19 for each head.)
template <int D>
__global__ void __launch_bounds__(tiles::kRows) join_kernel(const AttnArgs a) {
  follow<true>();
  constexpr int PIECES = D / 4 / kQuads;
  const int piece = blockIdx.x % PIECES, h = blockIdx.x / PIECES % a.geo.H;
  const int slot = blockIdx.x / PIECES / a.geo.H, r = threadIdx.x;
  const tiles::Pair p = tiles::pair_of_slot<true>(a, slot);
  if (!p.units) return;
  const int row = p.rt * tiles::kRows + r;
  if (row >= p.q.n * a.group || !row_in_bounds(a, p.q.row0, h, row)) return;
  const int4 item = a.items[static_cast<size_t>(slot) * a.geo.H + h];
  const int first = item.x, c0 = item.y, n = item.z;
  // (where row_start or group_start falls, or a wait ran out, nothing was left here)
  if (n <= 0 || n > kMaxTileCtas || c0 < 0 || c0 > kMaxTileCtas - n || first < 0 || first >= 2 * kMaxTileCtas) return;
  const float ninf = __int_as_float(0xff800000);
  float o[4 * kQuads], mm = ninf, ll = 0.f;
#pragma unroll
  for (int k = 0; k < 4 * kQuads; ++k) o[k] = 0.f;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const int sl = i == 0 ? first : 2 * (c0 + i);
    const float4 *src = reinterpret_cast<const float4 *>(a.tile_o) +
                        (static_cast<size_t>(sl) * (D / 4) + piece * kQuads) * tiles::kRows + r;
    const float2 e = a.tile_ml[sl * tiles::kRows + r];
    float4 x[kQuads];
#pragma unroll
    for (int k = 0; k < kQuads; ++k) x[k] = src[static_cast<size_t>(k) * tiles::kRows];
    const Join j = join(make_float2(mm, ll), e);
    mm = fmaxf(mm, e.x);
    ll = j.sum;
#pragma unroll
    for (int k = 0; k < kQuads; ++k) {
      o[4 * k] = fmaf(o[4 * k], j.x, x[k].x * j.y);
      o[4 * k + 1] = fmaf(o[4 * k + 1], j.x, x[k].y * j.y);
      o[4 * k + 2] = fmaf(o[4 * k + 2], j.x, x[k].z * j.y);
      o[4 * k + 3] = fmaf(o[4 * k + 3], j.x, x[k].w * j.y);
    }
  }
  const int tok = row / a.group;
  const size_t at = carry_at(a, p.q.row0 + tok, h * a.group + row - tok * a.group);
  float4 *dst = reinterpret_cast<float4 *>(a.carry_o + at * D) + piece * kQuads;
#pragma unroll
  for (int k = 0; k < kQuads; ++k) dst[k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
  if (piece == 0) a.carry_ml[at] = make_float2(mm == ninf ? mm : mm - tiles::kShift, ll);
}

}  // namespace shared

cudaError_t launch_segments(const AttnArgs &a, cudaStream_t stream) {
  const int n = a.groups + a.geo.S;
  shared::segments_kernel<<<(n + shared::kSegThreads - 1) / shared::kSegThreads, shared::kSegThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_join(const AttnArgs &a, cudaStream_t stream) {
  const long long slots = static_cast<long long>(a.rows) * a.group / kTileRows + a.segs;
  const long long grid = slots * a.geo.H * (a.geo.D / 4 / shared::kQuads);
  if (grid > 2147483647LL) return cudaErrorInvalidConfiguration;
  return launch_after(a.geo.D == 128 ? shared::join_kernel<128> : shared::join_kernel<64>, static_cast<unsigned>(grid),
                      kTileRows, 0, stream, a);
}

}  // namespace kv8
