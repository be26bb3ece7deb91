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

// Positions of each row on several axes, and the axis that each pair of channels
// turns by: two bits per pair.
struct Axes {
  const int *positions;  // [axes][stride]
  long long stride;
  int table_rows;
  uint32_t map[4];
};

cudaError_t launch_append(const Geo &geo, const Rows &k, const Rows &v, const Rows &q, const Rows &q_out, int Hq,
                          const int *row_start, int rows, int max_new, const float *rope, int rot_dim,
                          int interleaved, cudaStream_t stream, uint64_t *launches);
cudaError_t launch_append_axes(const Geo &geo, const Rows &k, const Rows &v, const Rows &q, const Rows &q_out, int Hq,
                               const int *row_start, int rows, int max_new, const float *rope, int rot_dim,
                               int interleaved, const Axes &axes, cudaStream_t stream, uint64_t *launches);

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
// kernel comes first, and a second set for the launches over shared blocks, at
// places that do not depend on the call: what a call of one shape leaves of its
// partial results is never another's counter.  Rows
// kernel: partial outputs [2 kMaxCtas][16][D] and their (max, sum).  Tile
// kernel, where a sequence can bring enough rows: the same for
// [2 kMaxTileCtas][256].
constexpr size_t kCounters = 3328;  // bytes of a set: kMaxCtas and kMaxTileCtas counters, to 256
struct AttnPlan {
  size_t off_cnt, off_tile_cnt, off_o, off_ml, off_tile_o, off_tile_ml, bytes;
  bool tiles;
};
AttnPlan plan_attn(int D, long long rows_per_head);

// Attention with shared blocks.  What lies behind them comes first: its kernels
// leave partial results (carry) for the rows whose group shares blocks.  The
// kernels over the shared blocks join them and write the outputs.  They need not
// wait for the others until then, so each has regions of its own.
struct SharedPlan {
  size_t off_prefix, off_segs, off_items, off_falls, off_ml, off_o, bytes;
  long long carry_blocks;
  bool own_tiles, prefix_tiles;
};
SharedPlan plan_shared(int D, int S, int H, int num_q_heads, long long rows, long long max_new,
                       long long max_group_rows);

// Threads of a CTA of the kernel that looks up the segments, its CTAs, and the
// words in which its warps say whether row_start or group_start falls.
constexpr int kSegThreads = 128;
inline int seg_ctas(int groups, int S) { return (groups + S + kSegThreads - 1) / kSegThreads; }
inline int fall_words(int groups, int S) { return seg_ctas(groups, S) * (kSegThreads / 32); }

// What one launch attends to, segment by segment.
enum {
  kWhole,   // sequences: their whole length
  kOwn,     // sequences: what lies behind the blocks shared with their group; leaves partial results
  kPrefix,  // groups of sequences: the blocks that they share, for the rows of all; joins the partial results
};

struct AttnArgs {
  Geo geo;
  int Hq, group;
  int part;    // kWhole, kPrefix or kOwn
  int fine;    // 1: the kernels whose segments are looked up before
  int causal;  // 1: a row sees up to its own position, 0: all of its segment
  int segs;    // segments: sequences or groups
  const int *group_start, *prefix_len;  // [groups + 1], [groups]; with kPrefix and kOwn
  int groups, max_group_rows;
  int4 *plan;        // two per segment: the groups', then the sequences'
  int4 *items;       // [kMaxTileCtas][2]: what the join kernel joins, by the first CTA of its parts
  int *falls;        // [fall_words]: whether row_start or group_start falls
  int fall_words;
  int first;         // the first launch behind the lookup of the segments
  // Partial results over what lies behind the shared blocks, of the rows of each
  // KV head, (tensor row, query head of the KV head):
  long long carry_blocks;  // per KV head: the rows, in blocks of 32
  float4 *carry_o;         // [H][carry_blocks] of [32][D / 4], or of [D / 4][32]: unnormalized outputs
  float2 *carry_ml;        // [H][carry_blocks][32]: (max, sum) in log2 units; sum -1: not to be written
  int carry_wide;          // 1: rows side by side
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
  int group_rows_max; // and a group
  long long wait_limit;  // SM cycles that a wait of the tile kernel may last before it gives up
  int wait_test;         // test aid: a wait of the tile kernel that nothing completes
};

// A segment: its tokens and rows.  A sequence whose row range is invalid has
// no rows and is not ok, as are all of a group whose shared blocks or rows are invalid.
struct Seg {
  int L, n, row0;  // tokens behind `base`; rows, and the first one
  int base;        // blocks in front, which another launch has seen
  int entry;       // the sequence whose blocks these are
  bool ok;
};

// A group's first sequence, its shared blocks and its rows.  Not ok: bad bounds,
// more rows than announced, or a first sequence whose stored tokens end within them.
struct Group {
  int first, blocks, row0, n;
  bool ok;
};
__device__ __forceinline__ Group load_group(const AttnArgs &a, int g) {
  Group x;
  x.first = a.group_start[g];
  const int end = a.group_start[g + 1], prefix = a.prefix_len[g];
  x.blocks = x.row0 = x.n = 0;
  x.ok = x.first >= 0 && end >= x.first && end <= a.geo.S;
  if (!x.ok || end == x.first) return x;
  x.ok = prefix >= 0 && prefix <= a.max_len;
  if (!x.ok) return x;
  int r0 = x.first, r1 = end, own = r0 + 1;
  if (a.row_start) {
    r0 = a.row_start[r0];
    r1 = a.row_start[r1];
    own = a.row_start[own];
  }
  x.blocks = prefix / a.geo.B;
  x.ok = r0 >= 0 && r1 >= r0 && r1 <= a.rows && r1 - r0 <= a.max_group_rows && own >= r0 && own <= r1 &&
         (x.blocks == 0 || a.geo.seq_len[x.first] - static_cast<long long>(own - r0) >= x.blocks * a.geo.B);
  x.row0 = r0;
  x.n = x.ok ? r1 - r0 : 0;
  return x;
}

// The sequence's segment, behind the blocks that it shares with its group.
// `shut`: the group has shared blocks, but this sequence's rows have no part in them.
__device__ __forceinline__ Seg own_seg(const AttnArgs &a, int s, bool &shut) {
  const Seq q = load_seq(a.geo, a.row_start, a.rows, a.max_new, s);
  Seg x = {q.L, q.n, q.row0, 0, s, q.ok};
  const int g = last_at_or_below(a.groups, s, [&](int i) { return a.group_start[i]; });
  if (a.group_start[g] <= s && s < a.group_start[g + 1]) {
    const Group of = load_group(a, g);
    const bool bounded = q.L <= a.max_len;  // (else zeros)
    if (!of.ok || (q.n > 0 && bounded && of.blocks && (q.L <= 0 || q.L - q.n < of.blocks * a.geo.B))) {
      x.ok = false;
      x.n = 0;
    } else if (q.n > 0 && bounded) {
      x.base = of.blocks;
      x.L -= of.blocks * a.geo.B;
    }
    shut = of.ok && of.blocks && !x.base;
  }
  return x;
}
__device__ __forceinline__ Seg group_seg(const AttnArgs &a, int g) {
  const Group x = load_group(a, g);
  const int L = x.blocks * a.geo.B;
  return {L, L ? x.n : 0, x.row0, 0, x.ok ? x.first : 0, x.ok};
}

// FINE: kernels whose segments have been looked up by a kernel before, two int4
// each.  With shared blocks each is a chain of six loads, which every CTA would
// wait for, for every sequence; and what a CTA runs once comes from far, so that
// the code counts too (a branch for whole sequences beside this one: 2 to 4 us).
struct Plan {
  int full, units, tiles;  // for the rows kernel: units of complete blocks, all units, row tiles per KV head
};
__device__ __forceinline__ void store_plan(const AttnArgs &a, int i, const Seg &x, const Plan &w) {
  a.plan[2 * i] = make_int4(x.L, x.n, x.row0, x.base);
  a.plan[2 * i + 1] = make_int4(x.ok ? x.entry : -1, w.full, w.units, w.tiles);
}
__device__ __forceinline__ Seg load_plan(const AttnArgs &a, int s, Plan &w) {
  if (!KVQ_IN_BOUNDS(a.geo.status, s, a.segs)) s = 0;
  const int4 *p = a.plan + 2 * (static_cast<size_t>(a.part == kOwn ? a.groups : 0) + s);
  const int4 x = a.first ? p[0] : __ldcg(p), y = a.first ? p[1] : __ldcg(p + 1);
  w = {y.y, y.z, y.w};
  return {x.x, x.y, x.z, x.w, max(y.x, 0), y.x >= 0};
}
template <bool FINE>
__device__ __forceinline__ Seg load_seg(const AttnArgs &a, int s) {
  if (FINE) {
    Plan w;
    return load_plan(a, s, w);
  }
  const Seq q = load_seq(a.geo, a.row_start, a.rows, a.max_new, s);
  return {q.L, q.n, q.row0, 0, s, q.ok};
}

// The kernels of one call of cross attention or with shared blocks start while the
// ones before still run.  Each lets the next one start once the segments are there: the first waits
// for them, and the others start behind it.  Each waits for the one before it
// at the latest before it ends, so that the end of one is the end of all before.
//
// A wait makes the writes of the grid before visible, and the first launch waits
// for the lookup.  The later ones read the lookup's words without a wait of their
// own.  They rely on two things: all CTAs of the first launch have waited, that is,
// the lookup's writes have been performed, before any of theirs starts; and their
// loads go past the first-level cache (load_plan), which may hold lines from before.
// (In the first launch that would cost beams 0.9 us and a batch's cross attention
// 1.4; a fence at the start of the later ones costs calls with shared blocks 0.7.)
__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <bool FINE>
__device__ __forceinline__ void start(const AttnArgs &a) {
  if (FINE) {
    if (a.first) wait_before();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
}
template <bool FINE>
__device__ __forceinline__ void finish() {
  if (FINE) wait_before();
}
template <typename... A>
cudaError_t launch_after(void (*kernel)(A...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream,
                         A... args) {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t config = {};
  config.gridDim = dim3(grid);
  config.blockDim = dim3(threads);
  config.dynamicSmemBytes = smem;
  config.stream = stream;
  config.attrs = &attr;
  config.numAttrs = 1;
  return cudaLaunchKernelEx(&config, kernel, args...);
}

// The last position of the segment that rows of its new token `tok` see.
template <typename T>
__device__ __forceinline__ int last_seen(const AttnArgs &a, const T &q, int tok) {
  return a.causal ? q.L - q.n + tok : q.L - 1;
}

// A row of KV head h among the partial results: (max, sum), and channels 4 c
// to 4 c + 3.  A thread of the tile kernel has a row, and a warp 32 neighbours:
// with rows side by side its accesses are 512 bytes each (six questions of 100 to
// 500 tokens behind 8192 shared ones: 312 us, 315 the other way).  The rows kernel
// has a row's channels side by side, and its order is taken where no sequence's rows
// are many (12 groups of drafts: 54 us, 55.8 the other way).
struct CarryRow {
  float2 *ml;
  float4 *o;
  int step;
  __device__ __forceinline__ float4 &at(int c) const { return o[step * c]; }
};
template <int D>
__device__ __forceinline__ CarryRow carry_row(const AttnArgs &a, int h, int row0, int row) {
  const long long r = static_cast<long long>(row0) * a.group + row;
  size_t at = static_cast<size_t>(h * a.carry_blocks) * 32 + r;
  if (!KVQ_IN_BOUNDS(a.geo.status, r, a.carry_blocks * 32) || !KVQ_IN_BOUNDS(a.geo.status, h, a.geo.H)) at = 0;
  const int lane = static_cast<int>(r & 31);
  return {a.carry_ml + at, a.carry_o + (a.carry_wide ? (at - lane) * (D / 4) + lane : at * (D / 4)),
          a.carry_wide ? 32 : 1};
}

// The factors that join two partial results (max, sum), and what their weighted
// sum is divided by: out = o x + other y over z.
struct Join {
  float x, y, sum;
};
__device__ __forceinline__ Join join(float2 own, float2 other) {
  const float top = fmaxf(own.x, other.x), base = top == __int_as_float(0xff800000) ? 0.f : top;
  const float h = kvq::fast_exp2(0.5f * (own.x - base)), k = kvq::fast_exp2(0.5f * (other.x - base));
  return {h * h, k * k, fmaf(own.y * h, h, other.y * k * k)};
}

// Debug builds: the tensors' row and head of a KV head's row are in range.
__device__ __forceinline__ bool row_in_bounds(const AttnArgs &a, int row0, int h, int row) {
  return KVQ_IN_BOUNDS(a.geo.status, static_cast<long long>(row0) + row / a.group, a.rows) &&
         KVQ_IN_BOUNDS(a.geo.status, static_cast<long long>(h) * a.group + row % a.group, a.Hq);
}

cudaError_t launch_attn(const AttnArgs &a, bool tiles, cudaStream_t stream, uint64_t *launches);
// looks up the segments of a call with shared blocks
cudaError_t launch_segments(const AttnArgs &a, cudaStream_t stream);
// joins the parts of the tile kernel's items over shared blocks
cudaError_t launch_join(const AttnArgs &a, cudaStream_t stream);
// the kernels for one head dimension (one translation unit each)
cudaError_t launch_rows_128(const AttnArgs &a, cudaStream_t stream);
cudaError_t launch_rows_64(const AttnArgs &a, cudaStream_t stream);
cudaError_t launch_tiles_128(const AttnArgs &a, cudaStream_t stream);
cudaError_t launch_tiles_64(const AttnArgs &a, cudaStream_t stream);
cudaError_t launch_rows_128_shared(const AttnArgs &a, cudaStream_t stream);
cudaError_t launch_rows_64_shared(const AttnArgs &a, cudaStream_t stream);
cudaError_t launch_tiles_128_shared(const AttnArgs &a, cudaStream_t stream);
cudaError_t launch_tiles_64_shared(const AttnArgs &a, cudaStream_t stream);

}  // namespace kv8
