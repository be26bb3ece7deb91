// Append to the 8-bit paged cache: rotate the new queries and keys to their
// positions, keep the newest tokens in the 16-bit window, and quantize each
// block of tokens that fills.
//
// One kernel.  A CTA takes one block of one sequence, for one or eight KV
// heads, keys and values or one of them (see launch_append): its tokens come
// from the window (stored before) and from the new rows, stay in registers
// while amax is reduced over the CTA, and leave as codes, so every byte is
// read and written once.  The CTA of the sequence's first block also writes
// the window tail, after it has read the window; no other CTA touches that
// window of that tensor, so nothing is ordered between CTAs.  Further CTAs
// rotate the queries: eight threads share a row, so that each table value that
// they load turns several heads.
//
// Bound: HBM for prompts (2 bytes read and 1 written per key or value element,
// 4 per query element): 16 sequences x 4096 tokens x 32 + 2 x 8 heads x 128
// take 467 us, 5.8 TB/s.  A single token per sequence is a launch and four
// dependent loads: 2.6 us.
#include <cuda_fp8.h>

#include "kv8_internal.cuh"

namespace kv8 {
namespace {

struct AppendArgs {
  Geo geo;
  Rows k, v, q, q_out;
  int Hq;
  const int *row_start;
  int rows, max_new;
  const float *rope;
  int rot, interleaved;
  int kv_tasks;     // CTAs that store keys and values
  int slots;        // block slots per group of heads (0: one per sequence)
  int heads;        // KV heads per CTA, one after the other
  int head_groups;  // groups of heads
  int split;        // 1: keys and values by CTAs of their own
  int lanes;        // threads that share a query row's chunk pair: 1 << lanes
};

// The two 8-channel chunks of chunk pair `pi` (of D / 16): the halves that
// turn together while pi < rot / 16, neighbours behind them.
__device__ __forceinline__ int2 chunk_pair(int pi, int rot) {
  const int rp = rot >> 4;
  if (pi < rp) return make_int2(pi, pi + rp);
  const int a = (rot >> 3) + 2 * (pi - rp);
  return make_int2(a, a + 1);
}

template <bool BF16>
__device__ __forceinline__ void turn(uint32_t &wa, uint32_t &wb, float c0, float c1, float s0, float s1) {
  const float2 a = unpack2<BF16>(wa), b = unpack2<BF16>(wb);
  wa = pack2<BF16>(__fsub_rn(__fmul_rn(a.x, c0), __fmul_rn(b.x, s0)),
                   __fsub_rn(__fmul_rn(a.y, c1), __fmul_rn(b.y, s1)));
  wb = pack2<BF16>(__fadd_rn(__fmul_rn(b.x, c0), __fmul_rn(a.x, s0)),
                   __fadd_rn(__fmul_rn(b.y, c1), __fmul_rn(a.y, s1)));
}

// One word holds a whole (even, odd) pair.
template <bool BF16>
__device__ __forceinline__ uint32_t turn_adjacent(uint32_t w, float c, float s) {
  const float2 x = unpack2<BF16>(w);
  return pack2<BF16>(__fsub_rn(__fmul_rn(x.x, c), __fmul_rn(x.y, s)),
                     __fadd_rn(__fmul_rn(x.y, c), __fmul_rn(x.x, s)));
}

// The 16 table values that turn chunk pair `pi` at position `pos`: cosines and
// sines of its angles (interleaved: chunk a's four, then chunk b's).
struct Turn {
  float4 c0, c1, s0, s1;
};
__device__ __forceinline__ Turn load_turn(int pi, int pos, const AppendArgs &a) {
  const int2 ch = chunk_pair(pi, a.rot);
  const float *first = a.rope + static_cast<size_t>(pos) * a.rot + (a.interleaved ? 4 * ch.x : 8 * pi);
  const int second = a.interleaved ? 4 * (ch.y - ch.x) : 4, half = a.rot >> 1;
  Turn t;
  t.c0 = __ldg(reinterpret_cast<const float4 *>(first));
  t.c1 = __ldg(reinterpret_cast<const float4 *>(first + second));
  t.s0 = __ldg(reinterpret_cast<const float4 *>(first + half));
  t.s1 = __ldg(reinterpret_cast<const float4 *>(first + half + second));
  return t;
}

// Rotates a chunk pair of one head.  Each product and sum is rounded on its
// own, so the result is a function of the table alone.
template <bool BF16>
__device__ __forceinline__ void rotate(uint4 &ca, uint4 &cb, const Turn &t, bool interleaved) {
  if (!interleaved) {
    turn<BF16>(ca.x, cb.x, t.c0.x, t.c0.y, t.s0.x, t.s0.y);
    turn<BF16>(ca.y, cb.y, t.c0.z, t.c0.w, t.s0.z, t.s0.w);
    turn<BF16>(ca.z, cb.z, t.c1.x, t.c1.y, t.s1.x, t.s1.y);
    turn<BF16>(ca.w, cb.w, t.c1.z, t.c1.w, t.s1.z, t.s1.w);
  } else {
    ca.x = turn_adjacent<BF16>(ca.x, t.c0.x, t.s0.x);
    ca.y = turn_adjacent<BF16>(ca.y, t.c0.y, t.s0.y);
    ca.z = turn_adjacent<BF16>(ca.z, t.c0.z, t.s0.z);
    ca.w = turn_adjacent<BF16>(ca.w, t.c0.w, t.s0.w);
    cb.x = turn_adjacent<BF16>(cb.x, t.c1.x, t.s1.x);
    cb.y = turn_adjacent<BF16>(cb.y, t.c1.y, t.s1.y);
    cb.z = turn_adjacent<BF16>(cb.z, t.c1.z, t.s1.z);
    cb.w = turn_adjacent<BF16>(cb.w, t.c1.w, t.s1.w);
  }
}

__device__ __forceinline__ uint4 load16(const uint16_t *p) { return *reinterpret_cast<const uint4 *>(p); }
__device__ __forceinline__ void store16(uint16_t *p, uint4 v) { *reinterpret_cast<uint4 *>(p) = v; }

// Largest magnitude bits of the eight 16-bit floats, in both halves' lanes:
// magnitudes order like unsigned integers, infinities and NaNs on top.
__device__ __forceinline__ uint32_t mag_max(uint32_t m, const uint4 &v) {
  m = __vmaxu2(m, v.x & 0x7fff7fffu);
  m = __vmaxu2(m, v.y & 0x7fff7fffu);
  m = __vmaxu2(m, v.z & 0x7fff7fffu);
  return __vmaxu2(m, v.w & 0x7fff7fffu);
}

// scale and the factor that takes an element to code units, from the block's
// largest magnitude.
template <int FMT>
__device__ __forceinline__ float2 scale_and_factor(float amax) {
  amax = fmaxf(amax, exp2_int(-100));
  if (FMT == KV8_INT8) return make_float2(__fdiv_rn(amax, 127.f), __fdiv_rn(127.f, amax));
  // the smallest power of two with amax <= 448 * 2^k = 1.75 * 2^(k + 8)
  const int bits = __float_as_int(amax);
  const int k = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
  return make_float2(exp2_int(k), exp2_int(-k));
}

// Four elements (two words) to four code bytes.  int8: adding 1.5 * 2^23 in
// one fused operation rounds the exact product half-even to a whole number,
// whose low byte is the code.
template <int FMT, bool BF16>
__device__ __forceinline__ uint32_t code4(uint32_t w0, uint32_t w1, float f) {
  const float2 a = unpack2<BF16>(w0), b = unpack2<BF16>(w1);
  if (FMT == KV8_INT8) {
    const float magic = 12582912.f;
    const uint32_t x0 = __float_as_uint(__fmaf_rn(a.x, f, magic)), x1 = __float_as_uint(__fmaf_rn(a.y, f, magic));
    const uint32_t x2 = __float_as_uint(__fmaf_rn(b.x, f, magic)), x3 = __float_as_uint(__fmaf_rn(b.y, f, magic));
    return __byte_perm(__byte_perm(x0, x1, 0x0040), __byte_perm(x2, x3, 0x0040), 0x5410);
  }
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a.x * f, a.y * f), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(b.x * f, b.y * f), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

template <int FMT, bool BF16>
__device__ __forceinline__ uint2 code8(const uint4 &v, float f, bool bad) {
  if (bad) return make_uint2(0u, 0u);
  return make_uint2(code4<FMT, BF16>(v.x, v.y, f), code4<FMT, BF16>(v.z, v.w, f));
}

// Queries: a thread turns one chunk pair of every (1 << lanes)-th head of a row,
// two heads at a time, with one set of table values.
template <int D, bool BF16, int T>
__device__ __forceinline__ void rotate_queries(const AppendArgs &a, int cta) {
  constexpr int PAIRS = D / 16;
  const int lanes = 1 << a.lanes, at = threadIdx.x / PAIRS;
  const int pi = threadIdx.x % PAIRS, lane = at & (lanes - 1);
  const int row = cta * ((T / PAIRS) >> a.lanes) + (at >> a.lanes);
  if (row >= a.rows || lane >= a.Hq) return;
  int s = row;
  if (a.row_start) s = last_at_or_below(a.geo.S, row, [&](int j) { return a.row_start[j]; });
  if (s >= a.geo.S) return;
  const Seq sq = load_seq(a.geo, a.row_start, a.rows, a.max_new, s);
  if (!sq.ok || row < sq.row0 || row >= sq.row0 + sq.n || sq.L < sq.n || sq.L > a.geo.capacity) return;
  if (!KVQ_IN_BOUNDS(a.geo.status, sq.L - sq.n + row - sq.row0, a.geo.capacity)) return;
  const bool turns = pi < (a.rot >> 4);
  Turn t;
  if (turns) t = load_turn(pi, sq.L - sq.n + row - sq.row0, a);
  const int2 ch = chunk_pair(pi, a.rot);
  const uint16_t *src = a.q.p + row * a.q.row + lane * a.q.head;
  uint16_t *dst = a.q_out.p + row * a.q_out.row + lane * a.q_out.head;
  const long long in = a.q.head << a.lanes, out = a.q_out.head << a.lanes;
#pragma unroll 1
  for (int h = lane; h < a.Hq; h += 2 * lanes, src += 2 * in, dst += 2 * out) {
    const bool two = h + lanes < a.Hq;
    uint4 x = load16(src + 8 * ch.x), y = load16(src + 8 * ch.y), z, w;
    if (two) {
      z = load16(src + in + 8 * ch.x);
      w = load16(src + in + 8 * ch.y);
    }
    if (turns) rotate<BF16>(x, y, t, a.interleaved);
    store16(dst + 8 * ch.x, x);
    store16(dst + 8 * ch.y, y);
    if (two) {
      if (turns) rotate<BF16>(z, w, t, a.interleaved);
      store16(dst + out + 8 * ch.x, z);
      store16(dst + out + 8 * ch.y, w);
    }
  }
}

// T threads, and NI chunk pairs of a block's keys (or values) per thread.
template <int D, int FMT, bool BF16, int T, int NI>
__global__ void __launch_bounds__(T, NI == 4 ? 3 : 1024 / T) append_kernel(const AppendArgs a) {
  constexpr int PAIRS = D / 16;
  if (static_cast<int>(blockIdx.x) >= a.kv_tasks) {
    if (a.slots && blockIdx.x == gridDim.x - 1) {
      // a sequence whose row range is invalid may own no slot
      for (int j = threadIdx.x; j < a.geo.S; j += T)
        if (!load_seq(a.geo, a.row_start, a.rows, a.max_new, j).ok) set_status(a.geo.status, KVQ_STATUS_BAD_LEN);
      return;
    }
    rotate_queries<D, BF16, T>(a, blockIdx.x - a.kv_tasks);
    return;
  }
  const Geo &geo = a.geo;
  const int B = geo.B, tid = threadIdx.x;
  int task = blockIdx.x, which = 0;  // 0: keys, 1: values
  if (a.split) {
    which = task & 1;
    task >>= 1;
  }
  const int h0 = task % a.head_groups * a.heads, h1 = min(h0 + a.heads, geo.H);
  int s = task / a.head_groups, t = 0;
  if (a.slots) {
    // slot -> (sequence, block): sequence s owns the slots from
    // row_start[s] / B + s on, at least as many as blocks it can complete
    const int slot = s;
    s = last_at_or_below(geo.S, slot, [&](int j) { return max(a.row_start[j], 0) / B + j; });
    t = slot - (max(a.row_start[s], 0) / B + s);
  }
  const Seq sq = load_seq(geo, a.row_start, a.rows, a.max_new, s);
  if (!sq.ok || sq.n > sq.L) {
    if (t == 0 && h0 == 0 && tid == 0) set_status(geo.status, KVQ_STATUS_BAD_LEN);
    return;
  }
  if (sq.L > geo.capacity) {
    if (t == 0 && h0 == 0 && tid == 0) set_status(geo.status, KVQ_STATUS_CAPACITY);
    return;
  }
  if (sq.n == 0) return;
  const int L = sq.L, old = L - sq.n, first = old / B, done = L / B - first;
  if (t < 0 || t >= max(done, 1)) return;
  const int p0 = (first + t) * B;  // position of the block's slot 0
  if (t < done && !KVQ_IN_BOUNDS(geo.status, first + t, geo.max_blocks)) return;
  const int blk = t < done ? geo.table[static_cast<size_t>(s) * geo.max_blocks + first + t] : -1;
  const int from = max(old, L / B * B);  // first new token that stays in the window
  const int items = B * PAIRS;
  const int2 ch = chunk_pair(tid % PAIRS, a.rot);
  const int apart = 8 * (ch.y - ch.x);
  __shared__ uint32_t red[2][T / 32];
  int phase = 0;

#pragma unroll 1
  for (;; ++which) {
    const Rows &rows = which ? a.v : a.k;
    const bool turns = !which && tid % PAIRS < (a.rot >> 4);
    uint16_t *const win = (which ? geo.v_win : geo.k_win) + static_cast<size_t>(s) * geo.H * B * D + 8 * ch.x;
    const uint16_t *const fresh = rows.p + (static_cast<long long>(sq.row0) - old) * rows.row + 8 * ch.x;
#pragma unroll 1
    for (int h = h0; h < h1; ++h, phase ^= 1) {
      if (t < done) {
        uint4 x[NI], y[NI];
        uint32_t m = 0;
        // a token's chunk pair from its window slot or new row
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int it = tid + i * T, slot = it / PAIRS, p = p0 + slot;
          if (it < items && (p < old || KVQ_IN_BOUNDS(geo.status, sq.row0 + p - old, a.rows))) {
            const uint16_t *src = p < old ? win + (static_cast<size_t>(h) * B + slot) * D
                                          : fresh + p * rows.row + h * rows.head;
            x[i] = load16(src);
            y[i] = load16(src + apart);
          }
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int it = tid + i * T, p = p0 + it / PAIRS;
          if (it < items) {
            if (turns && p >= old && KVQ_IN_BOUNDS(geo.status, p, geo.capacity))
              rotate<BF16>(x[i], y[i], load_turn(tid % PAIRS, p, a), a.interleaved);
            m = mag_max(mag_max(m, x[i]), y[i]);
          }
        }
        m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
        if ((tid & 31) == 0) red[phase][tid >> 5] = m;  // the other half may still be read
        __syncthreads();  // also: every window slot of the block has been read
#pragma unroll
        for (int w = 0; w < T / 32; ++w) m = max(m, red[phase][w]);
        if (blk < 0 || blk >= geo.num_blocks) {
          if (tid == 0) set_status(geo.status, KVQ_STATUS_BAD_BLOCK);
        } else {
          const bool bad = m >= nonfinite_bits<BF16>();
          const float2 sc = scale_and_factor<FMT>(bad ? 0.f : unpack2<BF16>(m).x);
          const size_t bh = (static_cast<size_t>(blk) * geo.H + h) * 2 + which;
          uint8_t *codes = geo.codes + bh * B * D + 8 * ch.x;
          if (tid == 0) geo.scales[bh] = bad ? __int_as_float(0x7fc00000) : sc.x;
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const int it = tid + i * T;
            if (it < items) {
              uint8_t *dst = codes + it / PAIRS * D;
              *reinterpret_cast<uint2 *>(dst) = code8<FMT, BF16>(x[i], sc.y, bad);
              *reinterpret_cast<uint2 *>(dst + apart) = code8<FMT, BF16>(y[i], sc.y, bad);
            }
          }
        }
      }
      if (t > 0) continue;

      // the tokens that stay in the window: all new ones when nothing filled,
      // else those behind the last complete block
      for (int it = tid; it < (L - from) * PAIRS; it += T) {
        const int p = from + it / PAIRS, slot = p & (B - 1);
        if (!KVQ_IN_BOUNDS(geo.status, sq.row0 + p - old, a.rows) || !KVQ_IN_BOUNDS(geo.status, p, geo.capacity)) continue;
        const uint16_t *src = fresh + p * rows.row + h * rows.head;
        uint4 x = load16(src), y = load16(src + apart);
        if (turns) rotate<BF16>(x, y, load_turn(tid % PAIRS, p, a), a.interleaved);
        uint16_t *dst = win + (static_cast<size_t>(h) * B + slot) * D;
        store16(dst, x);
        store16(dst + apart, y);
      }
    }
    if (a.split || which) break;
  }
}

template <int D, int FMT, bool BF16>
cudaError_t launch_ni(const AppendArgs &a, unsigned grid, cudaStream_t stream) {
  const int items = a.geo.B * D / 16;
  if (items == 128)
    append_kernel<D, FMT, BF16, 128, 1><<<grid, 128, 0, stream>>>(a);
  else if (items == 256)
    append_kernel<D, FMT, BF16, 256, 1><<<grid, 256, 0, stream>>>(a);
  else if (items == 512)
    append_kernel<D, FMT, BF16, 256, 2><<<grid, 256, 0, stream>>>(a);
  else
    append_kernel<D, FMT, BF16, 256, 4><<<grid, 256, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const AppendArgs &a, unsigned grid, cudaStream_t stream) {
  if (a.geo.fmt == KV8_INT8)
    return a.geo.bf16 ? launch_ni<D, KV8_INT8, true>(a, grid, stream) : launch_ni<D, KV8_INT8, false>(a, grid, stream);
  return a.geo.bf16 ? launch_ni<D, KV8_E4M3, true>(a, grid, stream) : launch_ni<D, KV8_E4M3, false>(a, grid, stream);
}

}  // namespace

cudaError_t launch_append(const Geo &geo, const Rows &k, const Rows &v, const Rows &q, const Rows &q_out, int Hq,
                          const int *row_start, int rows, int max_new, const float *rope, int rot_dim,
                          int interleaved, cudaStream_t stream, uint64_t *launches) {
  AppendArgs a;
  a.geo = geo;
  a.k = k;
  a.v = v;
  a.q = q;
  a.q_out = q_out;
  a.Hq = Hq;
  a.row_start = row_start;
  a.rows = rows;
  a.max_new = max_new;
  a.rope = rope;
  a.rot = rot_dim;
  a.interleaved = interleaved;
  // up to B new tokens complete at most one block of a sequence, and without
  // row_start, whatever max_new allows, each brings one
  a.slots = row_start && max_new > geo.B ? rows / geo.B + geo.S : 0;
  // With many blocks keys and values have CTAs of their own (prompts 467
  // against 543 us), and a CTA takes eight heads, so that the table's values, as
  // many bytes per token as a head's keys and values together, come from the
  // first-level cache for seven of them.  With few, a head's keys and values
  // share a CTA: less to start (ragged chunks of 356 blocks 18.5 against 20.0
  // us, a decode step of 64 x 8 heads 4.2 against 5.6).
  // Around the borders (int8 bf16, D 128, block 64, 8 x 4 heads; one head per CTA
  // with keys and values together, one apart, eight): blocks x heads of 544:
  // 17.0, 18.2, 31.7 us; 1056: 33.9, 35.7, 43.9; 2080: 64.6, 68.0, 60.1; 4160:
  // 127, 136, 119; 8320: not timed, 274, 234.  One token each for 256 sequences,
  // 2048: 10.3, 13.1, 6.1.  So eight heads pay from 2048 on, where keys and values
  // apart by themselves do not: between the borders this rule is 12% off, in that
  // decode step twofold.
  const long long blocks = a.slots ? a.slots : geo.S;
  a.split = blocks * geo.H >= 2048;
  a.heads = blocks * geo.H >= 8192 && rot_dim ? 8 : 1;
  a.head_groups = (geo.H + a.heads - 1) / a.heads;
  const long long tasks = blocks * a.head_groups * (a.split ? 2 : 1);
  // eight threads share a query row's chunk pair, fewer where there are fewer
  // heads (four: that decode step takes 5.0 us; sixteen: prompts 483)
  a.lanes = Hq >= 8 ? 3 : Hq >= 4 ? 2 : Hq >= 2 ? 1 : 0;
  const int per = (min(geo.B * geo.D / 16, 256) / (geo.D / 16)) >> a.lanes;  // query rows of a CTA, see launch_ni
  // and one CTA checks the row ranges where there are slots
  const long long grid = tasks + (Hq ? (static_cast<long long>(rows) + per - 1) / per : 0) + (a.slots ? 1 : 0);
  if (grid > 2147483647LL) return cudaErrorInvalidConfiguration;
  a.kv_tasks = static_cast<int>(tasks);
  ++*launches;
  return geo.D == 128 ? launch_d<128>(a, static_cast<unsigned>(grid), stream)
                      : launch_d<64>(a, static_cast<unsigned>(grid), stream);
}

}  // namespace kv8
