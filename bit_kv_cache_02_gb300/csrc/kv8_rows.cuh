// Attention over the 8-bit paged cache for few rows per sequence: single
// tokens, drafts (a "row" is one query head of one new token; the rows of a
// KV head share its keys).
//
// Mathematics: for each row an online softmax over 32-token units (16 in the
// 16-bit window), in log2 units: z = q.k scale_k softmax_scale log2(e) +
// log2(scale_v), m the running maximum of z, w = 2^(z - m + 15), o the sum of
// w v_code, l the sum of w / scale_v, out = o / l.  With scale_v in the
// exponent, o accumulates codes of blocks with different scales in the mma's
// own registers.  A block of zeros, which has no scale to speak of, enters m
// with kZeroLog for it and its weights, formed without, go into l alone.
//
// Both products run on mma.sync m16n8k16 with fp32 accumulators.  Up to eight
// rows are N, tokens (then channels) M: the codes become A fragments and the
// weights B fragments by 8 x 8 transposes.  Up to sixteen rows are M: the
// accumulators of the scores are the A operand of the second product as they
// lie in registers.  int8 keys enter as (code + 128) 2^-24, fp16 subnormals
// that are two byte permutes away from the code; the 128 sum(q) that this adds
// to a score is taken off in its fused multiply-add.  Values enter as they
// are: their sums nearly cancel over a long context, and 128 sum(w) would drown
// what is left.
//
// Roundings to 16 bits: w to fp16 (the factor 2^15 keeps weights down to 2^-29
// of the largest at full precision).  One part is enough here: a weight's 2^-11
// is at most what an fp16 output's own rounding adds, and less in the mean (the
// error against 64 bits grows from 2.1e-4 to 2.4e-4 in fp16, 2.6e-4 over long
// contexts, and from 1.7e-3 by 0.1e-3 at most in bf16), where the 8-bit tokens
// are off by 9e-3; a second part would double the products with the values.
// (The 2/4-bit kernels keep two: there a token's scale multiplies its weight.)
// And bf16 queries, which a power of two
// per row brings into fp16's range: a rounding only of elements 2^-29 below
// the row's largest.  Window tokens in bf16 are multiplied as they are (mma in
// bf16), so that no token's size touches another's; their weights go in as a
// bf16 part and the bf16 remainder, 2^-17 of themselves off.  Their weights have
// no scale in the exponent, but in m they count like a block's of their size, or
// the weights of blocks with small values would leave fp16's range beside them.
//
// The units of all (sequence, KV head, 16-row tile) triples form one line,
// cut into one equal range per CTA whatever the sequences' lengths.  The four
// warps of a CTA take the units of a triple in turn, each with its own ring of
// shared-memory slots filled by asynchronous copies, and merge their softmax
// states through shared memory when the triple (or the CTA's part of it)
// ends.  A triple cut by CTA borders is merged by the last CTA that finishes.
//
// Bound: HBM for one row per query head (2 D bytes per token and KV head).
// Measured, D 128, reading 4097 tokens x 16 sequences x 32 heads: 88 us, 6.1
// TB/s; 64 sequences x 8 heads of four rows, 1024 to 8192 tokens, e4m3: 111 us,
// 6.0 TB/s; one sequence of 2^20 tokens x 8 heads: 304 us, 7.1 TB/s.  With 12
// to 32 rows (16 sequences, 2000 to 6000 tokens, 8 heads, 3 to 8 drafts x 4)
// the keys are read once or twice and the chain of a unit's instructions
// bounds it, at two warps per scheduler: 43.5 us; three warps, at 168 registers,
// were no faster.
//
// 16-byte chunks are XOR swizzled by the token so that neither operand's
// shared-memory reads conflict: a lane's 16-byte read covers 16 channels of one
// token, which is four k-steps of the first product, or one channel of each of
// 16 n-tiles of the second; the channel order within the products is free as
// long as both operands agree on it.
#pragma once

#include <atomic>
#include <type_traits>

#include "kv8_internal.cuh"

namespace kv8 {
namespace rows {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 4;
constexpr int kUnit = 32;     // tokens of a unit of quantized blocks
constexpr int kWinUnit = 16;  // tokens of a unit of the window
// Ring slots of a warp for D 128 (twice as many of half the size for D 64).
// Three or four cost resident CTAs and were slower.
constexpr int kSlots = 2;

template <int D, int HALVES>
struct Smem {
  static constexpr int SLOTS = D == 128 ? kSlots : 2 * kSlots;
  static constexpr int HALF = kUnit * D;   // bytes of a unit's keys (and of its values)
  static constexpr int SLOT = 2 * HALF;    // a window unit has the same size
  static constexpr int NT = D / 8;         // n-tiles of the output
  static constexpr int META = kWarps * SLOTS * SLOT;                 // scales of each slot: float2
  static constexpr int ML = META + kWarps * SLOTS * 8;               // [kWarps][16] float2
  // the merge buffer; before the merge, sixteen rows' queries
  static constexpr int XCH = (ML + kWarps * kRowTile * 8 + 15) / 16 * 16;
  static_assert(HALVES == 1 || kWarps * 3 * (NT / 4) * 32 * 4 >= D / 16 * 512, "queries");
  static constexpr int FLAG = XCH + kWarps * 3 * (NT / 4) * 32 * 4;
  static constexpr int BYTES = FLAG + 16;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, or zeros when `full` is false
__device__ __forceinline__ void cp16z(uint32_t dst, const void *src, bool full) {
  const int n = full ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// d = a * b + c with c = 0; a B fragment is one 64-bit register pair
__device__ __forceinline__ void mma_zero(float (&d)[4], const uint32_t (&a)[4], uint64_t b) {
  asm volatile(
      "{\n\t.reg .b32 x, y;\n\tmov.b64 {x, y}, %8;\n\t"
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {x,y}, {%9,%9,%9,%9};\n\t}"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "l"(b), "f"(0.f));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint64_t b) {
  asm volatile(
      "{\n\t.reg .b32 x, y;\n\tmov.b64 {x, y}, %8;\n\t"
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {x,y}, {%0,%1,%2,%3};\n\t}"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "l"(b));
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  kvq::mma16816(d, a[0], a[1], a[2], a[3], b0, b1);
}

// Bytes 2 h and 2 h + 1 of two code words as fp16 pairs: the codes' values or,
// for int8 keys, (code + 128) 2^-24.  int8 words have their sign bits flipped.
template <int FMT, bool KEYS>
__device__ __forceinline__ uint64_t widen(uint32_t w0, int h0, uint32_t w1, int h1) {
  uint64_t r;
  if (FMT == KV8_INT8 && KEYS) {
    asm("{\n\t.reg .b32 x, y;\n\tprmt.b32 x, %1, 0, %3;\n\tprmt.b32 y, %2, 0, %4;\n\tmov.b64 %0, {x, y};\n\t}"
        : "=l"(r)
        : "r"(w0), "r"(w1), "r"(h0 ? 0x4342 : 0x4140), "r"(h1 ? 0x4342 : 0x4140));
  } else if (FMT == KV8_INT8) {
    // 0x64 above a byte makes 1024 + 128 + code
    asm("{\n\t.reg .b32 x, y;\n\tprmt.b32 x, %1, %5, %3;\n\tprmt.b32 y, %2, %5, %4;\n\t"
        "sub.rn.f16x2 x, x, %6;\n\tsub.rn.f16x2 y, y, %6;\n\tmov.b64 %0, {x, y};\n\t}"
        : "=l"(r)
        : "r"(w0), "r"(w1), "r"(h0 ? 0x4342 : 0x4140), "r"(h1 ? 0x4342 : 0x4140), "r"(0x64646464u), "r"(0x64806480u));
  } else {
    const uint16_t c0 = static_cast<uint16_t>(h0 ? w0 >> 16 : w0), c1 = static_cast<uint16_t>(h1 ? w1 >> 16 : w1);
    asm("{\n\t.reg .b32 x, y;\n\tcvt.rn.f16x2.e4m3x2 x, %1;\n\tcvt.rn.f16x2.e4m3x2 y, %2;\n\t"
        "mov.b64 %0, {x, y};\n\t}"
        : "=l"(r)
        : "h"(c0), "h"(c1));
  }
  return r;
}
// d = a * b + d with A from code words: fragment registers 0..3 are bytes 2 h
// and 2 h + 1 of w0..w3.
template <int FMT, bool KEYS>
__device__ __forceinline__ void mma_a(float (&d)[4], uint32_t w0, int h0, uint32_t w1, int h1, uint32_t w2, int h2,
                                      uint32_t w3, int h3, const uint32_t (&b)[2]) {
  const uint64_t x = widen<FMT, KEYS>(w0, h0, w1, h1), y = widen<FMT, KEYS>(w2, h2, w3, h3);
  asm volatile(
      "{\n\t.reg .b32 a, b, c, d;\n\tmov.b64 {a, b}, %4;\n\tmov.b64 {c, d}, %5;\n\t"
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {a,b,c,d}, {%6,%7}, {%0,%1,%2,%3};\n\t}"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "l"(x), "l"(y), "r"(b[0]), "r"(b[1]));
}

// The 8 x 8 matrix of 16-bit numbers held two to a lane, transposed.
__device__ __forceinline__ uint32_t transpose(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// int8 codes to offset binary
template <int FMT>
__device__ __forceinline__ uint32_t flip(uint32_t w) {
  return FMT == KV8_INT8 ? w ^ 0x80808080u : w;
}

// d = a * b + d in bf16
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Weights are formed as 2^15 w.
constexpr float kShift = 15.f, kUnshift = 1.f / 32768.f;

// A power-of-two pair (f, 1/f) that brings bf16 magnitudes up to `bits` to
// just below 2^15.  Magnitudes below 2^-107 count as that.
__device__ __forceinline__ float2 bf16_norm(uint32_t bits) {
  const int e = max(static_cast<int>(bits >> 7), 20);  // biased exponent of the largest, <= 254
  return make_float2(__int_as_float((268 - e) << 23), __int_as_float((e - 14) << 23));
}

// A word of two bf16, scaled, as a word of two fp16.
__device__ __forceinline__ uint32_t bf16_to_fp16(uint32_t w, float f) {
  const float2 x = unpack2<true>(w);
  return kvq::h2_as_u32(__floats2half2_rn(x.x * f, x.y * f));
}

// Largest finite magnitude of two 16-bit floats, folded into m.
__device__ __forceinline__ uint32_t finite_max(uint32_t m, uint32_t w, uint32_t limit) {
  const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
  m = max(m, lo < limit ? lo : 0u);
  return max(m, hi < limit ? hi : 0u);
}

// The larger of each half of two words over the eight lanes with the same q4,
// which hold all channels of a token between them.
__device__ __forceinline__ void all_channels(uint32_t &a, uint32_t &b) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    a = __vmaxu2(a, __shfl_xor_sync(kAll, a, o));
    b = __vmaxu2(b, __shfl_xor_sync(kAll, b, o));
  }
}

// What a bf16 window token whose largest value has these bits adds to its score
// in the maximum: log2 of the scale that a block of such values would have, but
// no more than 0, nor less than kZeroLog.
__device__ __forceinline__ float value_log(uint32_t bits) {
  return static_cast<float>(min(max(static_cast<int>(bits >> 7) - 133, static_cast<int>(kZeroLog)), 0));
}

// Work of one sequence: its units per (KV head, row tile) pair, and pairs.
struct Work {
  Seq q;
  int full;   // units of complete blocks
  int units;  // all units
  int tiles;  // row tiles per KV head
};

__device__ __forceinline__ Work seq_work(const AttnArgs &a, int s) {
  Work w;
  w.q = load_seq(a.geo, a.row_start, a.rows, a.max_new, s);
  const int L = w.q.L;
  const bool some = w.q.n > 0 && w.q.n * a.group <= a.rows_max && L > 0 && L <= a.max_len;
  const int nb = L / a.geo.B;
  w.full = some ? nb * (a.geo.B / kUnit) : 0;
  w.units = some ? w.full + (L - nb * a.geo.B + kWinUnit - 1) / kWinUnit : 0;
  w.tiles = some ? (w.q.n * a.group + kRowTile - 1) / kRowTile : 0;
  return w;
}
__device__ __forceinline__ long long line_of(const Work &w, int H) {
  return static_cast<long long>(w.units) * w.tiles * H;
}

// Walks a CTA's range of the line, one part of a (sequence, head, tile)
// triple at a time.
struct Walk {
  Work w;
  int s, h, tile;
  long long at, end;  // line position and end of the range
  int u0, u1;         // units of the current part
  long long start;    // line position of the triple's unit 0

  __device__ __forceinline__ void part() {
    u1 = static_cast<int>(min(static_cast<long long>(w.units), u0 + (end - at)));
    start = at - u0;
  }
  // the sequence that holds line position `pos`, whose own line starts at `base`
  __device__ __forceinline__ void enter(const AttnArgs &a, int seq, long long base, long long pos, long long end_) {
    s = seq;
    w = seq_work(a, s);
    at = pos;
    end = end_;
    const int pair = static_cast<int>(divide(pos - base, w.units));
    u0 = static_cast<int>((pos - base) - static_cast<long long>(pair) * w.units);
    h = pair / w.tiles;
    tile = pair - h * w.tiles;
    part();
  }
  // the next part; false at the end of the range
  __device__ __forceinline__ bool next(const AttnArgs &a) {
    at += u1 - u0;
    if (at >= end) return false;
    u0 = 0;
    if (++tile >= w.tiles) {
      tile = 0;
      if (++h >= a.geo.H) {
        h = 0;
        do {
          if (++s >= a.geo.S) return false;
          w = seq_work(a, s);
        } while (w.units == 0);
      }
    }
    part();
    return true;
  }
};

template <int D, int FMT, bool BF16, int HALVES>
__global__ void __launch_bounds__(kWarps * 32) rows_kernel(const AttnArgs a) {
  using SM = Smem<D, HALVES>;
  constexpr int NT = SM::NT;  // output n-tiles
  constexpr int KS = D / 16;  // k-steps of the scores
  extern __shared__ __align__(128) unsigned char smem[];
  const Geo &geo = a.geo;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
  const int B = geo.B, H = geo.H;
  const float ninf = __int_as_float(0xff800000);

  // The line's length.  On the way, a CTA writes the zero rows of its share of
  // the sequences with rows and nothing to see.
  long long total = 0, triples = 0;
  for (int s0 = 0; s0 < geo.S; s0 += 32) {
    Work w = {};
    bool blind = false;
    if (s0 + lane < geo.S) {
      w = seq_work(a, s0 + lane);
      blind = !w.q.ok || (w.q.n > 0 && (w.q.L <= 0 || w.q.L > a.max_len));
    }
    total += line_of(w, H);
    triples += static_cast<long long>(w.tiles) * H;
    for (unsigned m = __ballot_sync(kAll, blind); m; m &= m - 1) {
      const int s = s0 + __ffs(m) - 1;
      if (s % gridDim.x != blockIdx.x) continue;
      const Seq sq = load_seq(geo, a.row_start, a.rows, a.max_new, s);
      if (tid == 0 && (!sq.ok || sq.L != 0)) set_status(geo.status, sq.ok ? KVQ_STATUS_MAX_LEN : KVQ_STATUS_BAD_LEN);
      const int per_row = a.Hq * (D / 8);  // (a bad sequence has no rows)
      for (long long i = tid; i < static_cast<long long>(sq.n) * per_row; i += kWarps * 32) {
        const int row = static_cast<int>(i / per_row), c = static_cast<int>(i % per_row);
        *reinterpret_cast<uint4 *>(a.out.p + (sq.row0 + row) * a.out.row + (c / (D / 8)) * a.out.head +
                                   (c % (D / 8)) * 8) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    total += __shfl_xor_sync(kAll, total, o);
    triples += __shfl_xor_sync(kAll, triples, o);
  }
  // This CTA's range of the line.  Two units for each warp at least.  A multiple of the triples where that
  // costs little, for then triples of one length are cut alike, and one CTA for
  // each where they are short: merging parts takes as long as four units of a
  // warp (one sequence of 300 tokens, 8 KV heads: 9.1 us instead of 13.9).
  long long want = min(static_cast<long long>(gridDim.x), (total + 2 * kWarps - 1) / (2 * kWarps));
  if (want >= 4 * triples)
    want = triples ? divide(want, triples) * triples : want;
  else if (triples <= gridDim.x && total <= triples * 4 * kWarps)
    want = triples;
  const int ctas = static_cast<int>(min(want, total));
  if (static_cast<int>(blockIdx.x) >= ctas) return;
  const long long lo = divide(blockIdx.x * total, ctas), hi = divide((blockIdx.x + 1) * total, ctas);
  Walk use;
  {
    long long base = 0;
    for (int s0 = 0;; s0 += 32) {
      const long long mine = s0 + lane < geo.S ? line_of(seq_work(a, s0 + lane), H) : 0;
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(kAll, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned past = __ballot_sync(kAll, base + incl > lo);
      if (past) {
        const int j = __ffs(past) - 1;
        use.enter(a, s0 + j, base + __shfl_sync(kAll, incl - mine, j), lo, hi);
        break;
      }
      base += __shfl_sync(kAll, incl, 31);
    }
  }

  // ---- fetch: the warp's units, in the order it will use them
  Walk get = use;
  bool more = true;
  int gu = get.u0 + warp;  // next unit to fetch
  const uint32_t ring = kvq::smem_u32(smem) + warp * SM::SLOTS * SM::SLOT;
  const uint32_t meta = kvq::smem_u32(smem) + SM::META + warp * SM::SLOTS * 8;
  const int ushift = 26 - __clz(B);  // units per block: 1 << ushift
  // lane -> (row, chunk) of the copies, the swizzled place included
  constexpr int CPR = D / 16;                 // 16-byte chunks of a code row
  constexpr int RPI = 32 / CPR;               // code rows per instruction
  const int cr = lane / CPR, cc = lane % CPR;

  auto settle = [&]() {  // move to a part that has a unit for this warp
    while (more && gu >= get.u1) {
      more = get.next(a);
      gu = get.u0 + warp;
    }
  };
  auto table_entry = [&]() -> int {
    if (!more || gu >= get.w.full) return 0;
    if (!KVQ_IN_BOUNDS(geo.status, gu >> ushift, geo.max_blocks) || !KVQ_IN_BOUNDS(geo.status, get.s, geo.S)) return -1;
    return geo.table[static_cast<size_t>(get.s) * geo.max_blocks + (gu >> ushift)];
  };
  settle();
  int entry = table_entry();

  auto fetch = [&](int slot) {
    if (more) {
      const uint32_t kdst = ring + slot * SM::SLOT, vdst = kdst + SM::HALF;
      if (gu < get.w.full) {
        const bool good = entry >= 0 && entry < geo.num_blocks;
        const size_t bh = static_cast<size_t>(good ? entry : 0) * H + get.h;
        const uint8_t *ks = geo.codes + (bh * 2 * B + (gu & ((1 << ushift) - 1)) * kUnit) * D + lane * 16;
        const uint8_t *vs = ks + static_cast<size_t>(B) * D;
#pragma unroll
        for (int i = 0; i < kUnit / RPI; ++i) {
          const int row = i * RPI + cr;
          const int sw = D == 128 ? (row & 7) : ((row >> 1) & 3);
          const uint32_t off = row * D + ((cc ^ sw) << 4);
          cp16(kdst + off, ks + i * 512);
          cp16(vdst + off, vs + i * 512);
        }
        if (good) {
          if (lane == 0) cp8(meta + slot * 8, geo.scales + bh * 2);
        } else if (lane == 0) {
          set_status(geo.status, KVQ_STATUS_BAD_BLOCK);
          const float nan = __int_as_float(0x7fc00000);
          *reinterpret_cast<float2 *>(smem + SM::META + (warp * SM::SLOTS + slot) * 8) = make_float2(nan, nan);
        }
      } else {
        const int t0 = (gu - get.w.full) * kWinUnit;
        const int r = get.w.q.L % B - t0;  // tokens of the window from t0 on
        const size_t row0 = (static_cast<size_t>(get.s) * H + get.h) * B + t0;
#pragma unroll
        for (int i = 0; i < kWinUnit * CPR * 2 / 32; ++i) {
          const int c = i * 32 + lane, row = c / (2 * CPR), col = c % (2 * CPR);
          const uint32_t off = row * 2 * D + ((col ^ (row & 7)) << 4);
          // slots past the sequence's end are not read: zeros
          const size_t src = (row0 + (row < r ? row : 0)) * D + col * 8;
          if (!KVQ_IN_BOUNDS(geo.status, t0 + (row < r ? row : 0), B) ||
              !KVQ_IN_BOUNDS(geo.status, static_cast<long long>(get.s) * H + get.h, static_cast<long long>(geo.S) * H))
            continue;
          cp16z(kdst + off, geo.k_win + src, row < r);
          cp16z(vdst + off, geo.v_win + src, row < r);
        }
      }
      gu += kWarps;
      settle();
      entry = table_entry();
    }
    cp_commit();
  };

#pragma unroll
  for (int i = 0; i < SM::SLOTS; ++i) fetch(i);
  int slot = 0;

  for (bool live = true; live; live = use.next(a)) {
    const Work &w = use.w;
    const int n_rows = w.q.n * a.group;  // rows of this KV head
    const int r0 = use.tile * kRowTile;  // first row of the tile

    bool whole;
    // what a window value times its weight counts in the output's sum
    constexpr float kWin = BF16 ? 32768.f : 1.f;

    if constexpr (HALVES == 1) {
      // ================ up to eight rows: tokens (then channels) are M, rows N.
      // Lane (g, q4) holds 16 channels per 64 of row g as B fragments, and
      // rows 2 q4, 2 q4 + 1 of the results.
      uint32_t qb[KS][2];
      float rf[2], r128[2] = {0.f, 0.f};  // of rows 2 q4, 2 q4 + 1: score factor, 128 sum(q)
      int lim[2];                         // last position they see
      {
        const int row = r0 + g;
        const bool valid = row < n_rows && row_in_bounds(a, w.q, use.h, row);
        const int tok = valid ? row / a.group : 0;
        const uint16_t *src =
            a.q.p + (static_cast<long long>(w.q.row0) + tok) * a.q.row +
            (static_cast<long long>(use.h) * a.group + (valid ? row - tok * a.group : 0)) * a.q.head;
        uint32_t big = 0;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
          if (valid) {
            x = *reinterpret_cast<const uint4 *>(src + (c * 4 + q4) * 16);
            y = *reinterpret_cast<const uint4 *>(src + (c * 4 + q4) * 16 + 8);
          }
          const uint32_t e[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            qb[c * 4 + i / 2][i & 1] = e[i];
            if (BF16) big = finite_max(big, e[i], 0x7f80u);
          }
        }
        float f = a.zscale, sum = 0.f;
        if (BF16) {
          big = max(big, __shfl_xor_sync(kAll, big, 1));
          big = max(big, __shfl_xor_sync(kAll, big, 2));
          const float2 n = bf16_norm(big);
          f *= n.y;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            qb[k][0] = bf16_to_fp16(qb[k][0], n.x);
            qb[k][1] = bf16_to_fp16(qb[k][1], n.x);
          }
        }
        if (FMT == KV8_INT8) {
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const float2 x = unpack2<false>(qb[k][0]), y = unpack2<false>(qb[k][1]);
            sum += (x.x + x.y) + (y.x + y.y);
          }
          sum += __shfl_xor_sync(kAll, sum, 1);
          sum += __shfl_xor_sync(kAll, sum, 2);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          rf[i] = __shfl_sync(kAll, f, 4 * (2 * q4 + i));
          if (FMT == KV8_INT8) r128[i] = 128.f * __shfl_sync(kAll, sum, 4 * (2 * q4 + i));
          const int rr = r0 + 2 * q4 + i;
          lim[i] = rr < n_rows ? w.q.L - w.q.n + rr / a.group : -1;
        }
      }
      const int seen_by_all = w.q.L - w.q.n + r0 / a.group;
      constexpr int MT = D / 16;  // m-tiles of the output
      float acc[MT][4], m[2] = {ninf, ninf}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;

      // Scores of NB m-tiles of 16 tokens from position t0 to weights 2^15 w.
      // Row g of a tile is token g ^ 4 (g & 1), row g + 8 the same behind 8.
      const int tok0 = g ^ ((g & 1) << 2);
      auto softmax = [&](auto nb, float (*sc)[4], const float (&ka)[2], const float (&kb)[2], float inv, bool none,
                         int t0, bool window, uint32_t bad, const float *off) {
        constexpr int NB = decltype(nb)::value;
        float mx[2] = {m[0], m[1]};
#pragma unroll
        for (int t = 0; t < NB; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[t][i] = fmaf(sc[t][i], ka[i & 1], kb[i & 1]);
        if (window || bad || t0 + 16 * NB - 1 > seen_by_all) {
#pragma unroll
          for (int t = 0; t < NB; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int col = 16 * t + 8 * (i >> 1) + tok0;
              float z = sc[t][i];
              if (window) z += z - z;  // an infinite score becomes NaN
              if (bad >> col & 1u) z = __int_as_float(0x7fc00000);
              sc[t][i] = t0 + col > lim[i & 1] ? ninf : z;
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int t = 0; t < NB; ++t)
            mx[r] = off ? fmaxf(fmaxf(mx[r], sc[t][r] + off[0]), sc[t][r + 2] + off[1])
                        : fmaxf(fmaxf(mx[r], sc[t][r]), sc[t][r + 2]);
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(kAll, mx[r], 4));
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(kAll, mx[r], 8));
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(kAll, mx[r], 16));
        }
        if (__any_sync(kAll, mx[0] != m[0] || mx[1] != m[1])) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float h = mx[r] == m[r] ? 1.f : kvq::fast_exp2(0.5f * (m[r] - mx[r]));  // -inf before the first token
            const float f = h * h;
            m[r] = mx[r];
            l[r] = l[r] * h * h;  // (zeros' sums may outlive a factor that fp32 cannot hold)
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              acc[j][r] *= f;
              acc[j][r + 2] *= f;
            }
          }
        }
        if (none)
#pragma unroll
          for (int t = 0; t < NB; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[t][i] -= kZeroLog;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float ms = m[r] == ninf ? 0.f : m[r] - kShift;
          float sum = 0.f;
#pragma unroll
          for (int t = 0; t < NB; ++t) {
            sc[t][r] = kvq::fast_exp2(sc[t][r] - ms);
            sc[t][r + 2] = kvq::fast_exp2(sc[t][r + 2] - ms);
            sum += sc[t][r] + sc[t][r + 2];
          }
          l[r] = fmaf(sum, inv, l[r]);
        }
      };

      for (int u = use.u0 + warp; u < use.u1; u += kWarps) {
        cp_wait<SM::SLOTS - 1>();
        __syncwarp();
        const uint32_t kt = ring + slot * SM::SLOT, vt = kt + SM::HALF;
        if (u < w.full) {
          const float2 sc2 = *reinterpret_cast<const float2 *>(smem + SM::META + (warp * SM::SLOTS + slot) * 8);
          float sc[2][4];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[t][i] = 0.f;
            const int row = 16 * t + tok0;  // and row + 8: the same swizzle
            const int sw0 = D == 128 ? (row & 7) : ((row >> 1) & 3), sw1 = D == 128 ? sw0 : (((row + 8) >> 1) & 3);
#pragma unroll
            for (int c = 0; c < D / 64; ++c) {
              const uint4 x = lds16(kt + row * D + (((c * 4 + q4) ^ sw0) << 4));
              const uint4 y = lds16(kt + (row + 8) * D + (((c * 4 + q4) ^ sw1) << 4));
              const uint32_t e[4] = {x.x, x.y, x.z, x.w}, f[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint32_t w0 = flip<FMT>(e[i]), w1 = flip<FMT>(f[i]);
                mma_a<FMT, true>(sc[t], w0, 0, w1, 0, w0, 1, w1, 1, qb[c * 4 + i]);
              }
            }
          }
          const float inf = __int_as_float(0x7f800000);
          // scales that are not finite make the rows that see the block NaN;
          // zeros may have any scale
          const bool bad = !(fabsf(sc2.x) < inf && fabsf(sc2.y) < inf), none = sc2.y < kZeroScale;
          const float ks = bad ? 1.f : sc2.x, vs = bad || none ? 1.f : sc2.y;
          const float lv = none ? kZeroLog : __log2f(vs);
          float ka[2], kb[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float f = ks * rf[r];
            ka[r] = FMT == KV8_INT8 ? f * 16777216.f : f;
            kb[r] = FMT == KV8_INT8 ? fmaf(-r128[r], f, lv) : lv;
          }
          softmax(std::integral_constant<int, 2>{}, sc, ka, kb, __fdividef(1.f, vs), none, u * kUnit, false,
                  bad ? kAll : 0u, nullptr);
          uint32_t p[2][2];  // weights as B fragments of the two k-steps
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            p[t][0] = transpose(kvq::h2_as_u32(__floats2half2_rn(sc[t][0], sc[t][1])));
            p[t][1] = transpose(kvq::h2_as_u32(__floats2half2_rn(sc[t][2], sc[t][3])));
            if (none) p[t][0] = p[t][1] = 0u;
          }
          // values: lane (g, q4) reads its channels of the k-step's tokens 2 q4,
          // (2 q4 + 1) ^ 4 and those 8 behind
          constexpr int VW = D / 32;  // words per token
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            uint32_t v[4][VW];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = 16 * t + 8 * (i >> 1) + ((i & 1) ? ((2 * q4 + 1) ^ 4) : 2 * q4);
              if (D == 128) {
                const uint4 x = lds16(vt + row * D + ((g ^ (row & 7)) << 4));
                v[i][0] = x.x;
                v[i][1] = x.y;
                v[i][VW > 2 ? 2 : 0] = VW > 2 ? x.z : x.x;
                v[i][VW > 3 ? 3 : 0] = VW > 3 ? x.w : x.x;
              } else {
                const uint2 x = lds8(vt + row * D + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8);
                v[i][0] = x.x;
                v[i][1] = x.y;
              }
            }
#pragma unroll
            for (int j = 0; j < VW; ++j) {
              // two tokens' codes interleaved: channels 0, 1 and 2, 3 of the word
              const uint32_t a0 = flip<FMT>(__byte_perm(v[0][j], v[1][j], 0x5140));
              const uint32_t a1 = flip<FMT>(__byte_perm(v[0][j], v[1][j], 0x7362));
              const uint32_t b0 = flip<FMT>(__byte_perm(v[2][j], v[3][j], 0x5140));
              const uint32_t b1 = flip<FMT>(__byte_perm(v[2][j], v[3][j], 0x7362));
              mma_a<FMT, false>(acc[2 * j], a0, 0, a0, 1, b0, 0, b0, 1, p[t]);
              mma_a<FMT, false>(acc[2 * j + 1], a1, 0, a1, 1, b1, 0, b1, 1, p[t]);
            }
          }
        } else {
          // ---- 16 window tokens in 16 bits
          const int t0 = (u - w.full) * kWinUnit;
          float sc[1][4] = {{0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const uint32_t at = kt + tok0 * 2 * D + ((((c * 4 + q4) * 2 + hf) ^ (tok0 & 7)) << 4);
              const uint4 x = lds16(at), y = lds16(at + 16 * D);
              const uint32_t e[4] = {x.x, x.y, x.z, x.w}, f[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int k = c * 4 + 2 * hf + i;
                const uint32_t av[4] = {e[2 * i], f[2 * i], e[2 * i + 1], f[2 * i + 1]};
                if (BF16) {  // the queries in bf16: exact, they came from it
                  const float2 q0 = unpack2<false>(qb[k][0]), q1 = unpack2<false>(qb[k][1]);
                  mma_bf16(sc[0], av, pack2<true>(q0.x, q0.y), pack2<true>(q1.x, q1.y));
                } else {
                  mma(sc[0], av, qb[k][0], qb[k][1]);
                }
              }
            }
          constexpr int VW = D / 16;  // words of the lane's channels per token (2 channels each)
          uint32_t v[4][VW], mag[4];  // mag: the largest magnitude of the lane's channels
          uint32_t bad = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 8 * (i >> 1) + ((i & 1) ? ((2 * q4 + 1) ^ 4) : 2 * q4);
            uint32_t big = 0;
#pragma unroll
            for (int k = 0; k < VW / 4; ++k) {
              const uint4 x = lds16(vt + row * 2 * D + (((g * (VW / 4) + k) ^ (row & 7)) << 4));
              const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                v[i][4 * k + c] = e[c];
                big = __vmaxu2(big, e[c] & 0x7fff7fffu);
              }
            }
            mag[i] = max(big & 0xffffu, big >> 16);
            if (mag[i] >= nonfinite_bits<BF16>()) bad |= 1u << row;
          }
          bad = __reduce_or_sync(kAll, bad);
          const float zero[2] = {0.f, 0.f};
          float off[2];  // of tokens tok0 and tok0 + 8, which lanes with q4 = g / 2 have read
          if (BF16) {
            uint32_t lo = mag[0] | mag[1] << 16, hi = mag[2] | mag[3] << 16;
            all_channels(lo, hi);
            lo = __shfl_sync(kAll, lo, g >> 1);
            hi = __shfl_sync(kAll, hi, g >> 1);
            off[0] = value_log(g & 1 ? lo >> 16 : lo & 0xffffu);
            off[1] = value_log(g & 1 ? hi >> 16 : hi & 0xffffu);
          }
          softmax(std::integral_constant<int, 1>{}, sc, rf, zero, 1.f, false, w.full * kUnit + t0, true, bad,
                  BF16 ? off : nullptr);
          if (bad) {  // their weights are NaN where they are seen, and 0 elsewhere
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = 8 * (i >> 1) + ((i & 1) ? ((2 * q4 + 1) ^ 4) : 2 * q4);
              if (bad >> row & 1u)
#pragma unroll
                for (int k = 0; k < VW; ++k) v[i][k] = 0u;
            }
          }
          uint32_t p[2], rest[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float x = sc[0][2 * i] * (BF16 ? kUnshift : 1.f), y = sc[0][2 * i + 1] * (BF16 ? kUnshift : 1.f);
            const uint32_t hi = pack2<BF16>(x, y);
            p[i] = transpose(hi);
            if (BF16) {
              const float2 f = unpack2<true>(hi);
              rest[i] = transpose(pack2<true>(x - f.x, y - f.y));
            }
          }
#pragma unroll
          for (int j = 0; j < VW; ++j) {
            const uint32_t av[4] = {__byte_perm(v[0][j], v[1][j], 0x5410), __byte_perm(v[0][j], v[1][j], 0x7632),
                                    __byte_perm(v[2][j], v[3][j], 0x5410), __byte_perm(v[2][j], v[3][j], 0x7632)};
            float o[4] = {0.f, 0.f, 0.f, 0.f};
            if (BF16) {
              mma_bf16(o, av, p[0], p[1]);
              mma_bf16(o, av, rest[0], rest[1]);
            } else {
              mma(o, av, p[0], p[1]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[j][i] = fmaf(o[i], kWin, acc[j][i]);
          }
        }
        __syncwarp();  // every lane has read the slot
        fetch(slot);
        slot = slot + 1 == SM::SLOTS ? 0 : slot + 1;
      }

      // ---- merge the four warps' states; warp w ends up with quarter w of the
      // m-tiles
      float2 *ml = reinterpret_cast<float2 *>(smem + SM::ML);
      float *xch = reinterpret_cast<float *>(smem + SM::XCH);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(kAll, l[r], 4);
        l[r] += __shfl_xor_sync(kAll, l[r], 8);
        l[r] += __shfl_xor_sync(kAll, l[r], 16);
        l[r] *= kUnshift;
        if (g == 0) ml[warp * kRowTile + 2 * q4 + r] = make_float2(m[r], l[r]);
      }
      __syncthreads();
      whole = use.u0 == 0 && use.u1 == w.units;
      const int part = 2 * blockIdx.x + (use.start + use.u0 == lo ? 0 : 1);
      constexpr int QT = MT / 4;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float mm = ninf, ll = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) mm = fmaxf(mm, ml[i * kRowTile + 2 * q4 + r].x);
        const float base = mm == ninf ? 0.f : mm;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          const float2 e = ml[i * kRowTile + 2 * q4 + r];
          const float h = kvq::fast_exp2(0.5f * (e.x - base));
          ll += e.y * h * h;
        }
        const float f = kvq::fast_exp2(m[r] - base);
        if (r) __syncthreads();  // the buffer of the first row has been read
        float2 o[QT];
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          const float x[2] = {f * (acc[j][r] * kUnshift), f * (acc[j][r + 2] * kUnshift)};
          const int dst = j / QT;
          if (dst != warp) {
            float *b = xch + ((dst * 3 + ((warp - dst - 1) & 3)) * QT + j % QT) * 64 + lane;
            b[0] = x[0];
            b[32] = x[1];
          } else {
            o[j % QT] = make_float2(x[0], x[1]);
          }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < QT; ++j)
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            const float *b = xch + ((warp * 3 + i) * QT + j) * 64 + lane;
            o[j].x += b[0];
            o[j].y += b[32];
          }
        // m-tile j holds channels (D / 8) g + 2 j and the next one
        const int ch = (D / 8) * g + 2 * QT * warp, row = r0 + 2 * q4 + r;
        if (row < n_rows && row_in_bounds(a, w.q, use.h, row) && KVQ_IN_BOUNDS(geo.status, part, 2 * kMaxCtas)) {
          if (whole) {
            const float inv = inverse_sum(ll, lim[r]);
            const int tok = row / a.group;
            uint16_t *dst = a.out.p + (static_cast<long long>(w.q.row0) + tok) * a.out.row +
                            (static_cast<long long>(use.h) * a.group + row - tok * a.group) * a.out.head + ch;
#pragma unroll
            for (int j = 0; j < QT; ++j)
              *reinterpret_cast<uint32_t *>(dst + 2 * j) = pack2<BF16>(o[j].x * inv, o[j].y * inv);
          } else {
            float *dst = a.part_o + (static_cast<size_t>(part) * kRowTile + 2 * q4 + r) * D + ch;
#pragma unroll
            for (int j = 0; j < QT; ++j) *reinterpret_cast<float2 *>(dst + 2 * j) = o[j];
            if (warp == 0 && g == 0) a.part_ml[part * kRowTile + 2 * q4 + r] = make_float2(mm, ll);
          }
        }
      }
    } else {
      // ================ up to sixteen rows are M, tokens (then channels) N.
      // ---- the tile's queries as A fragments; lane (g, q4) holds 16 channels
      // of rows g and g + 8 per 64 channels
      uint32_t qa[KS][4];
      float qf[2], q128[2] = {0.f, 0.f};
      int lim[2];  // last position each row sees
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = r0 + g + 8 * r;
        const bool valid = row < n_rows && row_in_bounds(a, w.q, use.h, row);
        const int tok = valid ? row / a.group : 0;
        lim[r] = valid ? w.q.L - w.q.n + tok : -1;
        const uint16_t *src = a.q.p + (static_cast<long long>(w.q.row0) + tok) * a.q.row +
                              (static_cast<long long>(use.h) * a.group + (valid ? row - tok * a.group : 0)) * a.q.head;
        uint32_t big = 0;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint4 x = make_uint4(0u, 0u, 0u, 0u), y = x;
          if (valid) {
            x = *reinterpret_cast<const uint4 *>(src + (c * 4 + q4) * 16);
            y = *reinterpret_cast<const uint4 *>(src + (c * 4 + q4) * 16 + 8);
          }
          const uint32_t e[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            qa[c * 4 + i / 2][r + 2 * (i & 1)] = e[i];
            if (BF16) big = finite_max(big, e[i], 0x7f80u);
          }
        }
        qf[r] = a.zscale;
        if (BF16) {
          big = max(big, __shfl_xor_sync(kAll, big, 1));
          big = max(big, __shfl_xor_sync(kAll, big, 2));
          const float2 f = bf16_norm(big);
          qf[r] *= f.y;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            qa[k][r] = bf16_to_fp16(qa[k][r], f.x);
            qa[k][r + 2] = bf16_to_fp16(qa[k][r + 2], f.x);
          }
        }
        if (FMT == KV8_INT8) {
          float sum = 0.f;
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const float2 x = unpack2<false>(qa[k][r]), y = unpack2<false>(qa[k][r + 2]);
            sum += (x.x + x.y) + (y.x + y.y);
          }
          sum += __shfl_xor_sync(kAll, sum, 1);
          sum += __shfl_xor_sync(kAll, sum, 2);
          q128[r] = 128.f * sum;
        }
      }
      // They wait in shared memory, alike for all warps: in registers they cost
      // spills (16 sequences with 3 to 8 drafts: 3 us).
      const uint32_t qs = kvq::smem_u32(smem) + SM::XCH + lane * 16;
#pragma unroll
      for (int k = 0; k < KS; ++k)
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(qs + k * 512), "r"(qa[k][0]), "r"(qa[k][1]),
                     "r"(qa[k][2]), "r"(qa[k][3])
                     : "memory");
      __syncwarp();
      auto query = [&](uint32_t (&r)[4], int k) {
        const uint4 x = lds16(qs + k * 512);
        r[0] = x.x;
        r[1] = x.y;
        r[2] = x.z;
        r[3] = x.w;
      };
      // every row of the tile sees at least the tokens up to here
      const int seen_by_all = w.q.L - w.q.n + r0 / a.group;

      float acc[NT][4], m[2] = {ninf, ninf}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[j][r] = 0.f;

      // Scores of one unit to weights 2^15 w: NB n-tiles of 8 tokens from position
      // t0; column 2 q4 of a tile is token 2 q4, column 2 q4 + 1 token (2 q4 + 1) ^ 4.
      // z = s a + b for the two rows; `bad`: tokens that turn what sees them to NaN.
      auto softmax = [&](auto nb, float (*sc)[4], const float (&ka)[2], const float (&kb)[2], float inv, bool none,
                         int t0, bool window, uint32_t bad, const float *off) {
        constexpr int NB = decltype(nb)::value;
        float mx[2] = {m[0], m[1]};
#pragma unroll
        for (int t = 0; t < NB; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[t][i] = fmaf(sc[t][i], ka[i >> 1], kb[i >> 1]);
        if (window || bad || t0 + 8 * NB - 1 > seen_by_all) {
#pragma unroll
          for (int t = 0; t < NB; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int col = 8 * t + ((i & 1) ? ((2 * q4 + 1) ^ 4) : 2 * q4);
              float z = sc[t][i];
              if (window) z += z - z;  // an infinite score becomes NaN
              if (bad >> col & 1u) z = __int_as_float(0x7fc00000);
              sc[t][i] = t0 + col > lim[i >> 1] ? ninf : z;
            }
        }
#pragma unroll
        for (int t = 0; t < NB; ++t)
#pragma unroll
          for (int i = 0; i < 4; i += 2)
            mx[i >> 1] = off ? fmaxf(fmaxf(mx[i >> 1], sc[t][i] + off[2 * t]), sc[t][i + 1] + off[2 * t + 1])
                             : fmaxf(fmaxf(mx[i >> 1], sc[t][i]), sc[t][i + 1]);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(kAll, mx[r], 1));
          mx[r] = fmaxf(mx[r], __shfl_xor_sync(kAll, mx[r], 2));
        }
        if (__any_sync(kAll, mx[0] != m[0] || mx[1] != m[1])) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float h = mx[r] == m[r] ? 1.f : kvq::fast_exp2(0.5f * (m[r] - mx[r]));  // -inf before the first token
            const float f = h * h;
            m[r] = mx[r];
            l[r] = l[r] * h * h;  // (zeros' sums may outlive a factor that fp32 cannot hold)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              acc[j][2 * r] *= f;
              acc[j][2 * r + 1] *= f;
            }
          }
        }
        if (none)
#pragma unroll
          for (int t = 0; t < NB; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[t][i] -= kZeroLog;
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float ms = m[r] == ninf ? 0.f : m[r] - kShift;
#pragma unroll
          for (int t = 0; t < NB; ++t) {
            sc[t][2 * r] = kvq::fast_exp2(sc[t][2 * r] - ms);
            sc[t][2 * r + 1] = kvq::fast_exp2(sc[t][2 * r + 1] - ms);
            sum[r] += sc[t][2 * r] + sc[t][2 * r + 1];
          }
          l[r] = fmaf(sum[r], inv, l[r]);
        }
      };
      // the weights of n-tiles 2 k, 2 k + 1 as the A operand of k-step k
      auto weights = [&](uint32_t (&p)[4], const float *lo, const float *hi) {
        p[0] = kvq::h2_as_u32(__floats2half2_rn(lo[0], lo[1]));
        p[1] = kvq::h2_as_u32(__floats2half2_rn(lo[2], lo[3]));
        p[2] = kvq::h2_as_u32(__floats2half2_rn(hi[0], hi[1]));
        p[3] = kvq::h2_as_u32(__floats2half2_rn(hi[2], hi[3]));
      };

      for (int u = use.u0 + warp; u < use.u1; u += kWarps) {
        cp_wait<SM::SLOTS - 1>();
        __syncwarp();
        const uint32_t kt = ring + slot * SM::SLOT, vt = kt + SM::HALF;
        if (u < w.full) {
          const float2 sc2 = *reinterpret_cast<const float2 *>(smem + SM::META + (warp * SM::SLOTS + slot) * 8);
          float sc[4][4];
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            uint32_t e[4][4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const int row = 8 * t + (g ^ ((g & 1) << 2));
              const int sw = D == 128 ? (row & 7) : ((row >> 1) & 3);
              const uint4 x = lds16(kt + row * D + (((c * 4 + q4) ^ sw) << 4));
              e[t][0] = flip<FMT>(x.x);
              e[t][1] = flip<FMT>(x.y);
              e[t][2] = flip<FMT>(x.z);
              e[t][3] = flip<FMT>(x.w);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t qa[4];
              query(qa, c * 4 + i);
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                const uint64_t b = widen<FMT, true>(e[t][i], 0, e[t][i], 1);
                if (c == 0 && i == 0)
                  mma_zero(sc[t], qa, b);
                else
                  mma(sc[t], qa, b);
              }
            }
          }
          const float inf = __int_as_float(0x7f800000);
          // scales that are not finite make the rows that see the block NaN;
          // zeros may have any scale
          const bool bad = !(fabsf(sc2.x) < inf && fabsf(sc2.y) < inf), none = sc2.y < kZeroScale;
          const float ks = bad ? 1.f : sc2.x, vs = bad || none ? 1.f : sc2.y;
          const float lv = none ? kZeroLog : __log2f(vs);
          float ka[2], kb[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float f = ks * qf[r];
            ka[r] = FMT == KV8_INT8 ? f * 16777216.f : f;
            kb[r] = FMT == KV8_INT8 ? fmaf(-q128[r], f, lv) : lv;
          }
          softmax(std::integral_constant<int, 4>{}, sc, ka, kb, __fdividef(1.f, vs), none, u * kUnit, false,
                  bad ? kAll : 0u, nullptr);
          uint32_t p[2][4];
          weights(p[0], sc[0], sc[1]);
          weights(p[1], sc[2], sc[3]);
          if (none)
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i >> 2][i & 3] = 0u;
          // values: lane (g, q4) reads its channels of the 8 tokens of its k indices
          constexpr int VW = D / 32;  // words per token
          uint32_t v[8][VW];
#pragma unroll
          for (int i = 0; i < 8; ++i) {  // token: k-step i / 4, k index 2 q4 + (i & 1) + 8 (i / 2 & 1)
            const int row = 16 * (i >> 2) + 8 * (i >> 1 & 1) + ((i & 1) ? ((2 * q4 + 1) ^ 4) : 2 * q4);
            if (D == 128) {
              const uint4 x = lds16(vt + row * D + ((g ^ (row & 7)) << 4));
              v[i][0] = x.x;
              v[i][1] = x.y;
              v[i][VW > 2 ? 2 : 0] = VW > 2 ? x.z : x.x;
              v[i][VW > 3 ? 3 : 0] = VW > 3 ? x.w : x.x;
            } else {
              const uint2 x = lds8(vt + row * D + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8);
              v[i][0] = x.x;
              v[i][1] = x.y;
            }
          }
#pragma unroll
          for (int j = 0; j < VW; ++j) {
            // two tokens' codes interleaved: channels 0, 1 and 2, 3 of the word
            uint32_t lo[4], hi[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              lo[i] = flip<FMT>(__byte_perm(v[2 * i][j], v[2 * i + 1][j], 0x5140));
              hi[i] = flip<FMT>(__byte_perm(v[2 * i][j], v[2 * i + 1][j], 0x7362));
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              mma(acc[4 * j], p[k], widen<FMT, false>(lo[2 * k], 0, lo[2 * k + 1], 0));
              mma(acc[4 * j + 1], p[k], widen<FMT, false>(lo[2 * k], 1, lo[2 * k + 1], 1));
              mma(acc[4 * j + 2], p[k], widen<FMT, false>(hi[2 * k], 0, hi[2 * k + 1], 0));
              mma(acc[4 * j + 3], p[k], widen<FMT, false>(hi[2 * k], 1, hi[2 * k + 1], 1));
            }
          }
        } else {
          // ---- 16 window tokens in 16 bits
          const int t0 = (u - w.full) * kWinUnit;
          float sc[2][4];
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) sc[t][i] = 0.f;
#pragma unroll
          for (int k = 0; k < KS; k += 2) {
            uint32_t q0[4], q1[4];
            query(q0, k);
            query(q1, k + 1);
            if (BF16) {  // the queries in bf16: exact, they came from it
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 x = unpack2<false>(q0[i]), y = unpack2<false>(q1[i]);
                q0[i] = pack2<true>(x.x, x.y);
                q1[i] = pack2<true>(y.x, y.y);
              }
            }
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int row = 8 * t + (g ^ ((g & 1) << 2));
              const uint4 x = lds16(kt + row * 2 * D + ((((k & ~3) * 2 + q4 * 2 + (k >> 1 & 1)) ^ (row & 7)) << 4));
              if (BF16) {
                mma_bf16(sc[t], q0, x.x, x.y);
                mma_bf16(sc[t], q1, x.z, x.w);
              } else {
                mma(sc[t], q0, x.x, x.y);
                mma(sc[t], q1, x.z, x.w);
              }
            }
          }
          constexpr int VW = D / 16;  // words of the lane's channels per token (2 channels each)
          uint32_t v[4][VW], mag[4];  // mag: the largest magnitude of the lane's channels
          uint32_t bad = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 8 * (i >> 1) + ((i & 1) ? ((2 * q4 + 1) ^ 4) : 2 * q4);
            uint32_t big = 0;
#pragma unroll
            for (int k = 0; k < VW / 4; ++k) {
              const uint4 x = lds16(vt + row * 2 * D + (((g * (VW / 4) + k) ^ (row & 7)) << 4));
              const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                v[i][4 * k + c] = e[c];
                big = __vmaxu2(big, e[c] & 0x7fff7fffu);
              }
            }
            mag[i] = max(big & 0xffffu, big >> 16);
            if (mag[i] >= nonfinite_bits<BF16>()) bad |= 1u << row;
          }
          bad = __reduce_or_sync(kAll, bad);
          const float zero[2] = {0.f, 0.f};
          float off[4];  // of the tokens of v
          if (BF16) {
            uint32_t lo = mag[0] | mag[1] << 16, hi = mag[2] | mag[3] << 16;
            all_channels(lo, hi);
            off[0] = value_log(lo & 0xffffu);
            off[1] = value_log(lo >> 16);
            off[2] = value_log(hi & 0xffffu);
            off[3] = value_log(hi >> 16);
          }
          softmax(std::integral_constant<int, 2>{}, sc, qf, zero, 1.f, false, w.full * kUnit + t0, true, bad,
                  BF16 ? off : nullptr);
          uint32_t p[4], rest[4];
          if (BF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float x = sc[i >> 1][2 * (i & 1)] * kUnshift, y = sc[i >> 1][2 * (i & 1) + 1] * kUnshift;
              p[i] = pack2<true>(x, y);
              const float2 f = unpack2<true>(p[i]);
              rest[i] = pack2<true>(x - f.x, y - f.y);
            }
          } else {
            weights(p, sc[0], sc[1]);
          }
          if (bad) {  // their weights are NaN where they are seen, and 0 elsewhere
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int row = 8 * (i >> 1) + ((i & 1) ? ((2 * q4 + 1) ^ 4) : 2 * q4);
              if (bad >> row & 1u)
#pragma unroll
                for (int k = 0; k < VW; ++k) v[i][k] = 0u;
            }
          }
#pragma unroll
          for (int k = 0; k < VW; ++k) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t b0 = __byte_perm(v[0][k], v[1][k], c ? 0x7632 : 0x5410);
              const uint32_t b1 = __byte_perm(v[2][k], v[3][k], c ? 0x7632 : 0x5410);
              float o[4] = {0.f, 0.f, 0.f, 0.f};
              if (BF16) {
                mma_bf16(o, p, b0, b1);
                mma_bf16(o, rest, b0, b1);
              } else {
                mma(o, p, b0, b1);
              }
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[2 * k + c][r] = fmaf(o[r], kWin, acc[2 * k + c][r]);
            }
          }
        }
        __syncwarp();  // every lane has read the slot
        fetch(slot);
        slot = slot + 1 == SM::SLOTS ? 0 : slot + 1;
      }

      // ---- merge the four warps' states; warp w ends up with quarter w of the
      // n-tiles
      float2 *ml = reinterpret_cast<float2 *>(smem + SM::ML);
      float *xch = reinterpret_cast<float *>(smem + SM::XCH);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(kAll, l[r], 1);
        l[r] += __shfl_xor_sync(kAll, l[r], 2);
        l[r] *= kUnshift;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            acc[j][2 * r + i] *= kUnshift;
        if (q4 == 0) ml[warp * kRowTile + g + 8 * r] = make_float2(m[r], l[r]);
      }
      __syncthreads();
      whole = use.u0 == 0 && use.u1 == w.units;
      const int part = 2 * blockIdx.x + (use.start + use.u0 == lo ? 0 : 1);
      constexpr int QT = NT / 4;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float mm = ninf, ll = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) mm = fmaxf(mm, ml[i * kRowTile + g + 8 * r].x);
        const float base = mm == ninf ? 0.f : mm;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          const float2 e = ml[i * kRowTile + g + 8 * r];
          const float h = kvq::fast_exp2(0.5f * (e.x - base));
          ll += e.y * h * h;
        }
        const float f = kvq::fast_exp2(m[r] - base);
        float o[2][QT];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (r || c) __syncthreads();  // the buffer has been read
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const float x = acc[j][2 * r + c] * f;
            const int dst = j / QT;
            if (dst != warp)
              xch[((dst * 3 + ((warp - dst - 1) & 3)) * QT + j % QT) * 32 + lane] = x;
            else
              o[c][j % QT] = x;
          }
          __syncthreads();
#pragma unroll
          for (int j = 0; j < QT; ++j)
#pragma unroll
            for (int i = 0; i < 3; ++i) o[c][j] += xch[((warp * 3 + i) * QT + j) * 32 + lane];
        }
        const float (&o0)[QT] = o[0], (&o1)[QT] = o[1];
        // n-tile j, column c holds channel (D / 8) c + j
        const int ch0 = (D / 8) * (2 * q4) + warp * QT, ch1 = ch0 + D / 8;
        const int row = r0 + g + 8 * r;
        if (row < n_rows && row_in_bounds(a, w.q, use.h, row) && KVQ_IN_BOUNDS(geo.status, part, 2 * kMaxCtas)) {
          if (whole) {
            const float inv = inverse_sum(ll, lim[r]);
            const int tok = row / a.group;
            uint16_t *dst = a.out.p + (static_cast<long long>(w.q.row0) + tok) * a.out.row +
                            (static_cast<long long>(use.h) * a.group + row - tok * a.group) * a.out.head;
#pragma unroll
            for (int j = 0; j < QT; j += 2) {
              *reinterpret_cast<uint32_t *>(dst + ch0 + j) = pack2<BF16>(o0[j] * inv, o0[j + 1] * inv);
              *reinterpret_cast<uint32_t *>(dst + ch1 + j) = pack2<BF16>(o1[j] * inv, o1[j + 1] * inv);
            }
          } else {
            float *dst = a.part_o + (static_cast<size_t>(part) * kRowTile + g + 8 * r) * D;
#pragma unroll
            for (int j = 0; j < QT; j += 2) {
              *reinterpret_cast<float2 *>(dst + ch0 + j) = make_float2(o0[j], o0[j + 1]);
              *reinterpret_cast<float2 *>(dst + ch1 + j) = make_float2(o1[j], o1[j + 1]);
            }
            if (warp == 0 && q4 == 0) a.part_ml[part * kRowTile + g + 8 * r] = make_float2(mm, ll);
          }
        }
      }
    }

    if (!whole) {
      // ---- the last CTA with a part of this triple merges them all, a warp's rows
      // at once (one after the other the drafts take 47 us instead of 44)
      const long long s0 = use.start, s1 = s0 + w.units;  // the triple's place on the line
      auto owner = [&](long long pos) { return static_cast<int>(divide((pos + 1) * ctas - 1, total)); };
      const int c0 = owner(s0), c1 = owner(s1 - 1);
      int *flag = reinterpret_cast<int *>(smem + SM::FLAG);
      __syncthreads();
      if (tid == 0) {
        // releases the CTA's stores, which the barrier has ordered before, and
        // acquires the others' for the reads behind the next barrier
        const bool counted = KVQ_IN_BOUNDS(geo.status, c0, kMaxCtas) && KVQ_IN_BOUNDS(geo.status, c1, kMaxCtas);
        const bool last = counted && kvq::atom_add_acq_rel(a.counters + c0, 1) == c1 - c0;
        if (last) a.counters[c0] = 0;
        *flag = last;
      }
      __syncthreads();
      const int rows = min(kRowTile, n_rows - r0);
      if (*flag && warp < rows) {
        const int first = 2 * c0 + (divide(c0 * total, ctas) < s0 ? 1 : 0);  // later CTAs begin with their part
        const int parts = c1 - c0 + 1;
        constexpr int W = D / 32;                // channels per lane
        constexpr int NR = HALVES == 1 ? 2 : 4;  // rows per warp, at once: warp + 4 k, or again the last one
        float mm[NR], ll[NR], o[NR][W];
        int row[NR];
#pragma unroll
        for (int k = 0; k < NR; ++k) {
          row[k] = min(warp + kWarps * k, rows - 1);
          mm[k] = ninf;
          ll[k] = 0.f;
#pragma unroll
          for (int j = 0; j < W; ++j) o[k][j] = 0.f;
        }
#pragma unroll(HALVES == 1 ? 4 : 2)
        for (int i = 0; i < parts; ++i) {
          const int sl = i == 0 ? first : 2 * (c0 + i);
          float2 e[NR];
          float x[NR][W];
#pragma unroll
          for (int k = 0; k < NR; ++k) {
            e[k] = __ldcg(&a.part_ml[sl * kRowTile + row[k]]);
            const float *src = a.part_o + (static_cast<size_t>(sl) * kRowTile + row[k]) * D + lane * W;
#pragma unroll
            for (int j = 0; j < W; j += 2) {
              const float2 y = __ldcg(reinterpret_cast<const float2 *>(src + j));
              x[k][j] = y.x;
              x[k][j + 1] = y.y;
            }
          }
#pragma unroll
          for (int k = 0; k < NR; ++k) {
            const float top = fmaxf(mm[k], e[k].x), base = top == ninf ? 0.f : top;
            const float wh = kvq::fast_exp2(0.5f * (mm[k] - base)), fh = kvq::fast_exp2(0.5f * (e[k].x - base));
            const float was = wh * wh, f = fh * fh;
            mm[k] = top;
            ll[k] = fmaf(ll[k] * wh, wh, e[k].y * fh * fh);
#pragma unroll
            for (int j = 0; j < W; ++j) o[k][j] = fmaf(o[k][j], was, x[k][j] * f);
          }
        }
#pragma unroll
        for (int k = 0; k < NR; ++k) {
          if (warp + kWarps * k >= rows || !row_in_bounds(a, w.q, use.h, r0 + row[k])) break;
          const int tok = (r0 + row[k]) / a.group;
          const float inv = inverse_sum(ll[k], w.q.L - w.q.n + tok);
          uint16_t *dst = a.out.p + (static_cast<long long>(w.q.row0) + tok) * a.out.row +
                          (static_cast<long long>(use.h) * a.group + r0 + row[k] - tok * a.group) * a.out.head + lane * W;
#pragma unroll
          for (int j = 0; j < W; j += 2)
            *reinterpret_cast<uint32_t *>(dst + j) = pack2<BF16>(o[k][j] * inv, o[k][j + 1] * inv);
        }
      }
    }
    __syncthreads();  // the merge buffers are free for the next part
  }
  cp_wait<0>();
}

template <int D, int FMT, bool BF16, int HALVES>
cudaError_t launch_one(const AttnArgs &a, cudaStream_t stream) {
  auto kernel = rows_kernel<D, FMT, BF16, HALVES>;
  // resident CTAs and SMs of each device, once looked up
  static std::atomic<int> resident[64], sm_count[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int per = dev < 64 ? resident[dev].load() : 0, sms = dev < 64 ? sm_count[dev].load() : 0;
  if (per == 0 || sms == 0) {
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D, HALVES>::BYTES)) != cudaSuccess)
      return e;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kWarps * 32, Smem<D, HALVES>::BYTES)) != cudaSuccess)
      return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    // Three CTAs fit an SM where at most eight rows share the keys.  Few
    // instructions per byte (int8) keep HBM busy with two, and a third only
    // spreads the reads (a million tokens x 8 heads: 304 us against 331); the
    // conversions of e4m3 want it (64 x 8 heads ragged: 111 us against 116).
    per = min(max(per, 1), FMT == KV8_INT8 ? 2 : 3);
    if (dev < 64) {
      sm_count[dev].store(sms);
      resident[dev].store(per);
    }
  }
  // no more CTAs than units for their warps, as far as the host can tell
  const long long most = min(static_cast<long long>(a.max_new) * a.group, static_cast<long long>(a.rows_max));
  const long long tiles = (most + kRowTile - 1) / kRowTile;
  const long long units = (a.max_len / kUnit + a.geo.B / kWinUnit) * tiles * a.geo.H * a.geo.S;
  long long grid = min(static_cast<long long>(kMaxCtas), static_cast<long long>(sms) * per);
  grid = max(1LL, min(grid, (units + kWarps - 1) / kWarps));
  kernel<<<static_cast<unsigned>(grid), kWarps * 32, Smem<D, HALVES>::BYTES, stream>>>(a);
  return cudaGetLastError();
}

template <int D, int FMT, bool BF16>
cudaError_t launch_halves(const AttnArgs &a, cudaStream_t stream) {
  return static_cast<long long>(a.max_new) * a.group <= 8 ? launch_one<D, FMT, BF16, 1>(a, stream)
                                                          : launch_one<D, FMT, BF16, 2>(a, stream);
}

template <int D>
cudaError_t launch_dim(const AttnArgs &a, cudaStream_t stream) {
  if (a.geo.fmt == KV8_INT8)
    return a.geo.bf16 ? launch_halves<D, KV8_INT8, true>(a, stream) : launch_halves<D, KV8_INT8, false>(a, stream);
  return a.geo.bf16 ? launch_halves<D, KV8_E4M3, true>(a, stream) : launch_halves<D, KV8_E4M3, false>(a, stream);
}

}  // namespace rows
}  // namespace kv8
