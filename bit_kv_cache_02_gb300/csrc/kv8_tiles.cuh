// Attention over the 8-bit paged cache for many rows per sequence (chunks of
// prompts), on the tcgen05 tensor cores.
//
// A work item is 256 rows -- (new token, query head) pairs of one KV head, two
// tiles of 128 -- against the keys they see, 128 at a time.  Roles of a CTA:
//
//   warps 0-7, 8-15  softmax of row tile 0 and 1: two threads per row, for 64
//                    keys of a unit each (the instructions of one thread per
//                    row depend on each other too much to keep the SM busy).
//                    S comes from tensor memory, the weights go back there as
//                    fp16.
//   warps 16-19      bring 128 tokens' codes from the blocks (prefetched one
//                    tile ahead in registers), widen them to fp16 and store them
//                    in the 128-byte-swizzled layout the tensor core reads:
//                    tokens as rows for keys (K-major) and values (MN-major).
//   warp 20          issues the products: S = Q K^T, then O += P V with P in
//                    tensor memory.  The two row tiles alternate, so one tile's
//                    softmax runs under the other's products.
//   warp 21          walks the CTA's share of the work: a ring of Parts.
//   warp 22          looks up blocks and scales: a ring of Metas, one per unit.
//
// Parts and Metas live in shared memory so that the other roles keep their
// registers for data: a spilled register costs an L2 round trip here, as the
// tiles leave no first-level cache to speak of.  (The 28 bytes that kv8_attn's
// forms spill do not show: a chunk of 2048 tokens over 8192 takes 215 us, the form
// without spills before 218, prompts from position 0 561 and 560.)
//
// Mathematics, in log2 units per row: z_t = q.k_t scale_k softmax_scale log2(e),
// w_t = 2^(z_t + log2(scale_v) - M + 9), O = sum w_t v_code_t, l = sum w_t /
// scale_v, out = O / l.  Folding scale_v into the exponent lets O accumulate
// codes of blocks with different scales in tensor memory (blocks of zeros enter
// M with kZeroLog, and their weights, formed without, l alone).  M follows the row's
// maximum of z + log2(scale_v) lazily: O is rescaled only when it grew by more
// than 2^6, so w stays below 2^15 and weights down to 2^-23 of the largest
// keep fp16's full precision.  Roundings: w to fp16, as in the rows kernel; bf16
// queries scaled to fp16's range as there; bf16 window tokens scaled token by
// token (the factors enter z and M like the blocks' scales), which the rows
// kernel need not do: an element 2^-29 below its token's largest loses bits, in
// all 2^-39 of the largest, and the token's weight, for its values stand 2^8 above
// a block's codes, where it is 2^-15 or less of a block's of that size.
//
// The keys of all items form one line of 128-token units, with kOver more for
// what an item costs by itself, which is cut into one equal range per SM; items
// cut by a border are merged by the last CTA that finishes (fp32 partial O, M
// and l in the workspace).
//
// SHARED: the kernels of cross attention and of attention with shared blocks, whose
// segments have been looked up before.  They start beside the rows kernel; joining
// partial results costs them registers, and long calls 3 to 4% (16 entries x 16
// heads of 200 to 448 rows over 1500 tokens, D 64: 115 us replayed, 112 without),
// but short ones gain a quarter (27.5 against 21 us).  Over shared blocks, few rows make
// few items, which are cut into parts of two units: 256 rows x 8 KV heads over 4096
// shared tokens take 21 us, of which the second unit is 1.2: the rest comes once
// (3.3 until the line is cut, 3.6 until the part is known, 4.1 for queries, 1 for
// the first scores, 5 for the first unit, 4 for outputs and the end).  1830 rows x 32 query heads
// over 8192: 240 us, 1.02 PFLOP/s.
//
// Bound: the chain of a row tile.  Per unit it works on its softmax for about
// 2350 clocks and waits 1800 for its products, which take 1270 where no others
// are in the way: S (u + 1) goes where the weights of u lie, so Q K^T of the
// next unit comes after P V, and tensor memory (two S, two O of 128 columns)
// has no place for a second S.  The other tile fills the gaps: the tensor pipe
// is busy for 47% of the time, the issue slots for 54%, and most of the
// softmax's instructions take two slots (exp2 four).  2048 tokens x 32 query
// heads over 8192 tokens, D 128: 224 us, 1.07 PFLOP/s; an item costs 11,000
// clocks besides its units (queries 3500, first S 1600, outputs 4500), so
// prompts from position 0 (4 x 32 heads, 1500 to 4096 tokens) take 550 us, 0.78
// PFLOP/s counting visible pairs only.
#pragma once

#include <atomic>
#include <type_traits>

#include "kv8_internal.cuh"

namespace kv8 {
namespace tiles {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 768;
constexpr int kRows = kTileRows;  // 256 rows of an item
constexpr int kKeys = 128;        // tokens of a unit
constexpr int kMetas = 8, kParts = 4, kCols = 4;
constexpr int kOver = 3;          // queries and outputs of an item cost about as much as three units
constexpr float kGrow = 6.f;      // how far the maximum may pass M
constexpr float kShift = 9.f;     // w = 2^(z' - M + kShift) <= 2^15

template <int D>
struct Smem {
  static constexpr int HALF = 128 * 128;          // 128 rows of 64 channels in fp16
  static constexpr int TILE = HALF * (D / 64);    // 128 rows of D channels
  static constexpr int Q = 0;                     // two row tiles
  static constexpr int K = Q + 2 * TILE;          // two stages
  static constexpr int V = K + 2 * TILE;          // two stages
  static constexpr int META = V + 2 * TILE;       // [kMetas] Meta
  static constexpr int PART = META + kMetas * 128;  // [kParts] Part
  static constexpr int COL = PART + kParts * 64;  // [kCols] window columns: scale_k, log2 scale_v, - log2 scale_v or 0
  static constexpr int ROW = COL + kCols * 3 * kKeys * 4;  // per row: maxima of both halves, two units; exponents, sums
  static constexpr int BAR = ROW + 6 * kRows * 4;
  static constexpr int MISC = BAR + 48 * 8;
  static constexpr int BYTES = MISC + 384 + 1024;  // and the alignment of the base
};

// What the roles need to know of one unit.  A ring of eight: warp 22 reuses a
// slot once keys are stored three units later, which means that the products
// two units before those are done, and the softmax of the unit before that.
enum { kPacked, kWindow, kEnd };
struct Meta {
  long long off[4];           // pool offset of each group of 32 tokens' keys
  float k[4], lv[4], inv[4];  // scales of keys, log2 and inverse of those of values
  long long win;              // window offset of the (sequence, head)
  int kind;                   // kPacked, kWindow or kEnd
  int valid;                  // tokens of a window unit
  int flush;                  // groups whose values count as zeros (without a block, their offset is 0)
  int pad[7];
};
static_assert(sizeof(Meta) == 128, "Meta");

// One part of an item: units u0 .. u1 - 1 for 256 rows of one KV head.
struct Part {
  int u0, u1;           // u0 == u1: the end
  int packed, stored;   // units and tokens of complete blocks
  int L, n, row0;       // the sequence's tokens, new rows and first row
  int row;              // the item's first row among the sequence's rows of a KV head
  int h, s;             // KV head, and the sequence whose blocks these are
  int slot;             // partial slot, or -1: the part is the whole item
  int first, c0, cuts;  // the item's first partial slot, its first CTA, and how many CTAs follow
  int end0;             // end of the units that row tile 0 sees, in u0 .. u1
  int base;             // blocks in front of the segment's
};
static_assert(sizeof(Part) == 64, "Part");

// Over shared blocks: whether an item of so many cuts is left to the join kernel.
// Its last CTA would read the parts alone, but a few it has read before that
// kernel has started (six questions of 100 to 500 tokens behind 8192 shared ones,
// most items cut once: 306 us, 311 with all of them left).
__device__ __forceinline__ bool joined_later(int cuts) { return cuts >= 4; }

// All 512 columns of tensor memory are one CTA's: the address is 0.  Each row
// tile has 128 columns for S and 128 for O, of which D 64 leaves the second half
// free: there P has a place of its own, and the next unit's S need not wait for
// P V.  For D 128 the weights of 64 tokens lie over the start of their half of S.
constexpr uint32_t kS = 0, kO = 256;
template <int D>
struct Weights {
  static constexpr bool kApart = D == 64;
  static constexpr uint32_t kAt = kApart ? kO + 64 : kS;    // first column, and the tile's 128 t
  static constexpr uint32_t kHalf = kApart ? 32 : 64;       // columns from one half's weights to the other's
};

enum Bar {
  kQFull, kKFull, kKEmpty = kKFull + 2, kVFull = kKEmpty + 2, kVEmpty = kVFull + 2, kSFull = kVEmpty + 2,
  kPFull = kSFull + 2, kOFull = kPFull + 2, kPartFull = kOFull + 2, kPartFree = kPartFull + kParts,
  kMetaFull = kPartFree + kParts, kMetaFree = kMetaFull + kMetas, kDrained = kMetaFree + kMetas, kBars
};
static_assert(kBars <= 48, "barriers");

// ------------------------------------------------------------ tcgen05 in PTX

__device__ __forceinline__ void tmem_alloc(uint32_t smem_dst) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_dst) : "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Shared-memory matrix descriptors, 128-byte swizzle: 8-row groups of 1024
// bytes follow each other; `lead` is the step between 64-element halves of an
// MN-major operand (K-major operands do not use it).  The high words are the
// same for all; desc_lo gives the low one, to which byte offsets / 16 add.
constexpr uint32_t kDescHi = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lead) {
  return ((addr >> 4) & 0x3fff) | (lead >> 4 << 16);
}

// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)), "n"(kDescHi)
      : "memory");
}
// D[tmem] (+)= A[tmem] B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.u32 p, %4, 0;\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(static_cast<uint32_t>(add)), "n"(kDescHi)
      : "memory");
}

#define KV8_R8(v, i) "=r"(v[i]), "=r"(v[i + 1]), "=r"(v[i + 2]), "=r"(v[i + 3]), "=r"(v[i + 4]), "=r"(v[i + 5]), "=r"(v[i + 6]), "=r"(v[i + 7])
#define KV8_X8(v, i) "+r"(v[i]), "+r"(v[i + 1]), "+r"(v[i + 2]), "+r"(v[i + 3]), "+r"(v[i + 4]), "+r"(v[i + 5]), "+r"(v[i + 6]), "+r"(v[i + 7])
#define KV8_W8(v, i) "r"(v[i]), "r"(v[i + 1]), "r"(v[i + 2]), "r"(v[i + 3]), "r"(v[i + 4]), "r"(v[i + 5]), "r"(v[i + 6]), "r"(v[i + 7])

// Waits for this thread's loads from tensor memory; the registers go through
// it, so that nothing touches them before.
__device__ __forceinline__ void wait_ld32(uint32_t *v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : KV8_X8(v, 0), KV8_X8(v, 8), KV8_X8(v, 16), KV8_X8(v, 24)::"memory");
}
__device__ __forceinline__ void wait_ld16(uint32_t *v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : KV8_X8(v, 0), KV8_X8(v, 8)::"memory");
}

// 32 columns of the warp's 32 lanes
__device__ __forceinline__ void tmem_ld32(uint32_t *v, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : KV8_R8(v, 0), KV8_R8(v, 8), KV8_R8(v, 16), KV8_R8(v, 24)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t *v, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : KV8_R8(v, 0), KV8_R8(v, 8)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      KV8_W8(v, 0), KV8_W8(v, 8)
      : "memory");
}

// kind::f16 with fp16 operands and fp32 accumulators, M = 128
__host__ __device__ constexpr uint32_t instr_desc(int n, bool b_mn_major) {
  return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(n / 8) << 17) | (8u << 24);
}

__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// A barrier of `threads` threads that says whether `ok` held for all of them.
__device__ __forceinline__ bool bar_all(int id, int threads, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(ok))
      : "memory");
  return r != 0;
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void sts16(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t pack64(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack64(uint64_t v, float &x, float &y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Place of 16-byte chunk cc (8 channels) of row `row` in a tile.
__device__ __forceinline__ uint32_t place(int row, int cc) {
  return (cc >> 3) * 16384 + row * 128 + (((cc & 7) ^ (row & 7)) << 4);
}

// ------------------------------------------------------------------- the line

// A (sequence, row tile pair): what its items share.
struct Pair {
  Seg q;
  int s, rt;
  int last_seen;  // last position that any of its rows sees (at least 0)
  int stored;     // tokens in complete blocks
  int packed;     // units of complete blocks
  int units;      // and one for the window, where seen; 0: not a pair
  int units0;     // those that row tile 0 sees
};

// (SHARED: a start behind the rows, where a range is invalid, must not move the
// slots of others)
template <bool SHARED>
__device__ __forceinline__ int row_start_of(const AttnArgs &a, int s) {
  if (SHARED && a.part == kPrefix) s = min(max(a.group_start[s], 0), a.geo.S);
  if (!a.row_start) return s;
  return SHARED ? min(max(a.row_start[s], 0), a.rows) : max(a.row_start[s], 0);
}

template <bool SHARED>
__device__ __forceinline__ Pair make_pair(const AttnArgs &a, int s, int rt) {
  Pair p;
  p.s = s;
  p.rt = rt;
  p.units = 0;
  if (!KVQ_IN_BOUNDS(a.geo.status, s, a.segs)) return p;
  p.q = load_seg<SHARED>(a, s);
  const int L = p.q.L;
  const int n_rows = p.q.n * a.group;
  if (n_rows <= kRowsMax || L <= 0 || L > a.max_len || rt < 0 || rt * kRows >= n_rows) return p;
  const int last_row = min((rt + 1) * kRows, n_rows) - 1;
  p.last_seen = max(last_seen(a, p.q, last_row / a.group), 0);
  p.stored = L / a.geo.B * a.geo.B;
  p.packed = min(p.last_seen / kKeys + 1, (p.stored + kKeys - 1) / kKeys);
  p.units = p.packed + (p.last_seen >= p.stored ? 1 : 0);
  const int last_seen0 = max(last_seen(a, p.q, min(rt * kRows + 127, last_row) / a.group), 0);
  p.units0 = min(last_seen0 / kKeys + 1, p.packed) + (last_seen0 >= p.stored ? 1 : 0);
  return p;
}

// Sequence s owns the slots from row_start[s] * group / 256 + s on: at least
// as many as row tile pairs.
template <bool SHARED>
__device__ __forceinline__ Pair pair_of_slot(const AttnArgs &a, int slot) {
  auto base = [&](int s) {
    return static_cast<int>(static_cast<long long>(row_start_of<SHARED>(a, s)) * a.group / kRows) + s;
  };
  const int s = last_at_or_below(a.segs, slot, base);
  return make_pair<SHARED>(a, s, slot - base(s));
}

static_assert(64 + 8 * (kThreads / 32) + sizeof(Pair) <= 384, "a pair's place beside the barriers");

// An item's kOver + units line positions; unit u is at start + kOver + u.
template <bool SHARED>
struct Walk {
  Pair p;
  int h, u0, u1;    // KV head and units of the current part
  long long start;  // the item's first line position
  long long lo, end;

  // the part of the range in this item; false: the range ends before its units
  __device__ __forceinline__ bool part() {
    const long long first = start + kOver;
    u0 = static_cast<int>(max(lo - first, 0ll));
    u1 = static_cast<int>(min(static_cast<long long>(p.units), end - first));
    return u1 > u0;
  }
  __device__ __forceinline__ bool next(const AttnArgs &a) {
    start += kOver + p.units;
    if (start + kOver >= end) return false;
    if (++h >= a.geo.H) {
      h = 0;
      int s = p.s, rt = p.rt + 1;
      for (;;) {
        p = make_pair<SHARED>(a, s, rt);
        if (p.units) break;
        rt = 0;
        if (++s >= a.segs) return false;
      }
    }
    return part();
  }
};
// Line positions of a pair's items.
__device__ __forceinline__ long long line_of(const Pair &p, int H) {
  return p.units ? static_cast<long long>(p.units + kOver) * H : 0;
}

// Sum over the CTA, and each thread's exclusive prefix.
__device__ __forceinline__ long long cta_scan(long long v, long long &before, long long *buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(kAll, incl, o);
    if (lane >= o) incl += x;
  }
  __syncthreads();
  if (lane == 31) buf[warp] = incl;
  __syncthreads();
  long long total = 0;
  before = incl - v;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += buf[w];
    total += buf[w];
  }
  return total;
}

// --------------------------------------------------------------- code widening

template <int FMT>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi) {
  if (FMT == KV8_INT8) {
    const uint32_t u = w ^ 0x80808080u;
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __floats2half2_rn(1152.f, 1152.f);
    lo = kvq::h2_as_u32(__hsub2(*reinterpret_cast<__half2 *>(&a), off));
    hi = kvq::h2_as_u32(__hsub2(*reinterpret_cast<__half2 *>(&b), off));
  } else {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

// Bits of the largest magnitude of eight bf16 numbers (a row with an infinity
// or a NaN gives NaN whatever its scale).
__device__ __forceinline__ uint32_t mag_max8(const uint4 &x) {
  const uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                              __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}

// Eight bf16 numbers, scaled, as fp16.
__device__ __forceinline__ uint4 bf16_row_to_fp16(uint4 x, float f) {
  uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = unpack2<true>(e[i]);
    e[i] = kvq::h2_as_u32(__floats2half2_rn(y.x * f, y.y * f));
  }
  return make_uint4(e[0], e[1], e[2], e[3]);
}

// The largest z' = S k + log2(scale_v) of 64 columns of a row, from group g of 32
// on (EDGE: of the first cmax).  In a window S holds z' already.
template <bool EDGE>
__device__ __forceinline__ float unit_max(std::integral_constant<bool, EDGE>, uint32_t s_at, int g, const Meta &meta,
                                          float qf, bool window, int cmax) {
  const float ninf = __int_as_float(0xff800000);
  float mx = ninf;
#pragma unroll 1
  for (int c = g; c < g + 2; ++c) {
    uint32_t s[32];
    tmem_ld32(s, s_at + 32 * c);
    wait_ld32(s);
    const float k = EDGE && window ? 1.f : meta.k[c] * qf, lv = EDGE && window ? 0.f : meta.lv[c];
    float m[4] = {ninf, ninf, ninf, ninf};
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      float x = __uint_as_float(s[i]), y = __uint_as_float(s[i + 1]);
      if (EDGE) {
        const int col = 32 * c + i;
        x = col < cmax ? x : ninf;
        y = col + 1 < cmax ? y : ninf;
      }
      m[i / 2 & 3] = fmaxf(fmaxf(m[i / 2 & 3], x), y);
    }
    mx = fmaxf(mx, fmaf(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), k, lv));
  }
  return mx;
}

// Weights 2^(z' - ref) of those columns as fp16 from column p_at on; their sum
// over scale_v.  (A unit with values that count as zeros is EDGE too.)
template <bool EDGE>
__device__ __forceinline__ float unit_weights(std::integral_constant<bool, EDGE>, uint32_t s_at, uint32_t p_at, int g,
                                              const Meta &meta, float qf, float ref, bool window, int cmax) {
  const float ninf = __int_as_float(0xff800000);
  float l = 0.f;
#pragma unroll 1
  for (int c = g; c < g + 2; ++c) {
    uint32_t s[32];
    tmem_ld32(s, s_at + 32 * c);
    wait_ld32(s);
    const float k = EDGE && window ? 1.f : meta.k[c] * qf;
    // values that count as zeros (their place in V holds zeros): no scale, and
    // weights that fp16 need not hold
    const bool zero = EDGE && !window && (meta.flush >> c & 1);
    const float bias = (EDGE && window ? 0.f : EDGE && zero ? meta.lv[c] - kZeroLog : meta.lv[c]) - ref;
    const uint64_t a2 = pack64(k, k), b2 = pack64(bias, bias);
    uint64_t sum[2] = {pack64(0.f, 0.f), pack64(0.f, 0.f)};
    uint32_t pk[16];
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      float x, y;
      unpack64(fma2(pack64(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), a2, b2), x, y);
      if (EDGE) {
        const int col = 32 * c + i;
        x = col < cmax ? x : ninf;
        y = col + 1 < cmax ? y : ninf;
      }
      x = kvq::fast_exp2(x);
      y = kvq::fast_exp2(y);
      pk[i / 2] = kvq::h2_as_u32(__floats2half2_rn(x, y));
      sum[i / 2 & 1] = add2(sum[i / 2 & 1], pack64(x, y));
    }
    float x, y;
    unpack64(add2(sum[0], sum[1]), x, y);
    l = fmaf(x + y, EDGE && window ? 1.f : meta.inv[c], l);
    if (EDGE && zero) {
#pragma unroll
      for (int i = 0; i < 16; ++i) pk[i] = 0u;
    }
    tmem_st16(p_at + 16 * (c - g), pk);
  }
  return l;
}

template <int D, int FMT, bool BF16, bool SHARED>
__global__ void __launch_bounds__(kThreads, 1) tiles_kernel(const AttnArgs a) {
  using SM = Smem<D>;
  extern __shared__ unsigned char raw[];
  start<SHARED>(a);
  unsigned char *smem = raw + ((1024 - (kvq::smem_u32(raw) & 1023)) & 1023);
  const uint32_t base = kvq::smem_u32(smem);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + SM::BAR);
  volatile int *dead = reinterpret_cast<volatile int *>(smem + SM::MISC);       // a wait gave up
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + SM::MISC + 8);
  int *flag = reinterpret_cast<int *>(smem + SM::MISC + 16);
  long long *found = reinterpret_cast<long long *>(smem + SM::MISC + 32);       // where the range begins in its pair
  Pair *found_pair = reinterpret_cast<Pair *>(smem + SM::MISC + 64 + 8 * (kThreads / 32));
  long long *scan_buf = reinterpret_cast<long long *>(smem + SM::MISC + 64);    // [kThreads / 32]
  const Geo &geo = a.geo;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = geo.B, H = geo.H;
  const float ninf = __int_as_float(0xff800000), nan = __int_as_float(0x7fc00000);

  // ---- this CTA's range of the line
  long long total = 0, before = 0;
  const long long last_row = min(row_start_of<SHARED>(a, a.segs), a.rows);
  const int slots = static_cast<int>(last_row * a.group / kRows) + a.segs;
  Pair mine;
  {
    // The slots below need row_start, and group_start, to rise: the line is counted
    // by slots and walked by segments, and where the two differ CTAs disagree on
    // an item's parts, counters stay set and places lie behind the last.
    // (SHARED: the lookup has found out.  Its words are asked for first and used
    // last, and a fall makes the line's sum longer than any line: no wait and no
    // barrier of its own, which would cost short calls 1 us)
    constexpr long long kFalls = 1ll << 53;
    int fell = SHARED && tid < a.fall_words ? __ldcg(a.falls + tid) : 0;
    bool falls = false;
    if (!SHARED && a.row_start)
      for (int s = tid; s < geo.S; s += kThreads)
        falls |= a.row_start[s] < 0 || a.row_start[s + 1] < a.row_start[s] || a.row_start[s + 1] > a.rows;
    if (!SHARED && __syncthreads_or(falls)) return;  // the rows kernel has set the status
    long long sum = 0;
    for (int i = tid; i < slots; i += kThreads) {
      mine = pair_of_slot<SHARED>(a, i);
      sum += line_of(mine, H);
    }
    if (SHARED) {
      for (int i = tid + kThreads; i < a.fall_words; i += kThreads) fell |= __ldcg(a.falls + i);
      if (fell) sum = kFalls;
    }
    total = cta_scan(sum, before, scan_buf);
    if (SHARED && total >= kFalls) total = 0;
  }
  if (total == 0) return finish<SHARED>();
  // Eight line positions per CTA at least.  Long lines, from 1216 on, do not
  // meet this; short ones would be faster with four (8 KV heads x 4 queries,
  // D 128: a prompt of 256 tokens 28.9 against 20.6 us, of 512 34.6 against 25.4,
  // a chunk of 128 over 2000 42.1 against 35.2) and slower with sixteen (47.6,
  // 49.8, 55.9); kv8_attn keeps the parts, and with them the bits, that it had.
  // The other calls take four (10 sequences of 37 to 63 rows x 4 KV heads x 7 over
  // 1 to 4 tokens: 32 against 22 us).  Over shared blocks two: their parts are
  // joined by another kernel, by all SMs.
  const int least = !SHARED ? 8 : a.part == kPrefix ? 2 : 4;
  const int ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), (total + least - 1) / least));
  if (static_cast<int>(blockIdx.x) >= ctas) return finish<SHARED>();
  const long long lo = divide(blockIdx.x * total, ctas), hi = divide((blockIdx.x + 1) * total, ctas);
  {
    long long at = 0;
    for (int i0 = 0; i0 < slots; i0 += kThreads) {
      long long sum = total;
      if (slots > kThreads) {  // else each thread has its only pair, and its place on the line
        if (i0 + tid < slots) mine = pair_of_slot<SHARED>(a, i0 + tid);
        sum = cta_scan(i0 + tid < slots ? line_of(mine, H) : 0, before, scan_buf);
      }
      const long long u = i0 + tid < slots ? line_of(mine, H) : 0;
      if (lo >= at + before && lo < at + before + u) {
        *found = lo - (at + before);
        *found_pair = mine;
      }
      at += sum;
      if (lo < at) break;
    }
  }
  if (tid == 0) {
    *dead = 0;
    kvq::mbar_init(bars + kQFull, 512);
    kvq::mbar_init(bars + kDrained, 1);
    for (int i = 0; i < kParts; ++i) {
      kvq::mbar_init(bars + kPartFull + i, 1);
      kvq::mbar_init(bars + kPartFree + i, 18);  // sixteen softmax warps, the products, the tables
    }
    for (int i = 0; i < kMetas; ++i) {
      kvq::mbar_init(bars + kMetaFull + i, 1);
      kvq::mbar_init(bars + kMetaFree + i, 1);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      kvq::mbar_init(bars + kKFull + i, 128);
      kvq::mbar_init(bars + kKEmpty + i, 1);
      kvq::mbar_init(bars + kVFull + i, 128);
      kvq::mbar_init(bars + kVEmpty + i, 1);
      kvq::mbar_init(bars + kSFull + i, 1);
      kvq::mbar_init(bars + kPFull + i, 256);
      kvq::mbar_init(bars + kOFull + i, 1);
    }
    kvq::fence_mbar_init();
  }
  if (warp == 20) {
    tmem_alloc(kvq::smem_u32(tmem_slot));
    tmem_relinquish();
  }
  fence_before();
  __syncthreads();
  fence_after();

  Part *const parts = reinterpret_cast<Part *>(smem + SM::PART);
  Meta *const metas = reinterpret_cast<Meta *>(smem + SM::META);
  // A wait of a role; false ends the role (another one's wait ran out, or this).
  // A limit below a poll's 100 us holds to within that.
  // The polls suspend the warp for long: what it issues is missing to others
  // (a chunk of 2048 tokens over 8192: 229 against 243 us with short polls).
  auto wait = [&](int bar, uint32_t parity) -> bool {
    if (kvq::mbar_try_wait(bars + bar, parity)) return true;
    const long long since = clock64();
    while (!kvq::mbar_try_wait_hint(bars + bar, parity, 100000u)) {
      if (*dead) return false;
      if (clock64() - since > a.wait_limit) {
        *dead = 1;
        set_status(geo.status, KVQ_STATUS_TIMEOUT);
        return false;
      }
    }
    return true;
  };
  // The same for all `threads` threads of a role: its first warp polls, the
  // others wait at barrier `id`.  Most roles wait most of the time, and what a
  // polling warp issues is missing to the working ones.
  auto wait_all = [&](int bar, uint32_t parity, bool first, int id, int threads, bool ok) -> bool {
    if (first) ok = ok && wait(bar, parity);
    return bar_all(id, threads, ok);
  };

  if (warp >= 20) {
    // 4 x 80 + 112 + 48 = 6 x 80, what the CTA was launched with
    regs_dec<48>();
    if (warp == 20) {
      // ================================================= the products
      // The whole warp goes through the loop, so that addresses and
      // descriptors are uniform, and one lane issues.  The loops over the
      // k-steps stay rolled: unrolled, their code is fetched anew for every
      // unit, among eleven other warps' code (385 against 315 us a chunk).
      const bool leader = elect_one();
      constexpr uint32_t id_qk = instr_desc(kKeys, false), id_pv = instr_desc(D, true);
      uint32_t n_unit = 0;      // units issued so far
      uint32_t np0 = 0, np1 = 0;  // weights consumed, per row tile
      auto qk = [&](int t, uint32_t unit) {
        if (leader) {
          const uint32_t qd = desc_lo(base + SM::Q + t * SM::TILE, 16);
          const uint32_t kd = desc_lo(base + SM::K + (unit & 1) * SM::TILE, 16);
#pragma unroll 2
          for (int i = 0; i < D / 16; ++i) {
            const uint32_t off = ((i >> 2) * SM::HALF + (i & 3) * 32) >> 4;
            mma_ss(kS + t * 128, qd + off, kd + off, id_qk, i != 0);
          }
          commit(base + SM::BAR + (kSFull + t) * 8);
        }
      };
      auto pv = [&](int t, uint32_t unit, bool add) {
        if (leader) {
          const uint32_t vd = desc_lo(base + SM::V + (unit & 1) * SM::TILE, SM::HALF);
#pragma unroll 2
          for (int i = 0; i < kKeys / 16; ++i)
            mma_ts(kO + t * 128, Weights<D>::kAt + t * 128 + (i >> 2) * Weights<D>::kHalf + (i & 3) * 8, vd + i * (2048 >> 4), id_pv, add || i != 0);
          commit(base + SM::BAR + (kOFull + t) * 8);
        }
      };
      auto free_stage = [&](int bar) {
        if (leader) commit(base + SM::BAR + bar * 8);
      };
      bool ok = true;
      for (uint32_t n_part = 0; ok; ++n_part) {
        ok = __all_sync(kAll, wait(kPartFull + n_part % kParts, (n_part / kParts) & 1));
        if (!ok) break;
        const Part &p = parts[n_part % kParts];
        const int units = p.u1 - p.u0, units0 = p.end0 - p.u0;  // of both row tiles, of row tile 0
        const int tiles = p.n * a.group - p.row > 128 ? 2 : 1;
        __syncwarp();
        if (leader) kvq::mbar_arrive(bars + kPartFree + n_part % kParts);
        if (units == 0) break;
        ok = __all_sync(kAll, wait(kQFull, n_part & 1) && wait(kKFull + (n_unit & 1), (n_unit >> 1) & 1));
        if (!ok) break;
        fence_after();
        for (int t = 0; t < tiles; ++t)
          if (t || units0) qk(t, n_unit);
        free_stage(kKEmpty + (n_unit & 1));
        for (int u = 0; u < units && ok; ++u, ++n_unit) {
          const bool more = u + 1 < units;
          ok = wait(kVFull + (n_unit & 1), (n_unit >> 1) & 1);
          if (more) ok = ok && wait(kKFull + ((n_unit + 1) & 1), ((n_unit + 1) >> 1) & 1);
          ok = __all_sync(kAll, ok);
          for (int t = 0; t < tiles && ok; ++t) {
            const int here = t ? units : units0;
            if (u >= here) continue;
            uint32_t &np = t ? np1 : np0;
            ok = __all_sync(kAll, wait(kPFull + t, np & 1));
            if (!ok) break;
            ++np;
            fence_after();
            if (Weights<D>::kApart && u + 1 < here) qk(t, n_unit + 1);
            pv(t, n_unit, u != 0);
            if (!Weights<D>::kApart && u + 1 < here) qk(t, n_unit + 1);
          }
          if (!ok) break;
          free_stage(kVEmpty + (n_unit & 1));
          if (more) free_stage(kKEmpty + ((n_unit + 1) & 1));
        }
      }
      if (!ok) {  // a wait ran out: no product may be left when tensor memory is given back
        if (leader) commit(base + SM::BAR + kDrained * 8);
        for (int i = 0; i < 100000 && !kvq::mbar_try_wait(bars + kDrained, 0); ++i) {
        }
      }
    } else if (warp == 21 && lane == 0) {
      // ================================================= the walk
      Walk<SHARED> use;
      use.p = *found_pair;
      use.h = static_cast<int>(divide(*found, use.p.units + kOver));
      use.start = lo - (*found - static_cast<long long>(use.h) * (use.p.units + kOver));
      use.lo = lo;
      use.end = hi;
      bool more = use.part();
      for (uint32_t n_part = 0;; ++n_part) {
        if (n_part >= kParts && !wait(kPartFree + n_part % kParts, ((n_part / kParts) & 1) ^ 1)) break;
        Part &p = parts[n_part % kParts];
        p.u0 = more ? use.u0 : 0;
        p.u1 = more ? use.u1 : 0;
        if (more) {
          p.packed = use.p.packed;
          p.stored = use.p.stored;
          p.L = use.p.q.L;
          p.n = use.p.q.n;
          p.row0 = use.p.q.row0;
          p.row = use.p.rt * kRows;
          p.h = use.h;
          p.s = use.p.q.entry;
          p.base = SHARED ? use.p.q.base : 0;
          p.slot = -1;
          p.end0 = max(min(use.u1, use.p.units0), use.u0);
          if (use.u0 != 0 || use.u1 != use.p.units) {
            const long long unit0 = use.start + kOver;
            auto owner = [&](long long pos) { return static_cast<int>(divide((pos + 1) * ctas - 1, total)); };
            const int c0 = owner(unit0);
            p.c0 = c0;
            p.cuts = owner(unit0 + use.p.units - 1) - c0;
            // a CTA has partial slots for its range's first part and its last one
            p.slot = 2 * blockIdx.x + (lo < use.start ? 1 : 0);
            p.first = 2 * c0 + (divide(c0 * total, ctas) < use.start ? 1 : 0);
          }
          // for the kernel that joins them (a CTA begins one such item at most, its last)
          if (SHARED && a.part == kPrefix && use.u0 == 0 && p.slot >= 0 && joined_later(p.cuts)) {
            a.items[2 * blockIdx.x] = make_int4(p.first, p.cuts + 1, p.h, p.row);
            a.items[2 * blockIdx.x + 1] = make_int4(p.row0, p.n * a.group, 0, 0);
          }
        }
        kvq::mbar_arrive(bars + kPartFull + n_part % kParts);
        if (!more) break;
        more = use.next(a);
      }
    } else if (warp == 22) {
      // ================================================= blocks and scales
      uint32_t n_unit = 0;
      bool ok = true;
      auto slot_free = [&]() {
        if (n_unit >= kMetas) ok = __all_sync(kAll, wait(kMetaFree + n_unit % kMetas, ((n_unit / kMetas) & 1) ^ 1));
        return ok;
      };
      auto publish = [&]() {
        __syncwarp();
        if (lane == 0) kvq::mbar_arrive(bars + kMetaFull + n_unit % kMetas);
        ++n_unit;
      };
      for (uint32_t n_part = 0; ok; ++n_part) {
        ok = __all_sync(kAll, wait(kPartFull + n_part % kParts, (n_part / kParts) & 1));
        if (!ok) break;
        const Part p = parts[n_part % kParts];
        __syncwarp();
        if (lane == 0) kvq::mbar_arrive(bars + kPartFree + n_part % kParts);
        // eight units at a time, a lane per group of 32 tokens
        for (int u = p.u0; u < p.u1 && ok; u += 8) {
          const int mu = u + (lane >> 2), tok = mu * kKeys + (lane & 3) * 32;
          long long off = 0;
          bool none = true;
          float2 sc = make_float2(1.f, 1.f);
          if (mu < min(p.packed, p.u1) && tok < p.stored) {
            const int at = SHARED ? p.base + tok / B : tok / B;
            const bool listed = KVQ_IN_BOUNDS(geo.status, p.s, geo.S) && KVQ_IN_BOUNDS(geo.status, at, geo.max_blocks);
            const int e = listed ? geo.table[static_cast<size_t>(p.s) * geo.max_blocks + at] : -1;
            if (e >= 0 && e < geo.num_blocks) {
              const long long bh = static_cast<long long>(e) * H + p.h;
              off = bh * 2 * B * D + (tok & (B - 1)) * D;
              none = false;
              sc = *reinterpret_cast<const float2 *>(geo.scales + bh * 2);
            } else {
              set_status(geo.status, KVQ_STATUS_BAD_BLOCK);
              sc = make_float2(nan, nan);
            }
          }
          const float inf = __int_as_float(0x7f800000);
          const bool bad = !(fabsf(sc.x) < inf && fabsf(sc.y) < inf);
          // zeros may have any scale
          const bool zero = !bad && sc.y < kZeroScale;
          const unsigned flushes = __ballot_sync(kAll, none || zero);
          const float lv = bad ? nan : zero ? kZeroLog : log2f(sc.y), inv = bad || zero ? 1.f : 1.f / sc.y;
          for (int i = 0; i < 8 && u + i < p.u1; ++i) {
            if (!slot_free()) break;
            Meta &m = metas[n_unit % kMetas];
            if (lane >> 2 == i) {
              const int gr = lane & 3;
              m.off[gr] = off;
              m.k[gr] = bad ? 1.f : sc.x;
              m.lv[gr] = lv;
              m.inv[gr] = inv;
              if (gr == 0) {
                m.kind = mu < p.packed ? kPacked : kWindow;
                m.valid = p.L - p.stored;
                m.flush = (flushes >> (4 * i)) & 15;
                m.win = (static_cast<long long>(p.s) * H + p.h) * B * D;
              }
            }
            publish();
          }
        }
        if (p.u0 == p.u1) {
          if (slot_free()) {
            if (lane == 0) metas[n_unit % kMetas].kind = kEnd;
            publish();
          }
          break;
        }
      }
    }
  } else if (warp >= 16) {
    // =================================================== keys and values
    regs_inc<112>();
    const int ct = tid & 127;
    // Four threads take 64 bytes of a token, a warp eight tokens: with the
    // swizzle, eight threads' 16-byte stores meet eight bank groups.
    constexpr int CH = D / 64;                 // 64-byte pieces of a token's codes
    constexpr int NI = 4 * CH;                 // pieces per thread
    const int cr = ct >> 2, cc = ct & 3;       // token among 32, 16-byte chunk of the piece
    const uint32_t at0 = place(cr, 2 * cc), at1 = place(cr, 2 * cc + 1);
    uint4 kb[NI], vb[NI];

    const uint8_t *const codes = geo.codes + cr * D + cc * 16;
    auto load = [&](uint4 *buf, const Meta &m, int values) {
      const uint8_t *src = codes + values * B * D;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (!KVQ_IN_BOUNDS(geo.status, m.off[i / CH] + (values * B + cr) * D + cc * 16 + (i % CH) * 64,
                           static_cast<long long>(geo.num_blocks) * H * 2 * B * D - 15))
          continue;
        buf[i] = __ldg(reinterpret_cast<const uint4 *>(src + m.off[i / CH] + (i % CH) * 64));
      }
    };
    auto store = [&](uint32_t dst, const uint4 *buf) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        uint32_t e[8];
        widen4<FMT>(buf[i].x, e[0], e[1]);
        widen4<FMT>(buf[i].y, e[2], e[3]);
        widen4<FMT>(buf[i].z, e[4], e[5]);
        widen4<FMT>(buf[i].w, e[6], e[7]);
        const uint32_t at = dst + (i / CH) * 4096 + (i % CH) * SM::HALF;
        sts16(at + at0, e[0], e[1], e[2], e[3]);
        sts16(at + at1, e[4], e[5], e[6], e[7]);
      }
    };
    // One window token (thread ct's) of keys or values: what scales it.
    auto window_row = [&](const uint16_t *src, bool valid, float &f, bool &bad) {
      uint32_t big = 0;
      bad = false;
      f = 1.f;
      if (!valid) return;
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        const uint4 x = *reinterpret_cast<const uint4 *>(src + 8 * c);
        const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t lo16 = e[i] & 0x7fffu, hi16 = (e[i] >> 16) & 0x7fffu;
          if (lo16 >= nonfinite_bits<BF16>() || hi16 >= nonfinite_bits<BF16>()) bad = true;
          big = max(big, lo16 < nonfinite_bits<BF16>() ? lo16 : 0u);
          big = max(big, hi16 < nonfinite_bits<BF16>() ? hi16 : 0u);
        }
      }
      // a power of two that brings the largest element to [2^14, 2^15); elements
      // below 2^-67, zeros too, count as that, so that sums of f times weights
      // stay finite
      if (BF16) f = __int_as_float((268 - max(static_cast<int>(big >> 7), 60)) << 23);
    };
    auto store_window = [&](uint32_t dst, const uint16_t *src, bool zero, float f) {
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (!zero) x = *reinterpret_cast<const uint4 *>(src + 8 * c);
        if (BF16) x = bf16_row_to_fp16(x, f);
        sts16(dst + place(ct, c), x.x, x.y, x.z, x.w);
      }
    };

    const bool first = warp == 16;
    bool ok = true;
    int kind = kEnd;
    if (wait_all(kMetaFull, 0, first, 1, 128, true)) {
      kind = metas[0].kind;
      if (kind == kPacked) {
        load(kb, metas[0], 0);
        load(vb, metas[0], 1);
      }
    }
    for (uint32_t n_unit = 0; kind != kEnd; ++n_unit) {
      const int st = n_unit & 1;
      const uint32_t reuse = ((n_unit >> 1) & 1) ^ 1;  // the stage's previous user must be done
      const uint32_t kd = base + SM::K + st * SM::TILE, vd = base + SM::V + st * SM::TILE;
      const Meta &m = metas[n_unit % kMetas], &m1 = metas[(n_unit + 1) % kMetas];
      float vf = 1.f;
      bool vzero = true;
      if (n_unit >= 2 && !wait_all(kKEmpty + st, reuse, first, 1, 128, true)) break;
      // test aid: the second unit's keys wait for what only a give-up brings about
      if (n_unit == 1 && a.wait_test && !wait_all(kDrained, 0, first, 1, 128, true)) break;
      if (kind == kPacked) {
        store(kd, kb);
      } else {
        float *col = reinterpret_cast<float *>(smem + SM::COL) + (n_unit % kCols) * 3 * kKeys + ct;
        const uint16_t *ks = geo.k_win + m.win + ct * D, *vs = geo.v_win + m.win + ct * D;
        const bool valid = ct < m.valid && KVQ_IN_BOUNDS(geo.status, ct, B) &&
                           KVQ_IN_BOUNDS(geo.status, m.win / (B * D), static_cast<long long>(geo.S) * H);
        float kf;
        bool kbad, vbad;
        window_row(ks, valid, kf, kbad);
        window_row(vs, valid, vf, vbad);
        store_window(kd, ks, !valid, kf);
        vzero = !valid || vbad;
        col[0] = 1.f / kf;
        // tokens that are not finite turn the rows that see them to NaN
        col[kKeys] = kbad || vbad ? nan : -log2f(vf);
        col[2 * kKeys] = kbad || vbad ? 0.f : log2f(vf);
      }
      kvq::fence_proxy_async();
      kvq::mbar_arrive(bars + kKFull + st);
      if (ct == 0 && n_unit >= 3) kvq::mbar_arrive(bars + kMetaFree + (n_unit - 3) % kMetas);
      // the next unit's keys, and its values once this one's are stored
      if (first) {
        ok = wait(kMetaFull + (n_unit + 1) % kMetas, ((n_unit + 1) / kMetas) & 1);
        if (ok && n_unit >= 2) ok = wait(kVEmpty + st, reuse);
      }
      if (!bar_all(1, 128, ok)) break;
      const int next = m1.kind;
      if (next == kPacked) load(kb, m1, 0);
      if (kind == kPacked) {
        const int flush = m.flush;  // groups of 32 tokens whose values are stored as zeros
        if (flush) {
#pragma unroll
          for (int i = 0; i < NI; ++i)
            if (flush >> (i / CH) & 1) vb[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        store(vd, vb);
      } else {
        store_window(vd, geo.v_win + m.win + ct * D, vzero, vf);
      }
      kvq::fence_proxy_async();
      kvq::mbar_arrive(bars + kVFull + st);
      if (next == kPacked) load(vb, m1, 1);
      kind = next;
    }
  } else {
    // =================================================== softmax
    const int t = warp >> 3;         // row tile
    const int hf = warp >> 2 & 1;    // half of a unit's keys, of a row's channels, of the warp's rows
    const int r = tid & 127;         // row of the tile = lane of tensor memory
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const uint32_t s_at = lanes + kS + t * 128, o_at = lanes + kO + t * 128;
    const uint32_t p_at = lanes + Weights<D>::kAt + t * 128 + hf * Weights<D>::kHalf;
    uint32_t n_unit = 0;  // units so far
    uint32_t n_own = 0;   // units of this row tile so far
    // copies of whole rows: LPR lanes a row, RPI rows at a time, NQ times for the warp's 32
    // (two warps share the 32 rows)
    constexpr int LPR = D / 8, RPI = 32 / LPR, NQ = 16 / RPI;
    const int i0 = hf * NQ;
    float *const maxima = reinterpret_cast<float *>(smem + SM::ROW) + t * 128 + r;  // [unit parity][half][kRows]
    int *const exps = reinterpret_cast<int *>(smem + SM::ROW) + 4 * kRows + t * 128;
    float *const sums = reinterpret_cast<float *>(smem + SM::ROW) + 4 * kRows + t * 128 + r;  // [half][kRows]
    bool ok = true;
    for (uint32_t n_part = 0;; ++n_part) {
      // all sixteen warps go on together, or leave together
      ok = wait_all(kPartFull + n_part % kParts, (n_part / kParts) & 1, warp == 0, 2, 512, ok);
      if (!ok) break;
      const Part &p = parts[n_part % kParts];
      const int u0 = p.u0, u1 = p.u1;
      if (u0 == u1) break;
      const int end = t ? u1 : p.end0;  // behind the units that the row tile sees
      const int n_rows = p.n * a.group;
      const int row = p.row + t * 128 + r;
      const bool active = n_rows - p.row > t * 128;  // the tile has rows
      const bool valid = row < n_rows;
      const int some = min(row, n_rows - 1);  // rows behind the last one compute what it does
      const int tok = some / a.group;
      const int lim = valid ? last_seen(a, p, tok) : -1;  // last position the row sees

      // ---- the warp's 32 queries to shared memory: LPR lanes bring a row
      const long long head = static_cast<long long>(p.h) * a.group + some - tok * a.group;
      const bool inside = row_in_bounds(a, p.row0, p.h, some);
      const long long q_off = inside ? (static_cast<long long>(p.row0) + tok) * a.q.row + head * a.q.head : 0;
      float qf = a.zscale;
      if (active) {
        const uint32_t dst = base + SM::Q + t * SM::TILE;
        // (half of them at a time: their code runs once per item, and comes from far)
        constexpr int NB = NQ / 2;
#pragma unroll 1
        for (int i1 = i0; i1 < i0 + NQ; i1 += NB) {
          uint4 x[NB];
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            const long long off = __shfl_sync(kAll, q_off, (i1 + i) * RPI + lane / LPR);
            x[i] = *reinterpret_cast<const uint4 *>(a.q.p + off + lane % LPR * 8);
          }
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            const int at = 32 * (warp & 3) + (i1 + i) * RPI + lane / LPR;  // row of the tile
            if (BF16) {
              uint32_t big = mag_max8(x[i]);
#pragma unroll
              for (int o = 1; o < LPR; o <<= 1) big = max(big, __shfl_xor_sync(kAll, big, o));
              const int e = big ? min(max(static_cast<int>(big >> 7), 20), 254) : 141;
              x[i] = bf16_row_to_fp16(x[i], __int_as_float((268 - e) << 23));
              if (lane % LPR == 0) exps[at] = e;
            }
            sts16(dst + place(at, lane % LPR), x[i].x, x[i].y, x[i].z, x[i].w);
          }
        }
        if (BF16) {
          bar_sync(3 + t, 256);
          qf *= __int_as_float((exps[r] - 14) << 23);
        }
        kvq::fence_proxy_async();
      }
      fence_before();
      kvq::mbar_arrive(bars + kQFull);

      float M = ninf, l = 0.f;
      if (active) {
        // every row of the tile sees at least the tokens up to here
        const int seen_by_all = last_seen(a, p, (p.row + t * 128) / a.group);
        for (int u = u0; u < end; ++u, ++n_unit, ++n_own) {
          ok = wait_all(kSFull + t, n_own & 1, (warp & 7) == 0, 3 + t, 256, true);
          if (!ok) break;
          fence_after();
          const Meta &meta = metas[n_unit % kMetas];
          const bool window = meta.kind == kWindow;
          const int t0 = window ? p.stored : u * kKeys;
          const int here = min(kKeys, window ? meta.valid : p.stored - t0);  // tokens of the unit
          const float *col = reinterpret_cast<const float *>(smem + SM::COL) + (n_unit % kCols) * 3 * kKeys;
          const bool edge = window || here < kKeys || t0 + kKeys - 1 > seen_by_all || meta.flush;
          const int cmax = min(here, lim - t0 + 1);  // columns below it are seen
          if (window) {
            // each token has its own scales: S becomes z + log2 scale_v in place
#pragma unroll 1
            for (int c = 64 * hf; c < 64 * hf + 64; c += 16) {
              uint32_t z[16];
              tmem_ld16(z, s_at + c);
              wait_ld16(z);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                float x = __uint_as_float(z[i]) * (col[c + i] * qf) + col[kKeys + c + i];
                x += x - x;  // an infinite score becomes NaN
                z[i] = __float_as_uint(c + i < cmax ? x : ninf);
              }
              tmem_st16(s_at + c, z);
            }
            wait_st();
          }
          // ---- the maximum
          float mx = edge ? unit_max(std::true_type{}, s_at, 2 * hf, meta, qf, window, cmax)
                          : unit_max(std::false_type{}, s_at, 2 * hf, meta, qf, window, cmax);
          float *const both = maxima + (n_own & 1) * 2 * kRows;
          both[hf * kRows] = mx;
          // the products with the last weights are done before new ones are stored
          // (given up here, the next wait for S gives up for the whole tile)
          if (Weights<D>::kApart && (warp & 7) == 0 && u > u0) wait(kOFull + t, (n_own - 1) & 1);
          bar_sync(3 + t, 256);
          if (Weights<D>::kApart) fence_after();  // orders the stores of new weights behind that wait
          mx = fmaxf(mx, both[(hf ^ 1) * kRows]);
          // ---- the reference M, and O where it moved
          const bool move = mx > M + kGrow || (M == ninf && mx > ninf);
          if (__any_sync(kAll, move)) {
            const float to = move ? mx : M;
            const float h = M == ninf ? (move ? 0.f : 1.f) : kvq::fast_exp2(0.5f * (M - to));
            const float f = h * h;
            M = to;
            l = l * h * h;  // (zeros' sums may outlive a factor that fp32 cannot hold)
            if (u > u0) {
              // (given up here, the next wait for S gives up for the whole tile)
              if (!__all_sync(kAll, wait(kOFull + t, (n_own - 1) & 1))) continue;
              fence_after();
#pragma unroll 1
              for (int c = hf * (D / 32); c < (hf + 1) * (D / 32); ++c) {
                uint32_t o[16];
                tmem_ld16(o, o_at + 16 * c);
                wait_ld16(o);
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st16(o_at + 16 * c, o);
              }
            }
          }
          const float ref = M == ninf ? 0.f : M - kShift;
          if (window) {
#pragma unroll 1
            for (int c = 64 * hf; c < 64 * hf + 64; c += 16) {
              uint32_t z[16];
              tmem_ld16(z, s_at + c);
              wait_ld16(z);
#pragma unroll
              for (int i = 0; i < 16; ++i)
                l += c + i < cmax ? kvq::fast_exp2(__uint_as_float(z[i]) - ref + col[2 * kKeys + c + i]) : 0.f;
            }
          }
          // ---- weights
          const float sum = edge ? unit_weights(std::true_type{}, s_at, p_at, 2 * hf, meta, qf, ref, window, cmax)
                                 : unit_weights(std::false_type{}, s_at, p_at, 2 * hf, meta, qf, ref, window, cmax);
          if (!window) l += sum;
          wait_st();
          fence_before();
          kvq::mbar_arrive(bars + kPFull + t);
        }
        n_unit += u1 - end;
      } else {
        n_unit += u1 - u0;
      }

      // ---- the part's result
      const int slot = p.slot;
      const bool whole = slot < 0;
      float4 *part = reinterpret_cast<float4 *>(a.tile_o) + static_cast<size_t>(max(slot, 0)) * (D / 4) * kRows +
                     t * 128 + r;
      const long long out_off = valid && inside ? (static_cast<long long>(p.row0) + tok) * a.out.row + head * a.out.head : -1;
      // Outputs go through the queries' place, which the products are done
      // with, so that whole rows are stored: 32 channels of the thread's row
      // from channel 32 c on, then the warp's rows.
      const uint32_t stage = base + SM::Q + t * SM::TILE;
      auto put = [&](int c, const float *o, float f) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          sts16(stage + place(r, 4 * c + k), pack2<BF16>(o[8 * k] * f, o[8 * k + 1] * f),
                pack2<BF16>(o[8 * k + 2] * f, o[8 * k + 3] * f), pack2<BF16>(o[8 * k + 4] * f, o[8 * k + 5] * f),
                pack2<BF16>(o[8 * k + 6] * f, o[8 * k + 7] * f));
      };
      // With shared blocks: 32 channels of the row's partial result, left for the
      // other launch, or joined with what that has left.
      auto carry_of = [&]() { return carry_row<D>(a, p.h, p.row0, min(p.row + t * 128 + r, p.n * a.group - 1)); };
      const bool leaves = SHARED && p.base, joins = SHARED && a.part == kPrefix;
      auto finish_row = [&](int c, float *o, float top, float sum) {
        if (leaves) {
          if (!valid || !inside) return;
          const CarryRow carry = carry_of();
#pragma unroll
          for (int k = 0; k < 8; ++k)
            carry.at(8 * c + k) = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          if (c == 0) *carry.ml = make_float2(top == ninf ? top : top - kShift, sum);
          return;
        }
        if (joins) wait_before();
        if (joins && valid && inside) {
          const CarryRow carry = carry_of();
          const Join n = join(make_float2(top == ninf ? top : top - kShift, sum), *carry.ml);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float4 x = carry.at(8 * c + k);
            o[4 * k] = fmaf(o[4 * k], n.x, x.x * n.y);
            o[4 * k + 1] = fmaf(o[4 * k + 1], n.x, x.y * n.y);
            o[4 * k + 2] = fmaf(o[4 * k + 2], n.x, x.z * n.y);
            o[4 * k + 3] = fmaf(o[4 * k + 3], n.x, x.w * n.y);
          }
          sum = n.sum;
        }
        put(c, o, inverse_sum(sum, lim));
      };
      auto store_rows = [&]() {
        bar_sync(3 + t, 256);
        // (a row that is not to be written)
        const bool shut = joins && out_off >= 0 && carry_of().ml->y < 0.f;
#pragma unroll 4
        for (int i = 0; i < NQ; ++i) {
          const long long off = __shfl_sync(kAll, shut ? -1 : out_off, (i0 + i) * RPI + lane / LPR);
          const uint4 x = lds16(stage + place(32 * (warp & 3) + (i0 + i) * RPI + lane / LPR, lane % LPR));
          if (off >= 0) *reinterpret_cast<uint4 *>(a.out.p + off + lane % LPR * 8) = x;
        }
      };
      if (active) {
        sums[hf * kRows] = l;
        ok = wait_all(kOFull + t, (n_own - 1) & 1, (warp & 7) == 0 && end > u0, 3 + t, 256, ok);
        l += sums[(hf ^ 1) * kRows];
      }
      if (active && ok && (whole || KVQ_IN_BOUNDS(geo.status, slot, 2 * kMaxTileCtas))) {
        fence_after();
#pragma unroll 1
        for (int c = hf * (D / 64); c < (hf + 1) * (D / 64); ++c) {
          uint32_t o[32];
          tmem_ld32(o, o_at + 32 * c);
          wait_ld32(o);
          if (whole) {
            float x[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = l == 0.f ? 0.f : __uint_as_float(o[i]);
            finish_row(c, x, M, l);
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              part[static_cast<size_t>(8 * c + i / 4) * kRows] =
                  end > u0 ? make_float4(__uint_as_float(o[i]), __uint_as_float(o[i + 1]), __uint_as_float(o[i + 2]),
                                         __uint_as_float(o[i + 3]))
                           : make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
        if (whole && !leaves)
          store_rows();
        else if (!whole && hf == 0)
          a.tile_ml[slot * kRows + t * 128 + r] = make_float2(M, l);
        fence_before();
      }
      if (!whole && !(SHARED && a.part == kPrefix && joined_later(p.cuts))) {
        ok = bar_all(2, 512, ok);
        if (!ok) break;
        if (tid == 0) {
          // releases the CTA's stores, which the barrier has ordered before, and
          // acquires the others' for the reads behind the next barrier
          const bool counted = KVQ_IN_BOUNDS(geo.status, p.c0, kMaxTileCtas) &&
                               KVQ_IN_BOUNDS(geo.status, p.c0 + p.cuts, kMaxTileCtas) &&
                               KVQ_IN_BOUNDS(geo.status, p.first, 2 * kMaxTileCtas);
          const bool last = counted && kvq::atom_add_acq_rel(a.tile_counters + p.c0, 1) == p.cuts;
          if (last) a.tile_counters[p.c0] = 0;
          *flag = last;
        }
        bar_sync(2, 512);
        const bool merge = *flag;
        bar_sync(2, 512);  // read before it is set again
        if (merge && active) {
          const int first = p.first, c0 = p.c0, n = p.cuts + 1;
#pragma unroll 1
          for (int c = hf * (D / 64); c < (hf + 1) * (D / 64); ++c) {
            float o[32], mm = ninf, ll = 0.f;
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = 0.f;
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
              const int sl = i == 0 ? first : 2 * (c0 + i);
              const float4 *src = reinterpret_cast<const float4 *>(a.tile_o) +
                                  (static_cast<size_t>(sl) * (D / 4) + 8 * c) * kRows + t * 128 + r;
              const float2 e = __ldcg(&a.tile_ml[sl * kRows + t * 128 + r]);
              float4 x[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) x[k] = __ldcg(src + static_cast<size_t>(k) * kRows);
              const float top = fmaxf(mm, e.x), ref = top == ninf ? 0.f : top;
              const float wh = kvq::fast_exp2(0.5f * (mm - ref)), fh = kvq::fast_exp2(0.5f * (e.x - ref));
              const float was = wh * wh, f = fh * fh;
              mm = top;
              ll = fmaf(ll * wh, wh, e.y * fh * fh);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                o[4 * k] = fmaf(o[4 * k], was, x[k].x * f);
                o[4 * k + 1] = fmaf(o[4 * k + 1], was, x[k].y * f);
                o[4 * k + 2] = fmaf(o[4 * k + 2], was, x[k].z * f);
                o[4 * k + 3] = fmaf(o[4 * k + 3], was, x[k].w * f);
              }
            }
            finish_row(c, o, mm, ll);
          }
          if (!leaves) store_rows();
        }
      }
      __syncwarp();
      if (lane == 0) kvq::mbar_arrive(bars + kPartFree + n_part % kParts);
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == 20) {
    fence_after();
    tmem_free(*tmem_slot);
  }
  finish<SHARED>();
}

template <int D, int FMT, bool BF16, bool SHARED>
cudaError_t launch_one(const AttnArgs &a, cudaStream_t stream) {
  auto kernel = tiles_kernel<D, FMT, BF16, SHARED>;
  static std::atomic<int> sm_count[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int sms = dev < 64 ? sm_count[dev].load() : 0;
  if (sms == 0) {
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::BYTES)) != cudaSuccess)
      return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if (dev < 64) sm_count[dev].store(sms);
  }
  if (SHARED) return launch_after(kernel, min(sms, kMaxTileCtas), kThreads, Smem<D>::BYTES, stream, a);
  kernel<<<min(sms, kMaxTileCtas), kThreads, Smem<D>::BYTES, stream>>>(a);
  return cudaGetLastError();
}

template <int D, bool SHARED>
cudaError_t launch_dim(const AttnArgs &a, cudaStream_t stream) {
  if (a.geo.fmt == KV8_INT8)
    return a.geo.bf16 ? launch_one<D, KV8_INT8, true, SHARED>(a, stream)
                      : launch_one<D, KV8_INT8, false, SHARED>(a, stream);
  return a.geo.bf16 ? launch_one<D, KV8_E4M3, true, SHARED>(a, stream)
                    : launch_one<D, KV8_E4M3, false, SHARED>(a, stream);
}

}  // namespace tiles
}  // namespace kv8
