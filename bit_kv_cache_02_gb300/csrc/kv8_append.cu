// Append to the 8-bit paged cache: rotate the new queries and keys to their
// positions, keep the newest tokens in the 16-bit window, and quantize each
// block of tokens that fills.
//
// One kernel.  A CTA takes one block of one (sequence, KV head), keys and
// values: its tokens come from the window (stored before) and from the new
// rows, stay in registers while amax is reduced over the CTA, and leave as
// codes, so every byte is read and written once.  The CTA of the first block
// also writes the window tail, after it has read the window; no other CTA
// touches that window, so nothing is ordered between CTAs.  Further CTAs
// rotate the queries.
//
// Bound: HBM.  6 bytes per key or value element of a prompt (2 + 1 moved
// twice), 4 per query element.
#include <cuda_fp8.h>

#include "kv8_internal.cuh"

namespace kv8 {
namespace {

constexpr int kThreads = 256;
constexpr int kQueryItems = 4;  // (row, head, chunk pair) items per thread of a query CTA

struct AppendArgs {
  Geo geo;
  Rows k, v, q, q_out;
  int Hq;
  const int *row_start;
  int rows, max_new;
  const float *rope;
  int rot, interleaved;
  int kv_tasks;     // CTAs that store keys and values
  int slots;        // block slots per KV head (0: one per sequence)
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

// Rotates chunk pair `pi` of one head to position `pos`.  Each product and
// sum is rounded on its own, so the result is a function of the table alone.
template <bool BF16>
__device__ __forceinline__ void rotate(uint4 &ca, uint4 &cb, int pi, int pos, const AppendArgs &a) {
  if (pi >= (a.rot >> 4)) return;
  const float *row = a.rope + static_cast<size_t>(pos) * a.rot;
  const int half = a.rot >> 1;
  if (!a.interleaved) {
    const float4 *c = reinterpret_cast<const float4 *>(row + 8 * pi);
    const float4 *s = reinterpret_cast<const float4 *>(row + half + 8 * pi);
    const float4 c0 = __ldg(c), c1 = __ldg(c + 1), s0 = __ldg(s), s1 = __ldg(s + 1);
    turn<BF16>(ca.x, cb.x, c0.x, c0.y, s0.x, s0.y);
    turn<BF16>(ca.y, cb.y, c0.z, c0.w, s0.z, s0.w);
    turn<BF16>(ca.z, cb.z, c1.x, c1.y, s1.x, s1.y);
    turn<BF16>(ca.w, cb.w, c1.z, c1.w, s1.z, s1.w);
  } else {
    const int2 ch = chunk_pair(pi, a.rot);
    const float4 ac = __ldg(reinterpret_cast<const float4 *>(row + 4 * ch.x));
    const float4 as = __ldg(reinterpret_cast<const float4 *>(row + half + 4 * ch.x));
    const float4 bc = __ldg(reinterpret_cast<const float4 *>(row + 4 * ch.y));
    const float4 bs = __ldg(reinterpret_cast<const float4 *>(row + half + 4 * ch.y));
    ca.x = turn_adjacent<BF16>(ca.x, ac.x, as.x);
    ca.y = turn_adjacent<BF16>(ca.y, ac.y, as.y);
    ca.z = turn_adjacent<BF16>(ca.z, ac.z, as.z);
    ca.w = turn_adjacent<BF16>(ca.w, ac.w, as.w);
    cb.x = turn_adjacent<BF16>(cb.x, bc.x, bs.x);
    cb.y = turn_adjacent<BF16>(cb.y, bc.y, bs.y);
    cb.z = turn_adjacent<BF16>(cb.z, bc.z, bs.z);
    cb.w = turn_adjacent<BF16>(cb.w, bc.w, bs.w);
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

// Queries: thread items (row, head, chunk pair), four in flight.
template <int D, bool BF16>
__device__ void rotate_queries(const AppendArgs &a, int cta) {
  constexpr int PAIRS = D / 16;
  const long long items = static_cast<long long>(a.rows) * a.Hq * PAIRS;
  const long long base = static_cast<long long>(cta) * kThreads * kQueryItems + threadIdx.x;
  uint4 x[kQueryItems], y[kQueryItems];
  long long off[kQueryItems];
  int pos[kQueryItems];
#pragma unroll
  for (int i = 0; i < kQueryItems; ++i) {
    const long long it = base + static_cast<long long>(i) * kThreads;
    pos[i] = -1;
    if (it >= items) continue;
    const int pi = static_cast<int>(it % PAIRS);
    const long long rh = it / PAIRS;
    const int row = static_cast<int>(rh / a.Hq), head = static_cast<int>(rh % a.Hq);
    int s = row;
    if (a.row_start) s = last_at_or_below(a.geo.S, row, [&](int j) { return a.row_start[j]; });
    if (s >= a.geo.S) continue;
    const Seq sq = load_seq(a.geo, a.row_start, a.rows, a.max_new, s);
    if (!sq.ok || row < sq.row0 || row >= sq.row0 + sq.n || sq.L < sq.n || sq.L > a.geo.capacity) continue;
    pos[i] = sq.L - sq.n + row - sq.row0;
    const int2 ch = chunk_pair(pi, a.rot);
    const uint16_t *src = a.q.p + row * a.q.row + head * a.q.head;
    x[i] = load16(src + 8 * ch.x);
    y[i] = load16(src + 8 * ch.y);
    off[i] = row * a.q_out.row + head * a.q_out.head;
  }
#pragma unroll
  for (int i = 0; i < kQueryItems; ++i) {
    if (pos[i] < 0) continue;
    const int pi = static_cast<int>((base + static_cast<long long>(i) * kThreads) % PAIRS);
    const int2 ch = chunk_pair(pi, a.rot);
    rotate<BF16>(x[i], y[i], pi, pos[i], a);
    store16(a.q_out.p + off[i] + 8 * ch.x, x[i]);
    store16(a.q_out.p + off[i] + 8 * ch.y, y[i]);
  }
}

// NI: chunk pairs of a block's keys (and of its values) per thread.
template <int D, int FMT, bool BF16, int NI>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs a) {
  constexpr int PAIRS = D / 16;
  if (static_cast<int>(blockIdx.x) >= a.kv_tasks) {
    rotate_queries<D, BF16>(a, blockIdx.x - a.kv_tasks);
    return;
  }
  const Geo &geo = a.geo;
  const int B = geo.B, tid = threadIdx.x;
  const int h = blockIdx.x % geo.H;
  int s = blockIdx.x / geo.H, t = 0;
  if (a.slots) {
    // slot -> (sequence, block): sequence s owns the slots from
    // row_start[s] / B + s on, at least as many as blocks it can complete
    const int slot = s;
    s = last_at_or_below(geo.S, slot, [&](int j) { return max(a.row_start[j], 0) / B + j; });
    t = slot - (max(a.row_start[s], 0) / B + s);
  }
  const Seq sq = load_seq(geo, a.row_start, a.rows, a.max_new, s);
  if (!sq.ok || sq.n > sq.L) {
    if (t == 0 && h == 0 && tid == 0) set_status(geo.status, KVQ_STATUS_BAD_LEN);
    return;
  }
  if (sq.L > geo.capacity) {
    if (t == 0 && h == 0 && tid == 0) set_status(geo.status, KVQ_STATUS_CAPACITY);
    return;
  }
  if (sq.n == 0) return;
  const int L = sq.L, old = L - sq.n, first = old / B, done = L / B - first;
  if (t < 0 || t >= max(done, 1)) return;
  const int p0 = (first + t) * B;  // position of the block's slot 0
  const size_t win0 = (static_cast<size_t>(s) * geo.H + h) * B * D;
  const uint16_t *kr = a.k.p + h * a.k.head, *vr = a.v.p + h * a.v.head;

  // one token's chunk pair of the block: window slot or new row, rotated
  auto load_key = [&](int slot, int pi, uint4 &x, uint4 &y) {
    const int p = p0 + slot;
    const int2 ch = chunk_pair(pi, a.rot);
    const uint16_t *src =
        p < old ? geo.k_win + win0 + slot * D : kr + static_cast<long long>(sq.row0 + p - old) * a.k.row;
    x = load16(src + 8 * ch.x);
    y = load16(src + 8 * ch.y);
  };
  auto load_value = [&](int slot, int pi, uint4 &x, uint4 &y) {
    const int p = p0 + slot;
    const uint16_t *src =
        p < old ? geo.v_win + win0 + slot * D : vr + static_cast<long long>(sq.row0 + p - old) * a.v.row;
    x = load16(src + 8 * pi);
    y = load16(src + 8 * (pi + PAIRS));
  };

  if (t < done) {
    __shared__ uint32_t red[2][kThreads / 32];
    uint4 ka[NI], kb[NI], va[NI], vb[NI];
    const int items = B * PAIRS;
    uint32_t km = 0, vm = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int it = tid + i * kThreads;
      if (it < items) {
        load_key(it / PAIRS, it % PAIRS, ka[i], kb[i]);
        load_value(it / PAIRS, it % PAIRS, va[i], vb[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int it = tid + i * kThreads;
      if (it < items) {
        const int p = p0 + it / PAIRS;
        if (p >= old) rotate<BF16>(ka[i], kb[i], it % PAIRS, p, a);
        km = mag_max(mag_max(km, ka[i]), kb[i]);
        vm = mag_max(mag_max(vm, va[i]), vb[i]);
      }
    }
    km = __reduce_max_sync(0xffffffffu, max(km & 0xffffu, km >> 16));
    vm = __reduce_max_sync(0xffffffffu, max(vm & 0xffffu, vm >> 16));
    if ((tid & 31) == 0) {
      red[0][tid >> 5] = km;
      red[1][tid >> 5] = vm;
    }
    __syncthreads();  // also: every window slot of the block has been read
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      km = max(km, red[0][w]);
      vm = max(vm, red[1][w]);
    }
    const int blk = geo.table[static_cast<size_t>(s) * geo.max_blocks + first + t];
    if (blk < 0 || blk >= geo.num_blocks) {
      if (tid == 0) set_status(geo.status, KVQ_STATUS_BAD_BLOCK);
    } else {
      const bool kbad = km >= nonfinite_bits<BF16>(), vbad = vm >= nonfinite_bits<BF16>();
      const float2 ks = scale_and_factor<FMT>(kbad ? 0.f : unpack2<BF16>(km).x);
      const float2 vs = scale_and_factor<FMT>(vbad ? 0.f : unpack2<BF16>(vm).x);
      const size_t bh = static_cast<size_t>(blk) * geo.H + h;
      uint8_t *kc = geo.codes + bh * 2 * B * D, *vc = kc + B * D;
      if (tid == 0) {
        const float nan = __int_as_float(0x7fc00000);
        *reinterpret_cast<float2 *>(geo.scales + bh * 2) = make_float2(kbad ? nan : ks.x, vbad ? nan : vs.x);
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int it = tid + i * kThreads;
        if (it < items) {
          const int slot = it / PAIRS, pi = it % PAIRS;
          const int2 ch = chunk_pair(pi, a.rot);
          *reinterpret_cast<uint2 *>(kc + slot * D + 8 * ch.x) = code8<FMT, BF16>(ka[i], ks.y, kbad);
          *reinterpret_cast<uint2 *>(kc + slot * D + 8 * ch.y) = code8<FMT, BF16>(kb[i], ks.y, kbad);
          *reinterpret_cast<uint2 *>(vc + slot * D + 8 * pi) = code8<FMT, BF16>(va[i], vs.y, vbad);
          *reinterpret_cast<uint2 *>(vc + slot * D + 8 * (pi + PAIRS)) = code8<FMT, BF16>(vb[i], vs.y, vbad);
        }
      }
    }
  }
  if (t > 0) return;

  // the tokens that stay in the window: all new ones when nothing filled,
  // else those behind the last complete block
  const int from = max(old, L / B * B);
  for (int it = tid; it < (L - from) * PAIRS; it += kThreads) {
    const int p = from + it / PAIRS, pi = it % PAIRS, slot = p % B;
    const long long row = sq.row0 + p - old;
    const int2 ch = chunk_pair(pi, a.rot);
    uint4 x = load16(kr + row * a.k.row + 8 * ch.x), y = load16(kr + row * a.k.row + 8 * ch.y);
    const uint4 z = load16(vr + row * a.v.row + 8 * pi), w = load16(vr + row * a.v.row + 8 * (pi + PAIRS));
    rotate<BF16>(x, y, pi, p, a);
    store16(geo.k_win + win0 + slot * D + 8 * ch.x, x);
    store16(geo.k_win + win0 + slot * D + 8 * ch.y, y);
    store16(geo.v_win + win0 + slot * D + 8 * pi, z);
    store16(geo.v_win + win0 + slot * D + 8 * (pi + PAIRS), w);
  }
}

template <int D, int FMT, bool BF16>
cudaError_t launch_ni(const AppendArgs &a, unsigned grid, cudaStream_t stream) {
  const int items = a.geo.B * D / 16;
  if (items <= kThreads)
    append_kernel<D, FMT, BF16, 1><<<grid, kThreads, 0, stream>>>(a);
  else if (items <= 2 * kThreads)
    append_kernel<D, FMT, BF16, 2><<<grid, kThreads, 0, stream>>>(a);
  else
    append_kernel<D, FMT, BF16, 4><<<grid, kThreads, 0, stream>>>(a);
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
  // up to B new tokens complete at most one block of a sequence
  a.slots = max_new > geo.B ? rows / geo.B + geo.S : 0;
  const long long tasks = static_cast<long long>(a.slots ? a.slots : geo.S) * geo.H;
  const long long items = static_cast<long long>(rows) * Hq * (geo.D / 16);
  const long long grid = tasks + (items + kThreads * kQueryItems - 1) / (kThreads * kQueryItems);
  if (grid > 2147483647LL) return cudaErrorInvalidConfiguration;
  a.kv_tasks = static_cast<int>(tasks);
  ++*launches;
  return geo.D == 128 ? launch_d<128>(a, static_cast<unsigned>(grid), stream)
                      : launch_d<64>(a, static_cast<unsigned>(grid), stream);
}

}  // namespace kv8
