// C ABI of the 8-bit paged KV cache (include/kv8.h): argument validation,
// sizing and dispatch.  Every entry point checks its arguments before
// anything is enqueued and returns a KVQ_ERR_* code.
#include <math.h>

#include "kv8_internal.cuh"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_geometry(const kv8_cache *c) {
  if (!c) return KVQ_ERR_INVALID_ARG;
  if (c->num_seqs < 1 || c->num_kv_heads < 1 || c->capacity < 1 || c->num_blocks < 0) return KVQ_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return KVQ_ERR_UNSUPPORTED;
  if (c->block != 32 && c->block != 64 && c->block != 128) return KVQ_ERR_UNSUPPORTED;
  if (c->format != KV8_INT8 && c->format != KV8_E4M3) return KVQ_ERR_UNSUPPORTED;
  if (c->dtype != KV8_F16 && c->dtype != KV8_BF16) return KVQ_ERR_UNSUPPORTED;
  if (c->num_seqs > 65535 || c->num_kv_heads > 65535) return KVQ_ERR_UNSUPPORTED;
  if (c->capacity > KV8_MAX_CAPACITY) return KVQ_ERR_UNSUPPORTED;  // positions are counted in 32 bits
  // (sequence, KV head) pairs are counted in 32 bits
  if (static_cast<int64_t>(c->num_seqs) * c->num_kv_heads > 2147483647LL / 2) return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

int check_buffers(const kv8_cache *c) {
  int e = check_geometry(c);
  if (e) return e;
  if (!c->k_win || !c->v_win || !c->seq_len) return KVQ_ERR_INVALID_ARG;
  if (c->capacity >= c->block && (!c->codes || !c->scales || !c->block_table || c->num_blocks < 1))
    return KVQ_ERR_INVALID_ARG;
  if (!aligned(c->codes, 16) || !aligned(c->scales, 8) || !aligned(c->k_win, 16) || !aligned(c->v_win, 16) ||
      !aligned(c->seq_len, 4) || !aligned(c->block_table, 4) || !aligned(c->status, 4))
    return KVQ_ERR_ALIGNMENT;
  return KVQ_OK;
}

int check_rows(const kv8_rows *t, int heads, int rows, int head_dim, bool written) {
  if (!t || !t->data) return KVQ_ERR_INVALID_ARG;
  if (!aligned(t->data, 16) || t->row_stride % 8 != 0 || t->head_stride % 8 != 0) return KVQ_ERR_ALIGNMENT;
  if (written && ((heads > 1 && llabs(t->head_stride) < head_dim) || (rows > 1 && llabs(t->row_stride) < head_dim)))
    return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

int check_row_range(const kv8_cache *c, const int32_t *row_start, int32_t rows, int32_t max_new) {
  if (rows < 0 || max_new < 0) return KVQ_ERR_INVALID_ARG;
  if (max_new > c->capacity) return KVQ_ERR_CAPACITY;
  if (!aligned(row_start, 4)) return KVQ_ERR_ALIGNMENT;
  // without row_start every sequence brings one row
  if (!row_start && (rows < c->num_seqs || max_new < 1)) return KVQ_ERR_INVALID_ARG;
  return KVQ_OK;
}

kv8::Geo make_geo(const kv8_cache *c) {
  kv8::Geo g;
  g.S = c->num_seqs;
  g.H = c->num_kv_heads;
  g.D = c->head_dim;
  g.B = c->block;
  g.fmt = c->format;
  g.bf16 = c->dtype == KV8_BF16;
  g.capacity = c->capacity;
  g.max_blocks = c->capacity / c->block;
  g.num_blocks = c->num_blocks;
  g.codes = c->codes;
  g.scales = c->scales;
  g.k_win = c->k_win;
  g.v_win = c->v_win;
  g.seq_len = c->seq_len;
  g.table = c->block_table;
  g.status = c->status;
  return g;
}

kv8::Rows make_rows(const kv8_rows *t) { return {t->data, t->row_stride, t->head_stride}; }

int from_cuda(cudaError_t e, uint64_t launched) {
  kvq::count_launches(launched);
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

// Hq is a multiple of Hkv and the rows of a KV head are countable in 32 bits.
int check_heads(const kv8_cache *c, int32_t num_q_heads, int32_t max_new) {
  if (num_q_heads < 1 || num_q_heads % c->num_kv_heads != 0) return KVQ_ERR_INVALID_ARG;
  const int64_t per = static_cast<int64_t>(num_q_heads / c->num_kv_heads) * max_new;
  return per > 2147483647LL / 2 ? KVQ_ERR_UNSUPPORTED : KVQ_OK;
}

// Both appends; positions NULL: tokens stand at their places in the cache.
int append(const kv8_cache *cache, const kv8_rows *k, const kv8_rows *v, const kv8_rows *q, const kv8_rows *q_out,
           int32_t num_q_heads, const int32_t *row_start, int32_t rows, int32_t max_new, const float *rope,
           int32_t rope_rows, int32_t rot_dim, int32_t interleaved, const kv8::Axes *axes, void *stream) {
  int e = check_buffers(cache);
  if (e) return e;
  if ((e = check_row_range(cache, row_start, rows, max_new))) return e;
  const bool with_q = num_q_heads != 0;
  if (num_q_heads < 0 || with_q != (q != nullptr) || with_q != (q_out != nullptr)) return KVQ_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return KVQ_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim > cache->head_dim || rot_dim % 16 != 0) return KVQ_ERR_UNSUPPORTED;
  if (rot_dim && !rope) return KVQ_ERR_INVALID_ARG;
  if (!axes && rot_dim && rope_rows < cache->capacity) return KVQ_ERR_CAPACITY;
  if (!aligned(rope, 16)) return KVQ_ERR_ALIGNMENT;
  if (rows == 0 || max_new == 0) return KVQ_OK;
  if ((e = check_rows(k, cache->num_kv_heads, rows, cache->head_dim, false))) return e;
  if ((e = check_rows(v, cache->num_kv_heads, rows, cache->head_dim, false))) return e;
  if (with_q) {
    if ((e = check_rows(q, num_q_heads, rows, cache->head_dim, false))) return e;
    if ((e = check_rows(q_out, num_q_heads, rows, cache->head_dim, true))) return e;
    if (q->data == q_out->data && (q->row_stride != q_out->row_stride || q->head_stride != q_out->head_stride))
      return KVQ_ERR_INVALID_ARG;
  }
  const kv8::Rows none = {nullptr, 0, 0};
  const kv8::Rows qr = with_q ? make_rows(q) : none, os = with_q ? make_rows(q_out) : none;
  const kv8::Geo geo = make_geo(cache);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint64_t n = 0;
  const cudaError_t ce =
      axes ? kv8::launch_append_axes(geo, make_rows(k), make_rows(v), qr, os, num_q_heads, row_start, rows, max_new,
                                     rope, rot_dim, interleaved, *axes, st, &n)
           : kv8::launch_append(geo, make_rows(k), make_rows(v), qr, os, num_q_heads, row_start, rows, max_new, rope,
                                rot_dim, interleaved, st, &n);
  return from_cuda(ce, n);
}

// What the attention calls have in common: checks, and the arguments of a launch
// over the sequences' whole lengths.
int attn_args(kv8::AttnArgs &a, const kv8_cache *cache, int32_t num_q_heads, const kv8_rows *q, const kv8_rows *out,
              const int32_t *row_start, int32_t rows, int32_t max_new, float softmax_scale, int32_t max_len) {
  int e;
  if (max_new < 1 || max_len < 1) return KVQ_ERR_INVALID_ARG;
  if ((e = check_heads(cache, num_q_heads, max_new))) return e;
  if (max_len > cache->capacity) return KVQ_ERR_CAPACITY;
  if (rows == 0) return KVQ_OK;
  if ((e = check_rows(q, num_q_heads, rows, cache->head_dim, false))) return e;
  if ((e = check_rows(out, num_q_heads, rows, cache->head_dim, true))) return e;
  if (q->data == out->data && (q->row_stride != out->row_stride || q->head_stride != out->head_stride))
    return KVQ_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || !isfinite(softmax_scale))
    softmax_scale = 1.f / sqrtf(static_cast<float>(cache->head_dim));
  a = kv8::AttnArgs{};
  a.geo = make_geo(cache);
  a.Hq = num_q_heads;
  a.group = num_q_heads / cache->num_kv_heads;
  a.part = kv8::kWhole;
  a.causal = 1;
  a.segs = cache->num_seqs;
  a.q = make_rows(q);
  a.out = make_rows(out);
  a.row_start = row_start;
  a.rows = rows;
  a.max_new = max_new;
  a.max_len = max_len;
  a.zscale = softmax_scale * 1.4426950408889634f;
  const kvq::WaitTest wt = kvq::wait_test();
  a.wait_limit = wt.limit;
  a.wait_test = wt.before_fetch;
  return KVQ_OK;
}

// The regions of one launch's workspace.
void place(kv8::AttnArgs &a, const kv8::AttnPlan &plan, void *counters, void *regions) {
  uint8_t *ws = static_cast<uint8_t *>(regions), *cnt = static_cast<uint8_t *>(counters);
  a.part_o = reinterpret_cast<float *>(ws + plan.off_o);
  a.part_ml = reinterpret_cast<float2 *>(ws + plan.off_ml);
  a.counters = reinterpret_cast<int *>(cnt + plan.off_cnt);
  a.tile_counters = reinterpret_cast<int *>(cnt + plan.off_tile_cnt);
  a.tile_o = reinterpret_cast<float *>(ws + plan.off_tile_o);
  a.tile_ml = reinterpret_cast<float2 *>(ws + plan.off_tile_ml);
  a.rows_max = plan.tiles ? kv8::kRowsMax : 2147483647;
}

int check_workspace(const void *workspace, size_t given, size_t needed) {
  if (!workspace || given < needed) return KVQ_ERR_WORKSPACE;
  return aligned(workspace, 256) ? KVQ_OK : KVQ_ERR_ALIGNMENT;
}

// The segments of whole sequences, two int4 each, and the words behind them.
size_t seg_bytes(const kv8_cache *c) {
  return (static_cast<size_t>(c->num_seqs) * 32 + kv8::fall_words(0, c->num_seqs) * sizeof(int) + 255) / 256 * 256;
}

// Attention over whole sequences in one pass.
int attend(const kv8_cache *cache, int32_t num_q_heads, const kv8_rows *q, const kv8_rows *out,
           const int32_t *row_start, int32_t rows, int32_t max_new, float softmax_scale, void *workspace,
           size_t workspace_bytes, int32_t max_len, bool causal, void *stream) {
  kv8::AttnArgs a;
  int e = attn_args(a, cache, num_q_heads, q, out, row_start, rows, max_new, softmax_scale, max_len);
  if (e || rows == 0) return e;
  const kv8::AttnPlan plan = kv8::plan_attn(cache->head_dim, static_cast<int64_t>(a.group) * max_new);
  const size_t segs = causal ? 0 : seg_bytes(cache);
  if ((e = check_workspace(workspace, workspace_bytes, plan.bytes + segs))) return e;
  a.causal = causal;
  place(a, plan, workspace, workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint64_t n = 0;
  cudaError_t ce = cudaSuccess;
  if (!causal) {
    a.plan = reinterpret_cast<int4 *>(static_cast<uint8_t *>(workspace) + plan.bytes);
    a.falls = reinterpret_cast<int *>(a.plan + 2 * static_cast<size_t>(cache->num_seqs));
    a.fall_words = kv8::fall_words(0, cache->num_seqs);
    a.fine = a.first = 1;
    ++n;
    ce = kv8::launch_segments(a, st);
  }
  if (ce == cudaSuccess) ce = kv8::launch_attn(a, plan.tiles, st, &n);
  return from_cuda(ce, n);
}

// The rows of one segment and the tensors' rows of calls without a bound by the capacity.
int check_ranges(const kv8_cache *c, const int32_t *row_start, int32_t rows, int32_t max_rows) {
  if (rows < 0 || max_rows < 0) return KVQ_ERR_INVALID_ARG;
  if (!aligned(row_start, 4)) return KVQ_ERR_ALIGNMENT;
  return !row_start && rows < c->num_seqs ? KVQ_ERR_INVALID_ARG : KVQ_OK;
}

}  // namespace

extern "C" {

int32_t kv8_max_blocks(const kv8_cache *cache) {
  if (check_geometry(cache)) return -1;
  return cache->capacity / cache->block;
}

int64_t kv8_buffer_bytes(const kv8_cache *c, int32_t which) {
  if (check_geometry(c)) return -1;
  const int64_t pool = static_cast<int64_t>(c->num_blocks) * c->num_kv_heads;
  const int64_t win = static_cast<int64_t>(c->num_seqs) * c->num_kv_heads * c->block * c->head_dim * 2;
  switch (which) {
    case KV8_BUF_CODES: return pool * 2 * c->block * c->head_dim;
    case KV8_BUF_SCALES: return pool * 2 * 4;
    case KV8_BUF_K_WIN:
    case KV8_BUF_V_WIN: return win;
    case KV8_BUF_SEQ_LEN: return static_cast<int64_t>(c->num_seqs) * 4;
    case KV8_BUF_BLOCK_TABLE: return static_cast<int64_t>(c->num_seqs) * (c->capacity / c->block) * 4;
    default: return -1;
  }
}

int kv8_append(const kv8_cache *cache, const kv8_rows *k, const kv8_rows *v, const kv8_rows *q, const kv8_rows *q_out,
               int32_t num_q_heads, const int32_t *row_start, int32_t rows, int32_t max_new, const float *rope,
               int32_t rope_rows, int32_t rot_dim, int32_t interleaved, void *stream) {
  return append(cache, k, v, q, q_out, num_q_heads, row_start, rows, max_new, rope, rope_rows, rot_dim, interleaved,
                nullptr, stream);
}

int kv8_append_axes(const kv8_cache *cache, const kv8_axes_append *x, void *stream) {
  if (!x) return KVQ_ERR_INVALID_ARG;
  if (x->num_axes < 1 || x->num_axes > KV8_MAX_AXES || x->rot_dim % 16 != 0 || x->rot_dim > 128)
    return KVQ_ERR_UNSUPPORTED;
  if (x->rot_dim < 16 || x->rope_rows < 1 || (x->rows > 0 && !x->positions)) return KVQ_ERR_INVALID_ARG;
  if (!aligned(x->positions, 4)) return KVQ_ERR_ALIGNMENT;
  kv8::Axes axes = {x->positions, x->num_axes > 1 ? x->axis_stride : 0, x->rope_rows, {0, 0, 0, 0}};
  for (int i = 0; i < x->rot_dim / 2; ++i) {
    if (x->axis_of_pair[i] >= x->num_axes) return KVQ_ERR_INVALID_ARG;
    axes.map[i / 16] |= static_cast<uint32_t>(x->axis_of_pair[i]) << (2 * (i % 16));
  }
  // (without rows the queries' tensors may have no data either)
  const bool with_q = x->num_q_heads != 0;
  return append(cache, &x->k, &x->v, with_q || x->q.data ? &x->q : nullptr,
                with_q || x->q_out.data ? &x->q_out : nullptr, x->num_q_heads, x->row_start, x->rows, x->max_new,
                x->rope, x->rope_rows, x->rot_dim, x->interleaved, &axes, stream);
}

int64_t kv8_attn_workspace_bytes(const kv8_cache *cache, int32_t num_q_heads, int32_t max_new) {
  if (check_geometry(cache) || max_new < 1 || max_new > cache->capacity || check_heads(cache, num_q_heads, max_new))
    return -1;
  const int64_t group = num_q_heads / cache->num_kv_heads;
  return static_cast<int64_t>(kv8::plan_attn(cache->head_dim, group * max_new).bytes);
}

int kv8_attn(const kv8_cache *cache, int32_t num_q_heads, const kv8_rows *q, const kv8_rows *out,
             const int32_t *row_start, int32_t rows, int32_t max_new, float softmax_scale, void *workspace,
             size_t workspace_bytes, int32_t max_len, void *stream) {
  int e = check_buffers(cache);
  if (e) return e;
  if ((e = check_row_range(cache, row_start, rows, max_new))) return e;
  return attend(cache, num_q_heads, q, out, row_start, rows, max_new, softmax_scale, workspace, workspace_bytes,
                max_len, true, stream);
}

int64_t kv8_cross_attn_workspace_bytes(const kv8_cache *cache, int32_t num_q_heads, int32_t max_rows) {
  if (check_geometry(cache) || max_rows < 1 || check_heads(cache, num_q_heads, max_rows)) return -1;
  const int64_t group = num_q_heads / cache->num_kv_heads;
  return static_cast<int64_t>(kv8::plan_attn(cache->head_dim, group * max_rows).bytes + seg_bytes(cache));
}

int kv8_cross_attn(const kv8_cache *cache, int32_t num_q_heads, const kv8_rows *q, const kv8_rows *out,
                   const int32_t *row_start, int32_t rows, int32_t max_rows, float softmax_scale, void *workspace,
                   size_t workspace_bytes, int32_t max_len, void *stream) {
  int e = check_buffers(cache);
  if (e) return e;
  if ((e = check_ranges(cache, row_start, rows, max_rows))) return e;
  return attend(cache, num_q_heads, q, out, row_start, rows, max_rows, softmax_scale, workspace, workspace_bytes,
                max_len, false, stream);
}

int64_t kv8_shared_attn_workspace_bytes(const kv8_cache *cache, int32_t num_q_heads, int32_t rows, int32_t max_new,
                                        int32_t max_group_rows) {
  if (check_geometry(cache) || rows < 0 || max_new < 1 || max_new > cache->capacity || max_group_rows < 1 ||
      check_heads(cache, num_q_heads, max_new) || check_heads(cache, num_q_heads, max_group_rows))
    return -1;
  return static_cast<int64_t>(kv8::plan_shared(cache->head_dim, cache->num_seqs, cache->num_kv_heads, num_q_heads,
                                               rows, max_new, max_group_rows)
                                  .bytes);
}

int kv8_shared_attn(const kv8_cache *cache, int32_t num_q_heads, const kv8_rows *q, const kv8_rows *out,
                    const int32_t *row_start, int32_t rows, int32_t max_new, const int32_t *group_start,
                    const int32_t *prefix_len, int32_t num_groups, int32_t max_group_rows, float softmax_scale,
                    void *workspace, size_t workspace_bytes, int32_t max_len, void *stream) {
  int e = check_buffers(cache);
  if (e) return e;
  if ((e = check_row_range(cache, row_start, rows, max_new))) return e;
  if (num_groups < 1 || num_groups > cache->num_seqs || max_group_rows < 1 || !group_start || !prefix_len)
    return KVQ_ERR_INVALID_ARG;
  if (!aligned(group_start, 4) || !aligned(prefix_len, 4)) return KVQ_ERR_ALIGNMENT;
  kv8::AttnArgs a;
  if ((e = attn_args(a, cache, num_q_heads, q, out, row_start, rows, max_new, softmax_scale, max_len))) return e;
  if ((e = check_heads(cache, num_q_heads, max_group_rows))) return e;
  if (rows == 0) return KVQ_OK;
  const int64_t group = a.group;
  const kv8::SharedPlan plan = kv8::plan_shared(cache->head_dim, cache->num_seqs, cache->num_kv_heads, num_q_heads, rows,
                                                max_new, max_group_rows);
  if ((e = check_workspace(workspace, workspace_bytes, plan.bytes))) return e;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  a.group_start = group_start;
  a.prefix_len = prefix_len;
  a.groups = num_groups;
  a.max_group_rows = max_group_rows;
  a.plan = reinterpret_cast<int4 *>(ws + plan.off_segs);
  a.items = reinterpret_cast<int4 *>(ws + plan.off_items);
  a.falls = reinterpret_cast<int *>(ws + plan.off_falls);
  a.fall_words = kv8::fall_words(num_groups, cache->num_seqs);
  a.carry_ml = reinterpret_cast<float2 *>(ws + plan.off_ml);
  a.carry_o = reinterpret_cast<float4 *>(ws + plan.off_o);
  a.carry_blocks = plan.carry_blocks;
  a.carry_wide = plan.own_tiles;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint64_t n = 1;
  a.rows_max = plan.own_tiles ? kv8::kRowsMax : 2147483647;
  a.group_rows_max = plan.prefix_tiles ? kv8::kRowsMax : 2147483647;
  cudaError_t ce = kv8::launch_segments(a, st);
  if (ce != cudaSuccess) return from_cuda(ce, n);
  a.part = kv8::kOwn;
  a.first = a.fine = 1;
  place(a, kv8::plan_attn(cache->head_dim, group * max_new), ws, ws);
  ce = kv8::launch_attn(a, plan.own_tiles, st, &n);
  if (ce == cudaSuccess) {
    a.part = kv8::kPrefix;
    a.first = 0;
    a.causal = 0;
    a.segs = num_groups;
    place(a, kv8::plan_attn(cache->head_dim, group * max_group_rows), ws + kv8::kCounters, ws + plan.off_prefix);
    ce = kv8::launch_attn(a, plan.prefix_tiles, st, &n);
  }
  if (ce == cudaSuccess && plan.prefix_tiles) {
    ++n;
    ce = kv8::launch_join(a, st);
  }
  return from_cuda(ce, n);
}

}  // extern "C"

namespace kv8 {

AttnPlan plan_attn(int D, long long rows_per_head) {
  AttnPlan p;
  auto align = [](size_t x) { return (x + 255) / 256 * 256; };
  p.tiles = rows_per_head > kRowsMax;
  // the counters first, at offsets that no argument moves
  p.off_cnt = 0;
  p.off_tile_cnt = align(kMaxCtas * sizeof(int));
  static_assert(kCounters >= (kMaxCtas * sizeof(int) + 255) / 256 * 256 + kMaxTileCtas * sizeof(int), "counters");
  p.off_o = 2 * kCounters;
  p.off_ml = p.off_o + static_cast<size_t>(2) * kMaxCtas * kRowTile * D * sizeof(float);
  p.off_tile_o = align(p.off_ml + static_cast<size_t>(2) * kMaxCtas * kRowTile * sizeof(float2));
  p.off_tile_ml = p.off_tile_o + static_cast<size_t>(2) * kMaxTileCtas * kTileRows * D * sizeof(float);
  p.bytes = p.tiles ? align(p.off_tile_ml + static_cast<size_t>(2) * kMaxTileCtas * kTileRows * sizeof(float2))
                    : p.off_tile_o;
  return p;
}

SharedPlan plan_shared(int D, int S, int H, int num_q_heads, long long rows, long long max_new,
                       long long max_group_rows) {
  SharedPlan p;
  auto align = [](size_t x) { return (x + 255) / 256 * 256; };
  const int group = num_q_heads / H;
  const AttnPlan own = plan_attn(D, group * max_new), prefix = plan_attn(D, group * max_group_rows);
  p.own_tiles = own.tiles;
  p.prefix_tiles = prefix.tiles;
  p.off_prefix = own.bytes;
  p.off_segs = own.bytes + prefix.bytes;
  p.off_items = align(p.off_segs + static_cast<size_t>(2) * S * 2 * sizeof(int4));
  p.off_falls = p.off_items + static_cast<size_t>(2) * kMaxTileCtas * sizeof(int4);
  p.off_ml = align(p.off_falls + fall_words(S, S) * sizeof(int));
  p.carry_blocks = (rows * group + 31) / 32;
  const size_t n = static_cast<size_t>(H) * p.carry_blocks * 32;
  p.off_o = align(p.off_ml + n * sizeof(float2));
  p.bytes = align(p.off_o + n * D * sizeof(float));
  return p;
}

cudaError_t launch_attn(const AttnArgs &a, bool tiles, cudaStream_t stream, uint64_t *launches) {
  const bool wide = a.geo.D == 128;
  auto rows_kernel = [&](const AttnArgs &a) {
    ++*launches;
    return a.fine ? (wide ? launch_rows_128_shared(a, stream) : launch_rows_64_shared(a, stream))
                  : (wide ? launch_rows_128(a, stream) : launch_rows_64(a, stream));
  };
  auto tile_kernel = [&](const AttnArgs &a) {
    ++*launches;
    return a.fine ? (wide ? launch_tiles_128_shared(a, stream) : launch_tiles_64_shared(a, stream))
                  : (wide ? launch_tiles_128(a, stream) : launch_tiles_64(a, stream));
  };
  if (!tiles) return rows_kernel(a);
  // Over shared blocks the tile kernel goes first: the CTAs of the other one, which
  // wait for all before them, would keep it from the SMs.
  cudaError_t e = a.part == kPrefix ? tile_kernel(a) : rows_kernel(a);
  if (e != cudaSuccess) return e;
  AttnArgs second = a;
  second.first = 0;
  return a.part == kPrefix ? rows_kernel(second) : tile_kernel(second);
}

}  // namespace kv8
