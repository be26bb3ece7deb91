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
  int e = check_buffers(cache);
  if (e) return e;
  if ((e = check_row_range(cache, row_start, rows, max_new))) return e;
  const bool with_q = num_q_heads != 0;
  if (num_q_heads < 0 || with_q != (q != nullptr) || with_q != (q_out != nullptr)) return KVQ_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return KVQ_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim > cache->head_dim || rot_dim % 16 != 0) return KVQ_ERR_UNSUPPORTED;
  if (rot_dim && !rope) return KVQ_ERR_INVALID_ARG;
  if (rot_dim && rope_rows < cache->capacity) return KVQ_ERR_CAPACITY;
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
  uint64_t n = 0;
  const cudaError_t ce = kv8::launch_append(make_geo(cache), make_rows(k), make_rows(v), with_q ? make_rows(q) : none,
                                            with_q ? make_rows(q_out) : none, num_q_heads, row_start, rows, max_new,
                                            rope, rot_dim, interleaved, static_cast<cudaStream_t>(stream), &n);
  return from_cuda(ce, n);
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
  if (max_new < 1 || max_len < 1) return KVQ_ERR_INVALID_ARG;
  if ((e = check_heads(cache, num_q_heads, max_new))) return e;
  if (max_len > cache->capacity) return KVQ_ERR_CAPACITY;
  if (rows == 0) return KVQ_OK;
  if ((e = check_rows(q, num_q_heads, rows, cache->head_dim, false))) return e;
  if ((e = check_rows(out, num_q_heads, rows, cache->head_dim, true))) return e;
  if (q->data == out->data && (q->row_stride != out->row_stride || q->head_stride != out->head_stride))
    return KVQ_ERR_INVALID_ARG;
  const int64_t group = num_q_heads / cache->num_kv_heads;
  const kv8::AttnPlan plan = kv8::plan_attn(cache->head_dim, group * max_new);
  if (!workspace || workspace_bytes < plan.bytes) return KVQ_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return KVQ_ERR_ALIGNMENT;
  if (!(softmax_scale > 0.f) || !isfinite(softmax_scale))
    softmax_scale = 1.f / sqrtf(static_cast<float>(cache->head_dim));
  kv8::AttnArgs a;
  a.geo = make_geo(cache);
  a.Hq = num_q_heads;
  a.group = static_cast<int>(group);
  a.q = make_rows(q);
  a.out = make_rows(out);
  a.row_start = row_start;
  a.rows = rows;
  a.max_new = max_new;
  a.max_len = max_len;
  a.zscale = softmax_scale * 1.4426950408889634f;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  a.part_o = reinterpret_cast<float *>(ws + plan.off_o);
  a.part_ml = reinterpret_cast<float2 *>(ws + plan.off_ml);
  a.counters = reinterpret_cast<int *>(ws + plan.off_cnt);
  a.tile_counters = reinterpret_cast<int *>(ws + plan.off_tile_cnt);
  a.tile_o = reinterpret_cast<float *>(ws + plan.off_tile_o);
  a.tile_ml = reinterpret_cast<float2 *>(ws + plan.off_tile_ml);
  a.rows_max = plan.tiles ? kv8::kRowsMax : 2147483647;
  const kvq::WaitTest wt = kvq::wait_test();
  a.wait_limit = wt.limit;
  a.wait_test = wt.before_fetch;
  uint64_t n = 0;
  const cudaError_t ce = kv8::launch_attn(a, plan.tiles, static_cast<cudaStream_t>(stream), &n);
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
  p.off_o = p.off_tile_cnt + align(kMaxTileCtas * sizeof(int));
  p.off_ml = p.off_o + static_cast<size_t>(2) * kMaxCtas * kRowTile * D * sizeof(float);
  p.off_tile_o = align(p.off_ml + static_cast<size_t>(2) * kMaxCtas * kRowTile * sizeof(float2));
  p.off_tile_ml = p.off_tile_o + static_cast<size_t>(2) * kMaxTileCtas * kTileRows * D * sizeof(float);
  p.bytes = p.tiles ? align(p.off_tile_ml + static_cast<size_t>(2) * kMaxTileCtas * kTileRows * sizeof(float2))
                    : p.off_tile_o;
  return p;
}

cudaError_t launch_attn(const AttnArgs &a, bool tiles, cudaStream_t stream, uint64_t *launches) {
  ++*launches;
  cudaError_t e = a.geo.D == 128 ? launch_rows_128(a, stream) : launch_rows_64(a, stream);
  if (e != cudaSuccess || !tiles) return e;
  ++*launches;
  return a.geo.D == 128 ? launch_tiles_128(a, stream) : launch_tiles_64(a, stream);
}

}  // namespace kv8
