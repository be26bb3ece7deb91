/*
 * kv8.h -- C ABI of the 8-bit paged KV cache (part of libkvq.so, sm_103a).
 *
 * The sibling of the 2/4-bit cache of kvq.h for callers that want half the
 * memory of 16 bits: keys and values in 8 bits with one fp32 scale per (block
 * of tokens, KV head, keys or values), pages shared by all heads of a sequence,
 * fp16 or bf16 activations, and attention for any number of new tokens per
 * sequence (one while decoding, a few when checking drafts, many in a prompt's
 * chunk).  Normal values come back with an error of 0.9% (int8) or 2.7% (e4m3)
 * of their size, root mean square, and attention over 4096 such tokens with
 * 1.3% or 3.8%; where four key channels of 128 are six times as large, with 4%
 * or 8%.
 *
 *   kv8_append  rotates queries and keys to their positions, stores the keys
 *               and values, and quantizes every block that fills.
 *   kv8_attn    attention of the new tokens' queries over the cache, causal.
 *
 * A step of a serving loop raises seq_len by the new tokens of each sequence,
 * calls kv8_append, then kv8_attn with the same seq_len and row_start.
 *
 * Conventions are those of kvq.h: all buffers are device memory owned by the
 * caller; nothing is allocated and nothing synchronizes; work is enqueued on
 * `stream`, on the current device; arguments are checked before anything is
 * launched and give KVQ_OK or a KVQ_ERR_* code (kvq_strerror has the
 * messages); errors that only the device can see are OR-ed into the
 * optional word `status` (KVQ_STATUS_*); no C++ exception or abort crosses
 * the boundary; kvq_launch_count counts these kernels too.  Calls on the same
 * cache or the same workspace must not overlap on the GPU: order them by
 * stream or event.
 */
#ifndef KV8_H
#define KV8_H

#include <stddef.h>
#include <stdint.h>

#include "kvq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define KV8_INT8 0  /* codes -127..127 */
#define KV8_E4M3 1  /* 8-bit floating point, 4 exponent and 3 mantissa bits */

#define KV8_F16  0  /* IEEE binary16 */
#define KV8_BF16 1  /* bfloat16 */

#define KV8_MAX_CAPACITY (1 << 30)

/* which buffer for kv8_buffer_bytes() */
#define KV8_BUF_CODES       0
#define KV8_BUF_SCALES      1
#define KV8_BUF_K_WIN       2
#define KV8_BUF_V_WIN       3
#define KV8_BUF_SEQ_LEN     4
#define KV8_BUF_BLOCK_TABLE 5

/*
 * Cache descriptor.  Plain data; every pointer is a caller-owned device
 * buffer sized by kv8_buffer_bytes().
 *
 *   codes    [num_blocks][Hkv][2][block][D], 16-byte aligned: the pool.
 *            [..][0] are keys, [..][1] values, one byte per element, tokens
 *            in order.
 *   scales   [num_blocks][Hkv][2] fp32, 8-byte aligned; element = code * scale.
 *   k_win, v_win  [S][Hkv][block][D] in 16 bits, 16-byte aligned: the tokens
 *            of each sequence's last, incomplete block; token p in slot
 *            p mod block.
 *   seq_len  [S] int32, read only: tokens of each sequence INCLUDING the new
 *            ones of the call.  The caller advances it.
 *   block_table  [S][max_blocks] int32, max_blocks = floor(capacity / block):
 *            pool block of each complete block, the same for all heads.  The
 *            caller assigns an entry before the append that completes the
 *            block; entries past the complete blocks are never read.
 *            Sequences may share blocks that are complete.  An entry outside
 *            [0, num_blocks) is never dereferenced: KVQ_STATUS_BAD_BLOCK is
 *            set, kv8_append leaves its block out and kv8_attn gives NaN in
 *            the rows that see it.
 *   status   optional int32 (may be NULL).
 *
 * With L = seq_len[s], tokens below floor(L / block) * block are in the pool
 * and the rest in the window.  A caller that takes tokens back (rejected
 * drafts) may lower L while floor(L / block) stays the same.
 */
typedef struct kv8_cache {
  int32_t  num_seqs;      /* S, 1 .. 65535                       */
  int32_t  num_kv_heads;  /* Hkv, 1 .. 65535                     */
  int32_t  head_dim;      /* D: 64 or 128                        */
  int32_t  block;         /* tokens per block: 32, 64 or 128     */
  int32_t  format;        /* KV8_INT8 or KV8_E4M3                */
  int32_t  dtype;         /* KV8_F16 or KV8_BF16: 16-bit tensors */
  int32_t  capacity;      /* max tokens, 1 .. KV8_MAX_CAPACITY   */
  int32_t  num_blocks;    /* pool size, >= 1 when capacity >= block */
  uint8_t  *codes;
  float    *scales;
  uint16_t *k_win, *v_win;
  const int32_t *seq_len;
  const int32_t *block_table;
  int32_t  *status;
} kv8_cache;

/*
 * A 16-bit tensor [rows][heads][D] with its own strides (in elements); the D
 * elements of a head are contiguous.  Rows are the new tokens of all
 * sequences, one sequence after the other.  data is 16-byte aligned and the
 * strides are multiples of 8, so that slices of a fused projection's output
 * can be passed as they are.
 */
typedef struct kv8_rows {
  uint16_t *data;
  int64_t  row_stride;
  int64_t  head_stride;
} kv8_rows;

/* floor(capacity / block), or -1 on bad geometry. */
int32_t kv8_max_blocks(const kv8_cache *cache);

/* Size in bytes of buffer `which` (KV8_BUF_*), -1 on bad geometry. */
int64_t kv8_buffer_bytes(const kv8_cache *cache, int32_t which);

/*
 * kv8_append -- store the new tokens of every sequence, rotated to their
 * positions.
 *
 *   k, v       [rows][Hkv][D].  Read only.
 *   q, q_out   [rows][Hq][D]: queries to rotate along, and where they go
 *              (may be the same tensor).  Both NULL, or num_q_heads 0: none.
 *   row_start  device int32 [S + 1]: sequence s brings rows row_start[s] ..
 *              row_start[s + 1] - 1.  NULL: one row per sequence, row s.
 *   rows       rows of the tensors; those that belong to no sequence are
 *              neither read nor written.
 *   max_new    host bound on the new rows of one sequence, 0 .. capacity.
 *   rope       device fp32 [rope_rows][rot_dim], 16-byte aligned: row p holds
 *              the cosines, then the sines, of the rot_dim / 2 angles of
 *              position p.  The first rot_dim channels of each head are
 *              rotated (rot_dim: a multiple of 16, at most D), the others
 *              kept.  rope_rows >= capacity.  rot_dim 0: no rotation, rope
 *              may be NULL.
 *   interleaved  0: channel i turns with channel i + rot_dim / 2; 1: channel
 *              2 i with 2 i + 1.
 *
 * A pair (a, b) becomes (a c - b s, b c + a s) in fp32, each product and sum
 * rounded on its own, then rounded to the 16-bit type.  The n new tokens of
 * sequence s take positions seq_len[s] - n .. seq_len[s] - 1.
 *
 * A block that fills is quantized from its 16-bit tokens: amax = the largest
 * magnitude of its block * D elements (at least 2^-100), then
 *   int8: scale = fl32(amax / 127), code = round-half-even(x * fl32(127 / amax));
 *   e4m3: scale = 2^k with the smallest k for which amax <= 448 * 2^k, code =
 *         x / scale rounded half-even to e4m3.
 * A block with a NaN or an infinity gets scale NaN and codes 0.  The result
 * does not depend on how a token stream is split into appends.
 *
 * A sequence whose row range is not within [0, rows], longer than max_new or
 * than seq_len[s], or whose seq_len[s] exceeds the capacity, is left alone
 * (its rows of q_out too) and sets KVQ_STATUS_BAD_LEN or
 * KVQ_STATUS_CAPACITY.  row_start must not decrease: where it does,
 * KVQ_STATUS_BAD_LEN is set and other sequences may be left alone too.  One
 * kernel.
 */
int kv8_append(const kv8_cache *cache, const kv8_rows *k, const kv8_rows *v,
               const kv8_rows *q, const kv8_rows *q_out, int32_t num_q_heads,
               const int32_t *row_start, int32_t rows, int32_t max_new,
               const float *rope, int32_t rope_rows, int32_t rot_dim,
               int32_t interleaved, void *stream);

/*
 * kv8_attn_workspace_bytes -- scratch size for kv8_attn calls with at most
 * max_new rows per sequence (a multiple of 256); -1 on invalid arguments.
 * About 10 MiB for D = 128, and 50 MiB where max_new * Hq / Hkv > 48: there a
 * second kernel, on the tcgen05 tensor cores, takes the sequences with more
 * than 48 rows per KV head.  A size that serves a larger max_new serves a
 * smaller one.
 */
int64_t kv8_attn_workspace_bytes(const kv8_cache *cache, int32_t num_q_heads,
                                 int32_t max_new);

/*
 * kv8_attn -- softmax attention of the new tokens' queries over the cache.
 *
 *   q, out     [rows][Hq][D]; query head j reads KV head j / (Hq / Hkv), Hq a
 *              multiple of Hkv.  Queries are already rotated.  out may be q.
 *   row_start, rows, max_new  as in kv8_append (max_new >= 1).
 *   softmax_scale  multiplier of q.k; <= 0 selects 1/sqrt(D).
 *   workspace  at least kv8_attn_workspace_bytes() bytes, 256-byte aligned,
 *              zero-filled before its first use and written by kv8_attn
 *              only.  Every call leaves its counters zero again, at places
 *              that no argument moves: calls of other caches, head
 *              dimensions and bounds may follow each other on one workspace
 *              that is large enough for each (zero it after
 *              KVQ_STATUS_TIMEOUT, which a call that gave up sets, its rows
 *              being undefined).
 *   max_len    host bound on every seq_len, 1 .. capacity.
 *
 * Row i of the n rows of sequence s sits at position seq_len[s] - n + i and
 * sees the tokens up to its own position; a row at a negative position sees
 * none and gets zeros.  A sequence with seq_len[s] < 0 or above max_len gets
 * zero rows and sets KVQ_STATUS_MAX_LEN; one whose row range is invalid is
 * left alone and sets KVQ_STATUS_BAD_LEN, and so may others be where row_start
 * decreases.  Rows that belong to no sequence are left as they are.  A token
 * with a NaN or an infinity in its keys or values makes the rows that see it
 * NaN (through a whole block once the block is quantized), and no other row.
 * A query with a NaN or an infinity makes its own row NaN (zeros where the row
 * sees no token).
 * A block of values whose scale is below 2^-80 counts as zeros.  Weights are
 * rounded to fp16 relative to the row's largest weight times scale of values:
 * those 2^23 below it (2^15 for bf16 window tokens beside blocks) lose bits.
 * That is far below what the tokens' own 8 bits lose, but where values differ
 * by such factors: a block of large values takes bits of the others even if the
 * row sees only small ones of it, and in bf16 a block 2^125 below others may
 * lose its share of the weights.  In bf16 results may overflow where a window
 * token's keys or values are above 2^100 in magnitude.  Results do not depend on timing: the same call gives the same
 * bits.  One or two kernels, which read all lengths on the device: a captured
 * call can be replayed for other lengths within max_len, rows and max_new.
 */
int kv8_attn(const kv8_cache *cache, int32_t num_q_heads, const kv8_rows *q,
             const kv8_rows *out, const int32_t *row_start, int32_t rows,
             int32_t max_new, float softmax_scale, void *workspace,
             size_t workspace_bytes, int32_t max_len, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* KV8_H */
