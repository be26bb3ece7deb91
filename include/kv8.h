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
 *   kv8_append_axes   the append with positions that have several axes (time,
 *               height and width of image patches) or are not the tokens' places
 *               in the cache.
 *   kv8_cross_attn    attention to all tokens of each sequence: an encoder's
 *               states, by a decoder's rows of any number.
 *   kv8_shared_attn   kv8_attn for sequences of which groups share their first
 *               blocks, which it reads once per group.
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
#define KV8_MAX_AXES 4

/* a bit of the status word, beside KVQ_STATUS_*: a position outside the table */
#define KV8_STATUS_BAD_POSITION 64

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
 * kv8_append_axes -- kv8_append for positions that are given.  Its arguments are
 * one struct, which is read before the call returns: a call's host time is what a
 * one-token step waits for, and most of that is the passing of arguments.
 *
 *   k, v, q, q_out, num_q_heads, row_start, rows, max_new, interleaved  as in
 *              kv8_append (without queries: num_q_heads 0, q and q_out without
 *              data).
 *   positions  device int32: position of row r on axis x at
 *              positions[x * axis_stride + r].  Those of rows of no
 *              sequence may hold anything.
 *   axis_stride  any (0: all axes have the first one's); not used with one axis.
 *   num_axes   1 .. KV8_MAX_AXES.
 *   axis_of_pair  the first rot_dim / 2 count: channel pair i (as in kv8_append,
 *              i + rot_dim / 2 or 2 i + 1 beside it) turns by the angle i of the
 *              table's row positions[axis_of_pair[i]].  In order (the first pairs by
 *              the first axis, ...) or in turn, as the model has them; in order is
 *              faster where four aligned pairs have one axis.
 *   rope, rope_rows  as in kv8_append, for positions 0 .. rope_rows - 1, whatever
 *              the capacity.  The table's columns may have any angles: one
 *              sequence of frequencies over all pairs, or one anew for each axis.
 *   rot_dim    a multiple of 16, 16 .. D.
 *
 * All else is as in kv8_append: tokens are stored at places seq_len[s] - n ..
 * seq_len[s] - 1 of their sequence, whatever their positions.  A position outside
 * the table is not read at: the channels that turn by it become NaN, in queries
 * and keys, and KV8_STATUS_BAD_POSITION is set.  With one axis whose positions
 * are the tokens' places the results are kv8_append's, bit for bit.  One kernel.
 */
typedef struct kv8_axes_append {
  kv8_rows k, v, q, q_out;
  const int32_t *row_start;
  const float   *rope;
  const int32_t *positions;
  int64_t  axis_stride;
  int32_t  num_q_heads, rows, max_new;
  int32_t  rope_rows, rot_dim, interleaved;
  int32_t  num_axes;
  uint8_t  axis_of_pair[64];
} kv8_axes_append;

int kv8_append_axes(const kv8_cache *cache, const kv8_axes_append *args, void *stream);

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

/*
 * kv8_cross_attn -- softmax attention to all tokens of each sequence, without
 * order: a decoder's rows over an encoder's states, which kv8_append (without
 * rope, or kv8_append_axes) has stored.
 *
 *   q, out     [rows][Hq][D] as in kv8_attn.
 *   row_start  device int32 [S + 1]: rows row_start[s] .. row_start[s + 1] - 1
 *              attend to sequence s: tokens of the decoder, beams that share the
 *              states, or both.  Their number has nothing to do with seq_len[s].
 *              NULL: one row per sequence, row s.
 *   max_rows   host bound on the rows of one sequence, from 1 on; not bound by
 *              the capacity.  max_rows * Hq / Hkv is below 2^30.
 *   softmax_scale, workspace, max_len, and all else, as in kv8_attn; the
 *              workspace has at least kv8_cross_attn_workspace_bytes(), about 32
 *              bytes per sequence more than kv8_attn's, and may serve both.
 *
 * Every row sees the seq_len[s] tokens of its sequence.  Rows of a sequence
 * without tokens get zeros.  Two or three kernels.
 */
int64_t kv8_cross_attn_workspace_bytes(const kv8_cache *cache, int32_t num_q_heads, int32_t max_rows);
int kv8_cross_attn(const kv8_cache *cache, int32_t num_q_heads, const kv8_rows *q, const kv8_rows *out,
                   const int32_t *row_start, int32_t rows, int32_t max_rows, float softmax_scale, void *workspace,
                   size_t workspace_bytes, int32_t max_len, void *stream);

/*
 * kv8_shared_attn -- kv8_attn where groups of sequences share their first blocks
 * (a system prompt, a document, the prompt of several answers): the rows of all
 * sequences of a group attend to those blocks at once, and each sequence's rows
 * to what lies behind them; both results are joined in 32 bits.  It pays where many
 * sequences of few rows share a group's blocks.  Where each sequence's line of the
 * table names the shared blocks too, kv8_attn gives the same rows, and reads blocks
 * that others have read from L2: 64 single tokens behind 4096 shared ones 51 us
 * here and 76 there (8 KV heads of 4), but four behind 512 tokens 19 and 14, 12 groups
 * of 1 to 8 sequences with drafts 52 and 36, six chunks of 100 to 500 rows behind 8192
 * 294 and 274.
 *
 *   q, out, row_start, rows, max_new, softmax_scale, max_len  as in kv8_attn.
 *   group_start  device int32 [num_groups + 1]: group g is sequences
 *              group_start[g] .. group_start[g + 1] - 1.  Groups may be empty;
 *              sequences before the first or behind the last group share
 *              nothing.
 *   prefix_len  device int32 [num_groups]: tokens that a group shares, at most
 *              max_len, rounded down to whole blocks.  The blocks are those of the
 *              block table's line of the group's first sequence; the other
 *              sequences' entries for them are not read.  Each sequence of the
 *              group has stored them before the call's new tokens: prefix_len,
 *              rounded down, is at most seq_len[s] minus its new rows.
 *   num_groups 1 .. S.
 *   max_group_rows  host bound on the rows of one group's sequences together.
 *   workspace  at least kv8_shared_attn_workspace_bytes() for these rows, max_new
 *              and max_group_rows (a size that serves larger ones serves smaller
 *              ones), with the rules of kv8_attn's; it may serve kv8_attn and
 *              kv8_cross_attn too.  It is as large as kv8_attn's for max_new and
 *              kv8_attn's for max_group_rows rows of a sequence together, and 4 D + 8
 *              bytes per row and query head and about 70 per sequence more.
 *
 * A group with bad bounds, a bad prefix_len, more rows than max_group_rows or a
 * first sequence that ends within the shared blocks is invalid: the rows of its
 * sequences are left alone, as are those of a sequence that ends within them, and
 * KVQ_STATUS_BAD_LEN is set.  Neither row_start nor group_start may decrease:
 * where one does, that bit is set and the rows of all sequences are undefined
 * (nothing else is: the workspace serves the next call).
 * Otherwise results are as kv8_attn describes them, for a table in which all
 * sequences of a group have its first one's entries.  Three to six kernels.
 */
int64_t kv8_shared_attn_workspace_bytes(const kv8_cache *cache, int32_t num_q_heads, int32_t rows, int32_t max_new,
                                        int32_t max_group_rows);
int kv8_shared_attn(const kv8_cache *cache, int32_t num_q_heads, const kv8_rows *q, const kv8_rows *out,
                    const int32_t *row_start, int32_t rows, int32_t max_new, const int32_t *group_start,
                    const int32_t *prefix_len, int32_t num_groups, int32_t max_group_rows, float softmax_scale,
                    void *workspace, size_t workspace_bytes, int32_t max_len, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* KV8_H */
