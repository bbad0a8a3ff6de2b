/*
 * dg_paged.h — a key/value cache in pages, with the operators that fill and read it,
 * one layer at a time: for callers whose sequences have their own lengths (blocks
 * appended while other canvases are still denoised, prompts of mixed lengths in one
 * pass, single tokens), which the fixed-batch dg_kv handles of dg.h do not hold.
 *
 * A batch is B sequences.  Sequence b brings the rows q_start[b] .. q_start[b+1] - 1 of
 * the call's row tensors as its chunk of new tokens; kv_len[b] counts its positions
 * INCLUDING the chunk, so row i of the chunk stands at position
 *   p = kv_len[b] - (q_start[b+1] - q_start[b]) + i.
 * Position p lives in slot p % page_size of page page_table[b, p / page_size].
 *
 * Conventions are those of dg.h (device pointers unless stated, dg_status returns,
 * `stream` = cudaStream_t as void*, nothing thrown, arguments checked before any launch)
 * with these additions:
 *   - The three operators need no model handle, allocate nothing and may be captured into
 *     a graph.  They run on the current device; its first dg_paged_attention call there
 *     sets a kernel attribute.
 *   - What only the device can see is checked there.  err (nullable) is a device int32
 *     into which bits of dg_paged_error are OR'd; the library never clears it.  Whatever
 *     q_start, kv_len and page_table hold, nothing outside the described tensors is read
 *     or written.
 *   - Rows that belong to no sequence (before q_start[0], from q_start[B] on) are left as
 *     they were in every output, and so are the rows of a sequence with a bad length.
 *   - A call with no rows (n or n_tokens 0) or no sequence (B 0) does nothing, and looks at
 *     nothing on the device.
 */
#ifndef DG_PAGED_H
#define DG_PAGED_H

#include "dg.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum dg_elem { DG_ELEM_BF16 = 0, DG_ELEM_F16 = 1, DG_ELEM_F32 = 2 } dg_elem;

/* Bits of an operator's err word. */
typedef enum dg_paged_error {
  DG_PAGED_BAD_BATCH = 1, /* q_start leaves [0, n_tokens], a chunk longer than max_q, or
                             kv_len outside [0, max_pages * page_size]: the sequence is
                             skipped.  q_start decreases: dg_paged_attention skips the whole
                             batch, since its chunks may overlap, and of what belongs to it
                             dg_paged_append may write any part                         */
  DG_PAGED_BAD_PAGE = 2,  /* a page number outside [0, n_pages) where a row is stored (it
                             is not) or a key is read (the sequence's rows that see it are
                             NaN, and neighbours of theirs computed with them may be)   */
  DG_PAGED_TIMEOUT = 4    /* a bounded device-side wait gave up; outputs are undefined  */
} dg_paged_error;

/* Rows of heads: element (t, j, i) at p + t * token_stride + j * head_stride + i, strides
 * in elements.  p and both strides (in bytes) are multiples of 16. */
typedef struct dg_heads {
  void* p;
  int64_t token_stride, head_stride;
  int32_t n_heads;
} dg_heads;

/* The rotation's constants: turns[i] = base^(-2i/head_dim) / (2 pi) in units of 2^-64
 * turn, for pair (i, i + head_dim/2).  Position times turns[i], modulo 2^64, is the exact
 * fraction of a turn, so far positions lose nothing. */
typedef struct dg_rope {
  int32_t head_dim;
  int32_t reserved;
  uint64_t turns[128];
} dg_rope;

/* One layer's pages: key of slot t, head j of page g at
 * k + g * page_stride + t * token_stride + j * head_stride (elements; v alike).  Any order
 * of the axes will do; page_size is a power of two from 16 on. */
typedef struct dg_paged_cache {
  void *k, *v;   /* 16-byte aligned */
  int32_t dtype; /* dg_elem: DG_ELEM_BF16 or DG_ELEM_F16 */
  int32_t n_pages, page_size, n_kv_heads, head_dim;
  int64_t page_stride, token_stride, head_stride; /* multiples of 8 */
} dg_paged_cache;

typedef struct dg_paged_batch {
  int32_t B;
  int32_t n_tokens;          /* rows of the call's row tensors (any behind q_start[B] are padding) */
  int32_t max_q;             /* no chunk is longer                                     */
  int32_t max_pages;         /* columns of page_table                                  */
  const int32_t* q_start;    /* [B + 1], not decreasing                                */
  const int32_t* kv_len;     /* [B]                                                    */
  const int32_t* page_table; /* [B, max_pages]; entries that no position needs are not read */
} dg_paged_batch;

/* Fills *out (host memory) for a rotation by p * base^(-2i/head_dim).  Host only.
 * Requires base >= 1 and finite, head_dim a multiple of 16 in [16, 256]. */
dg_status dg_rope_init(double base, int32_t head_dim, dg_rope* out);

/* Per head row x of q and of k: y = x / sqrt(mean(x^2) + eps) * gain (eps < 0: y = x, and
 * the gains must be NULL; a NULL gain is 1), then the rotation of y to positions[t]
 * (rope: host pointer, NULL: none).  Squares, sums and angles in fp32 or better (a row
 * whose squares leave fp32's range, elements beyond 2^60, comes out as 0), one rounding at
 * the end.  q_out and k_out have q's and k's shapes and may be the same memory as their
 * inputs; otherwise they must not overlap them.  k->n_heads may be 0 (k_out then unused),
 * and so may q's.  q_gain, k_gain: [head_dim] of the rows' type, 16-byte aligned.
 * positions: [n] int32, any sign (needed when rope is given).
 * Requires n >= 0, head_dim a multiple of 16 in [16, 256], rope->head_dim == head_dim. */
dg_status dg_qk_norm_rope(int32_t dtype, int32_t n, int32_t head_dim, const dg_heads* q,
                          const dg_heads* k, const int32_t* positions, const dg_rope* rope,
                          const void* q_gain, const void* k_gain, float eps,
                          const dg_heads* q_out, const dg_heads* k_out, void* stream);

/* Stores every chunk row's keys (normalised and rotated to the row's position as in
 * dg_qk_norm_rope) and values (as they are) in their pages; the keys already stored stay.
 * With q (nullable) the query rows are normalised and rotated too, into q_out (may be q's
 * memory).  k, v: n_kv_heads heads of the cache's type.  A row with a negative position
 * (kv_len shorter than the chunk) is not stored.  Two rows of a call with the same slot
 * (sequences sharing a page that both write): either one's values end there. */
dg_status dg_paged_append(const dg_paged_cache* cache, const dg_paged_batch* batch,
                          const dg_heads* k, const dg_heads* v, const dg_rope* rope,
                          const void* k_gain, float eps, const dg_heads* q,
                          const void* q_gain, const dg_heads* q_out, int32_t* err,
                          void* stream);

/* Bytes of workspace a dg_paged_attention call on this cache, batch and n_q_heads needs: a
 * function of max_q, n_q_heads, n_kv_heads and head_dim (host only, no device memory read). */
dg_status dg_paged_attention_workspace(const dg_paged_cache* cache, const dg_paged_batch* batch,
                                       int32_t n_q_heads, size_t* bytes);

/* out[t, j] = sum_s softmax_s(scale q[t, j] . key(s)) value(s) over the positions s of the
 * row's sequence that the row sees; query head j reads key head j / (Hq / Hkv).
 *   causal (causal_seq[b] if causal_seq is given, else causal, != 0): a row at position p
 *     sees s <= p, with a window also s > p - window (the prompt and append passes of dg.h);
 *   else: every row of the chunk sees all of the chunk and the `window` positions before
 *     it (the canvas rows of dg.h).  window 0: no limit.
 * A row that sees nothing gets 0 and lse -inf.  lse (nullable): [n_tokens, Hq] fp32, the
 * natural log of the sum of exponentials.  out: [n_tokens, Hq, head_dim] of the cache's
 * type, contiguous, 16-byte aligned, overlapping no input.  Scores, softmax and sums are
 * fp32; the weights are rounded to the cache's type before they meet the values (f16: by at
 * most 2^-32 of the row's largest weight where that is more than half a step of the weight
 * itself).
 * Keys and values at positions no row of the sequence sees, slots past kv_len included,
 * may hold anything; a non-finite value that some row sees can reach other rows of the same
 * sequence.  workspace: 256-byte aligned, at least dg_paged_attention_workspace bytes, this
 * call's alone until it has finished; it needs no initial value.
 * Requires head_dim 64 or 128 (dg_paged_append stores heads of other sizes too, for other
 * readers), Hq a multiple of Hkv with Hq / Hkv <= 128, scale > 0 and scale log2(e) finite in
 * fp32, window >= 0, q's strides > 0 where it has more than one row or head, max_pages *
 * page_size at least 256 below 2^31, and fewer than 2^31 key tiles of 128 in all (chunk rows
 * by key heads, against the table's width: DG_ERR_UNSUPPORTED). */
dg_status dg_paged_attention(const dg_paged_cache* cache, const dg_paged_batch* batch,
                             const dg_heads* q, int32_t causal, const uint8_t* causal_seq,
                             int32_t window, float scale, void* out, float* lse,
                             void* workspace, size_t workspace_bytes, int32_t* err,
                             void* stream);

#ifdef __cplusplus
}
#endif
#endif /* DG_PAGED_H */
