/*
 * vqv_round.h - C ABI of libvqv's operators around the projections in a
 * verify round of block-wise speculative decoding on MI355X (gfx950):
 *
 *   vqv_rope_append    rotary positions of queries and keys; keys and values
 *                      are written to a paged cache.
 *   vqv_paged_attn     attention of every sequence's new rows over its pages
 *                      (causal; optionally a sliding window and a few first
 *                      tokens that stay visible).
 *   vqv_cache_*        pages: copy, fork, trim, reserve; and compact, which
 *                      keeps the confirmed rows of a block.
 *   vqv_logits_*       penalties, biases and grammar masks on logits, written
 *                      out or fused with the greedy verify of vqv.h.
 *
 * Memory, streams, errors and threads are as in vqv.h: device memory owned by
 * the caller, asynchronous launches on the caller's stream, arguments checked
 * on the host before the first launch, nothing allocated and nothing kept.
 * The structs below are host memory, read during the call only. All calls are
 * deterministic and can be captured into a HIP graph.
 *
 * Values that live on the device (tables, lengths, tokens) cannot be checked
 * on the host. The kernels check each of them where it is used as an index:
 * a bad one is treated as the comments say and never leaves the buffers.
 */
#ifndef VQV_ROUND_H
#define VQV_ROUND_H

#include "vqv.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Keys and values of all layers in pages of page_size tokens:
 * k and v [layers, pages, page_size, kv_heads, dim], bf16 or fp16, with the
 * strides below in elements (the same for k and v); dim is contiguous.
 *   dim        a multiple of 8, 8..256.
 *   strides    multiples of 8, >= 0; k and v 16-byte aligned.
 *   A layer's pages span less than 2^32 units of 16 bytes (64 GiB) per tensor.
 */
typedef struct {
  void* k;
  void* v;
  int layers, pages, page_size, kv_heads, dim;
  int dtype; /* VQV_BF16 or VQV_FP16 */
  int64_t layer_stride, page_stride, slot_stride, head_stride;
} vqv_cache;

/*
 * The rows of a call, sequence after sequence.
 *   row_start  [n_seqs + 1] int32, ascending from 0 to n_rows: sequence b's
 *              new rows are row_start[b] .. row_start[b+1]-1 (none is fine).
 *   kv_len     [n_seqs] int32: tokens of sequence b, its new rows among them:
 *              row i of n stands at position kv_len[b] - n + i.
 *   table      [n_seqs, table_width] int32, rows table_stride apart: page of
 *              token t of sequence b is table[b][t / page_size]. A token past
 *              the table or on a page outside [0, pages) is not stored by
 *              vqv_rope_append and is hidden from vqv_paged_attn.
 *   max_rows   at least the largest count of rows of a sequence, and
 *   max_kv     at least the largest kv_len: they size grids and workspaces.
 *              Rows past max_rows are not computed; tokens past max_kv are
 *              computed, but slower.
 */
typedef struct {
  const int32_t* row_start;
  const int32_t* kv_len;
  const int32_t* table;
  int64_t table_stride;
  int n_seqs, table_width, n_rows, max_rows, max_kv;
} vqv_seqs;

/*
 * Rotary positions of the first rot values of each head: pair i of position p
 * is turned by p * f_i, and cosine and sine are multiplied by mscale.
 *   interleaved  pairs are (2i, 2i+1), else (i, i + rot/2).
 *   scaling      f_i = base^(-2i/rot) and, over a factor:
 *     VQV_ROPE_NONE    as it is (factor is not used)
 *     VQV_ROPE_LINEAR  f_i / factor
 *     VQV_ROPE_NTK     base is multiplied by factor^(rot/(rot-2)) (rot > 2)
 *     VQV_ROPE_YARN    between f_i and f_i / factor along a ramp from the
 *                      pair that makes 32 turns in original_len positions
 *                      (floor) to the one that makes 1 (ceiling);
 *                      mscale = 0.1 ln(factor) + 1, or 1 where factor <= 1
 *     VQV_ROPE_SMOOTH  f_i where a pair makes 4 turns or more in
 *                      original_len, f_i / factor where it makes 1 or less,
 *                      and linear in the turns between them.
 * vqv_rope_plan fills the struct; `turns` holds f_i / (2 pi) in 64 bits, and
 * both it and mscale may be changed by the caller afterwards.
 */
enum { VQV_ROPE_NONE = 0, VQV_ROPE_LINEAR = 1, VQV_ROPE_NTK = 2, VQV_ROPE_YARN = 3,
       VQV_ROPE_SMOOTH = 4 };

typedef struct {
  int rot;          /* even, 2..256 */
  int interleaved;
  float mscale;
  int reserved;
  double turns[128];
} vqv_rope;

vqv_status vqv_rope_plan(vqv_rope* plan, int rot, double base, int interleaved, int scaling,
                         double factor, int original_len);

/*
 * q_out = rotated q, and the cache's rows of layer `layer` = rotated k and v.
 *   q, k, v    [n_rows, heads | kv_heads, dim] in in_dtype (bf16, fp16 or
 *              fp32), row and head strides in elements (dim contiguous), for
 *              example slices of one stacked projection. 16-byte aligned,
 *              strides multiples of 16 bytes.
 *   q_out      [n_rows, heads, dim] dense in the cache's type, 16-byte
 *              aligned; it may not overlap an input.
 *   heads      >= 1 (a multiple of kv_heads is not needed here).
 * Angles are formed in 64 bits and reduced to one turn before the 32-bit
 * sine and cosine, the rotation is in 32 bits, rounded once. Rows that no
 * sequence holds are left out.
 */
vqv_status vqv_rope_append(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                           const void* k, int64_t k_row_stride, int64_t k_head_stride,
                           const void* v, int64_t v_row_stride, int64_t v_head_stride,
                           vqv_dtype in_dtype, int heads, const vqv_cache* cache, int layer,
                           const vqv_seqs* seqs, const vqv_rope* rope, void* q_out,
                           void* hip_stream);

/*
 * out[r, e] = sum_j p_j v_j / sum_j p_j, p_j = exp(scale q[r, e] . k_j) over
 * the visible tokens j of the row's sequence and the key head e / (heads /
 * kv_heads): j <= the row's position, j < kv_len and, with window > 0, also
 * j > position - window or j < sinks. A row that sees nothing gives zeros.
 * Hidden tokens have no influence, whatever their slots hold.
 *   q, out     [n_rows, heads, dim] dense in the cache's type, 16-byte
 *              aligned; out may not overlap q.
 *   heads      a multiple of kv_heads, heads / kv_heads <= 1024.
 *   scale      finite and > 0.
 *   window     0 (none) or the tokens a row sees up to its own; sinks >= 0
 *              (used with a window only).
 *   dim        64, 80, 96, 128, 192 or 256 (else VQV_ERR_UNSUPPORTED).
 *   workspace  vqv_paged_attn_workspace_bytes bytes, 16-byte aligned; may be
 *              NULL when that is 0. Its contents on entry do not matter.
 * Scores, maxima, sums and the output are held in fp32. For the product with v
 * the weights p_j, relative to the largest so far, are held in two values of
 * the cache's type (to 2^-16 of a weight in bf16, 2^-22 in fp16) where max_rows
 * rows of a key head's queries are 64 or fewer, as in decoding and verify
 * blocks; for longer chunks they are rounded to one (half a step each, the
 * largest is exact). fp16 weights 2^29 below the largest are off by up to 2^-39
 * of it.
 */
size_t vqv_paged_attn_workspace_bytes(const vqv_cache* cache, const vqv_seqs* seqs, int heads,
                                      int window, int sinks);

vqv_status vqv_paged_attn(const void* q, const vqv_cache* cache, int layer, const vqv_seqs* seqs,
                          int heads, float scale, int window, int sinks, void* out,
                          void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * The book of a cache's pages.
 *   ref        [pages] int32: tables that hold the page; 0: free. Nothing is
 *              to be written to a page that several hold (vqv_rope_append and
 *              vqv_cache_compact do not see the book and cannot tell).
 *   table      [rows, width] int32, rows width apart; -1 where none.
 *   held       [rows] int32: pages of a row, table[row][0 .. held-1].
 *   length     [rows] int32: tokens of a row.
 */
typedef struct {
  int32_t* ref;
  int32_t* table;
  int32_t* held;
  int32_t* length;
  int pages, rows, width, page_size;
} vqv_pages;

/* Scratch of vqv_cache_fork and vqv_cache_reserve, 16-byte aligned. */
size_t vqv_cache_workspace_bytes(const vqv_pages* pages);

/*
 * Pages src[i] to dst[i] (int32, n of them), on all layers, k and v. No page
 * may be in dst twice or in both. A pair with a page outside the cache is
 * left out.
 */
vqv_status vqv_cache_copy(const vqv_cache* cache, const int32_t* src, const int32_t* dst, int n,
                          void* hip_stream);

/*
 * Gives back the pages of table rows past keep_len tokens: for each row i of
 * the n (row rows[i], or i when rows is NULL, then n <= pages->rows) the
 * pages from ceil(keep_len[i] / page_size) on lose one reference and leave
 * the table; held and length are cut, and never grow. A negative length is 0;
 * a row outside the table is left out; of a row that is named several times
 * the shortest length counts.
 */
vqv_status vqv_cache_trim(const vqv_pages* pages, const int32_t* keep_len, const int32_t* rows,
                          int n, void* hip_stream);

/*
 * Takes free pages until row i holds ceil(goal_len[i] / page_size) of them
 * (all pages->rows rows, or the first n). Rows are served in their order, a
 * row's pages in theirs, from the free pages in the order of their numbers.
 * ok[i] (int32) is 1, or 0 for a row that got none: its goal is wider than
 * the table, its goal is past `length` and token `length` falls on a page that
 * other rows hold too, or the free pages do not reach for it (and then not for
 * any row after it that needs some). `length` is not changed.
 *   Such a page is left by a trim to inside the pages that a row shares with
 *   its branches. To go on from there, fork the row once more (the branch gets
 *   a copy of its own of that page), trim the row to 0 and use the branch.
 */
vqv_status vqv_cache_reserve(const vqv_pages* pages, const int32_t* goal_len, int n, int32_t* ok,
                             void* workspace, size_t workspace_bytes, void* hip_stream);

/*
 * Row child[i] becomes a branch of row parent[i] (int32, n <= pages->rows of
 * them): it shares the parent's full pages (their references grow) and gets a
 * copy of its last, partly filled page on a free page (in the order of i, the
 * lowest free numbers first), all layers, k and v. held and length are the
 * parent's, cut to its last token's page. ok[i] is 1, or 0 where nothing was
 * done: a row outside the table, a child that holds pages, is named twice
 * (the first stands) or is a parent of this call, a parent whose last, partly
 * filled page is none of the cache, or no page free for it. Entries of full
 * pages that are none are passed on as they are.
 */
vqv_status vqv_cache_fork(const vqv_cache* cache, const vqv_pages* pages, const int32_t* parent,
                          const int32_t* child, int n, int32_t* ok, void* workspace,
                          size_t workspace_bytes, void* hip_stream);

/*
 * Of every sequence's new rows, those with keep[row] != 0 (int32 [n_rows])
 * move together to the first of the new rows' places, in their order, on all
 * layers, k and v. new_len[b] (int32) = kv_len[b] - rows + kept rows. What is
 * in the places behind stays as it was. A row on a bad page is not moved, and
 * a place on a bad page is not written.
 *   The bytes move as they are. A prefix of the rows, which is what a greedy
 * verify confirms, moves nothing: the call then only forms new_len. A row that
 * is kept behind one that is not keeps the key that was turned for its old
 * place (vqv_rope_append gives row i position kv_len - n + i), and its values
 * are of a block in which it saw the dropped rows (vqv_paged_attn is causal by
 * row order). Such a row is right only where neither matters; else feed it
 * again.
 */
vqv_status vqv_cache_compact(const vqv_cache* cache, const vqv_seqs* seqs, const int32_t* keep,
                             int32_t* new_len, void* hip_stream);

/*
 * What is done to the logits of each sequence b (rows b*T .. b*T+T-1 over n
 * tokens), in this order:
 *   penalties  where any of repetition, frequency, presence (fp32 [n_seqs])
 *              is given. count = counts[b][token] (int32 [n_seqs, n], NULL:
 *              0) plus how often the token is among the drafts fed at rows
 *              1..i; a token is used where count > 0. Where it is used or in
 *              the set `seen` (bits, int32 [n_seqs, ceil(n/32)], the lowest
 *              first; NULL: none), x = x > 0 ? x / repetition : x *
 *              repetition; then x -= frequency * count, and x -= presence
 *              where it is used. NULL: repetition 1, frequency and presence 0.
 *   biases     x += bias_value[e] for entries e = bias_start[b] ..
 *              bias_start[b+1]-1 with token bias_token[e]; of entries with the
 *              same token the last one counts; a token outside [0, n) is left
 *              out. n_bias is the length of the entries' arrays.
 *   mask       (per call) x = -inf where the row's bit is not set.
 * Each step is one rounding in fp32.
 */
typedef struct {
  int n_seqs, n;
  const int32_t* counts;
  const int32_t* seen;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int32_t* bias_start; /* [n_seqs + 1], or NULL: no biases */
  const int32_t* bias_token;
  const float* bias_value;
  int n_bias;
  int reserved;
} vqv_edits;

/*
 * out = edited logits [B*T, n] fp32; out may be logits itself (no other
 * overlap). draft as in vqv_verify (NULL: none are counted), mask int32
 * [B*T, ceil(n/32)] or NULL. B = edits->n_seqs, 1 <= T <= 64, B*T*n < 2^31,
 * n <= 2^31 - 4096 (else VQV_ERR_UNSUPPORTED).
 * 16-byte aligned logits and out.
 */
vqv_status vqv_logits_edit(const float* logits, const vqv_edits* edits, const int32_t* draft,
                           int T, const int32_t* mask, float* out, void* hip_stream);

/*
 * vqv_verify_ex of the edited logits, which are not written. draft (not NULL
 * when T > 1), draft_len, argmax, accept_len, margin and the workspace
 * (vqv_verify_workspace_bytes) as there. A row whose mask leaves nothing has
 * argmax 0 and margin 0 (+inf when n is 1).
 */
vqv_status vqv_logits_verify(const float* logits, const vqv_edits* edits, const int32_t* draft,
                             const int32_t* draft_len, int T, const int32_t* mask,
                             int32_t* argmax, int32_t* accept_len, float* margin,
                             void* workspace, size_t workspace_bytes, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* VQV_ROUND_H */
