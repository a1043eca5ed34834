/*
 * vqv_serve.h - C ABI of libvqv's operators for batches of many requests on
 * MI355X (gfx950), each with a history, a sampling and an adapter of its own:
 *
 *   vqv_rope_append_q4    vqv_rope_append into a paged cache held in 4 bits,
 *   vqv_cache_q4_read     the new rows as that cache holds them,
 *   vqv_paged_attn_q4     vqv_paged_attn over it.
 *   vqv_verify_sampled    drafted tokens verified against the target's
 *                         probabilities, from given random numbers.
 *   vqv_lora_add          low-rank adapters, one per row's request, added to a
 *                         projection's output.
 *
 * Memory, streams, errors and threads are as in vqv.h and vqv_round.h: device
 * memory owned by the caller, asynchronous launches on the caller's stream,
 * arguments checked on the host before the first launch, nothing allocated and
 * nothing kept. All calls are deterministic and can be captured into a HIP
 * graph. Calls that share a workspace must not overlap in time.
 */
#ifndef VQV_SERVE_H
#define VQV_SERVE_H

#include "vqv_round.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Keys and values of all layers in pages of page_size tokens, 4 bits a value:
 * k and v hold a record per token and key head, [layers, pages, page_size,
 * kv_heads] of them, with the strides below in bytes (the same for k and v).
 *   dim        64, 80, 96, 128, 192 or 256 (else VQV_ERR_UNSUPPORTED).
 *   strides    multiples of 16, >= 0; k and v 16-byte aligned.
 *   A layer's pages span less than 2^32 units of 16 bytes (64 GiB) per tensor.
 *
 * A record is vqv_q4_record_bytes(dim) bytes (48, 64, 64, 80, 128 or 160):
 * dim/2 bytes of codes, then a scale and a bias in fp16 for each group of 32
 * values (the last of 80 is a group of 16), then zeros. Word w of the codes
 * (32 bits) holds values 8w .. 8w+7: value 8w + 2i + j in bits 16j + 4i .. +3.
 *     value = scale * code + bias.
 * vqv_rope_append_q4 makes them, every step in fp32, from a group's values x,
 * cut to +-32768: bias is the least value and scale (largest - least) * (1/15),
 * both rounded to fp16 (a bias of zero is +0), and code = round((x - bias) * (1 / scale)), ties to
 * even, cut to 0..15 (0 where scale is 0). A group with a NaN is NaN.
 *
 * Calls that move records as bytes (vqv_cache_copy, vqv_cache_fork,
 * vqv_cache_compact) take a vqv_cache over the same memory with dtype
 * VQV_BF16, dim = record bytes / 2 and strides in units of 2 bytes.
 */
typedef struct {
  void* k;
  void* v;
  int layers, pages, page_size, kv_heads, dim;
  int reserved;
  int64_t layer_stride, page_stride, slot_stride, head_stride;
} vqv_cache_q4;

/* Bytes of a record, 0 for a dim that is not supported. */
size_t vqv_q4_record_bytes(int dim);

/*
 * vqv_rope_append with the rows going to a 4-bit cache: arguments as there, and
 *   q_dtype    type of q_out, VQV_BF16 or VQV_FP16.
 * Keys are turned in 64 bits, sine and cosine included, and rounded once to
 * fp32 before they are quantised, so that codes do not depend on how an
 * fp32 rotation rounds; queries as in vqv_rope_append.
 */
vqv_status vqv_rope_append_q4(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                              const void* k, int64_t k_row_stride, int64_t k_head_stride,
                              const void* v, int64_t v_row_stride, int64_t v_head_stride,
                              vqv_dtype in_dtype, int heads, const vqv_cache_q4* cache, int layer,
                              const vqv_seqs* seqs, const vqv_rope* rope, void* q_out,
                              vqv_dtype q_dtype, void* hip_stream);

/*
 * k_out, v_out [n_rows, kv_heads, dim] dense, 16-byte aligned = the sequences'
 * new rows as layer `layer` holds them, in out_dtype (bf16, fp16 or fp32; each
 * value is formed in fp32 and rounded once more). Either may be NULL. A row on
 * a page that the cache lacks is zeros; rows that no sequence holds are left
 * as they were. The outputs may not overlap the cache or each other.
 */
vqv_status vqv_cache_q4_read(const vqv_cache_q4* cache, int layer, const vqv_seqs* seqs,
                             void* k_out, void* v_out, vqv_dtype out_dtype, void* hip_stream);

/*
 * vqv_paged_attn over a 4-bit cache: arguments and formula as there, k_j and
 * v_j being the records' values, and
 *   dtype      type of q and out, VQV_BF16 or VQV_FP16.
 * Scores, maxima, sums and the output are held in fp32. The matrix products
 * take fp16: values rounded once from scale * code + bias (2^-12 of a value; they
 * are to stay below 65504), keys so for bf16 queries and in two such numbers (to
 * 2^-22) for fp16 ones, bf16 queries times a power of two per row (a query value
 * 2^27 below its row's largest loses bits). The weights p_j, relative to the
 * largest so far, are rounded once too; for fp16 outputs they are two numbers
 * (to 2^-22) where max_rows rows of a key head's queries are 64 or fewer.
 * Weights 2^29 below the largest are off by up to 2^-39 of it.
 * The workspace of large bf16 calls without a window (prompt chunks) holds the
 * tokens of their sequences in fp16, beside what other calls need. Where they
 * would take more than 1 GiB they have 1 GiB, and the sequences that do not fit it
 * are read as in smaller calls: this share does not fall as a call grows.
 * vqv_paged_attn_q4_workspace_bytes is enough for either type, ..type_workspace_bytes
 * for queries of `dtype` (fp16 calls hold no such tokens). A call refuses a
 * workspace that is smaller than its own type's.
 */
size_t vqv_paged_attn_q4_workspace_bytes(const vqv_cache_q4* cache, const vqv_seqs* seqs,
                                         int heads, int window, int sinks);
size_t vqv_paged_attn_q4_type_workspace_bytes(const vqv_cache_q4* cache, const vqv_seqs* seqs,
                                              vqv_dtype dtype, int heads, int window, int sinks);

vqv_status vqv_paged_attn_q4(const void* q, vqv_dtype dtype, const vqv_cache_q4* cache, int layer,
                             const vqv_seqs* seqs, int heads, float scale, int window, int sinks,
                             void* out, void* workspace, size_t workspace_bytes,
                             void* hip_stream);

/*
 * Verify of one block per sequence by sampling: drafts are accepted, and the
 * token behind them drawn, so that every token is distributed as the target
 * alone would draw it.
 *   p_i = softmax(logits row b*T+i / temperature[b]) is the target's
 * probability of what follows row i, q_i the drafter's at draft i (fed at row
 * i+1). Drafts are taken in their order: draft i is accepted if
 *     uniform[b, i] * q_i(draft) < p_i(draft).
 * At the first that is not, token is drawn from r = max(p_i - q_i, 0) (from
 * p_i where r is zero everywhere); where all are accepted, from r = p of the
 * row behind the last draft. A draw takes the lowest token j with r_j > 0 and
 *     r_0 + .. + r_j > uniform[b, T-1] * (r_0 + .. + r_(N-1)),
 * or, where there is none, the last token with r_j > 0.
 *   logits       [B*T, N] fp32, rows as in vqv_verify (edited ones: form them
 *                with vqv_logits_edit first). 16-byte aligned.
 *   draft        [B, T-1] int32 (may be NULL when T == 1). A token outside
 *                [0, N) is not accepted.
 *   draft_probs  [B, T-1, N] fp32, or NULL: the drafts were not drawn, q_i is 1
 *                at the draft and 0 elsewhere. 16-byte aligned. Rows are used as
 *                they are; a draft whose own entry is NaN is rejected, and a
 *                token whose entry is NaN is not drawn from r.
 *   draft_len    [B] int32 or NULL, as in vqv_verify_ex.
 *   temperature  [B] fp32, or NULL: 1. Where it is 0 or less (or NaN) the
 *                request is greedy: p is 1 at the row's argmax as vqv_verify
 *                finds it and 0 elsewhere. A row that holds a NaN or +inf, or
 *                nothing but -inf, is taken so whatever the temperature.
 *   uniform      [B, T] fp32 in [0, 1).
 *   token        [B] int32, written; accept_len [B] int32, written: the drafts
 *                accepted (tokens committed = accept_len + 1).
 *   logprob      [B, T] fp32 or NULL, written: log p of the committed tokens at
 *                entries 0 .. accept_len, 0 behind them.
 *   B >= 1, 1 <= T <= 64, N >= 1, B*T*N < 2^31; B <= 65535 and N <= 2^31 - 4096
 *   (else VQV_ERR_UNSUPPORTED).
 *   workspace    vqv_verify_sampled_workspace_bytes(B, T, N) bytes, 16-byte
 *                aligned; its contents on entry do not matter.
 * No output may overlap an input, another output or the workspace. Exponentials
 * and sums are formed in 64 bits: a drawn token lies next to the borders of its
 * neighbours, which among 10^5 tokens are as close as fp32 sums are off.
 */
size_t vqv_verify_sampled_workspace_bytes(int B, int T, int N);

vqv_status vqv_verify_sampled(const float* logits, const int32_t* draft, const float* draft_probs,
                              const int32_t* draft_len, const float* temperature,
                              const float* uniform, int B, int T, int N, int32_t* token,
                              int32_t* accept_len, float* logprob, void* workspace,
                              size_t workspace_bytes, void* hip_stream);

/*
 * Adapters of a projection: a [n, rank, K] and b [n, N, rank], dense, 16-byte
 * aligned, bf16 or fp16; scale [n] fp32 on the device; ranks [n] int32 on the
 * device or NULL (all `rank`): of adapter e the first ranks[e] are used (cut to
 * 0..rank); the others have no influence, whatever they hold, but are read: a call
 * costs what `rank` ranks cost.
 *   rank       a multiple of 8, 8..256; K a multiple of 8, 8 <= K <= 32768;
 *              1 <= N < 2^31 - 4096 (else VQV_ERR_ARG or, past the largest,
 *              VQV_ERR_UNSUPPORTED).
 */
typedef struct {
  const void* a;
  const void* b;
  const float* scale;
  const int32_t* ranks;
  int n, rank, K, N;
  int dtype; /* VQV_BF16 or VQV_FP16 */
  int reserved;
} vqv_adapters;

/*
 * out[m] = y[m] + scale[e] * (x[m] . a[e]^T) . b[e]^T, e = which[m]; rows whose
 * which[m] is outside [0, n) are out[m] = y[m].
 *   x          [M, K] dense in act_dtype: the adapters' type or VQV_FP32 (else
 *              VQV_ERR_UNSUPPORTED). 16-byte aligned.
 *   which      [M] int32, in any order; rows of one adapter next to one another
 *              read it once.
 *   y, out     [M, N] fp32, rows y_stride and out_stride elements apart (>= N):
 *              a projection's output or columns of a stacked one. 4-byte
 *              aligned (16-byte aligned rows are faster). out may be y itself
 *              with the same stride, else they may not overlap (other columns
 *              of the same rows do not).
 *   M          >= 0, M * N and M * K < 2^40, M < 2^22 (else
 *              VQV_ERR_UNSUPPORTED, as where a grid were too large: it is not
 *              while (M + 64) * min(n, 64) * (N + 1024) < 2^34).
 *   workspace  vqv_lora_add_workspace_bytes(adapters, M) bytes, 16-byte
 *              aligned; may be NULL when that is 0.
 * Products of 16-bit values are exact; sums, and the values between the two
 * products, are fp32.
 */
size_t vqv_lora_add_workspace_bytes(const vqv_adapters* adapters, int M);

vqv_status vqv_lora_add(const void* x, vqv_dtype act_dtype, const vqv_adapters* adapters,
                        const int32_t* which, int M, const float* y, int64_t y_stride, float* out,
                        int64_t out_stride, void* workspace, size_t workspace_bytes,
                        void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* VQV_SERVE_H */
