// Internal launch interface between the entry points of include/vqv_round.h
// (round_api.hip) and their kernels. Arguments here are already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/vqv_round.h"
#include "vqv_internal.h"

namespace vqv {

// A slice of a stacked projection: pointer and strides in elements.
struct RowsIn {
  const void* p;
  int64_t row_stride, head_stride;
};

hipError_t launch_rope_append(const RowsIn& q, const RowsIn& k, const RowsIn& v, int in_dtype,
                              int heads, const vqv_cache& cache, int layer, const vqv_seqs& seqs,
                              const vqv_rope& rope, void* q_out, hipStream_t stream);

// How an attention call is cut (attn.hip): the query rows of a work-group, the
// blocks of tokens of a split, and the splits that the longest sequence has
// (1: no partials and no second kernel).
struct AttnPlan {
  int mw, kw, kt;      // waves over query rows, over tokens; tokens per wave
  int groups;          // of 32 * mw (row, head) pairs per sequence and key head
  int split_blocks;    // blocks of kw * kt tokens per split
  int splits;
};
bool attn_dim_supported(int dim);
AttnPlan attn_plan(const vqv_cache& cache, const vqv_seqs& seqs, int heads, int window, int sinks);
size_t attn_partial_bytes(const vqv_cache& cache, const vqv_seqs& seqs, int heads,
                          const AttnPlan& plan);
hipError_t launch_paged_attn(const void* q, const vqv_cache& cache, int layer,
                             const vqv_seqs& seqs, int heads, float scale, int window, int sinks,
                             void* out, void* workspace, const AttnPlan& plan,
                             hipStream_t stream);

hipError_t launch_cache_copy(const vqv_cache& cache, const int32_t* src, const int32_t* dst,
                             int n, hipStream_t stream);
hipError_t launch_cache_trim(const vqv_pages& pages, const int32_t* keep_len, const int32_t* rows,
                             int n, hipStream_t stream);
hipError_t launch_cache_reserve(const vqv_pages& pages, const int32_t* goal_len, int n,
                                int32_t* ok, int32_t* scratch, hipStream_t stream);
// int32 entries of scratch per table row (fork takes the most).
constexpr int kCacheScratchPerRow = 5;
hipError_t launch_cache_fork(const vqv_cache& cache, const vqv_pages& pages,
                             const int32_t* parent, const int32_t* child, int n, int32_t* ok,
                             int32_t* scratch, hipStream_t stream);
hipError_t launch_cache_compact(const vqv_cache& cache, const vqv_seqs& seqs, const int32_t* keep,
                                int32_t* new_len, hipStream_t stream);

hipError_t launch_logits_edit(const float* logits, const vqv_edits& edits, const int32_t* draft,
                              int T, const int32_t* mask, float* out, hipStream_t stream);
// Partials as verify_stage1 leaves them: verify_chunks(n) per row.
hipError_t launch_logits_verify(const float* logits, const vqv_edits& edits, const int32_t* mask,
                                const VerifyArgs& va, hipStream_t stream);

}  // namespace vqv
