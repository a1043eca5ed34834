// Internal launch interface between the entry points of include/vqv_serve.h
// (serve_api.hip) and their kernels. Arguments here are already validated.
#pragma once

#include "../../include/vqv_serve.h"
#include "round_internal.h"

namespace vqv {

// Bytes of a record: codes, a scale and a bias per group of 32, whole pieces
// of 16 bytes.
constexpr int q4_record_bytes(int dim) { return (dim / 2 + (dim + 31) / 32 * 4 + 15) / 16 * 16; }

hipError_t launch_rope_append_q4(const RowsIn& q, const RowsIn& k, const RowsIn& v, int in_dtype,
                                 int heads, const vqv_cache_q4& cache, int layer,
                                 const vqv_seqs& seqs, const vqv_rope& rope, void* q_out,
                                 int q_dtype, hipStream_t stream);
hipError_t launch_cache_q4_read(const vqv_cache_q4& cache, int layer, const vqv_seqs& seqs,
                                void* k_out, void* v_out, int out_dtype, hipStream_t stream);

AttnPlan attn_q4_plan(const vqv_cache_q4& cache, const vqv_seqs& seqs, int heads, int window,
                      int sinks);
// The sequences that are not `copied`.
hipError_t launch_paged_attn_q4(const void* q, int dtype, const vqv_cache_q4& cache, int layer,
                                const vqv_seqs& seqs, int heads, float scale, int window,
                                int sinks, const Copied& copied, void* out, void* workspace,
                                const AttnPlan& plan, hipStream_t stream);

// The tokens of sequences of many rows as fp16, in the workspace.
struct CopyPlan {
  Copied copied;  // slots 0: nothing is
  int width;      // pages of a sequence
  size_t values;  // bytes of keys (values); the pages' table is behind them
  size_t bytes;   // in all
  AttnPlan attn;
};
CopyPlan copy_plan(const vqv_cache_q4& cache, const vqv_seqs& seqs, int heads, int window);
vqv_cache copy_cache(const vqv_cache_q4& cache, const CopyPlan& plan, void* workspace);
vqv_seqs copy_seqs(const vqv_seqs& seqs, const CopyPlan& plan, void* workspace);
hipError_t launch_copy_q4(const vqv_cache_q4& cache, int layer, const vqv_seqs& seqs, int heads,
                          const CopyPlan& plan, void* workspace, hipStream_t stream);

struct SampleArgs {
  const float* logits;
  const int32_t* draft;
  const float* probs;
  const int32_t* draft_len;
  const float* temperature;
  const float* uniform;
  int B, T, N;
  int32_t* token;
  int32_t* accept_len;
  float* logprob;
  void* workspace;
};
size_t sample_workspace_bytes(int B, int T, int N);
hipError_t launch_verify_sampled(const SampleArgs& a, hipStream_t stream);

// Rows of a block of 64 that share an adapter (-1: none do).
struct __attribute__((aligned(16))) LoraSlot {
  uint64_t rows;
  int adapter;
};
struct LoraArgs {
  const void* x;
  vqv_adapters ad;
  const int32_t* which;
  int M;
  const float* y;
  int64_t y_stride;
  float* out;
  int64_t out_stride;
  void* workspace;
  // In the workspace: the blocks' slots, and the values between the products.
  LoraSlot* slots;
  float* low;
};
// Whether a call's grids are within 32 bits.
bool lora_grids_fit(const vqv_adapters& ad, int M);
size_t lora_workspace_bytes(const vqv_adapters& ad, int M);
hipError_t launch_lora_add(const LoraArgs& a, int act_dtype, hipStream_t stream);

}  // namespace vqv
