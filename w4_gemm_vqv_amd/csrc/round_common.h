// Device helpers that the operators over a paged cache share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/vqv_round.h"

namespace vqv {

// Sequence of row r: how many of row_start[1..n_seqs] are <= r, counted by a
// whole wave (r uniform; a chain of one load where a search would have many).
// n_seqs where no sequence is left.
__device__ __forceinline__ int seq_of_row(const int32_t* __restrict__ row_start, int n_seqs,
                                          int r) {
  const int lane = threadIdx.x & 63;
  int b = 0;
  for (int c = 0; c < n_seqs; c += 64) {
    const int i = c + lane;
    b += __popcll(__ballot(i < n_seqs && row_start[i + 1] <= r));
  }
  return b;
}

// Page of token t of sequence b, or -1 where the table has none or a bad one.
__device__ __forceinline__ int page_of(const vqv_seqs& s, int b, int t, int page_size, int pages) {
  if (t < 0) return -1;
  const int j = t / page_size;
  if (j >= s.table_width) return -1;
  const int p = s.table[(int64_t)b * s.table_stride + j];
  return (unsigned)p < (unsigned)pages ? p : -1;
}

}  // namespace vqv
