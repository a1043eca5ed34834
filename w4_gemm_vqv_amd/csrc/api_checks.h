// Checks of arguments that the entry points of include/vqv_round.h and
// include/vqv_serve.h share.
#pragma once

#include <math.h>
#include <stdint.h>

#include "round_internal.h"

namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Whether every non-NULL pointer of the list can hold int32 or fp32 values.
template <typename... P>
bool words_aligned(const P*... p) {
  return (... && aligned(p, 4));
}

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a && b && na && nb && a0 < b0 + nb && b0 < a0 + na;
}

inline vqv_status check_seqs(const vqv_seqs* s) {
  if (!s || !s->row_start || !s->kv_len || !s->table) return VQV_ERR_ARG;
  if (s->n_seqs < 1 || s->table_width < 1 || s->n_rows < 0 || s->max_rows < 0 || s->max_kv < 0 ||
      s->table_stride < s->table_width)
    return VQV_ERR_ARG;
  if (s->n_seqs > 65535) return VQV_ERR_UNSUPPORTED;
  if (!words_aligned(s->row_start, s->kv_len, s->table)) return VQV_ERR_ALIGN;
  return VQV_OK;
}

inline vqv_status status_of(hipError_t e) { return e == hipSuccess ? VQV_OK : VQV_ERR_HIP; }

// Bytes that the rows of a rotary call's q, k or v span.
inline size_t rows_span(int n_rows, int64_t row_stride, int64_t head_stride, int heads, int dim,
                        int esz) {
  return (size_t)((n_rows - 1) * row_stride + (heads - 1) * head_stride + dim) * esz;
}

}  // namespace
