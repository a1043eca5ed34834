// Device helpers that the operators over a paged cache share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/vqv_round.h"

namespace vqv {

typedef __attribute__((ext_vector_type(8))) short s16x8;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;

template <typename T>
__device__ __forceinline__ f32x4 mfma16(s16x8 a, s16x8 b, f32x4 c);
template <>
__device__ __forceinline__ f32x4 mfma16<__bf16>(s16x8 a, s16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x4 mfma16<_Float16>(s16x8 a, s16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// 16 bytes per lane from global memory to LDS at `lds` (uniform) + 16 * lane, without
// registers between. These are no loads to the compiler, which would wait for them
// before every LDS read: the caller waits for them. The no-op covers the write of m0,
// which nothing else here uses.
__device__ __forceinline__ void load16_to_lds(const void* from, unsigned lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(lds), "v"(from)
               : "memory");
}

template <typename V>
__device__ __forceinline__ V lds_read(unsigned at) {
  return *(__attribute__((address_space(3))) V*)(uintptr_t)at;
}

__device__ __forceinline__ unsigned lds_offset(const void* p) {
  return (unsigned)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

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
