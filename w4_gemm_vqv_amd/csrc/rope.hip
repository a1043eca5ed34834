// Rotary positions and the append to a paged cache (vqv_rope_append).
//
// One work-group takes one row, all of its heads. Its first threads form the
// row's cosines and sines once, for all heads: the angle of position p in
// turns, p * f / (2 pi), in 64 bits, less its nearest whole number, is at
// most half a turn, so the 32-bit sine and cosine lose nothing to a far
// position. Then each thread takes 8 consecutive values of a head at a time,
// q, k and v alike, and writes them as 16 bytes: q to q_out, k and v to the
// row's slot of the cache.
//
// The bound is memory: each value is read once from HBM and written once. 4
// chunks of up to 2048 rows of 48 heads of 128, bf16, interleaved pairs: 28.8
// us, 4.0 TB/s; with a row's heads over three work-groups 20 % more, as each
// forms the angles. In the half layout the partner of a value is a second read
// of the same lines, in pieces of 2 bytes: such chunks take 50 us. A block of 8
// rows takes 8.1 us, the chain of a row's sequence, length, page and rotation.

#include "round_common.h"
#include "round_internal.h"

namespace vqv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxDim = 256;

struct RopeArgs {
  RowsIn q, k, v;
  void* q_out;
  vqv_cache cache;  // k and v point at the layer
  vqv_seqs seqs;
  int heads;
  vqv_rope rope;
};

template <typename T>
struct Vec8 {
  T v[8];
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* x) {
  const Vec8<T> r = *reinterpret_cast<const Vec8<T>*>(p);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = (float)r.v[e];
}

template <typename TIN, typename TC>
__global__ __launch_bounds__(kThreads) void rope_append(const RopeArgs a) {
  __shared__ float cs[kMaxDim], sn[kMaxDim];  // of the first rot values of a head
  const int r = blockIdx.x;
  const int b = seq_of_row(a.seqs.row_start, a.seqs.n_seqs, r);
  if (b >= a.seqs.n_seqs) return;
  const int first = a.seqs.row_start[b], next = a.seqs.row_start[b + 1];
  if (r < first) return;
  const int64_t at_pos = (int64_t)a.seqs.kv_len[b] - (next - first) + (r - first);
  const int pos = (int)(at_pos < -1 ? -1 : at_pos);  // of the cache: -1 is none
  const int D = a.cache.dim, rot = a.rope.rot, half = rot >> 1;
  const bool inter = a.rope.interleaved;

  for (int i = threadIdx.x; i < half; i += kThreads) {
    const double turns = (double)at_pos * a.rope.turns[i];
    const float part = (float)(turns - rint(turns));
    float s, c;
    sincospif(2.0f * part, &s, &c);
    s *= a.rope.mscale;
    c *= a.rope.mscale;
    const int e = inter ? 2 * i : i, o = inter ? 2 * i + 1 : i + half;
    cs[e] = c;
    cs[o] = c;
    sn[e] = -s;  // y_e = x_e cos - x_o sin,  y_o = x_o cos + x_e sin
    sn[o] = s;
  }
  const int page = page_of(a.seqs, b, pos, a.cache.page_size, a.cache.pages);
  const int64_t at = (int64_t)page * a.cache.page_stride +
                     (int64_t)(pos % a.cache.page_size) * a.cache.slot_stride;
  __syncthreads();

  const int per = D >> 3;  // 8-value pieces of a head
  const int hk = a.cache.kv_heads;
  for (int item = threadIdx.x; item < (a.heads + 2 * hk) * per; item += kThreads) {
    const int h = item / per, e0 = (item % per) * 8;
    const int kind = h < a.heads ? 0 : h < a.heads + hk ? 1 : 2;
    if (kind && page < 0) continue;
    const RowsIn& in = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const int hh = kind == 0 ? h : kind == 1 ? h - a.heads : h - a.heads - hk;
    const TIN* x = static_cast<const TIN*>(in.p) + (int64_t)r * in.row_stride +
                   (int64_t)hh * in.head_stride;
    float y[8];
    load8(x + e0, y);
    if (kind < 2 && e0 < rot) {
      float other[8];
      if (inter) {
#pragma unroll
        for (int e = 0; e < 8; ++e) other[e] = y[e ^ 1];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = e0 + e;
          other[e] = c < rot ? (float)x[c < half ? c + half : c - half] : 0.0f;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e0 + e < rot) y[e] = y[e] * cs[e0 + e] + other[e] * sn[e0 + e];
    }
    TC* out;
    if (kind == 0)
      out = static_cast<TC*>(a.q_out) + ((int64_t)r * a.heads + hh) * D;
    else
      out = static_cast<TC*>(kind == 1 ? a.cache.k : a.cache.v) + at +
            (int64_t)hh * a.cache.head_stride;
    Vec8<TC> w;
#pragma unroll
    for (int e = 0; e < 8; ++e) w.v[e] = (TC)y[e];
    *reinterpret_cast<Vec8<TC>*>(out + e0) = w;
  }
}

template <typename TIN, typename TC>
hipError_t launch_t(const RopeArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((rope_append<TIN, TC>), dim3(a.seqs.n_rows), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

template <typename TIN>
hipError_t launch_in(const RopeArgs& a, hipStream_t stream) {
  return a.cache.dtype == VQV_BF16 ? launch_t<TIN, __bf16>(a, stream)
                                   : launch_t<TIN, _Float16>(a, stream);
}

}  // namespace

hipError_t launch_rope_append(const RowsIn& q, const RowsIn& k, const RowsIn& v, int in_dtype,
                              int heads, const vqv_cache& cache, int layer, const vqv_seqs& seqs,
                              const vqv_rope& rope, void* q_out, hipStream_t stream) {
  RopeArgs a{q, k, v, q_out, cache, seqs, heads, rope};
  a.cache.k = static_cast<uint16_t*>(cache.k) + layer * cache.layer_stride;
  a.cache.v = static_cast<uint16_t*>(cache.v) + layer * cache.layer_stride;
  if (in_dtype == VQV_FP32) return launch_in<float>(a, stream);
  if (in_dtype == VQV_BF16) return launch_in<__bf16>(a, stream);
  return launch_in<_Float16>(a, stream);
}

}  // namespace vqv
