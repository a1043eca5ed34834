// Rotary positions and the append to a 4-bit paged cache (vqv_rope_append_q4),
// and the new rows read back from it (vqv_cache_q4_read).
//
// As in rope.hip one work-group takes one row, all of its heads, and forms the
// row's sines and cosines once. Here they are 64-bit values, and keys are turned
// in 64 bits and rounded once: a code changes where a value passes a border, and
// two fp32 rotations that round differently would end at different codes.
// Queries are turned in fp32. A thread takes 8 values of a head; four
// neighbouring threads hold a group of 32, exchange its least and largest value,
// and write its 16 bytes of codes, the first of them its scale and bias.
//
// What bounds it, with 32 query heads and 8 key heads of 128: 8 rows take 9 us, the
// chain of row, length, page, sine and rotation; 4 ragged chunks of up to 2048 rows
// 30 to 34 us, as a row's own values are asked for behind that chain; with the read of
// the new rows in fp32 (12 us) 45 us for 141 MB, 3.1 TB/s.

#include "round_common.h"
#include "serve_internal.h"

namespace vqv {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxDim = 256;

struct RopeArgs {
  RowsIn q, k, v;
  void* q_out;
  char* kc;  // of the layer
  char* vc;
  int64_t page_stride, slot_stride, head_stride;
  int pages, page_size, kv_heads, dim, record;
  vqv_seqs seqs;
  int heads;
  vqv_rope rope;
};

template <typename T>
struct Vec8 {
  T v[8];
};

// Where a row stands: its position, and its slot's offset in the layer
// (page < 0: none).
struct Place {
  int64_t pos, at;
  int page;
};

__device__ __forceinline__ bool find_row(const vqv_seqs& s, int r, int page_size, int pages,
                                         int64_t page_stride, int64_t slot_stride, Place& p) {
  const int b = seq_of_row(s.row_start, s.n_seqs, r);
  if (b >= s.n_seqs) return false;
  const int first = s.row_start[b], next = s.row_start[b + 1];
  if (r < first) return false;
  p.pos = (int64_t)s.kv_len[b] - (next - first) + (r - first);
  const int pos = (int)(p.pos < -1 ? -1 : p.pos);  // of the cache: -1 is none
  p.page = page_of(s, b, pos, page_size, pages);
  p.at = (int64_t)p.page * page_stride + (int64_t)(pos % page_size) * slot_stride;
  return true;
}

__device__ __forceinline__ float cut(float x) {
  return x > 32768.0f ? 32768.0f : x < -32768.0f ? -32768.0f : x;  // a NaN stays
}

// Writes 8 values of a group as codes; lanes 4i .. 4i+3 hold the group (those
// without values of it have none).
__device__ __forceinline__ void store_codes(const float* x, bool has, int piece, char* record,
                                            int dim, int zeros, int record_bytes) {
  float lo = __builtin_inff(), hi = -__builtin_inff();
  bool nan = false;
  if (has) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      lo = fminf(lo, x[e]);
      hi = fmaxf(hi, x[e]);
      nan |= x[e] != x[e];
    }
  }
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    lo = fminf(lo, __shfl_xor(lo, d));
    hi = fmaxf(hi, __shfl_xor(hi, d));
    nan |= __shfl_xor((int)nan, d) != 0;
  }
  if (!has) return;
  const float none = __uint_as_float(0x7FC00000u);
  float step = (hi - lo) * (1.0f / 15.0f);
  asm("" : "+v"(step));  // rounded to fp32 first: not one instruction with the next rounding
  const _Float16 scale = (_Float16)(nan ? none : step);
  const _Float16 bias = (_Float16)(nan ? none : lo) + (_Float16)0.0f;  // of zeros: +0
  const float s = (float)scale, b = (float)bias, inv = 1.0f / s;
  unsigned w = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float c = s > 0.0f ? fminf(fmaxf(rintf((x[e] - b) * inv), 0.0f), 15.0f) : 0.0f;
    w |= (unsigned)c << (16 * (e & 1) + 4 * (e >> 1));
  }
  *reinterpret_cast<unsigned*>(record + 4 * piece) = w;
  if (piece % 4 == 0) {
    typedef __attribute__((ext_vector_type(2))) _Float16 h2;
    *reinterpret_cast<h2*>(record + dim / 2 + piece) = h2{scale, bias};
  }
  if (piece < zeros) *reinterpret_cast<unsigned*>(record + record_bytes - 4 * (piece + 1)) = 0u;
}

template <typename TIN, typename TQ>
__global__ __launch_bounds__(kThreads) void rope_append_q4(const RopeArgs a) {
  __shared__ double cs[kMaxDim], sn[kMaxDim];  // of the first rot values of a head
  const int r = blockIdx.x;
  Place p;
  if (!find_row(a.seqs, r, a.page_size, a.pages, a.page_stride, a.slot_stride, p)) return;
  const int D = a.dim, rot = a.rope.rot, half = rot >> 1;
  const bool inter = a.rope.interleaved;

  for (int i = threadIdx.x; i < half; i += kThreads) {
    const double turns = (double)p.pos * a.rope.turns[i];
    double s, c;
    sincospi(2.0 * (turns - rint(turns)), &s, &c);
    s *= a.rope.mscale;
    c *= a.rope.mscale;
    const int e = inter ? 2 * i : i, o = inter ? 2 * i + 1 : i + half;
    cs[e] = c;
    cs[o] = c;
    sn[e] = -s;  // y_e = x_e cos - x_o sin,  y_o = x_o cos + x_e sin
    sn[o] = s;
  }
  __syncthreads();

  const int per = D >> 3;  // 8-value pieces of a head
  const auto partners = [&](const TIN* x, int e0, const float* y, float* other) {
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
  };
  const auto load8 = [](const TIN* x, float* y) {
    const Vec8<TIN> v = *reinterpret_cast<const Vec8<TIN>*>(x);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = (float)v.v[e];
  };

  // Keys and values; a head's pieces in sets of 4.
  const int hk = a.kv_heads, padded = (per + 3) & ~3;
  const int zeros = (a.record - D / 2 - (D + 31) / 32 * 4) / 4;
  if (p.page >= 0) {
    for (int item = threadIdx.x; item < 2 * hk * padded; item += kThreads) {
      const int h = item / padded, piece = item % padded, e0 = piece * 8;
      const bool has = piece < per, key = h < hk;
      const RowsIn& in = key ? a.k : a.v;
      const int hh = key ? h : h - hk;
      float y[8] = {};
      if (has) {
        const TIN* x = static_cast<const TIN*>(in.p) + (int64_t)r * in.row_stride +
                       (int64_t)hh * in.head_stride;
        load8(x + e0, y);
        if (key && e0 < rot) {
          float other[8];
          partners(x, e0, y, other);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e0 + e < rot) y[e] = (float)(y[e] * cs[e0 + e] + other[e] * sn[e0 + e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = cut(y[e]);
      }
      store_codes(y, has, piece, (key ? a.kc : a.vc) + p.at + (int64_t)hh * a.head_stride, D,
                  zeros, a.record);
    }
  }

  for (int item = threadIdx.x; item < a.heads * per; item += kThreads) {
    const int h = item / per, e0 = (item % per) * 8;
    const TIN* x = static_cast<const TIN*>(a.q.p) + (int64_t)r * a.q.row_stride +
                   (int64_t)h * a.q.head_stride;
    float y[8];
    load8(x + e0, y);
    if (e0 < rot) {
      float other[8];
      partners(x, e0, y, other);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e0 + e < rot) y[e] = y[e] * (float)cs[e0 + e] + other[e] * (float)sn[e0 + e];
    }
    Vec8<TQ> w;
#pragma unroll
    for (int e = 0; e < 8; ++e) w.v[e] = (TQ)y[e];
    *reinterpret_cast<Vec8<TQ>*>(static_cast<TQ*>(a.q_out) + ((int64_t)r * a.heads + h) * D + e0) =
        w;
  }
}

struct ReadArgs {
  const char* kc;
  const char* vc;
  int64_t page_stride, slot_stride, head_stride;
  int pages, page_size, kv_heads, dim;
  vqv_seqs seqs;
  void* k_out;
  void* v_out;
};

template <typename T>
__global__ __launch_bounds__(kThreads) void cache_q4_read(const ReadArgs a) {
  const int r = blockIdx.x;
  Place p;
  if (!find_row(a.seqs, r, a.page_size, a.pages, a.page_stride, a.slot_stride, p)) return;
  const int D = a.dim, per = D >> 3, hk = a.kv_heads;
  for (int item = threadIdx.x; item < 2 * hk * per; item += kThreads) {
    const int h = item / per, piece = item % per;
    const bool key = h < hk;
    const int hh = key ? h : h - hk;
    T* out = static_cast<T*>(key ? a.k_out : a.v_out);
    if (!out) continue;
    Vec8<T> w = {};
    if (p.page >= 0) {
      const char* rec = (key ? a.kc : a.vc) + p.at + (int64_t)hh * a.head_stride;
      const unsigned codes = *reinterpret_cast<const unsigned*>(rec + 4 * piece);
      typedef __attribute__((ext_vector_type(2))) _Float16 h2;
      const h2 sb = *reinterpret_cast<const h2*>(rec + D / 2 + piece / 4 * 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float x = fmaf((float)(codes >> (16 * (e & 1) + 4 * (e >> 1)) & 15u), (float)sb[0],
                       (float)sb[1]);
        asm("" : "+v"(x));  // rounded to fp32: an fp16 product and sum in one would not be
        w.v[e] = (T)x;
      }
    }
    *reinterpret_cast<Vec8<T>*>(out + ((int64_t)r * hk + hh) * D + 8 * piece) = w;
  }
}

template <typename TIN>
hipError_t launch_in(const RopeArgs& a, int q_dtype, hipStream_t stream) {
  const dim3 grid(a.seqs.n_rows), block(kThreads);
  if (q_dtype == VQV_BF16)
    hipLaunchKernelGGL((rope_append_q4<TIN, __bf16>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((rope_append_q4<TIN, _Float16>), grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope_append_q4(const RowsIn& q, const RowsIn& k, const RowsIn& v, int in_dtype,
                                 int heads, const vqv_cache_q4& c, int layer, const vqv_seqs& seqs,
                                 const vqv_rope& rope, void* q_out, int q_dtype,
                                 hipStream_t stream) {
  const RopeArgs a{q,
                   k,
                   v,
                   q_out,
                   static_cast<char*>(c.k) + layer * c.layer_stride,
                   static_cast<char*>(c.v) + layer * c.layer_stride,
                   c.page_stride,
                   c.slot_stride,
                   c.head_stride,
                   c.pages,
                   c.page_size,
                   c.kv_heads,
                   c.dim,
                   q4_record_bytes(c.dim),
                   seqs,
                   heads,
                   rope};
  if (in_dtype == VQV_FP32) return launch_in<float>(a, q_dtype, stream);
  if (in_dtype == VQV_BF16) return launch_in<__bf16>(a, q_dtype, stream);
  return launch_in<_Float16>(a, q_dtype, stream);
}

hipError_t launch_cache_q4_read(const vqv_cache_q4& c, int layer, const vqv_seqs& seqs,
                                void* k_out, void* v_out, int out_dtype, hipStream_t stream) {
  const ReadArgs a{static_cast<const char*>(c.k) + layer * c.layer_stride,
                   static_cast<const char*>(c.v) + layer * c.layer_stride,
                   c.page_stride,
                   c.slot_stride,
                   c.head_stride,
                   c.pages,
                   c.page_size,
                   c.kv_heads,
                   c.dim,
                   seqs,
                   k_out,
                   v_out};
  const dim3 grid(seqs.n_rows), block(kThreads);
  if (out_dtype == VQV_FP32)
    hipLaunchKernelGGL(cache_q4_read<float>, grid, block, 0, stream, a);
  else if (out_dtype == VQV_BF16)
    hipLaunchKernelGGL(cache_q4_read<__bf16>, grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL(cache_q4_read<_Float16>, grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace vqv
