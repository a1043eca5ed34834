// What the attention kernels over a paged cache share: matrix instructions and
// their operands, loads to LDS, the blocks of tokens that rows see, and the
// kernel that joins the partial sums of split sequences.
#pragma once

#include <limits.h>

#include "round_common.h"
#include "round_internal.h"

namespace vqv {
namespace {

typedef __attribute__((ext_vector_type(4))) unsigned u32x4;
typedef __attribute__((ext_vector_type(2))) unsigned u32x2;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(16))) float f32x16;

constexpr unsigned kNoPlace = ~0u;
constexpr float kLarge = 4096.0f;  // a shift below it is off by 2^-13 at most

// The sequences of a launch. Of a 4-bit cache those of many rows are read through
// a 16-bit copy (kCopied), the others from the cache itself.
enum { kAll, kCopied, kOthers };

// (row, head) pairs of one key head from which a sequence's tokens are copied.
constexpr int kCopiedPairs = 512;

struct AttnArgs {
  const void* q;
  void* out;
  const void* k;  // of the layer
  const void* v;
  vqv_seqs seqs;
  int page_size, pages, kv_heads, group;  // group: query heads per key head
  unsigned page_mul;                      // t / page_size = (t * page_mul) >> 32 >> page_shift
  int page_shift;                         // (page_mul 0: page_size is 1)
  unsigned page_units, slot_units, head_units;  // strides in 16-byte units
  float scale_log2;
  int window, sinks;
  int groups, split_blocks, splits;  // work-groups over a sequence's rows; of its tokens
  int which;                         // of kAll, kCopied, kOthers
  Copied copied;
  float* part;  // [n_rows * heads][splits][dim] sums, then [..][splits][2] (max, sum)
  float* part_ml;
};

template <typename T>
__device__ __forceinline__ f32x16 mfma(s16x8 a, s16x8 b, f32x16 c);
template <>
__device__ __forceinline__ f32x16 mfma<__bf16>(s16x8 a, s16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ f32x16 mfma<_Float16>(s16x8 a, s16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <typename T>
__device__ __forceinline__ unsigned pack2(float a, float b) {
  typedef __attribute__((ext_vector_type(2))) T t2;
  const t2 r = {(T)a, (T)b};
  return __builtin_bit_cast(unsigned, r);
}

template <typename T>
struct Bits;  // of a type: its exponent, 1, and log2 of the largest weight
template <>
struct Bits<__bf16> {
  static constexpr unsigned exponent = 0x7F80u, one = 0x3F80u;
  static constexpr float top = 0.0f;
};
template <>
struct Bits<_Float16> {
  static constexpr unsigned exponent = 0x7C00u, one = 0x3C00u;
  static constexpr float top = 15.0f;
};

// c + both values of w, in fp32.
template <typename T>
__device__ __forceinline__ float add2(unsigned w, float c);
template <>
__device__ __forceinline__ float add2<__bf16>(unsigned w, float c) {
  typedef __attribute__((ext_vector_type(2))) __bf16 t2;
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(t2, w),
                                         t2{(__bf16)1.0f, (__bf16)1.0f}, c, false);
}
template <>
__device__ __forceinline__ float add2<_Float16>(unsigned w, float c) {
  typedef __attribute__((ext_vector_type(2))) _Float16 t2;
  return __builtin_amdgcn_fdot2(__builtin_bit_cast(t2, w),
                                t2{(_Float16)1.0f, (_Float16)1.0f}, c, false);
}

// a and b (0 or more), cut to T, and what that leaves. The rest is never 0
// unless the weight is, so that the product of both with an infinity is one.
template <typename T>
__device__ __forceinline__ u32x2 split2(float a, float b);
template <>
__device__ __forceinline__ u32x2 split2<__bf16>(float a, float b) {
  constexpr float up = 1.0f + 0x1p-22f;
  const unsigned x = __float_as_uint(a), y = __float_as_uint(b);
  return u32x2{__builtin_amdgcn_perm(y, x, 0x07060302u),
               pack2<__bf16>(fmaf(a, up, -__uint_as_float(x & 0xFFFF0000u)),
                             fmaf(b, up, -__uint_as_float(y & 0xFFFF0000u)))};
}
template <>
__device__ __forceinline__ u32x2 split2<_Float16>(float a, float b) {
  constexpr float least = 0x1p-24f;
  const auto r = __builtin_amdgcn_cvt_pkrtz(a, b);
  return u32x2{__builtin_bit_cast(unsigned, r),
               pack2<_Float16>(__builtin_amdgcn_fmed3f(a - (float)r[0], least, a),
                               __builtin_amdgcn_fmed3f(b - (float)r[1], least, b))};
}

// The power of two that brings a bf16 row, of which `top` is the largest
// magnitude's bits, to between 2^10 and 2^11.
__device__ __forceinline__ int shift_to_half(unsigned top) {
  const int e = max((int)(top >> 7), 1) - 127;
  return top != 0 && top < 0x7F80u ? 10 - e : 0;
}

// 8 bf16 values as fp16 times 2^e.
__device__ __forceinline__ s16x8 scaled_to_half(s16x8 v, int e) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = ldexpf(__uint_as_float((unsigned)(unsigned short)v[2 * i] << 16), e);
    const float b = ldexpf(__uint_as_float((unsigned)(unsigned short)v[2 * i + 1] << 16), e);
    r[i] = pack2<_Float16>(a, b);
  }
  return __builtin_bit_cast(s16x8, r);
}

// The scale of the scores of a row that is 2^e times itself, within fp32's normal range: as 0 or an
// infinity it would turn a hidden score or a difference of 0 into NaN. At the bounds it stands for, all
// weights of a row are the same or all but the largest 0, as of the true scale.
__device__ __forceinline__ float scale_of_row(float scale_log2, int e) {
  return fminf(fmaxf(ldexpf(scale_log2, -e), 0x1p-126f), 0x1p127f);
}

// Not 0 where one of two packed values is an infinity or NaN: an exponent of
// ones carries into the sign's place.
template <typename T>
__device__ __forceinline__ unsigned not_finite(unsigned w) {
  constexpr unsigned e = Bits<T>::exponent, low = e & (0u - e);
  return ((w & (e | e << 16)) + (low | low << 16)) & 0x80008000u;
}

// Values with 0 in the place of infinities and NaN.
template <typename T>
__device__ __forceinline__ s16x8 finite(s16x8 v) {
  u32x4 w = __builtin_bit_cast(u32x4, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] &= ~((not_finite<T>(w[i]) >> 15) * 0xFFFFu);
  return __builtin_bit_cast(s16x8, w);
}

// Adds to o what the infinities and NaN of a column come to: where a row sees
// one, the infinity, or both (NaN). Which rows see one is a product of zeros
// and ones, over the 16-token steps of a block; `seen` holds a lane's bits of
// the tokens that its query row sees, 8 to a step.
template <typename T, int STEPS, typename F>
__device__ __forceinline__ void add_not_finite(F values, unsigned seen, f32x16& o) {
  constexpr unsigned e = Bits<T>::exponent;
  f32x16 a = {}, b = {};
#pragma unroll 1
  for (int u = 0; u < STEPS; ++u) {
    const s16x8 v = values(u);
    s16x8 up = {}, down = {}, see = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const unsigned w = (unsigned short)v[i];
      const bool out = (w & e) == e, nan = out && (w & 0x7FFFu) != e;
      up[i] = out && (nan || !(w & 0x8000u)) ? Bits<T>::one : 0;
      down[i] = out && (nan || (w & 0x8000u)) ? Bits<T>::one : 0;
      see[i] = seen >> (8 * u + i) & 1u ? Bits<T>::one : 0;
    }
    a = mfma<T>(up, see, a);
    b = mfma<T>(down, see, b);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (a[i] != 0.0f) o[i] += __builtin_inff();
    if (b[i] != 0.0f) o[i] -= __builtin_inff();
  }
}

// Which 16-byte piece of a staged row of DC pieces holds piece c. Without the
// exchange the rows that one LDS access touches would begin in the same
// banks. Keys are read 8 rows at a time, one piece each; values 4 rows at a
// time, 4 pieces each.
template <int DC>
__device__ __forceinline__ int k_piece(int row, int c) {
  if (DC % 8 == 0) return c ^ (row & 7);
  if (DC == 12) return c ^ (row >> 2 & 1);
  return c;
}
template <int DC>
__device__ __forceinline__ int v_piece(int row, int c) {
  if (DC % 16 == 0) return c ^ ((row & 3) << 2);
  if (DC % 8 == 0) return c ^ ((row >> 1 & 1) << 2);
  return c;
}

__device__ __forceinline__ int page_index(const AttnArgs& a, int t) {
  return a.page_mul ? (int)(__umulhi((unsigned)t, a.page_mul) >> a.page_shift) : t;
}

// 4 bytes per lane, as load16_to_lds; staged() waits for both.
__device__ __forceinline__ void load4_to_lds(const void* from, unsigned lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :
               : "s"(lds), "v"(from)
               : "memory");
}

// All but the last FLIGHT loads of this wave are there, and then every wave's.
template <int FLIGHT>
__device__ __forceinline__ void staged() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"(FLIGHT) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The order of a run of N matrix instructions that each take an LDS read: the
// reads of AHEAD of them go first, and then one's with each (left to itself the
// compiler waits for more of them in turn: a prompt chunk takes 388 us, not 369).
template <int N, int AHEAD>
__device__ __forceinline__ void pipelined() {
  constexpr int ahead = N < AHEAD ? N : AHEAD;
  __builtin_amdgcn_sched_group_barrier(0x100, ahead, 0);
#pragma unroll
  for (int i = 0; i < N - ahead; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, ahead, 0);
}

// exp2((x - top) * scale), 0 where x is -inf (also when both are).
__device__ __forceinline__ float exp_of(float x, float top, float scale) {
  return x == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f((x - top) * scale);
}

// The lane's number, which the compiler cannot compute with ahead of a loop:
// for code that seldom runs, so that what it needs does not take registers
// from the loop.
__device__ __forceinline__ int lane_here() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

__device__ __forceinline__ float max_of_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// LDS addresses of a lane's share of the keys and values of a staged block, for
// its first piece; the other pieces are a constant away, or an exclusive or
// where the exchange of pieces reaches (stages begin at multiples of a row).
template <int D>
__device__ __forceinline__ unsigned key_address(int lane) {
  const int row = lane & 31;
  return row * D * 2 + k_piece<D / 8>(row, lane >> 5) * 16;
}
template <int D>
__device__ __forceinline__ unsigned value_address(int lane) {
  const int row = 4 * (lane >> 5) + (lane >> 2 & 3);
  const int col = 16 * (lane >> 4 & 1) + 4 * (lane & 3);
  return row * D * 2 + v_piece<D / 8>(row, col >> 3) * 16 + (col & 7) * 2;
}

// Keys of 32 tokens (u) and 16 columns (x), as the A operand.
template <int D>
__device__ __forceinline__ s16x8 keys(unsigned at, int u, int x) {
  at = D / 8 % 8 == 0 ? (at ^ (x & 3) << 5) + (x >> 2) * 128 : at + x * 32;
  return *(__attribute__((address_space(3))) s16x8*)(at + u * 32 * D * 2);
}

// Values of 16 tokens (u) and 32 columns (d), as the A operand: lane l of 16
// reads 4 columns of token l / 4 and gets 4 tokens of column l % 16.
template <int D>
__device__ __forceinline__ s16x8 values(unsigned at, int u, int d) {
  at = D / 8 % 16 == 0  ? (at ^ (d & 3) << 6) + (d >> 2) * 256
       : D / 8 % 8 == 0 ? (at ^ (d & 1) << 6) + (d >> 1) * 128
                        : at + d * 64;
  s16x4 v[2];
#pragma unroll
  for (int y = 0; y < 2; ++y)
    v[y] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)(at + (16 * u + 8 * y) * D * 2));
  return __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7);
}

// A block whose values hold infinities or NaN, some rows not seeing all of its
// tokens. A function of its own: it seldom runs, and takes no registers from
// the loop. `seen` are the bits of the tokens that the lane's row sees.
// Weights of 16 tokens in one value each of the cache's type, or in two.
struct Weights {
  s16x8 high, low;
};

template <int DB, int SUB>
struct BadBlock {
  f32x16 o[DB];
  Weights weights[2 * SUB];
};

template <typename T, int D, int SUB, bool FINE>
__device__ __attribute__((noinline)) void product_with_bad_values(
    BadBlock<(D + 31) / 32, SUB>& x, unsigned seen, unsigned vs) {
  vs += value_address<D>(threadIdx.x & 63);
#pragma unroll
  for (int d = 0; d < (D + 31) / 32; ++d) {
    f32x16 o = x.o[d];
    add_not_finite<T, 2 * SUB>([&](int u) { return values<D>(vs, u, d); }, seen, o);
#pragma unroll
    for (int u = 0; u < 2 * SUB; ++u) {
      const s16x8 v = finite<T>(values<D>(vs, u, d));
      o = mfma<T>(v, x.weights[u].high, o);
      if (FINE) o = mfma<T>(v, x.weights[u].low, o);
    }
    x.o[d] = o;
  }
}

// The tokens that the rows of a tile see, as blocks of BT tokens: `sink`
// blocks from token 0 on, then those from block `first` on; `all` in total.
// Rows before the first token (a sequence shorter than its rows) see nothing;
// with the widest window their lower bound would pass 32 bits.
struct Blocks {
  int sink, first, all;
};

template <int BT>
__device__ __forceinline__ Blocks visible_blocks(int p0, int p1, int kv_len, int window,
                                                 int sinks) {
  const int hi = p1 < kv_len ? p1 + 1 : kv_len;
  if (hi <= 0) return Blocks{0, 0, 0};
  const int lo = window > 0 ? min(max(max(p0, 0) - window + 1, 0), hi) : 0;
  const int sink_end = min(sinks, lo);
  Blocks r;
  r.sink = window > 0 && sink_end > 0 ? (sink_end + BT - 1) / BT : 0;
  const int last = (hi + BT - 1) / BT;
  r.sink = min(r.sink, last);
  r.first = max(lo / BT, r.sink);
  r.all = r.sink + max(last - r.first, 0);
  return r;
}

// Tokens of a sequence that a table can hold; those past it are hidden. Places
// in blocks are counted in 32 bits, with room for a block more.
__device__ __forceinline__ int tokens_of(const AttnArgs& a, int kv_len) {
  const int64_t room = (int64_t)a.seqs.table_width * a.page_size;
  return (int)min((int64_t)kv_len, min(room, (int64_t)1 << 30));
}

__device__ __forceinline__ bool is_copied(const vqv_seqs& s, int b, int group, const Copied& c) {
  const int row0 = max(s.row_start[b], 0);
  const int n = min(min(s.row_start[b + 1], s.n_rows) - row0, s.max_rows);
  return n * group >= kCopiedPairs && s.kv_len[b] <= c.len &&
         (c.by_number ? b : row0 * group / kCopiedPairs) < c.slots;
}

__device__ __forceinline__ bool not_of_this_call(const AttnArgs& a, int b) {
  return a.which != kAll && is_copied(a.seqs, b, a.group, a.copied) != (a.which == kCopied);
}

// Blocks of a split: the plan's, or more where a sequence is longer than the
// plan was made for.
__device__ __forceinline__ int blocks_of_split(const AttnArgs& a, int all) {
  return max(a.split_blocks, (all + a.splits - 1) / a.splits);
}

// The rows of a work-group: tiles `first` and `second` (the same where there
// is no second), of `tiles` tiles of (row, head) pairs. PAIRS: two tiles, as
// far from the chunk's middle.
struct Tiles {
  int first, second;
};

template <bool PAIRS>
__device__ __forceinline__ Tiles tiles_of(int group, int tiles) {
  return Tiles{group, PAIRS ? tiles - 1 - group : group};
}
template <bool PAIRS>
__device__ __forceinline__ int group_of(int tile, int tiles) {
  return PAIRS ? min(tile, tiles - 1 - tile) : tile;
}

// Joins the partial sums of a (row, head): one work-group, 4 columns per
// thread, so that 1024 / D (rounded down) parts are read at the same time. SOME: the
// launch may be for some of the sequences.
template <typename T, int D, int BT, int ROWS, bool PAIRS, bool SOME>
__global__ __launch_bounds__(256) void paged_attn_join(const AttnArgs a) {
  constexpr int COLS = D / 4, SETS = 256 / COLS;
  __shared__ f32x4 sums[SETS][COLS];
  const int heads = a.kv_heads * a.group;
  const int r = blockIdx.x / heads, head = blockIdx.x % heads;
  const int b = seq_of_row(a.seqs.row_start, a.seqs.n_seqs, r);
  if (b >= a.seqs.n_seqs) return;
  const int row0 = max(a.seqs.row_start[b], 0);
  if (r < row0) return;
  const int n = min(min(a.seqs.row_start[b + 1], a.seqs.n_rows) - row0, a.seqs.max_rows);
  if (r - row0 >= n) return;
  const int g = a.group, tiles = (n * g + ROWS - 1) / ROWS;
  const int pos0 = max(a.seqs.kv_len[b], 0) - (a.seqs.row_start[b + 1] - a.seqs.row_start[b]);
  const int kv_len = tokens_of(a, a.seqs.kv_len[b]);
  if (SOME && not_of_this_call(a, b)) return;
  const Tiles tile =
      tiles_of<PAIRS>(group_of<PAIRS>(((r - row0) * g + head % g) / ROWS, tiles), tiles);
  const Blocks blocks =
      visible_blocks<BT>(pos0 + tile.first * ROWS / g,
                         pos0 + (min((tile.second + 1) * ROWS, n * g) - 1) / g, kv_len, a.window,
                         a.sinks);
  const int per_split = blocks_of_split(a, blocks.all);
  const int parts = (blocks.all + per_split - 1) / per_split;
  if (parts <= 1) return;  // written by the first kernel
  const int64_t at = (int64_t)blockIdx.x * a.splits;
  const float* ml = a.part_ml + 2 * at;
  const int lane = threadIdx.x & 63;
  float top = -__builtin_inff();
  for (int s = lane; s < parts; s += 64) top = fmaxf(top, ml[2 * s]);
#pragma unroll
  for (int d = 32; d; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
  float sum = 0.0f;
  for (int s = lane; s < parts; s += 64) sum += exp_of(ml[2 * s], top, a.scale_log2) * ml[2 * s + 1];
#pragma unroll
  for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);

  const int set = threadIdx.x / COLS, col = threadIdx.x % COLS;
  f32x4 o = {};
  if (set < SETS) {
    const float* part = a.part + at * D + 4 * col;
#pragma unroll 4
    for (int s = set; s < parts; s += SETS)
      o += exp_of(ml[2 * s], top, a.scale_log2) *
           *reinterpret_cast<const f32x4*>(part + (int64_t)s * D);
    sums[set][col] = o;
  }
  __syncthreads();
  if (set == 0) {
    for (int x = 1; x < SETS; ++x) o += sums[x][col];
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const u32x2 w = {pack2<T>(o[0] * inv, o[1] * inv), pack2<T>(o[2] * inv, o[3] * inv)};
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out) + (int64_t)blockIdx.x * D + 4 * col) =
        w;
  }
}

// What a call's arguments give the kernels, but for the cache's memory.
inline AttnArgs attn_args(const void* q, void* out, const vqv_seqs& seqs, int page_size, int pages,
                          int kv_heads, int heads, int dim, float scale, int window, int sinks,
                          void* workspace, const AttnPlan& plan) {
  AttnArgs a{};
  a.q = q;
  a.out = out;
  a.seqs = seqs;
  a.page_size = page_size;
  a.pages = pages;
  a.page_mul = 0;
  a.page_shift = 0;
  if (page_size > 1) {
    // ceil(2^(32 + shift) / page_size) with 2^shift < page_size <= 2^(shift + 1): exact for
    // tokens below 2^31.
    while ((2ll << a.page_shift) < page_size) ++a.page_shift;
    a.page_mul = (unsigned)(((1ull << (32 + a.page_shift)) + page_size - 1) / page_size);
  }
  a.kv_heads = kv_heads;
  a.group = heads / kv_heads;
  a.scale_log2 = fminf(scale * 1.4426950408889634f, 0x1p127f);
  a.window = window;
  a.sinks = window > 0 ? sinks : 0;
  a.groups = plan.groups;
  a.split_blocks = plan.split_blocks;
  a.splits = plan.splits;
  a.which = kAll;
  a.part = static_cast<float*>(workspace);
  a.part_ml = a.part + (size_t)seqs.n_rows * heads * plan.splits * dim;
  return a;
}

}  // namespace
}  // namespace vqv
