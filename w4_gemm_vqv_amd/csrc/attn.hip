// Attention of new rows over a paged cache (vqv_paged_attn).
//
// The query rows of a sequence that share a key head, (row, head) pairs with
// the head fastest, are cut into 32 per wave; a work-group of MW x KW waves
// walks over the visible tokens in blocks of KW * KT, staged in LDS STAGES
// deep, so that every wave reads each key and value once from there whatever
// the page size and layout. Wave (mw, kw) takes the mw-th 32 rows and the
// kw-th KT tokens of each block. With few query rows (plain decoding, verify
// blocks) the waves split the tokens (KW > 1), and long sequences are also
// split over work-groups, whose partial sums a second kernel joins. With many,
// eight waves share a block's loads: two tiles of 128 rows, one from the
// chunk's beginning and one from its end, so that all work-groups have as much
// to do (2048 rows of 32 heads over 10240 tokens: 369 us, with four waves and one
// tile 393). Under a window the two would not see the same tokens: one tile (3
// chunks of up to 1500 rows, window 1023: 75 us, with two tiles 105).
//
// Loads go to LDS without registers between, up to STAGES - 1 blocks ahead. A
// block's places in the cache are found before that: its entries of the page
// table are asked for 2 STAGES - 1 blocks ahead (to LDS too: a wait for a
// register would wait for all loads in flight), and turned into places STAGES
// blocks ahead, each block by another wave.
//
// A wave forms S^T = K Q^T with 32x32x16 matrix instructions: lane l holds 16
// scores of each 32 tokens for query row l % 32, so maxima and sums stay in
// the lane but for one exchange with lane l ^ 32. Accumulator rows of lane
// half h are the tokens 8i + 4h + 0..3; read as the B operand of O^T = V^T
// P^T these are the k slots 8h + 0..7 of a 16-token step if the step's tokens
// are taken in the order 4h..4h+3, 8+4h..8+4h+3. V^T is read in that order
// (the transposing LDS read gives a lane four tokens of one column), so P
// needs no exchange at all.
//
// Softmax runs with base-2 exponentials and a running maximum; scores, maxima,
// sums and outputs are fp32. P goes to the matrix instruction in the cache's
// type. Up to 64 (row, head) pairs, where memory bounds the kernel, it goes
// twice, cut to its bits and what that left over (to 2^-16 of a weight in bf16,
// 2^-22 in fp16): the outputs are then the fp32 form's but for the order of
// sums (decoding 349 us, rounded once 350; a block of 8 rows 15.6 and 15.2; 16
// blocks of 16 rows, dim 256, 78 and 76). Beyond that it is rounded once, an
// error of at most half a step of each weight, none of the largest, which the
// sum over tokens averages: a second product would take 478 us of a prompt
// chunk for 369, for an error of 1.66e-3 instead of 2.15e-3 (of which the
// output's own rounding is 1.66e-3). The largest weight is 1, in fp16 2^15 (the
// sum of weights is as much larger): with 1 a token 2^14 below it would lose
// bits, and thousands of them 2^25 below would be nothing.

#include <limits.h>

#include "round_common.h"
#include "round_internal.h"

namespace vqv {
namespace {

typedef __attribute__((ext_vector_type(4))) unsigned u32x4;
typedef __attribute__((ext_vector_type(2))) unsigned u32x2;
typedef __attribute__((ext_vector_type(4))) short s16x4;
typedef __attribute__((ext_vector_type(8))) short s16x8;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((ext_vector_type(4))) float f32x4;

constexpr unsigned kNoPlace = ~0u;
constexpr float kLarge = 4096.0f;  // a shift below it is off by 2^-13 at most

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

// 16 (4) bytes per lane from global memory to LDS at `lds` (uniform) + 16 (4)
// * lane, without registers between. These are no loads to the compiler, which
// would wait for them before every LDS read: staged() waits for them. The
// no-op covers the write of m0, which nothing else here uses.
__device__ __forceinline__ void load16_to_lds(const void* from, unsigned lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(lds), "v"(from)
               : "memory");
}
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

__device__ __forceinline__ unsigned lds_offset(const void* p) {
  return (unsigned)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
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

template <typename T, int D, int MW, int KW, int KT, int STAGES>
__global__ __launch_bounds__(MW * KW * 64, MW >= 4 && D <= 128 ? 2 : 1) void paged_attn(
    const AttnArgs a) {
  constexpr int NW = MW * KW, BT = KW * KT, DC = D / 8, DS = D / 16, DB = (D + 31) / 32;
  constexpr bool PAIRS = MW == 8;
  constexpr bool FINE = MW <= 2;
  constexpr int ROWS = PAIRS ? 128 : 32 * MW;        // (row, head) pairs of a tile
  constexpr int GROUPS = BT * DC / 64;               // of 64 pieces: a wave's access
  constexpr int LOADS = (GROUPS + NW - 1) / NW;      // per wave, of keys and of values
  constexpr int SUB = KT / 32;
  constexpr int STAGE = BT * D;                      // values of K (or V) of a block
  // Where D is not a multiple of 32 the last column block of V reads past its
  // row, at the end past its stage (the results are not used).
  constexpr int VSTAGE = STAGE + (D % 32 ? 32 : 0);
  constexpr int RING = 8;                            // blocks whose places are held
  static_assert(2 * STAGES - 1 <= RING && (STAGES & (STAGES - 1)) == 0, "");
  __shared__ __align__(1024) uint16_t lds[STAGES * (STAGE + VSTAGE)];
  __shared__ unsigned places[RING][BT];  // in the cache, in 16-byte units, or kNoPlace
  __shared__ int entries[RING][BT];      // of the page table
  __shared__ int holes;                  // not 0: a page was missing

  const int h = blockIdx.x % a.kv_heads;
  const int b = blockIdx.x / a.kv_heads % a.seqs.n_seqs;
  const int rest = blockIdx.x / a.kv_heads / a.seqs.n_seqs;
  const int group = a.groups - 1 - rest % a.groups;  // the longest first
  const int split = rest / a.groups;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int mw = wave % MW, kw = wave / MW;

  const int row0 = max(a.seqs.row_start[b], 0);
  const int n = min(min(a.seqs.row_start[b + 1], a.seqs.n_rows) - row0, a.seqs.max_rows);
  const int g = a.group, pairs = n * g;
  const int tiles = (pairs + ROWS - 1) / ROWS;
  if (n <= 0 || group >= (PAIRS ? (tiles + 1) / 2 : tiles)) return;
  const Tiles tile = tiles_of<PAIRS>(group, tiles);
  const int pos0 = max(a.seqs.kv_len[b], 0) - (a.seqs.row_start[b + 1] - a.seqs.row_start[b]);
  const int kv_len = tokens_of(a, a.seqs.kv_len[b]);
  const Blocks blocks =
      visible_blocks<BT>(pos0 + tile.first * ROWS / g,
                         pos0 + (min((tile.second + 1) * ROWS, pairs) - 1) / g, kv_len, a.window,
                         a.sinks);
  const int per_split = blocks_of_split(a, blocks.all);
  const int parts = max((blocks.all + per_split - 1) / per_split, 1);
  if (split >= parts) return;
  const int j0 = split * per_split, j1 = min(j0 + per_split, blocks.all);

  // This wave's rows, and this lane's with its values as the B operand.
  int m0 = (PAIRS ? mw < 4 ? tile.first : tile.second : tile.first) * ROWS + mw % (ROWS / 32) * 32;
  if (PAIRS && mw >= 4 && tile.first == tile.second) m0 = pairs;  // none
  const int p0 = pos0 + m0 / g, p1 = pos0 + (min(m0 + 32, pairs) - 1) / g;
  struct Row {
    bool real;
    int64_t index;  // of (row, head), densely
  };
  const auto row_of = [&](int lane) {
    const int m = m0 + (lane & 31), row = m / g;
    return Row{m < pairs, (int64_t)(row0 + row) * (a.kv_heads * g) + h * g + m - row * g};
  };
  const Row mine = row_of(lane);
  s16x8 qf[DS];
#pragma unroll
  for (int s = 0; s < DS; ++s) {
    qf[s] = s16x8{};
    if (mine.real)
      qf[s] = *reinterpret_cast<const s16x8*>(static_cast<const uint16_t*>(a.q) + mine.index * D +
                                              16 * s + 8 * (lane >> 5));
  }

  f32x16 o[DB];
#pragma unroll
  for (int d = 0; d < DB; ++d) o[d] = f32x16{};
  float mx = -__builtin_inff(), sum = 0.0f;

  const auto base_of = [&](int j) {
    return (j < blocks.sink ? j : blocks.first + j - blocks.sink) * BT;
  };

  const char* kbase = static_cast<const char*>(a.k) + (uint64_t)h * a.head_units * 16;
  const char* vbase = static_cast<const char*>(a.v) + (uint64_t)h * a.head_units * 16;
  const int32_t* table = a.seqs.table + (int64_t)b * a.seqs.table_stride;
  const auto place_of = [&](int t, int i, int entry) {
    if (t < kv_len && i < a.seqs.table_width && (unsigned)entry < (unsigned)a.pages)
      return (unsigned)entry * a.page_units + (unsigned)(t - i * a.page_size) * a.slot_units;
    if (t < kv_len) holes = 1;
    return kNoPlace;
  };
  // The wave whose turn block j is (or waves: 64 tokens each).
  constexpr int TURN = (BT + 63) / 64;
  const auto turn = [&](int j) { return (wave - (j - j0) * TURN) & (NW - 1); };
  const auto ask = [&](int j) {
    const int x = turn(j);
    if (j < j1 && x < TURN && (BT % 64 == 0 || lane < BT)) {
      const int i = min(page_index(a, base_of(j) + 64 * x + lane), a.seqs.table_width - 1);
      load4_to_lds(table + i,
                   __builtin_amdgcn_readfirstlane(lds_offset(&entries[(j - j0) % RING][64 * x])));
    }
  };
  const auto look_up = [&](int j) {
    const int x = turn(j);
    if (j < j1 && x < TURN && (BT % 64 == 0 || lane < BT)) {
      const int t = base_of(j) + 64 * x + lane;
      places[(j - j0) % RING][64 * x + lane] =
          place_of(t, page_index(a, t), entries[(j - j0) % RING][64 * x + lane]);
    }
  };
  // Piece p of a block's keys goes to LDS place p; it is piece k_piece(t, p %
  // DC) of token t = p / DC, and likewise for the values. A token that is none
  // is loaded from the cache's first place and masked.
  const auto load = [&](int j) {
    const int buf = (j - j0) % STAGES;
    const unsigned kl = lds_offset(lds) + buf * (STAGE + VSTAGE) * 2, vl = kl + STAGE * 2;
    const int lane = lane_here();
    unsigned place[LOADS];
#pragma unroll
    for (int x = 0; x < LOADS; ++x) {
      const int g0 = x * NW + wave;
      if (GROUPS % NW && g0 >= GROUPS) continue;
      place[x] = places[(j - j0) % RING][(g0 * 64 + lane) / DC];
    }
#pragma unroll
    for (int x = 0; x < LOADS; ++x) {
      const int g0 = x * NW + wave;
      if (GROUPS % NW && g0 >= GROUPS) continue;
      const int p = g0 * 64 + lane, t = p / DC, c = p % DC;
      const unsigned at = place[x] == kNoPlace ? 0u : place[x];
      load16_to_lds(kbase + (uint64_t)(at + k_piece<DC>(t, c)) * 16,
                    __builtin_amdgcn_readfirstlane(kl + g0 * 1024));
      load16_to_lds(vbase + (uint64_t)(at + v_piece<DC>(t, c)) * 16,
                    __builtin_amdgcn_readfirstlane(vl + g0 * 1024));
    }
  };

  // The waits for the query rows belong here, not in the loop behind loads.
#pragma unroll
  for (int x = 0; x < DS; ++x) asm volatile("" : "+v"(qf[x]));
  if (threadIdx.x == 0) holes = 0;
  __syncthreads();
  for (int x = threadIdx.x; x < (2 * STAGES - 1) * BT; x += NW * 64) {
    const int j = j0 + x / BT;
    if (j < j1) {
      const int t = base_of(j) + x % BT, i = page_index(a, t);
      places[x / BT][x % BT] =
          place_of(t, i, t < kv_len && i < a.seqs.table_width ? table[i] : -1);
    }
  }
  __syncthreads();
#pragma unroll
  for (int x = 0; x < STAGES - 1; ++x)
    if (j0 + x < j1) load(j0 + x);
  for (int j = j0; j < j1; ++j) {
    const int buf = (j - j0) % STAGES;
    // Block j is there for all, and all are done with block j - 1.
    if (STAGES > 2 && j + STAGES - 2 < j1)
      staged<(STAGES - 2) * 2 * (GROUPS / NW)>();
    else
      staged<0>();
    ask(j + 2 * STAGES - 1);
    if (j + STAGES - 1 < j1) load(j + STAGES - 1);
    if (j - j0 >= STAGES - 1) look_up(j + STAGES);

    const uint16_t* ks = lds + buf * (STAGE + VSTAGE) + kw * KT * D;
    const uint16_t* vs = lds + buf * (STAGE + VSTAGE) + STAGE + kw * KT * D;
    const int t0 = base_of(j) + kw * KT;
    // Nothing to see for these rows.
    if (t0 > p1 || m0 >= pairs ||
        (a.window > 0 && t0 + KT <= max(p0, 0) - a.window + 1 && t0 >= a.sinks))
      continue;

    f32x16 s[SUB];
    const unsigned ka = lds_offset(ks) + key_address<D>(lane);
    const unsigned va = lds_offset(vs) + value_address<D>(lane);
#pragma unroll
    for (int x = 0; x < DS; ++x)
#pragma unroll
      for (int u = 0; u < SUB; ++u)
        s[u] = mfma<T>(keys<D>(ka, u, x), qf[x], x ? s[u] : f32x16{});
    pipelined<SUB * DS, 4>();
    // Hidden tokens, and those without a page. Where every row sees every token
    // there is nothing to mask.
    bool full = t0 + KT - 1 <= p0 && (a.window == 0 || t0 > p1 - a.window);
    const bool whole = holes == 0;
    full = full && t0 + KT <= kv_len && whole;
    unsigned seen = 0;
    if (!full) {
      // Token t0 + 32 u + 8 (i / 4) + 4 half + i % 4, against the row's bounds.
      const int l = lane_here(), row = (m0 + (l & 31)) / g, half = l >> 5;
      const int hi = (m0 + (l & 31) < pairs ? pos0 + row : -1) - t0 - 4 * half;
      const int lo = a.window > 0 ? max(hi, -1) - a.window : INT_MIN;
      const int sink = a.sinks - t0 - 4 * half;
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        const unsigned paged =
            (unsigned)__ballot(places[(j - j0) % RING][kw * KT + 32 * u + (l & 31)] != kNoPlace) >>
            (4 * half);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int k = 8 * (i / 4) + (i & 3), r = 32 * u + k;
          const bool see = r <= hi && (r > lo || r < sink) && (paged >> k & 1u);
          s[u][i] = see ? s[u][i] : -__builtin_inff();
          seen |= (see ? 1u : 0u) << (16 * u + i);
        }
      }
    }
    float top = s[0][0];
#pragma unroll
    for (int u = 0; u < SUB; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[u][i]);
    top = max_of_halves(top);
    // The maximum that weights are relative to follows every score, so that
    // the largest weight is 1 and its rounding to the cache's type is exact.
    // (One that lags by up to 2^8 spares most blocks the scaling of the sums: 4 %
    // of a prompt chunk's time, 3 % of a windowed one's, nothing elsewhere; its
    // outputs are off by 9 to 18 % more, and a single large weight by half a step.)
    if (__any(top > mx)) {
      const float now = fmaxf(mx, top);
      const float back = exp_of(mx, now, a.scale_log2);
      mx = now;
      sum *= back;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= back;
    }
    const float base = mx == -__builtin_inff() ? 0.0f : mx;
    float shift = fmaf(base, a.scale_log2, -Bits<T>::top);
    // Of a large maximum the shift's rounding would be the weights' size: the
    // maximum is then taken off the scores first, which is exact near it.
    if (__any(fabsf(shift) > kLarge)) {
      shift = -Bits<T>::top;
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[u][i] -= base;
    }
    // The weights of 16 tokens, as the B operand of their product. FINE: in
    // two values each. Else the sum takes them as rounded, as the
    // product does.
    const auto weights = [&](int u) {
      u32x4 high, low = {};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float p[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          p[e] = __builtin_amdgcn_exp2f(
              fmaf(s[u / 2][8 * (u & 1) + 2 * i + e], a.scale_log2, -shift));
        if (FINE) {
          const u32x2 w = split2<T>(p[0], p[1]);
          high[i] = w[0];
          low[i] = w[1];
          sum += p[0] + p[1];
        } else {
          const unsigned w = pack2<T>(p[0], p[1]);
          high[i] = w;
          sum = add2<T>(w, sum);
        }
      }
      return Weights{__builtin_bit_cast(s16x8, high), __builtin_bit_cast(s16x8, low)};
    };

    // A hidden token's weight is 0, which an infinity or NaN of its values
    // would turn into NaN: where some rows do not see all tokens, such values
    // are looked for and left out of the product.
    bool bad = false;
    if (!full) {
      unsigned found = 0;
      for (int x = lane_here(); x < KT * DC; x += 64) {
        const u32x4 w = *reinterpret_cast<const u32x4*>(vs + x * 8);
#pragma unroll
        for (int e = 0; e < 4; ++e) found |= not_finite<T>(w[e]);
      }
      bad = __ballot(found != 0) != 0;
    }
    if (bad) {
      BadBlock<DB, SUB> x;
#pragma unroll
      for (int u = 0; u < 2 * SUB; ++u) x.weights[u] = weights(u);
#pragma unroll
      for (int d = 0; d < DB; ++d) x.o[d] = o[d];
      product_with_bad_values<T, D, SUB, FINE>(x, seen, lds_offset(vs));
#pragma unroll
      for (int d = 0; d < DB; ++d) o[d] = x.o[d];
    } else {
      // The next 16 tokens' weights are formed while the matrix unit works.
      Weights next = weights(0);
#pragma unroll
      for (int u = 0; u < 2 * SUB; ++u) {
        const Weights p = next;
#pragma unroll
        for (int d = 0; d < DB; ++d) {
          const s16x8 v = values<D>(va, u, d);
          o[d] = mfma<T>(v, p.high, o[d]);
          if (FINE) o[d] = mfma<T>(v, p.low, o[d]);
        }
        if (u + 1 < 2 * SUB) next = weights(u + 1);
      }
    }
  }
  sum += __shfl_xor(sum, 32);

  // Waves that split the tokens join their sums through LDS, half of them at
  // a time.
  if (KW > 1) {
    float* x = reinterpret_cast<float*>(lds);
    constexpr int PER = DB * 16 + 2;
#pragma unroll
    for (int w = KW / 2; w >= 1; w >>= 1) {
      __syncthreads();
      float* mine = x + (((kw % w) * MW + mw) * PER) * 64 + lane;
      if (kw >= w && kw < 2 * w) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) mine[(d * 16 + i) * 64] = o[d][i];
        mine[DB * 16 * 64] = mx;
        mine[(DB * 16 + 1) * 64] = sum;
      }
      __syncthreads();
      if (kw < w) {
        const float om = mine[DB * 16 * 64], os = mine[(DB * 16 + 1) * 64];
        const float top = fmaxf(mx, om);
        const float fa = exp_of(mx, top, a.scale_log2), fb = exp_of(om, top, a.scale_log2);
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[d][i] = o[d][i] * fa + mine[(d * 16 + i) * 64] * fb;
        sum = sum * fa + os * fb;
        mx = top;
      }
    }
    if (kw > 0) return;
  }

  const int l = lane_here(), half = l >> 5;
  const Row row = row_of(l);
  if (!row.real) return;
  if (parts == 1) {
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    uint16_t* out = static_cast<uint16_t*>(a.out) + row.index * D;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = 32 * d + 8 * i + 4 * half;
        if (col < D) {
          u32x2 w = {pack2<T>(o[d][4 * i] * inv, o[d][4 * i + 1] * inv),
                     pack2<T>(o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv)};
          *reinterpret_cast<u32x2*>(out + col) = w;
        }
      }
  } else {
    const int64_t at = row.index * a.splits + split;
    float* out = a.part + at * D;
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = 32 * d + 8 * i + 4 * half;
        if (col < D)
          *reinterpret_cast<f32x4*>(out + col) =
              f32x4{o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]};
      }
    if (half == 0) {
      a.part_ml[2 * at] = mx;
      a.part_ml[2 * at + 1] = sum;
    }
  }
}

// Joins the partial sums of a (row, head): one work-group, 4 columns per
// thread, so that 1024 / D (rounded down) parts are read at the same time.
template <typename T, int D, int BT, int ROWS, bool PAIRS>
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

template <typename T, int D, int MW, int KW, int KT, int STAGES>
hipError_t launch_shape(const AttnArgs& a, hipStream_t stream) {
  const int64_t grid = (int64_t)a.kv_heads * a.seqs.n_seqs * a.groups * a.splits;
  hipLaunchKernelGGL((paged_attn<T, D, MW, KW, KT, STAGES>), dim3((unsigned)grid),
                     dim3(MW * KW * 64), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL((paged_attn_join<T, D, KW * KT, MW == 8 ? 128 : 32 * MW, MW == 8>),
                     dim3((unsigned)(a.seqs.n_rows * a.kv_heads * a.group)), dim3(256), 0, stream,
                     a);
  return hipGetLastError();
}

// Waves that split the tokens of a block while there are few query rows. Two
// work-groups then fit a CU's LDS, and one's loads fill the other's pauses.
constexpr int token_waves(int dim) { return dim <= 64 ? 4 : dim <= 128 ? 2 : 1; }

template <typename T, int D>
hipError_t launch_dim(const AttnArgs& a, const AttnPlan& p, hipStream_t stream) {
  constexpr int kw = token_waves(D);
  if constexpr (D <= 128) {
    if (p.mw == 8) return launch_shape<T, D, 8, 1, 64, 4>(a, stream);
    if (p.mw == 4) return launch_shape<T, D, 4, 1, 64, 2>(a, stream);
  } else {
    if (p.mw == 4) return launch_shape<T, D, 4, 1, 32, 4>(a, stream);
  }
  if (p.mw == 2) return launch_shape<T, D, 2, kw < 2 ? kw : 2, 32, 2>(a, stream);
  return launch_shape<T, D, 1, kw, 32, 2>(a, stream);
}

template <typename T>
hipError_t launch_type(const AttnArgs& a, int dim, const AttnPlan& p, hipStream_t stream) {
  switch (dim) {
    case 64: return launch_dim<T, 64>(a, p, stream);
    case 80: return launch_dim<T, 80>(a, p, stream);
    case 96: return launch_dim<T, 96>(a, p, stream);
    case 128: return launch_dim<T, 128>(a, p, stream);
    case 192: return launch_dim<T, 192>(a, p, stream);
    default: return launch_dim<T, 256>(a, p, stream);
  }
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

}  // namespace

bool attn_dim_supported(int dim) {
  return dim == 64 || dim == 80 || dim == 96 || dim == 128 || dim == 192 || dim == 256;
}

AttnPlan attn_plan(const vqv_cache& c, const vqv_seqs& s, int heads, int window, int sinks) {
  const int64_t m = (int64_t)(s.max_rows < s.n_rows ? s.max_rows : s.n_rows) * (heads / c.kv_heads);
  const int kw = token_waves(c.dim);
  AttnPlan p;
  p.mw = m <= 32 ? 1 : m <= 64 ? 2 : m <= 128 || c.dim > 128 || window > 0 ? 4 : 8;
  p.kw = p.mw >= 4 ? 1 : p.mw == 2 && kw > 2 ? 2 : kw;
  p.kt = p.mw >= 4 && c.dim <= 128 ? 64 : 32;
  p.groups = ceil_div(m < 1 ? 1 : m, 32 * p.mw);
  const int bt = p.kw * p.kt;
  // The most blocks that a tile's rows see.
  int64_t tokens = s.max_kv;
  if (window > 0) {
    const int64_t rows_of_tile = 32 * p.mw / (heads / c.kv_heads) + 2;
    int64_t seen = (int64_t)window + rows_of_tile + 2 * bt;
    seen += sinks < s.max_kv ? (int64_t)sinks + bt : s.max_kv;
    tokens = seen < tokens ? seen : tokens;
  }
  const int blocks = ceil_div(tokens < 1 ? 1 : tokens, bt);
  const int64_t base = (int64_t)c.kv_heads * s.n_seqs * p.groups;
  // Blocks of a split. Full tiles: as many work-groups as fit the 256 CUs at
  // once, splits of 4 blocks at least. Few query rows: one work-group per
  // CU while that leaves splits of 16 blocks or fewer (a block of 8 rows over
  // 4096 tokens: 15.8 us, with two per CU 17.2, one for two CUs 18.6); then
  // splits of 16 or more, in 16 rounds as lengths differ (48 ragged sequences:
  // 350 us, in 8 rounds 361, in 4 407), but in two where a window makes them
  // alike (80 us, in 4 rounds 84).
  int64_t per;
  if (p.mw >= 4) {
    per = ceil_div(blocks * base, p.mw == 4 && c.dim <= 128 ? 512 : 256);
    if (per < 4) per = 4;
  } else {
    per = ceil_div(blocks * base, 256);
    if (per > 16) {
      per = ceil_div(blocks * base, window > 0 ? 512 : 4096);
      if (per < 16) per = 16;
    }
  }
  p.split_blocks = per < blocks ? (int)per : blocks;
  p.splits = ceil_div(blocks, p.split_blocks);
  return p;
}

size_t attn_partial_bytes(const vqv_cache& c, const vqv_seqs& s, int heads, const AttnPlan& p) {
  if (p.splits <= 1) return 0;
  return (size_t)s.n_rows * heads * p.splits * (c.dim + 2) * sizeof(float);
}

hipError_t launch_paged_attn(const void* q, const vqv_cache& c, int layer, const vqv_seqs& seqs,
                             int heads, float scale, int window, int sinks, void* out,
                             void* workspace, const AttnPlan& plan, hipStream_t stream) {
  AttnArgs a{};
  a.q = q;
  a.out = out;
  a.k = static_cast<const uint16_t*>(c.k) + layer * c.layer_stride;
  a.v = static_cast<const uint16_t*>(c.v) + layer * c.layer_stride;
  a.seqs = seqs;
  a.page_size = c.page_size;
  a.pages = c.pages;
  a.page_mul = 0;
  a.page_shift = 0;
  if (c.page_size > 1) {
    // ceil(2^(32 + shift) / page_size) with 2^shift < page_size <= 2^(shift + 1): exact for
    // tokens below 2^31.
    while ((2ll << a.page_shift) < c.page_size) ++a.page_shift;
    a.page_mul = (unsigned)(((1ull << (32 + a.page_shift)) + c.page_size - 1) / c.page_size);
  }
  a.kv_heads = c.kv_heads;
  a.group = heads / c.kv_heads;
  a.page_units = (unsigned)(c.page_stride >> 3);
  a.slot_units = (unsigned)(c.slot_stride >> 3);
  a.head_units = (unsigned)(c.head_stride >> 3);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.window = window;
  a.sinks = window > 0 ? sinks : 0;
  a.groups = plan.groups;
  a.split_blocks = plan.split_blocks;
  a.splits = plan.splits;
  a.part = static_cast<float*>(workspace);
  a.part_ml = a.part + (size_t)seqs.n_rows * heads * plan.splits * c.dim;
  return c.dtype == VQV_BF16 ? launch_type<__bf16>(a, c.dim, plan, stream)
                             : launch_type<_Float16>(a, c.dim, plan, stream);
}

}  // namespace vqv
