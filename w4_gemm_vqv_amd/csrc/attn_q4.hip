// Attention of new rows over a paged cache held in 4 bits (vqv_paged_attn_q4).
//
// As in attn.hip, the (row, head) pairs of a sequence that share a key head are
// cut into tiles, S^T = K Q^T and O^T = V^T P^T are formed with matrix
// instructions (here 16x16x32 in fp16) and a running maximum, and long sequences
// are split over work-groups whose sums a second kernel joins. What differs is how
// keys and values come: records of 4-bit codes with a scale and a bias per 32
// values (a token's record of 128 values is 80 bytes instead of 256).
//
// Each wave walks over its own blocks of 32 tokens, every KW-th one of the
// work-group's, for RT tiles of 16 rows: it copies their records to LDS as they
// are, two blocks deep, and waits for nobody else; a token's page is looked up
// three blocks ahead. Keys: a lane's codes become fp16 right where the A operand
// wants them (a matrix step's 32 columns are chunks of 8 codes that lie together,
// and the query rows are read in that order). Values: the transposing read of 4-bit
// elements gives a lane one column's codes of 16 tokens, that of 16-bit elements
// their scales and biases, so nothing but codes is moved. (Values made fp16 first,
// written to LDS and read transposed: decode took 229 us for 164.)
//
// A code becomes fp16 by placing it under an exponent (1024 + q, or 64 + q for
// those that stand 4 bits higher: no shift), subtracting that, which is exact,
// and one fused multiply-add: 13 instructions for 8 values, and a single
// rounding, 2^-12 of a value. bf16 queries become fp16 times a power of two per
// row, exact but for values 2^27 below the row's largest. Keys of fp16 queries
// stay in two fp16 values: rounded once, they would make the larger part of an
// fp16 output's error. Of bf16 calls keys, values and weights are one fp16 value
// each; over 4096 tokens they add 2.2e-4, 1.9e-4 and 2.0e-4 (in all 3.5e-4) to the
// 1.64e-3 that the output's own rounding is off by. Weights in two values would
// leave 2.9e-4 of that, for 173 us of decoding instead of 165. Of fp16 calls values
// are rounded once: 2.8e-4 in all, where a form in fp32 is off by 2.1e-4.
//
// All work-groups of a tile's or a split's tokens run on one XCD whatever their key
// head: with slots as the outer order the records of neighbouring heads share cache
// lines (decode took 229 us without that, 175 with).
//
// What bounds it, with 32 heads of 128 on 8 (a copy moves 4.8 TB/s here):
//   48 ragged sequences to 16383 tokens, one row each: 159 us for 565 MB, 3.6 TB/s:
//   the records' loads; the 16-bit cache takes 351 us for 1.8 GB.
//   8 rows over 4096 tokens: 15 us, two launches and a chain of waits, for 5 MB.
//   16 sequences of 16 rows, 16 heads of 256 on 4 in fp16, a window of 4096: 120 us
//   for 86 MB: forming keys and weights in two values for two tiles of rows.
// Large bf16 calls without a window go through copy_q4.hip instead.

#include "attn_common.h"
#include "serve_internal.h"

namespace vqv {
namespace {

typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;
typedef __attribute__((ext_vector_type(2))) int i32x2;

template <int I>
struct Index {
  static constexpr int value = I;
};

// f(0) .. f(N - 1), the number known to the compiler.
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F& f) {
  if constexpr (I < N) {
    f(Index<I>{});
    each<N, I + 1>(f);
  }
}

// Which 16-byte piece of a staged record of PC pieces holds piece c, so that
// the same piece of 8 records lies in different banks (an exchange is its own
// inverse).
template <int PC>
__device__ __forceinline__ int raw_piece(int row, int c) {
  if (PC == 4) return c ^ (row >> 1 & 3);
  if (PC == 8) return c ^ (row & 7);
  if (PC == 10) return c ^ (row >> 2 & 1);
  return c;  // 3 and 5 have no common factor with 8
}

// The exponents of 1024 and 64 in both halves, for values of which each is the
// offset. They are kept in vector registers: "and" and "or" are one instruction
// only where one of two constants is.
struct Offsets {
  unsigned ten, six;
  __device__ __forceinline__ Offsets() : ten(0x64006400u), six(0x54005400u) {
    asm volatile("" : "+v"(ten), "+v"(six));
  }
};

// Codes 2i and 2i + 1 of 8 (in the records' order), as fp16; w is shifted by 8
// for i of 2 and 3.
__device__ __forceinline__ f16x2 pair_of_codes(unsigned w, int i, const Offsets& at) {
  const f16x2 c10 = {(_Float16)1024.0f, (_Float16)1024.0f}, c6 = {(_Float16)64.0f, (_Float16)64.0f};
  return i & 1 ? __builtin_bit_cast(f16x2, (w & 0x00F000F0u) | at.six) - c6
               : __builtin_bit_cast(f16x2, (w & 0x000F000Fu) | at.ten) - c10;
}

// 8 values: scale * code + bias, rounded to fp16; FINE: what that left over.
template <bool FINE>
__device__ __forceinline__ Weights values_of_codes(unsigned w, unsigned meta, const Offsets& at) {
  const f16x2 sb = __builtin_bit_cast(f16x2, meta);
  const f16x2 scale = {sb[0], sb[0]}, bias = {sb[1], sb[1]};
  u32x4 high, low = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f16x2 n = pair_of_codes(w, i, at);
    const f16x2 v = __builtin_elementwise_fma(n, scale, bias);
    high[i] = __builtin_bit_cast(unsigned, v);
    if (FINE) {
      f16x2 rest;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        rest[e] = (_Float16)(fmaf((float)n[e], (float)scale[e], (float)bias[e]) - (float)v[e]);
      low[i] = __builtin_bit_cast(unsigned, rest);
    }
    if (i & 1) w >>= 8;
  }
  return Weights{__builtin_bit_cast(s16x8, high), __builtin_bit_cast(s16x8, low)};
}

// The keys' columns of a matrix step (s): lane quarter q has 8, those of chunk
// chunk(s, q), so that a quarter's codes are as near to one another as the
// groups allow. The query rows are read in the same order.
template <int D>
struct Keys {
  static constexpr int PC = q4_record_bytes(D) / 16;
  static constexpr int STEPS = (D + 31) / 32;
  static __device__ __forceinline__ int chunk(int s, int q) {
    if (D % 128 == 0) return s / 4 * 16 + 4 * q + s % 4;
    if (D == 80) return s < 2 ? 2 * q + s : 8 + q;
    return D / 32 * q + s;
  }
  static __device__ __forceinline__ bool has(int s, int q) { return D != 80 || s < 2 || q < 2; }

  unsigned codes[STEPS], meta[STEPS];

  // Of the record of staged row `row`, which begins at `at`.
  __device__ __forceinline__ void read(unsigned at, int row, int q) {
    const auto word = [&](int byte) { return at + raw_piece<PC>(row, byte / 16) * 16 + byte % 16; };
    const auto meta_of = [&](int s) { return lds_read<unsigned>(word(D / 2 + chunk(s, q) / 4 * 4)); };
    if (D % 128 == 0) {
#pragma unroll
      for (int s = 0; s < STEPS; s += 4) {
        const u32x4 w = lds_read<u32x4>(word(4 * chunk(s, q)));
        const unsigned m = meta_of(s);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          codes[s + e] = w[e];
          meta[s + e] = m;
        }
      }
    } else if (D == 96) {
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        codes[s] = lds_read<unsigned>(word(4 * chunk(s, q)));
        meta[s] = meta_of(s);
      }
    } else {
#pragma unroll
      for (int s = 0; s + 1 < STEPS; s += 2) {
        const u32x2 w = lds_read<u32x2>(word(4 * chunk(s, q)));
        codes[s] = w[0];
        codes[s + 1] = w[1];
        meta[s] = meta[s + 1] = meta_of(s);
      }
      if (STEPS % 2) {  // 80: the last half step
        const int x = q < 2 ? q : 0;
        codes[STEPS - 1] = lds_read<unsigned>(word(4 * (8 + x)));
        meta[STEPS - 1] = q < 2 ? lds_read<unsigned>(word(D / 2 + 8)) : 0u;
      }
    }
  }
};

// The values of 32 tokens as the A operand: rows are 16 columns, the k slots of
// quarter q are tokens 4q .. 4q+3 and 16+4q .. 16+4q+3. The codes are transposed
// as they lie in the records: of 16 lanes each gives 8 bytes of a row and gets
// the 16 codes of one column. Eight rows are the quarter's tokens for one tile of
// 16 columns, eight the same for the next tile, in an order that leaves pairs of
// tokens 4 codes apart. Their scales and biases are transposed too, which gives
// each lane four tokens of one group's scale or bias: the lane that has it passes
// it to the other 15.
template <int D>
struct Values {
  static constexpr int PC = q4_record_bytes(D) / 16, GROUPS = (D + 31) / 32;
  static __device__ __forceinline__ unsigned word(int row, int byte) {
    return row * PC * 16 + raw_piece<PC>(row, byte / 16) * 16 + byte % 16;
  }
  // Tiles of 16 columns of group g.
  static constexpr int tiles(int g) { return D - 32 * g >= 32 ? 2 : 1; }

  // Of this lane, from a stage's values on: its token of the codes (the same
  // for both tiles) and its row of the scales, the second one 16 rows on.
  static __device__ __forceinline__ int code_row(int lane) {
    const int i = lane & 7, t = i < 4 ? 2 * i : 2 * i - 7;
    return 16 * (t >> 2) + 4 * (lane >> 4) + (t & 3);
  }
  static __device__ __forceinline__ unsigned codes_at(int lane, int row, int g) {
    return word(row, 16 * g + (tiles(g) == 2 ? lane & 8 : 0));
  }
  static __device__ __forceinline__ unsigned meta_at(int lane, int y) {
    constexpr int cols = (GROUPS + 1) / 2;  // runs of four columns
    const int x = lane & 3;
    return word(16 * y + 4 * (lane >> 4) + (lane >> 2 & 3), D / 2 + 8 * (x < cols ? x : 0));
  }
};

// Scales and biases of 8 tokens, two to a register, from lane L of 16.
template <int L>
__device__ __forceinline__ u32x4 pass_to_16(u32x4 x) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = (unsigned)__builtin_amdgcn_update_dpp(0, (int)x[i], 0x150 + L, 0xF, 0xF, true);
  return r;
}

// 8 tokens of a column: scale * code + bias, rounded to fp16.
__device__ __forceinline__ s16x8 column_of_codes(unsigned w, u32x4 scale, u32x4 bias,
                                                 const Offsets& at) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f16x2 n = pair_of_codes(w, i, at);
    const unsigned by = scale[i], to = bias[i];  // (a cast of an element would be the first's)
    r[i] = __builtin_bit_cast(
        unsigned, __builtin_elementwise_fma(n, __builtin_bit_cast(f16x2, by),
                                            __builtin_bit_cast(f16x2, to)));
    if (i & 1) w >>= 8;
  }
  return __builtin_bit_cast(s16x8, r);
}

// The product of 16 columns whose values hold infinities or NaN, some rows not
// seeing all of the tokens: such values are left out of it and added apart for
// the rows that see them (bits `seen` of the lane's tokens). A function of its
// own: it seldom runs, and takes no registers from the loop.
template <bool FINE>
__device__ __attribute__((noinline)) f32x4 product_with_bad_values(s16x8 v, Weights w,
                                                                   unsigned seen, f32x4 o) {
  constexpr unsigned e = Bits<_Float16>::exponent, one = Bits<_Float16>::one;
  s16x8 up, down, see;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const unsigned x = (unsigned short)v[i];
    const bool out = (x & e) == e, nan = out && (x & 0x7FFFu) != e;
    up[i] = out && (nan || !(x & 0x8000u)) ? one : 0;
    down[i] = out && (nan || (x & 0x8000u)) ? one : 0;
    see[i] = seen >> i & 1u ? one : 0;
  }
  const f32x4 a = mfma16<_Float16>(up, see, f32x4{}), b = mfma16<_Float16>(down, see, f32x4{});
  const s16x8 f = finite<_Float16>(v);
  o = mfma16<_Float16>(f, w.high, o);
  if (FINE) o = mfma16<_Float16>(f, w.low, o);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (a[i] != 0.0f) o[i] += __builtin_inff();
    if (b[i] != 0.0f) o[i] -= __builtin_inff();
  }
  return o;
}

__device__ __forceinline__ float max_of_quarters(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return max_of_halves(fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1])));
}

template <typename T, int D, int RT, int KW, bool FINE>
__global__ __launch_bounds__(KW * 64, D > 128 ? 1 : RT == 1 ? 3 : 2) void paged_attn_q4(
    const AttnArgs a) {
  typedef _Float16 H;
  constexpr bool HALF = Bits<T>::exponent == Bits<H>::exponent;  // fp16 queries and outputs
  constexpr int BT = KW * 32, DT = D / 16, KS = Keys<D>::STEPS, VG = Values<D>::GROUPS;
  constexpr int R = q4_record_bytes(D), PC = R / 16;
  constexpr int ROWS = 16 * RT;
  constexpr int RAW = 64 * R;  // a stage: 32 records of keys, then of values
  constexpr int STAGES = 2;    // blocks of records in LDS
  constexpr int RING = 4;      // blocks whose places are held
  constexpr int OWN = STAGES * RAW + 2 * RING * 128;  // of a wave
  constexpr int PER = DT * 4 + 2;
  constexpr int JOIN = KW / 2 * PER * 256;
  static_assert(2 * STAGES - 1 <= RING, "");
  __shared__ __align__(256) char lds[KW * OWN > JOIN ? KW * OWN : JOIN];

  // Work-groups go to the 8 XCDs in turn: the heads of a part come 8 apart, so that those that
  // share cache lines (records of 80 bytes, side by side) share an L2.
  const int h = blockIdx.x / 8 % a.kv_heads;
  const int part = blockIdx.x / 8 / a.kv_heads * 8 + blockIdx.x % 8;
  const int rest = part / a.seqs.n_seqs;
  // A sequence's tiles and splits go round the XCDs, pairs of them to the same (two tiles read the
  // same tokens). By numbers alone those of an even number of sequences go to a few only: a chunk of
  // 256 rows beside 47 decoding rows 1390 us, so 404; 16 blocks of 16 rows to 16383 tokens 204 and 131.
  const int b = (part + (a.seqs.n_seqs % 2 ? 0 : rest / 2)) % a.seqs.n_seqs;
  const int group = a.groups - 1 - rest % a.groups;  // the longest first
  const int split = rest / a.groups;
  if (split >= a.splits) return;

  const int lane = threadIdx.x & 63, quarter = lane >> 4, tok = lane & 31;
  const int kw = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  const int row0 = max(a.seqs.row_start[b], 0);
  const int n = min(min(a.seqs.row_start[b + 1], a.seqs.n_rows) - row0, a.seqs.max_rows);
  const int g = a.group, pairs = n * g;
  const int tiles = (pairs + ROWS - 1) / ROWS;
  if (n <= 0 || group >= tiles) return;
  const int pos0 = max(a.seqs.kv_len[b], 0) - (a.seqs.row_start[b + 1] - a.seqs.row_start[b]);
  const int kv_len = tokens_of(a, a.seqs.kv_len[b]);
  if (not_of_this_call(a, b)) return;
  const int m0 = group * ROWS;
  const int p_last = pos0 + (min(m0 + ROWS, pairs) - 1) / g;
  const Blocks blocks = visible_blocks<BT>(pos0 + m0 / g, p_last, kv_len, a.window, a.sinks);
  const int per_split = blocks_of_split(a, blocks.all);
  const int parts = max((blocks.all + per_split - 1) / per_split, 1);
  if (split >= parts) return;
  const int j0 = split * per_split, j1 = min(j0 + per_split, blocks.all);

  struct Row {
    bool real;
    int64_t index;  // of (row, head), densely
  };
  const auto row_of = [&](int r, int lane) {
    const int m = m0 + 16 * r + (lane & 15), row = m / g;
    return Row{m < pairs, (int64_t)(row0 + row) * (a.kv_heads * g) + h * g + m - row * g};
  };

  // The query rows as B operands, in the order of the keys' columns.
  s16x8 qf[RT][KS];
  float scale[RT];  // of scores, to powers of two
  int shift_q[RT];  // the rows are 2^shift_q times themselves
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const Row mine = row_of(r, lane);
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + mine.index * D;
    unsigned top = 0;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      s16x8 v = {};
      if (mine.real && Keys<D>::has(s, quarter))
        v = *reinterpret_cast<const s16x8*>(q + 8 * Keys<D>::chunk(s, quarter));
      qf[r][s] = v;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, (unsigned)(unsigned short)v[e] & 0x7FFFu);
    }
    shift_q[r] = 0;
    if (!HALF) {
      top = max(top, (unsigned)__shfl_xor((int)top, 16));
      top = max(top, (unsigned)__shfl_xor((int)top, 32));
      shift_q[r] = shift_to_half(top);
#pragma unroll
      for (int x = 0; x < KS; ++x) qf[r][x] = scaled_to_half(qf[r][x], shift_q[r]);
    }
    scale[r] = scale_of_row(a.scale_log2, shift_q[r]);
  }

  f32x4 o[RT][DT];
  float mx[RT], sum[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
#pragma unroll
    for (int d = 0; d < DT; ++d) o[r][d] = f32x4{};
    mx[r] = -__builtin_inff();
    sum[r] = 0.0f;
  }

  const auto base_of = [&](int j) {
    return (j < blocks.sink ? j : blocks.first + j - blocks.sink) * BT + 32 * kw;
  };
  const char* kbase = static_cast<const char*>(a.k) + (uint64_t)h * a.head_units * 16;
  const char* vbase = static_cast<const char*>(a.v) + (uint64_t)h * a.head_units * 16;
  const int32_t* table = a.seqs.table + (int64_t)b * a.seqs.table_stride;
  // A wave's own LDS: stages, then the rings of places (in the cache, in 16-byte
  // units; 0 for a token that is none) and of entries of the page table.
  const unsigned own = lds_offset(lds) + kw * OWN;
  const unsigned places = own + STAGES * RAW, entries = places + RING * 128;
  const auto ring = [&](unsigned at, int j, int t) {
    return (__attribute__((address_space(3))) unsigned*)(at + ((j - j0) & (RING - 1)) * 128 +
                                                         t * 4);
  };
  bool holes = false;  // a page was missing
  const auto is_there = [&](int t, int i, int entry) {
    return t < kv_len && i < a.seqs.table_width && (unsigned)entry < (unsigned)a.pages;
  };
  const auto place_of = [&](int t, int i, int entry) {
    const bool good = is_there(t, i, entry);
    if (__ballot(t < kv_len && !good) != 0) holes = true;
    return good ? (unsigned)entry * a.page_units + (unsigned)(t - i * a.page_size) * a.slot_units
                : 0u;
  };
  const auto ask = [&](int j) {
    if (j < j1 && lane < 32) {
      const int i = min(page_index(a, base_of(j) + lane), a.seqs.table_width - 1);
      load4_to_lds(table + i,
                   __builtin_amdgcn_readfirstlane(entries + ((j - j0) & (RING - 1)) * 128));
    }
  };
  const auto look_up = [&](int j) {
    if (j < j1) {
      const int t = base_of(j) + tok;
      *ring(places, j, tok) = place_of(t, page_index(a, t), (int)*ring(entries, j, tok));
    }
  };
  // Piece p of a stage is place p of the staged records: keys, then values.
  const auto load = [&](int j) {
    const unsigned to = own + (unsigned)(j - j0) % STAGES * RAW;
    unsigned at[PC];
#pragma unroll
    for (int x = 0; x < PC; ++x) at[x] = *ring(places, j, (x * 64 + lane) / PC & 31);
#pragma unroll
    for (int x = 0; x < PC; ++x) {
      const int p = x * 64 + lane, t = p / PC, c = p % PC;
      load16_to_lds((t < 32 ? kbase : vbase) + (uint64_t)(at[x] + raw_piece<PC>(t & 31, c)) * 16,
                    __builtin_amdgcn_readfirstlane(to + x * 1024));
    }
  };
  const int code_row = Values<D>::code_row(lane);
  const Offsets offsets;

  // 32 tokens of a staged block. FULL: all rows see all of them; else hidden ones
  // are masked, and values that are not finite are looked for.
  const auto block = [&](auto which, int j, int t0) {
    constexpr bool FULL = decltype(which)::value;
    const unsigned ks = own + (unsigned)(j - j0) % STAGES * RAW, vs = ks + RAW / 2;
    f32x4 s[RT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      Keys<D> x;
      const int row = 16 * u + (lane & 15);
      x.read(ks + row * R, row, quarter);
#pragma unroll
      for (int e = 0; e < KS; ++e) {
        const Weights k = values_of_codes<HALF>(x.codes[e], x.meta[e], offsets);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          s[r][u] = mfma16<_Float16>(k.high, qf[r][e], e ? s[r][u] : f32x4{});
          if (HALF) s[r][u] = mfma16<_Float16>(k.low, qf[r][e], s[r][u]);
        }
      }
    }

    unsigned seen[RT] = {};
    if (!FULL) {
      // Token t0 + 16 u + 4 quarter + i, against the rows' bounds.
      const int l = lane_here(), qd = l >> 4, t = t0 + (l & 31);
      const unsigned paged =
          (unsigned)__ballot(is_there(t, page_index(a, t), (int)*ring(entries, j, l & 31))) >>
          (4 * qd);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int m = m0 + 16 * r + (l & 15);
        const int hi = (m < pairs ? pos0 + m / g : -1) - t0 - 4 * qd;
        const int lo = a.window > 0 ? max(hi, -1) - a.window : INT_MIN;
        const int sink = a.sinks - t0 - 4 * qd;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int k = 16 * (i / 4) + (i & 3);
          const bool see = k <= hi && (k > lo || k < sink) && (paged >> k & 1u);
          s[r][i / 4][i & 3] = see ? s[r][i / 4][i & 3] : -__builtin_inff();
          seen[r] |= (see ? 1u : 0u) << i;
        }
      }
    }

    // The maximum that weights are relative to follows every score.
    float top[RT], shift[RT];
    bool up = false, large = false;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      top[r] = s[r][0][0];
#pragma unroll
      for (int i = 1; i < 8; ++i) top[r] = fmaxf(top[r], s[r][i / 4][i & 3]);
      top[r] = max_of_quarters(top[r]);
      up |= top[r] > mx[r];
    }
    if (__any(up)) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const float now = fmaxf(mx[r], top[r]);
        const float back = exp_of(mx[r], now, scale[r]);
        mx[r] = now;
        sum[r] *= back;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[r][d][i] *= back;
      }
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      top[r] = mx[r] == -__builtin_inff() ? 0.0f : mx[r];
      shift[r] = fmaf(top[r], scale[r], -Bits<H>::top);
      large |= fabsf(shift[r]) > kLarge;
    }
    // Of a large maximum the shift's rounding would be the weights' size: the
    // maximum is then taken off the scores first, which is exact near it.
    if (__any(large)) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        shift[r] = -Bits<H>::top;
#pragma unroll
        for (int i = 0; i < 8; ++i) s[r][i / 4][i & 3] -= top[r];
      }
    }
    Weights w[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      u32x4 high, low = {};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float p[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          p[e] = __builtin_amdgcn_exp2f(
              fmaf(s[r][i / 2][2 * (i & 1) + e], scale[r], -shift[r]));
        if (FINE) {
          const u32x2 x = split2<H>(p[0], p[1]);
          high[i] = x[0];
          low[i] = x[1];
          sum[r] += p[0] + p[1];
        } else {
          const unsigned x = pack2<H>(p[0], p[1]);
          high[i] = x;
          sum[r] = add2<H>(x, sum[r]);
        }
      }
      w[r] = Weights{__builtin_bit_cast(s16x8, high), __builtin_bit_cast(s16x8, low)};
    }

    s16x4 half_meta[2];
#pragma unroll
    for (int y = 0; y < 2; ++y)
      half_meta[y] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) s16x4*)(vs + Values<D>::meta_at(lane, y)));
    const u32x4 meta = __builtin_bit_cast(
        u32x4, __builtin_shufflevector(half_meta[0], half_meta[1], 0, 1, 2, 3, 4, 5, 6, 7));
    const auto group_of = [&](auto index) {
      constexpr int i = decltype(index)::value;
      const auto codes = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
          (__attribute__((address_space(3))) i32x2*)(vs + Values<D>::codes_at(lane, code_row, i)));
      const u32x4 scale = pass_to_16<2 * i>(meta), bias = pass_to_16<2 * i + 1>(meta);
#pragma unroll
      for (int e = 0; e < Values<D>::tiles(i); ++e) {
        const s16x8 v = column_of_codes((unsigned)codes[e], scale, bias, offsets);
        bool bad = false;
        if (!FULL) {
          const u32x4 x = __builtin_bit_cast(u32x4, v);
          unsigned found = 0;
#pragma unroll
          for (int y = 0; y < 4; ++y) found |= not_finite<H>(x[y]);
          bad = __ballot(found != 0) != 0;
        }
#pragma unroll
        for (int r = 0; r < RT; ++r) {
          f32x4& to = o[r][2 * i + e];
          if (bad) {
            to = product_with_bad_values<FINE>(v, w[r], seen[r], to);
          } else {
            to = mfma16<_Float16>(v, w[r].high, to);
            if (FINE) to = mfma16<_Float16>(v, w[r].low, to);
          }
        }
      }
    };
    each<VG>(group_of);
  };

#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int x = 0; x < KS; ++x) asm volatile("" : "+v"(qf[r][x]));
#pragma unroll 1
  for (int x = 0; x < 2 * STAGES - 1; ++x) {  // the first blocks' places
    const int j = j0 + x;
    if (j < j1) {
      const int t = base_of(j) + tok, i = page_index(a, t);
      const int entry = t < kv_len && i < a.seqs.table_width ? table[i] : -1;
      *ring(entries, j, tok) = (unsigned)entry;
      *ring(places, j, tok) = place_of(t, i, entry);
    }
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
#pragma unroll
  for (int x = 0; x < STAGES - 1; ++x)
    if (j0 + x < j1) load(j0 + x);

  for (int j = j0; j < j1; ++j) {
    // Block j is there; this wave's reads of block j - 1 are done.
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    ask(j + 2 * STAGES - 1);
    if (j + STAGES - 1 < j1) load(j + STAGES - 1);
    if (j - j0 >= STAGES - 1) look_up(j + STAGES);

    const int t0 = base_of(j);
    if (t0 > p_last || t0 >= kv_len) continue;
    // Whether all rows see all tokens.
    const bool full = t0 + 31 <= pos0 + m0 / g && (a.window == 0 || t0 > p_last - a.window) &&
                      t0 + 32 <= kv_len && !holes;
    if (full)
      block(Index<1>{}, j, t0);
    else
      block(Index<0>{}, j, t0);
  }

#pragma unroll
  for (int r = 0; r < RT; ++r) {
    sum[r] += __shfl_xor(sum[r], 16);
    sum[r] += __shfl_xor(sum[r], 32);
    // Row 4 quarter + i of a tile is the column of the code at that place in 8 bytes: quarters
    // 2x and 2x + 1 have the even and the odd ones of 8 columns, and take four each in a row.
#pragma unroll
    for (int d = 0; d < DT; ++d) {
      const f32x4 x = o[r][d];
      const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x[0]), __float_as_uint(x[2]),
                                                      false, false);
      const auto q = __builtin_amdgcn_permlane16_swap(__float_as_uint(x[1]), __float_as_uint(x[3]),
                                                      false, false);
      o[r][d] = f32x4{__uint_as_float(p[0]), __uint_as_float(p[1]), __uint_as_float(q[0]),
                      __uint_as_float(q[1])};
    }
    // The waves join their sums through LDS, half of them at a time.
    float* x = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int w = KW / 2; w >= 1; w >>= 1) {
      __syncthreads();
      float* mine = x + (kw % w) * PER * 64 + lane;
      if (kw >= w && kw < 2 * w) {
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) mine[(d * 4 + i) * 64] = o[r][d][i];
        mine[DT * 4 * 64] = mx[r];
        mine[(DT * 4 + 1) * 64] = sum[r];
      }
      __syncthreads();
      if (kw < w) {
        const float om = mine[DT * 4 * 64], os = mine[(DT * 4 + 1) * 64];
        const float top = fmaxf(mx[r], om);
        const float fa = exp_of(mx[r], top, scale[r]), fb = exp_of(om, top, scale[r]);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[r][d][i] = o[r][d][i] * fa + mine[(d * 4 + i) * 64] * fb;
        sum[r] = sum[r] * fa + os * fb;
        mx[r] = top;
      }
    }
    if (kw > 0) continue;

    const int l = lane_here(), qd = l >> 4;
    const Row row = row_of(r, l);
    if (!row.real) continue;
    if (parts == 1) {
      const float inv = sum[r] == 0.0f ? 0.0f : 1.0f / sum[r];
      uint16_t* out = static_cast<uint16_t*>(a.out) + row.index * D + 4 * qd;
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const u32x2 x = {pack2<T>(o[r][d][0] * inv, o[r][d][1] * inv),
                         pack2<T>(o[r][d][2] * inv, o[r][d][3] * inv)};
        *reinterpret_cast<u32x2*>(out + 16 * d) = x;
      }
    } else {
      const int64_t at = row.index * a.splits + split;
      float* out = a.part + at * D + 4 * qd;
#pragma unroll
      for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4*>(out + 16 * d) = o[r][d];
      if (qd == 0) {
        a.part_ml[2 * at] = ldexpf(mx[r], -shift_q[r]);
        a.part_ml[2 * at + 1] = sum[r];
      }
    }
  }
}

// Waves of a work-group, each with blocks of its own.
constexpr int waves(int dim) { return dim <= 128 ? 4 : 2; }

template <typename T, int D, int RT, bool FINE>
hipError_t launch_shape(const AttnArgs& a, hipStream_t stream) {
  const int64_t grid = ((int64_t)a.seqs.n_seqs * a.groups * a.splits + 7) / 8 * 8 * a.kv_heads;
  hipLaunchKernelGGL((paged_attn_q4<T, D, RT, waves(D), FINE>), dim3((unsigned)grid),
                     dim3(waves(D) * 64), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL((paged_attn_join<T, D, waves(D) * 32, 16 * RT, false, true>),
                     dim3((unsigned)(a.seqs.n_rows * a.kv_heads * a.group)), dim3(256), 0, stream,
                     a);
  return hipGetLastError();
}

// Tiles of 16 (row, head) pairs of a work-group, at most. With four the
// registers of a wave hold no second block's work and spill (a prompt chunk of
// 2048 rows over 10240 tokens took 1425 us, with two it takes 730).
constexpr int kMostTiles = 2;

// Weights in two values: for fp16 outputs of up to 64 pairs. A bf16 output's own
// rounding is eight times that of a weight in one.
template <typename T, int D>
hipError_t launch_dim(const AttnArgs& a, const AttnPlan& p, bool few, hipStream_t stream) {
  constexpr bool HALF = Bits<T>::exponent == Bits<_Float16>::exponent;
  if constexpr (HALF) {
    if (!few) return launch_shape<T, D, 2, false>(a, stream);
  }
  return p.mw == 2 ? launch_shape<T, D, 2, HALF>(a, stream)
                   : launch_shape<T, D, 1, HALF>(a, stream);
}

template <typename T>
hipError_t launch_type(const AttnArgs& a, int dim, const AttnPlan& p, bool few,
                       hipStream_t stream) {
  switch (dim) {
    case 64: return launch_dim<T, 64>(a, p, few, stream);
    case 80: return launch_dim<T, 80>(a, p, few, stream);
    case 96: return launch_dim<T, 96>(a, p, few, stream);
    case 128: return launch_dim<T, 128>(a, p, few, stream);
    case 192: return launch_dim<T, 192>(a, p, few, stream);
    default: return launch_dim<T, 256>(a, p, few, stream);
  }
}

int64_t pairs_of(const vqv_seqs& s, int heads, int kv_heads) {
  return (int64_t)(s.max_rows < s.n_rows ? s.max_rows : s.n_rows) * (heads / kv_heads);
}

}  // namespace

AttnPlan attn_q4_plan(const vqv_cache_q4& c, const vqv_seqs& s, int heads, int window, int sinks) {
  const int64_t m = pairs_of(s, heads, c.kv_heads);
  AttnPlan p{};
  p.mw = m <= 16 ? 1 : kMostTiles;
  p.groups = ceil_div(m < 1 ? 1 : m, 16 * p.mw);
  const int bt = waves(c.dim) * 32;
  // The most blocks that a tile's rows see.
  int64_t tokens = s.max_kv;
  if (window > 0) {
    const int64_t rows_of_tile = 16 * p.mw / (heads / c.kv_heads) + 2;
    int64_t seen = (int64_t)window + rows_of_tile + 2 * bt;
    seen += sinks < s.max_kv ? (int64_t)sinks + bt : s.max_kv;
    tokens = seen < tokens ? seen : tokens;
  }
  const int blocks = ceil_div(tokens < 1 ? 1 : tokens, bt);
  // Work-groups that have rows, of all sequences.
  const int64_t grid = (int64_t)c.kv_heads * s.n_seqs * p.groups;
  const int64_t tiles = (int64_t)s.n_rows * (heads / c.kv_heads) / (16 * p.mw) + s.n_seqs;
  const int64_t base = c.kv_heads * tiles < grid ? c.kv_heads * tiles : grid;
  // Blocks of a split: as many as leave a work-group to each CU, and no more than
  // 1024 tokens' worth unless that were more than 16 rounds of work-groups (48
  // ragged sequences: 161 us, with 2048 tokens 167, with 4096 194).
  // Where the rows alone fill the GPU: all, unless few work-groups have long
  // sequences, of which the longest would end alone (ragged to 16383 tokens, one
  // row each, split and whole: 64 sequences 217 and 277 us, 128 453 and 550; 32 x 16
  // rows to 32768 413 and 630). Else the join costs more than it gives (2.7 ns a row
  // and head: 256 sequences of 4 rows to 4096 255 and 229 us, 128 of 8 rows to 8192
  // 296 and 276, a chunk of 512 rows over 4096 138 and 93).
  const int most = 1024 / bt;
  int64_t per = ceil_div(blocks * base, 256);
  const bool uneven = base < (p.mw == 1 ? 2048 : 1024) && s.n_seqs > 1 && blocks >= 8 * most;
  if (base >= 512 && !(uneven && window == 0)) {
    per = blocks;
  } else if (per > most) {
    per = ceil_div(blocks * base, window > 0 ? 512 : 4096);
    if (per < most) per = most;
    // Not more than a launch can count: a call is not refused for its splits.
    if (base >= 512 && (grid * ceil_div(blocks, per) >= (1 << 23) ||
                        (int64_t)s.n_rows * heads >= (1 << 24)))
      per = blocks;
  }
  p.split_blocks = per < blocks ? (int)per : blocks;
  p.splits = ceil_div(blocks, p.split_blocks);
  return p;
}

hipError_t launch_paged_attn_q4(const void* q, int dtype, const vqv_cache_q4& c, int layer,
                                const vqv_seqs& seqs, int heads, float scale, int window,
                                int sinks, const Copied& copied, void* out, void* workspace,
                                const AttnPlan& plan, hipStream_t stream) {
  AttnArgs a = attn_args(q, out, seqs, c.page_size, c.pages, c.kv_heads, heads, c.dim, scale,
                         window, sinks, workspace, plan);
  a.k = static_cast<const char*>(c.k) + layer * c.layer_stride;
  a.v = static_cast<const char*>(c.v) + layer * c.layer_stride;
  a.page_units = (unsigned)(c.page_stride >> 4);
  a.slot_units = (unsigned)(c.slot_stride >> 4);
  a.head_units = (unsigned)(c.head_stride >> 4);
  if (copied.slots > 0) a.which = kOthers;
  a.copied = copied;
  const bool few = pairs_of(seqs, heads, c.kv_heads) <= 64;
  return dtype == VQV_BF16 ? launch_type<__bf16>(a, c.dim, plan, few, stream)
                           : launch_type<_Float16>(a, c.dim, plan, few, stream);
}

}  // namespace vqv
