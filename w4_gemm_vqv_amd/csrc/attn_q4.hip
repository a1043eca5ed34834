// Attention of new rows over a paged cache held in 4 bits (vqv_paged_attn_q4).
//
// As in attn.hip, the (row, head) pairs of a sequence that share a key head are
// cut into tiles of 32, S^T = K Q^T and O^T = V^T P^T are formed with 32x32x16
// matrix instructions and a running maximum, and long sequences are split over
// work-groups whose sums a second kernel joins. What differs is how keys and
// values come: records of 4-bit codes with a scale and a bias per 32 values
// (a token's record of 128 values is 80 bytes instead of 256).
//
// Each wave walks over its own blocks of 32 tokens, every KW-th one of the
// work-group's, for RT tiles of rows: it loads their records to an LDS buffer
// of its own, STAGES deep, and waits for nobody else. A lane takes half of
// token l % 32's record: its keys become fp16 in registers, right where the A
// operand wants them (a matrix step's 16 columns are 8 of each lane half's
// group, and the query rows are read in that order), its values become fp16 in
// LDS, where the transposing read turns them.
//
// A code becomes fp16 by placing it under an exponent (1024 + q, or 64 + q for
// those that stand 4 bits higher: no shift), subtracting that, which is exact,
// and one fused multiply-add: 13 instructions for 8 values, and a single
// rounding, 2^-12 of a value. bf16 queries become fp16 times a power of two per
// row, exact but for values 2^24 below the row's largest.

#include "attn_common.h"
#include "serve_internal.h"

namespace vqv {
namespace {

typedef __attribute__((ext_vector_type(2))) _Float16 f16x2;

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

// 8 codes as fp16: scale * code + bias.
__device__ __forceinline__ s16x8 values_of_codes(unsigned w, f16x2 scale, f16x2 bias) {
  const f16x2 c10 = {(_Float16)1024.0f, (_Float16)1024.0f}, c6 = {(_Float16)64.0f, (_Float16)64.0f};
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const f16x2 a = __builtin_bit_cast(f16x2, (w & 0x000F000Fu) | 0x64006400u) - c10;
    const f16x2 b = __builtin_bit_cast(f16x2, (w & 0x00F000F0u) | 0x54005400u) - c6;
    r[i] = __builtin_bit_cast(unsigned, __builtin_elementwise_fma(a, scale, bias));
    r[i + 1] = __builtin_bit_cast(unsigned, __builtin_elementwise_fma(b, scale, bias));
    w >>= 8;
  }
  return __builtin_bit_cast(s16x8, r);
}

// A lane's share of token l % 32's record, for a pair of groups (i): lane half
// h has group 2i + h, or half of the last group where there is no other. The
// codes of 8 * steps(i) values, and the group's scale and bias.
template <int D>
struct Share {
  static constexpr int PC = q4_record_bytes(D) / 16;
  static constexpr int PAIRS = (D + 63) / 64;
  static constexpr int steps(int i) { return D - 64 * i >= 64 ? 4 : (D - 64 * i) / 16; }
  // The first column of half h's share.
  static __device__ __forceinline__ int column(int i, int h) { return 64 * i + 8 * steps(i) * h; }

  unsigned codes[4];
  f16x2 scale, bias;

  __device__ __forceinline__ void read(unsigned row_at, int row, int i, int h) {
    const int n = steps(i);
    const int byte = column(i, h) / 2;
    const unsigned at = row_at + raw_piece<PC>(row, byte / 16) * 16 + byte % 16;
    if (n == 4) {
      const u32x4 w = *(__attribute__((address_space(3))) u32x4*)at;
#pragma unroll
      for (int s = 0; s < 4; ++s) codes[s] = w[s];
    } else if (n == 2) {
      const u32x2 w = *(__attribute__((address_space(3))) u32x2*)at;
      codes[0] = w[0];
      codes[1] = w[1];
    } else {
      codes[0] = *(__attribute__((address_space(3))) unsigned*)at;
    }
    const int meta = D / 2 + 4 * (n == 4 ? 2 * i + h : 2 * i);
    const unsigned w = *(__attribute__((address_space(3))) unsigned*)(
        row_at + raw_piece<PC>(row, meta / 16) * 16 + meta % 16);
    const f16x2 sb = __builtin_bit_cast(f16x2, w);
    scale = f16x2{sb[0], sb[0]};
    bias = f16x2{sb[1], sb[1]};
  }
};

// 8 query values as fp16 times 2^e.
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

template <typename T, int D, int RT, int KW, int STAGES, bool FINE>
__global__ __launch_bounds__(KW * 64, RT * D <= 128 ? 2 : 1) void paged_attn_q4(const AttnArgs a) {
  typedef _Float16 H;
  constexpr int BT = KW * 32, DC = D / 8, DS = D / 16, DB = (D + 31) / 32;
  constexpr int R = q4_record_bytes(D), PC = R / 16;
  constexpr int ROWS = 32 * RT;
  constexpr int RAW = 64 * R;  // a stage: 32 records of keys, then of values
  // Where D is not a multiple of 32 the last column block of V reads past its
  // row (the results are not used).
  constexpr int VBUF = 32 * D * 2 + (D % 32 ? 64 : 0);
  constexpr int OWN = (STAGES * RAW + VBUF + 255) / 256 * 256;  // of a wave
  constexpr int RING = 8;  // blocks whose places are held
  constexpr int JOIN = KW / 2 * (DB * 16 + 2) * 256;
  static_assert(2 * STAGES - 1 <= RING, "");
  __shared__ __align__(1024) char lds[KW * OWN > JOIN ? KW * OWN : JOIN];
  __shared__ unsigned places[KW][RING][32];  // in the cache, in 16-byte units, or kNoPlace
  __shared__ int entries[KW][RING][32];      // of the page table

  const int h = blockIdx.x % a.kv_heads;
  const int b = blockIdx.x / a.kv_heads % a.seqs.n_seqs;
  const int rest = blockIdx.x / a.kv_heads / a.seqs.n_seqs;
  const int group = a.groups - 1 - rest % a.groups;  // the longest first
  const int split = rest / a.groups;

  const int lane = threadIdx.x & 63, half = lane >> 5, tok = lane & 31;
  const int kw = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  const int row0 = max(a.seqs.row_start[b], 0);
  const int n = min(min(a.seqs.row_start[b + 1], a.seqs.n_rows) - row0, a.seqs.max_rows);
  const int g = a.group, pairs = n * g;
  const int tiles = (pairs + ROWS - 1) / ROWS;
  if (n <= 0 || group >= tiles) return;
  const int pos0 = max(a.seqs.kv_len[b], 0) - (a.seqs.row_start[b + 1] - a.seqs.row_start[b]);
  const int kv_len = tokens_of(a, a.seqs.kv_len[b]);
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
    const int m = m0 + 32 * r + (lane & 31), row = m / g;
    return Row{m < pairs, (int64_t)(row0 + row) * (a.kv_heads * g) + h * g + m - row * g};
  };

  // The query rows as B operands, in the order of the keys' columns.
  s16x8 qf[RT][DS];
  float scale[RT];  // of scores, to powers of two
  int shift_q[RT];  // the rows are 2^shift_q times themselves
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const Row mine = row_of(r, lane);
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + mine.index * D;
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < Share<D>::PAIRS; ++i)
#pragma unroll
      for (int s = 0; s < Share<D>::steps(i); ++s) {
        s16x8 v = {};
        if (mine.real)
          v = *reinterpret_cast<const s16x8*>(q + Share<D>::column(i, half) + 8 * s);
        qf[r][4 * i + s] = v;
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, (unsigned)(unsigned short)v[e] & 0x7FFFu);
      }
    shift_q[r] = 0;
    if (sizeof(T) == 2 && Bits<T>::exponent == 0x7F80u) {
      const auto both = __builtin_amdgcn_permlane32_swap(top, top, false, false);
      top = max(both[0], both[1]);
      const int e = max((int)(top >> 7), 1) - 127;
      if (top != 0 && top < 0x7F80u) shift_q[r] = 10 - e;
#pragma unroll
      for (int x = 0; x < DS; ++x) qf[r][x] = scaled_to_half(qf[r][x], shift_q[r]);
    }
    scale[r] = ldexpf(a.scale_log2, -shift_q[r]);
  }

  f32x16 o[RT][DB];
  float mx[RT], sum[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
#pragma unroll
    for (int d = 0; d < DB; ++d) o[r][d] = f32x16{};
    mx[r] = -__builtin_inff();
    sum[r] = 0.0f;
  }

  const auto base_of = [&](int j) {
    return (j < blocks.sink ? j : blocks.first + j - blocks.sink) * BT + 32 * kw;
  };
  const char* kbase = static_cast<const char*>(a.k) + (uint64_t)h * a.head_units * 16;
  const char* vbase = static_cast<const char*>(a.v) + (uint64_t)h * a.head_units * 16;
  const int32_t* table = a.seqs.table + (int64_t)b * a.seqs.table_stride;
  bool holes = false;  // a page was missing
  const auto place_of = [&](int t, int i, int entry) {
    const bool in = t < kv_len;
    const bool good =
        in && i < a.seqs.table_width && (unsigned)entry < (unsigned)a.pages;
    if (__ballot(in && !good) != 0) holes = true;
    return good ? (unsigned)entry * a.page_units + (unsigned)(t - i * a.page_size) * a.slot_units
                : kNoPlace;
  };
  const auto ask = [&](int j) {
    if (j < j1 && lane < 32) {
      const int i = min(page_index(a, base_of(j) + lane), a.seqs.table_width - 1);
      load4_to_lds(table + i, __builtin_amdgcn_readfirstlane(
                                  lds_offset(&entries[kw][(j - j0) % RING][0])));
    }
  };
  const auto look_up = [&](int j) {
    if (j < j1) {
      const int t = base_of(j) + tok;
      places[kw][(j - j0) % RING][tok] =
          place_of(t, page_index(a, t), entries[kw][(j - j0) % RING][tok]);
    }
  };
  const unsigned own = lds_offset(lds) + kw * OWN;
  // Piece p of a stage is place p of the staged records: keys, then values.
  const auto load = [&](int j) {
    const unsigned to = own + (j - j0) % STAGES * RAW;
#pragma unroll
    for (int x = 0; x < PC; ++x) {
      const int p = x * 64 + lane, t = p / PC, c = p % PC;
      const unsigned place = places[kw][(j - j0) % RING][t & 31];
      const unsigned at = place == kNoPlace ? 0u : place;
      load16_to_lds((t < 32 ? kbase : vbase) + (uint64_t)(at + raw_piece<PC>(t & 31, c)) * 16,
                    __builtin_amdgcn_readfirstlane(to + x * 1024));
    }
  };

#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int x = 0; x < DS; ++x) asm volatile("" : "+v"(qf[r][x]));
#pragma unroll 1
  for (int x = 0; x < 2 * STAGES - 1; ++x) {
    const int j = j0 + x;
    if (j < j1) {
      const int t = base_of(j) + tok, i = page_index(a, t);
      const int entry = t < kv_len && i < a.seqs.table_width ? table[i] : -1;
      places[kw][x][tok] = place_of(t, i, entry);
    }
  }
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
#pragma unroll
  for (int x = 0; x < STAGES - 1; ++x)
    if (j0 + x < j1) load(j0 + x);

  for (int j = j0; j < j1; ++j) {
    // Block j is there; this wave's reads of block j - 1 are done.
    if (STAGES > 2 && j + STAGES - 2 < j1)
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"((STAGES - 2) * PC) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    ask(j + 2 * STAGES - 1);
    if (j + STAGES - 1 < j1) load(j + STAGES - 1);
    if (j - j0 >= STAGES - 1) look_up(j + STAGES);

    const int t0 = base_of(j);
    if (t0 > p_last || t0 >= kv_len) continue;
    const unsigned ks = own + (j - j0) % STAGES * RAW, vs = ks + RAW / 2;
    const unsigned vbuf = own + STAGES * RAW;
    const bool there = places[kw][(j - j0) % RING][tok] != kNoPlace;
    const unsigned paged = (unsigned)__ballot(there);

    // Values to fp16 rows. A token that is none is zeros.
#pragma unroll
    for (int i = 0; i < Share<D>::PAIRS; ++i) {
      Share<D> x;
      x.read(vs + tok * R, tok, i, half);
      if (!there) x.scale = x.bias = f16x2{};
#pragma unroll
      for (int s = 0; s < Share<D>::steps(i); ++s) {
        const int c = (Share<D>::column(i, half) >> 3) + s;
        *(__attribute__((address_space(3))) s16x8*)(vbuf + tok * D * 2 + v_piece<DC>(tok, c) * 16) =
            values_of_codes(x.codes[s], x.scale, x.bias);
      }
    }

    f32x16 s[RT];
#pragma unroll
    for (int i = 0; i < Share<D>::PAIRS; ++i) {
      Share<D> x;
      x.read(ks + tok * R, tok, i, half);
#pragma unroll
      for (int e = 0; e < Share<D>::steps(i); ++e) {
        const s16x8 k = values_of_codes(x.codes[e], x.scale, x.bias);
#pragma unroll
        for (int r = 0; r < RT; ++r)
          s[r] = mfma<H>(k, qf[r][4 * i + e], i || e ? s[r] : f32x16{});
      }
    }
    asm volatile("" ::: "memory");
    const unsigned va = vbuf + value_address<D>(lane);

#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const int mr = m0 + 32 * r;
      if (mr >= pairs) continue;
      const int p0 = pos0 + mr / g, p1 = pos0 + (min(mr + 32, pairs) - 1) / g;
      // Nothing to see for these rows.
      if (t0 > p1 || (a.window > 0 && t0 + 32 <= max(p0, 0) - a.window + 1 && t0 >= a.sinks))
        continue;
      const bool full = t0 + 31 <= p0 && (a.window == 0 || t0 > p1 - a.window) &&
                        t0 + 32 <= kv_len && !holes;
      unsigned seen = 0;
      if (!full) {
        // Token t0 + 8 (i / 4) + 4 half + i % 4, against the row's bounds.
        const int l = lane_here(), m = mr + (l & 31), hf = l >> 5;
        const int hi = (m < pairs ? pos0 + m / g : -1) - t0 - 4 * hf;
        const int lo = a.window > 0 ? max(hi, -1) - a.window : INT_MIN;
        const int sink = a.sinks - t0 - 4 * hf;
        const unsigned have = paged >> (4 * hf);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int k = 8 * (i / 4) + (i & 3);
          const bool see = k <= hi && (k > lo || k < sink) && (have >> k & 1u);
          s[r][i] = see ? s[r][i] : -__builtin_inff();
          seen |= (see ? 1u : 0u) << i;
        }
      }
      float top = s[r][0];
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[r][i]);
      top = max_of_halves(top);
      if (__any(top > mx[r])) {
        const float now = fmaxf(mx[r], top);
        const float back = exp_of(mx[r], now, scale[r]);
        mx[r] = now;
        sum[r] *= back;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[r][d][i] *= back;
      }
      const float base = mx[r] == -__builtin_inff() ? 0.0f : mx[r];
      float shift = fmaf(base, scale[r], -Bits<H>::top);
      if (__any(fabsf(shift) > kLarge)) {
        shift = -Bits<H>::top;
#pragma unroll
        for (int i = 0; i < 16; ++i) s[r][i] -= base;
      }
      const auto weights = [&](int u) {
        u32x4 high, low = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float p[2];
#pragma unroll
          for (int e = 0; e < 2; ++e)
            p[e] = __builtin_amdgcn_exp2f(fmaf(s[r][8 * u + 2 * i + e], scale[r], -shift));
          if (FINE) {
            const u32x2 w = split2<H>(p[0], p[1]);
            high[i] = w[0];
            low[i] = w[1];
            sum[r] += p[0] + p[1];
          } else {
            const unsigned w = pack2<H>(p[0], p[1]);
            high[i] = w;
            sum[r] = add2<H>(w, sum[r]);
          }
        }
        return Weights{__builtin_bit_cast(s16x8, high), __builtin_bit_cast(s16x8, low)};
      };
      bool bad = false;
      if (!full) {
        unsigned found = 0;
        for (int x = lane_here(); x < 32 * DC; x += 64) {
          const u32x4 w = *(__attribute__((address_space(3))) u32x4*)(vbuf + x * 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) found |= not_finite<H>(w[e]);
        }
        bad = __ballot(found != 0) != 0;
      }
      if (bad) {
        BadBlock<DB, 1> x;
#pragma unroll
        for (int u = 0; u < 2; ++u) x.weights[u] = weights(u);
#pragma unroll
        for (int d = 0; d < DB; ++d) x.o[d] = o[r][d];
        product_with_bad_values<H, D, 1, FINE>(x, seen, vbuf);
#pragma unroll
        for (int d = 0; d < DB; ++d) o[r][d] = x.o[d];
      } else {
        Weights next = weights(0);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const Weights p = next;
#pragma unroll
          for (int d = 0; d < DB; ++d) {
            const s16x8 v = values<D>(va, u, d);
            o[r][d] = mfma<H>(v, p.high, o[r][d]);
            if (FINE) o[r][d] = mfma<H>(v, p.low, o[r][d]);
          }
          if (u == 0) next = weights(1);
        }
      }
    }
  }

#pragma unroll
  for (int r = 0; r < RT; ++r) {
    sum[r] += __shfl_xor(sum[r], 32);
    // The waves join their sums through LDS, half of them at a time.
    float* x = reinterpret_cast<float*>(lds);
    constexpr int PER = DB * 16 + 2;
#pragma unroll
    for (int w = KW / 2; w >= 1; w >>= 1) {
      __syncthreads();
      float* mine = x + (kw % w) * PER * 64 + lane;
      if (kw >= w && kw < 2 * w) {
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) mine[(d * 16 + i) * 64] = o[r][d][i];
        mine[DB * 16 * 64] = mx[r];
        mine[(DB * 16 + 1) * 64] = sum[r];
      }
      __syncthreads();
      if (kw < w) {
        const float om = mine[DB * 16 * 64], os = mine[(DB * 16 + 1) * 64];
        const float top = fmaxf(mx[r], om);
        const float fa = exp_of(mx[r], top, scale[r]), fb = exp_of(om, top, scale[r]);
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            o[r][d][i] = o[r][d][i] * fa + mine[(d * 16 + i) * 64] * fb;
        sum[r] = sum[r] * fa + os * fb;
        mx[r] = top;
      }
    }
    if (kw > 0) continue;

    const int l = lane_here(), hf = l >> 5;
    const Row row = row_of(r, l);
    if (!row.real) continue;
    if (parts == 1) {
      const float inv = sum[r] == 0.0f ? 0.0f : 1.0f / sum[r];
      uint16_t* out = static_cast<uint16_t*>(a.out) + row.index * D;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = 32 * d + 8 * i + 4 * hf;
          if (col < D) {
            const u32x2 w = {pack2<T>(o[r][d][4 * i] * inv, o[r][d][4 * i + 1] * inv),
                             pack2<T>(o[r][d][4 * i + 2] * inv, o[r][d][4 * i + 3] * inv)};
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
          const int col = 32 * d + 8 * i + 4 * hf;
          if (col < D)
            *reinterpret_cast<f32x4*>(out + col) = f32x4{o[r][d][4 * i], o[r][d][4 * i + 1],
                                                         o[r][d][4 * i + 2], o[r][d][4 * i + 3]};
        }
      if (hf == 0) {
        a.part_ml[2 * at] = ldexpf(mx[r], -shift_q[r]);
        a.part_ml[2 * at + 1] = sum[r];
      }
    }
  }
}

constexpr int kWaves = 4;

template <typename T, int D, int RT, bool FINE>
hipError_t launch_shape(const AttnArgs& a, hipStream_t stream) {
  const int64_t grid = (int64_t)a.kv_heads * a.seqs.n_seqs * a.groups * a.splits;
  hipLaunchKernelGGL((paged_attn_q4<T, D, RT, kWaves, 2, FINE>), dim3((unsigned)grid),
                     dim3(kWaves * 64), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL((paged_attn_join<T, D, kWaves * 32, 32 * RT, false>),
                     dim3((unsigned)(a.seqs.n_rows * a.kv_heads * a.group)), dim3(256), 0, stream,
                     a);
  return hipGetLastError();
}

constexpr int row_tiles(int dim) { return dim <= 128 ? 2 : 1; }

template <typename T, int D>
hipError_t launch_dim(const AttnArgs& a, const AttnPlan& p, bool fine, hipStream_t stream) {
  if constexpr (row_tiles(D) == 2) {
    if (p.mw == 2)
      return fine ? launch_shape<T, D, 2, true>(a, stream) : launch_shape<T, D, 2, false>(a, stream);
    return launch_shape<T, D, 1, true>(a, stream);
  } else {
    return fine ? launch_shape<T, D, 1, true>(a, stream) : launch_shape<T, D, 1, false>(a, stream);
  }
}

template <typename T>
hipError_t launch_type(const AttnArgs& a, int dim, const AttnPlan& p, bool fine,
                       hipStream_t stream) {
  switch (dim) {
    case 64: return launch_dim<T, 64>(a, p, fine, stream);
    case 80: return launch_dim<T, 80>(a, p, fine, stream);
    case 96: return launch_dim<T, 96>(a, p, fine, stream);
    case 128: return launch_dim<T, 128>(a, p, fine, stream);
    case 192: return launch_dim<T, 192>(a, p, fine, stream);
    default: return launch_dim<T, 256>(a, p, fine, stream);
  }
}

int64_t pairs_of(const vqv_seqs& s, int heads, int kv_heads) {
  return (int64_t)(s.max_rows < s.n_rows ? s.max_rows : s.n_rows) * (heads / kv_heads);
}

}  // namespace

AttnPlan attn_q4_plan(const vqv_cache_q4& c, const vqv_seqs& s, int heads, int window, int sinks) {
  const int64_t m = pairs_of(s, heads, c.kv_heads);
  AttnPlan p;
  p.mw = m <= 32 ? 1 : row_tiles(c.dim);
  p.kw = kWaves;
  p.kt = 32;
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
  int64_t per = ceil_div(blocks * base, 256);
  if (per > 8) {
    per = ceil_div(blocks * base, window > 0 ? 512 : 4096);
    if (per < 8) per = 8;
  }
  p.split_blocks = per < blocks ? (int)per : blocks;
  p.splits = ceil_div(blocks, p.split_blocks);
  return p;
}

size_t attn_q4_partial_bytes(const vqv_cache_q4& c, const vqv_seqs& s, int heads,
                             const AttnPlan& p) {
  if (p.splits <= 1) return 0;
  return (size_t)s.n_rows * heads * p.splits * (c.dim + 2) * sizeof(float);
}

hipError_t launch_paged_attn_q4(const void* q, int dtype, const vqv_cache_q4& c, int layer,
                                const vqv_seqs& seqs, int heads, float scale, int window,
                                int sinks, void* out, void* workspace, const AttnPlan& plan,
                                hipStream_t stream) {
  AttnArgs a = attn_args(q, out, seqs, c.page_size, c.pages, c.kv_heads, heads, c.dim, scale,
                         window, sinks, workspace, plan);
  a.k = static_cast<const char*>(c.k) + layer * c.layer_stride;
  a.v = static_cast<const char*>(c.v) + layer * c.layer_stride;
  a.page_units = (unsigned)(c.page_stride >> 4);
  a.slot_units = (unsigned)(c.slot_stride >> 4);
  a.head_units = (unsigned)(c.head_stride >> 4);
  const bool fine = pairs_of(seqs, heads, c.kv_heads) <= 64;
  return dtype == VQV_BF16 ? launch_type<__bf16>(a, c.dim, plan, fine, stream)
                           : launch_type<_Float16>(a, c.dim, plan, fine, stream);
}

}  // namespace vqv
