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

#include "attn_common.h"

namespace vqv {
namespace {

// T is the type of the cache and of the matrix products, TO that of queries and
// outputs: the same, or bf16 over an fp16 cache (one that was held in 4 bits).
template <typename T, int D, int MW, int KW, int KT, int STAGES, typename TO>
__global__ __launch_bounds__(MW * KW * 64, MW >= 4 && D <= 128 ? 2 : 1) void paged_attn(
    const AttnArgs a) {
  constexpr int NW = MW * KW, BT = KW * KT, DC = D / 8, DS = D / 16, DB = (D + 31) / 32;
  constexpr bool SAME = Bits<T>::exponent == Bits<TO>::exponent;  // else only the sequences of a copy
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
  const int rest = blockIdx.x / a.kv_heads / a.seqs.n_seqs;
  // From one tile of a sequence to the next it is an odd number of sequences' places, so that the tiles
  // of one long chunk go round the parts of the GPU (by numbers alone those of a chunk of 2048 rows
  // among 48 sequences run on a quarter of each XCD's CUs: 2270 us, so 1140).
  const int b = (blockIdx.x / a.kv_heads + (a.seqs.n_seqs % 2 ? 0 : rest)) % a.seqs.n_seqs;
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
  if constexpr (!SAME) {
    if (not_of_this_call(a, b)) return;
  }
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

  // bf16 queries of fp16 products: times a power of two for each row, which the
  // scale of its scores takes back.
  int shift_q = 0;
  if constexpr (!SAME) {
    unsigned top = 0;
#pragma unroll
    for (int s = 0; s < DS; ++s)
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, (unsigned)(unsigned short)qf[s][e] & 0x7FFFu);
    const auto both = __builtin_amdgcn_permlane32_swap(top, top, false, false);
    shift_q = shift_to_half(max(both[0], both[1]));
#pragma unroll
    for (int s = 0; s < DS; ++s) qf[s] = scaled_to_half(qf[s], shift_q);
  }
  const float scale_log2 = SAME ? a.scale_log2 : scale_of_row(a.scale_log2, shift_q);

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
      const float back = exp_of(mx, now, scale_log2);
      mx = now;
      sum *= back;
#pragma unroll
      for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= back;
    }
    const float base = mx == -__builtin_inff() ? 0.0f : mx;
    float shift = fmaf(base, scale_log2, -Bits<T>::top);
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
              fmaf(s[u / 2][8 * (u & 1) + 2 * i + e], scale_log2, -shift));
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
        const float fa = exp_of(mx, top, scale_log2), fb = exp_of(om, top, scale_log2);
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
          u32x2 w = {pack2<TO>(o[d][4 * i] * inv, o[d][4 * i + 1] * inv),
                     pack2<TO>(o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv)};
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
      a.part_ml[2 * at] = SAME ? mx : ldexpf(mx, -shift_q);
      a.part_ml[2 * at + 1] = sum;
    }
  }
}

template <typename T, int D, int MW, int KW, int KT, int STAGES, typename TO = T>
hipError_t launch_shape(const AttnArgs& a, hipStream_t stream) {
  const int64_t grid = (int64_t)a.kv_heads * a.seqs.n_seqs * a.groups * a.splits;
  hipLaunchKernelGGL((paged_attn<T, D, MW, KW, KT, STAGES, TO>), dim3((unsigned)grid),
                     dim3(MW * KW * 64), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL((paged_attn_join<TO, D, KW * KT, MW == 8 ? 128 : 32 * MW, MW == 8,
                                      Bits<T>::exponent != Bits<TO>::exponent>),
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

// bf16 queries over the fp16 copy of a 4-bit cache: only the plans of many rows
// without a window.
template <int D>
hipError_t launch_copied_dim(const AttnArgs& a, hipStream_t stream) {
  if constexpr (D <= 128) {
    return launch_shape<_Float16, D, 8, 1, 64, 4, __bf16>(a, stream);
  } else {
    return launch_shape<_Float16, D, 4, 1, 32, 4, __bf16>(a, stream);
  }
}

hipError_t launch_copied(const AttnArgs& a, int dim, hipStream_t stream) {
  switch (dim) {
    case 64: return launch_copied_dim<64>(a, stream);
    case 80: return launch_copied_dim<80>(a, stream);
    case 96: return launch_copied_dim<96>(a, stream);
    case 128: return launch_copied_dim<128>(a, stream);
    case 192: return launch_copied_dim<192>(a, stream);
    default: return launch_copied_dim<256>(a, stream);
  }
}

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

size_t attn_partial_bytes(int dim, const vqv_seqs& s, int heads, const AttnPlan& p) {
  if (p.splits <= 1) return 0;
  return (size_t)s.n_rows * heads * p.splits * (dim + 2) * sizeof(float);
}

namespace {

AttnArgs args_of(const void* q, const vqv_cache& c, int layer, const vqv_seqs& seqs, int heads,
                 float scale, int window, int sinks, void* out, void* workspace,
                 const AttnPlan& plan) {
  AttnArgs a = attn_args(q, out, seqs, c.page_size, c.pages, c.kv_heads, heads, c.dim, scale,
                         window, sinks, workspace, plan);
  a.k = static_cast<const uint16_t*>(c.k) + layer * c.layer_stride;
  a.v = static_cast<const uint16_t*>(c.v) + layer * c.layer_stride;
  a.page_units = (unsigned)(c.page_stride >> 3);
  a.slot_units = (unsigned)(c.slot_stride >> 3);
  a.head_units = (unsigned)(c.head_stride >> 3);
  return a;
}

}  // namespace

hipError_t launch_paged_attn(const void* q, const vqv_cache& c, int layer, const vqv_seqs& seqs,
                             int heads, float scale, int window, int sinks, void* out,
                             void* workspace, const AttnPlan& plan, hipStream_t stream) {
  const AttnArgs a =
      args_of(q, c, layer, seqs, heads, scale, window, sinks, out, workspace, plan);
  return c.dtype == VQV_BF16 ? launch_type<__bf16>(a, c.dim, plan, stream)
                             : launch_type<_Float16>(a, c.dim, plan, stream);
}

hipError_t launch_paged_attn_copied(const void* q, const vqv_cache& c, const vqv_seqs& seqs,
                                    int heads, float scale, const Copied& copied, void* out,
                                    void* workspace, const AttnPlan& plan, hipStream_t stream) {
  AttnArgs a = args_of(q, c, 0, seqs, heads, scale, 0, 0, out, workspace, plan);
  a.which = kCopied;
  a.copied = copied;
  return launch_copied(a, c.dim, stream);
}

}  // namespace vqv
