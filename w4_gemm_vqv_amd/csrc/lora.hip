// Low-rank adapters of many requests beside a shared projection (vqv_lora_add):
// out[m] = y[m] + scale[e] (x[m] . a[e]^T) . b[e]^T, e = which[m].
//
// Rows are taken 64 at a time, and the rows of such a block that share an
// adapter (its slot) together, whatever their order, gathered into tiles of 16.
// First kernel: the products with a. A work-group takes a slot, up to 64 ranks
// and a part of K; its waves take tiles of rows and split that part further, and
// join through LDS. The parts' sums go to the workspace.
// Second kernel: the products with b. A work-group takes a slot and some
// columns; each wave joins the parts of its rows, and runs over its columns. The
// values between the two products are fp32: they go to the matrix instructions
// as three values of the adapters' type, which hold all of their bits, so that
// no rounding comes between.
//
// Weights are the A operand of both products, so that a lane ends with four
// neighbouring ranks (columns) of one row and moves them as 16 bytes.
//
// What bounds it, y not in a cache: 2100 rows of three adapters of rank 64, 5120 to
// 17408 columns in fp16, take 113 us, 19 of them in the first kernel, for 320 MB
// (2.8 TB/s; y and out are 292 MB of it); 64 rows of 40 adapters of rank 32, 2560 to
// 18432, 19 us for 51 MB (2.6 TB/s); 8 rows of rank 16 10.5 us, which are two
// launches and three waits for memory, one after the other, in each. Ranks of 72 to
// 128 take 83 KB of LDS, one work-group to a CU, and those past 128 16 columns at a time:
// 64 rows of 40 adapters of rank 64, 96, 128, 136 and 256 take 31, 80, 77, 235 and 295 us.

#include "round_common.h"
#include "serve_internal.h"

namespace vqv {
namespace {

constexpr int kBlock = 64;       // rows that are looked at together
constexpr int kShrinkWaves = 8;
constexpr int kExpandWaves = 4;

template <typename T>
constexpr bool kHalf = false;
template <>
constexpr bool kHalf<_Float16> = true;

// The adapter of a lane's row, -1 for none, and the slot-th distinct one of the
// block with the rows that have it (adapter -1: there is none).
typedef LoraSlot Slot;

__device__ __forceinline__ int adapter_of(const LoraArgs& a, int row) {
  const int e = row < a.M ? a.which[row] : -1;
  return (unsigned)e < (unsigned)a.ad.n ? e : -1;
}

__device__ __forceinline__ Slot find_slot(int mine, int slot) {
  uint64_t left = __ballot(mine >= 0);
  for (int s = 0; left != 0; ++s) {
    const int e = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
    const uint64_t rows = __ballot(mine == e);
    if (s == slot) return Slot{rows, e};
    left &= ~rows;
  }
  return Slot{0, -1};
}

// Place of the k-th set bit of rows (k < their count).
__device__ __forceinline__ int nth_row(uint64_t rows, int k) {
  int at = 0;
#pragma unroll
  for (int w = 32; w; w >>= 1) {
    const int c = __popcll(rows >> at & ((1ull << w) - 1));
    if (k >= c) {
      k -= c;
      at += w;
    }
  }
  return at;
}

__device__ __forceinline__ int rank_of(const LoraArgs& a, int e) {
  return a.ad.ranks ? min(max(a.ad.ranks[e], 0), a.ad.rank) : a.ad.rank;
}

// The wait for load16_to_lds.
__device__ __forceinline__ void loaded() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Which 16-byte piece of a staged row of `pieces` holds piece c, so that the
// same piece of 8 rows lies in different banks (an exchange is its own inverse).
__device__ __forceinline__ int piece_of(int pieces, int row, int c) {
  return pieces % 8 == 0   ? c ^ (row & 7)
         : pieces % 4 == 0 ? c ^ (row >> 1 & 3)
         : pieces % 2 == 0 ? c ^ (row >> 2 & 1)
                           : c;
}

// One step of 32 of K, as operands: weights of RT tiles of 16 ranks, and x.
template <typename T, typename X, int RT>
struct Step {
  s16x8 w[RT];
  f32x4 x[sizeof(X) / 2];

  // Lanes past K (TAIL: there may be some) have zeros.
  template <bool TAIL>
  __device__ __forceinline__ void load(const uint16_t* const* weights, const X* row, int k, int K) {
    const int at = TAIL && k >= K ? 0 : k;
#pragma unroll
    for (int t = 0; t < RT; ++t) w[t] = *reinterpret_cast<const s16x8*>(weights[t] + at);
#pragma unroll
    for (int e = 0; e < (int)sizeof(X) / 2; ++e)
      x[e] = *reinterpret_cast<const f32x4*>(row + at + 4 * e);
    if (TAIL && k >= K) {
#pragma unroll
      for (int t = 0; t < RT; ++t) w[t] = s16x8{};
#pragma unroll
      for (int e = 0; e < (int)sizeof(X) / 2; ++e) x[e] = f32x4{};
    }
  }

  // Tiles t0 .. t1 - 1 of ranks.
  __device__ __forceinline__ void add(f32x4* acc, int t0, int t1) const {
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      if (t < t0 || t >= t1) continue;
      if constexpr (sizeof(X) == 2) {
        acc[t] = mfma16<T>(w[t], __builtin_bit_cast(s16x8, x[0]), acc[t]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const short a = w[t][e];
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32((float)__builtin_bit_cast(T, a),
                                                        x[e / 4][e % 4], acc[t], 0, 0, 0);
        }
      }
    }
  }
};

// RT tiles of 16 ranks. X is the type of x (the adapters', or float). Ranks and
// rows that are none are loaded from those that are, and not used: no load
// waits for a condition. Few rows: the waves split K, four steps' loads in
// flight. Several tiles of rows: 128 of K at a time are staged in LDS for all of
// them, rows of 16 or 32 lanes, as the operands' own loads (16 rows at a time)
// take the address unit 64 cycles each.
template <typename T, typename X, int RT>
__global__ __launch_bounds__(kShrinkWaves * 64) void lora_shrink(const LoraArgs a, int slots,
                                                                 int splits, int rank_groups) {
  constexpr int KC = 128;                                // of K to a stage
  constexpr int XP = KC * (int)sizeof(X) / 16, WP = KC * 2 / 16;  // pieces of a row
  constexpr int XL = kBlock * XP / (64 * kShrinkWaves);  // loads of a wave: x, weights
  constexpr int WL = (16 * RT * WP + 64 * kShrinkWaves - 1) / (64 * kShrinkWaves);
  constexpr int STAGE = (XL + WL) * kShrinkWaves * 1024;
  constexpr int SUMS = kShrinkWaves * RT * 1024;
  __shared__ __align__(1024) char lds[2 * STAGE > SUMS ? 2 * STAGE : SUMS];
  int id = blockIdx.x;
  const int split = id % splits;
  id /= splits;
  const int r0 = id % rank_groups * 16 * RT;
  const bool first = split == 0 && r0 == 0;
  id /= rank_groups;
  const int slot = id % slots, block = id / slots;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quarter = lane >> 4;
  const Slot s = find_slot(adapter_of(a, block * kBlock + lane), slot);
  if (first && threadIdx.x == 0) a.slots[(int64_t)block * slots + slot] = s;
  if (s.adapter < 0) return;
  const int count = __popcll(s.rows), tiles = (count + 15) / 16;
  const int K = a.ad.K;

  // Waves to a tile of rows: all for one tile, or 2 for each of four.
  const int per_tile = tiles == 1 ? kShrinkWaves : kShrinkWaves / 4;
  const int tile = wave / per_tile, part = split * per_tile + wave % per_tile;
  const int parts = splits * per_tile;
  const int m = tile * 16 + col;
  const bool real = m < count;
  const int row = block * kBlock + nth_row(s.rows, real ? m : 0);

  f32x4 acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) acc[t] = f32x4{};
  const int steps = (K + 31) / 32, whole = K / 32;
  const X* x = static_cast<const X*>(a.x) + (int64_t)row * K;
  const uint16_t* weights = static_cast<const uint16_t*>(a.ad.a) + (int64_t)s.adapter * a.ad.rank * K;
  const uint16_t* w[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) w[t] = weights + (int64_t)min(r0 + 16 * t + col, a.ad.rank - 1) * K;
  if (tiles > 1) {
    const int half = wave % per_tile;  // of two: of the tiles of ranks, or of the steps
    const int u0 = (int)((int64_t)steps * split / splits);
    const int u1 = (int)((int64_t)steps * (split + 1) / splits);
    const int stages = max(min(u1, whole) - u0, 0) / (KC / 32);
    const char* from[XL + WL];
#pragma unroll
    for (int e = 0; e < XL; ++e) {
      const int p = (e * kShrinkWaves + wave) * 64 + lane, r = p / XP, c = p % XP;
      const int at = block * kBlock + nth_row(s.rows, min(r, count - 1));
      from[e] = reinterpret_cast<const char*>(static_cast<const X*>(a.x) + (int64_t)at * K + 32 * u0) +
                piece_of(XP, r, c) * 16;
    }
#pragma unroll
    for (int e = 0; e < WL; ++e) {
      const int p = (e * kShrinkWaves + wave) * 64 + lane, r = p / WP, c = p % WP;
      from[XL + e] = reinterpret_cast<const char*>(
                         weights + (int64_t)min(r0 + r, a.ad.rank - 1) * K + 32 * u0) +
                     piece_of(WP, r, c) * 16;
    }
    const unsigned base = lds_offset(lds);
    const auto stage = [&](int i) {
      const unsigned to = base + (i & 1) * STAGE + wave * 1024;
#pragma unroll
      for (int e = 0; e < XL + WL; ++e)
        load16_to_lds(from[e] + (int64_t)i * KC * (e < XL ? (int)sizeof(X) : 2),
                      __builtin_amdgcn_readfirstlane(to + e * kShrinkWaves * 1024));
    };
    if (stages > 0) stage(0);
    for (int i = 0; i < stages; ++i) {
      // Stage i is there for all, and all are done with stage i - 1.
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      if (i + 1 < stages) stage(i + 1);
      const unsigned xs = base + (i & 1) * STAGE, ws = xs + XL * kShrinkWaves * 1024;
      const int xr = tile * 16 + col;
#pragma unroll
      for (int u = 0; u < KC / 32; ++u) {
        if (RT == 1 && u / (KC / 64) != half) continue;
        Step<T, X, RT> step;
#pragma unroll
        for (int e = 0; e < (int)sizeof(X) / 2; ++e)
          step.x[e] = lds_read<f32x4>(
              xs + (xr * XP + piece_of(XP, xr, (4 * u + quarter) * (int)sizeof(X) / 2 + e)) * 16);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          const int wr = 16 * t + col;
          step.w[t] = lds_read<s16x8>(ws + (wr * WP + piece_of(WP, wr, 4 * u + quarter)) * 16);
        }
        if (RT == 1)
          step.add(acc, 0, 1);
        else
          step.add(acc, half * (RT / 2), (half + 1) * (RT / 2));
      }
    }
    if (tile < tiles) {
      for (int u = u0 + stages * (KC / 32) + half; u < u1; u += 2) {
        Step<T, X, RT> step;
        step.template load<true>(w, x, 32 * u + 8 * quarter, K);
        step.add(acc, 0, RT);
      }
    }
    __syncthreads();
  } else if (tile < tiles) {
    const int u0 = (int)((int64_t)steps * part / parts);
    const int u1 = (int)((int64_t)steps * (part + 1) / parts);
    int u = u0;
    for (; u + 4 <= min(u1, whole); u += 4) {
      Step<T, X, RT> step[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) step[e].template load<false>(w, x, 32 * (u + e) + 8 * quarter, K);
#pragma unroll
      for (int e = 0; e < 4; ++e) step[e].add(acc, 0, RT);
    }
    for (; u < u1; ++u) {
      Step<T, X, RT> step;
      step.template load<true>(w, x, 32 * u + 8 * quarter, K);
      step.add(acc, 0, RT);
    }
  }
  f32x4* sums = reinterpret_cast<f32x4*>(lds) + lane;  // [wave][t][64]
#pragma unroll
  for (int t = 0; t < RT; ++t) sums[(wave * RT + t) * 64] = acc[t];
  __syncthreads();
  if (tile >= tiles || wave % per_tile != 0 || !real) return;
  float* low = a.low + ((int64_t)split * a.M + row) * a.ad.rank + r0 + 4 * quarter;
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    for (int w = 1; w < per_tile; ++w) acc[t] += sums[((wave + w) * RT + t) * 64];
    if (r0 + 16 * t + 4 * quarter < a.ad.rank) *reinterpret_cast<f32x4*>(low + 16 * t) = acc[t];
  }
}

// x in three values of T, which hold all of its bits (in fp16 those down to 2^-24: 2^-38 of a
// row's largest value); an infinity or NaN in one. Finite values that T would round to an
// infinity are cut to its largest, and the rest is in the others.
template <typename T>
__device__ __forceinline__ void split3(float x, short* out) {
  constexpr float most = kHalf<T> ? 65504.0f : 0x1.FEp127f;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const bool real = fabsf(x) < __builtin_inff();
    const T t = (T)(real ? fminf(fmaxf(x, -most), most) : x);
    out[i] = __builtin_bit_cast(short, t);
    const float rest = x - (float)t;
    x = real ? rest : 0.0f;
  }
}

struct F4 {  // rows of any 4-byte alignment
  float v[4];
};

// RB blocks of 32 ranks. CT tiles of 16 columns are taken at a time, their
// loads before their products. The lanes of a matrix operand would read 16 rows
// at a time, 64 bytes of each, which the address unit takes one lane after the
// other: weights (whole rows, one after the other in memory) come through LDS,
// and so do the sums, so that y and out are moved in runs of 64 columns.
template <typename T, int RB, int CT>
__global__ __launch_bounds__(kExpandWaves * 64) void lora_expand(const LoraArgs a, int slots,
                                                                 int splits, int col_groups,
                                                                 int cols) {
  constexpr int COLS = 16 * CT;
  constexpr int SUMS = 16 * (COLS + 4);  // rows 4 apart begin in other banks
  __shared__ __align__(16) char staged[kExpandWaves][COLS * RB * 64 + SUMS * 4];
  // Work-groups go to the 8 XCDs in turn: each has columns of its own, whose weights its L2 holds.
  const int eighth = (col_groups + 7) / 8;
  int id = blockIdx.x / 8;
  const int c0 = (id % eighth * 8 + blockIdx.x % 8) * cols;
  id /= eighth;
  const int slot = id % slots, block = id / slots;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quarter = lane >> 4;
  const int N = a.ad.N, end = min(c0 + cols, N);
  if (c0 >= N) return;

  if (slot == 0 && a.out != a.y) {
    // Rows without an adapter stay as they are.
    const int row = block * kBlock + lane;
    uint64_t none = __ballot(row < a.M && adapter_of(a, row) < 0);
    while (none != 0) {
      const int64_t row = block * kBlock + __builtin_ctzll(none);
      for (int c = c0 + threadIdx.x; c < end; c += kExpandWaves * 64)
        a.out[row * a.out_stride + c] = a.y[row * a.y_stride + c];
      none &= none - 1;
    }
  }
  const Slot s = a.slots[(int64_t)block * slots + slot];
  if (s.adapter < 0) return;
  const int rank = rank_of(a, s.adapter);
  const float scale = a.ad.scale[s.adapter];
  const int count = __popcll(s.rows), tiles = (count + 15) / 16;
  // One tile of rows: the waves share its columns. More: a wave takes a tile
  // (and there are at most four).
  const int tile = tiles == 1 ? 0 : wave;
  if (tile >= tiles) return;
  const int m = tile * 16 + col;
  const bool real = m < count;
  const int64_t row = block * kBlock + nth_row(s.rows, real ? m : 0);

  const uint16_t* w = static_cast<const uint16_t*>(a.ad.b) + (int64_t)s.adapter * N * a.ad.rank;
  const unsigned wl = lds_offset(staged[wave]);
  float* sums = reinterpret_cast<float*>(staged[wave] + COLS * RB * 64);
  const int pieces = a.ad.rank / 8;
  // Pieces of the staged weights: place p has piece `from` of them, in bytes.
  // p / pieces = p * mul >> 16 for p below 2048.
  constexpr int LOADS = CT * RB;
  const int mul = (65535 + pieces) / pieces;
  int from[LOADS];
#pragma unroll
  for (int e = 0; e < LOADS; ++e) {
    const int p = min(e * 64 + lane, COLS * pieces - 1), r = p * mul >> 16, c = p - r * pieces;
    from[e] = (r * pieces + piece_of(pieces, r, c)) * 16;
  }
  // This lane's rows of y and out, and its 4 columns of them: a row to 4 CT lanes.
  const int of_row = lane / (4 * CT), of_col = lane % (4 * CT) * 4;
  int64_t rows[CT];
#pragma unroll
  for (int i = 0; i < CT; ++i) {
    const int r = 16 / CT * i + of_row;
    rows[i] = (int64_t)block * kBlock + __shfl((int)(row - (int64_t)block * kBlock), r);
  }
  const int step = tiles == 1 ? COLS * kExpandWaves : COLS;
  int n0 = c0 + (tiles == 1 ? COLS * wave : 0);
  // The weights and y of the next COLS columns are asked for while the last sums are
  // stored, the first while the row's values are formed (asked for as they are needed:
  // 150 us instead of 120 for 2100 rows of rank 64, y not in a cache).
  F4 v[CT];
  const auto ask = [&](int n0) {
    // COLS rows of weights, as they lie.
    const char* rows_at = reinterpret_cast<const char*>(w + (int64_t)n0 * a.ad.rank);
#pragma unroll
    for (int e = 0; e < LOADS; ++e)
      if (e * 64 < COLS * pieces)
        load16_to_lds(rows_at + from[e], __builtin_amdgcn_readfirstlane(wl + e * 1024));
#pragma unroll
    for (int i = 0; i < CT; ++i)
      __builtin_memcpy(&v[i], a.y + rows[i] * a.y_stride + n0 + of_col, 16);
  };
  if (n0 + COLS <= end) ask(n0);

  // The row's values between the products, as B operands.
  s16x8 low[RB][3];
  float back = scale;
  {
    float v[RB][8];
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int r = 32 * i + 8 * quarter;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
      if (real && r < rank) {
        const float* p = a.low + row * a.ad.rank + r;
        const int64_t part = (int64_t)a.M * a.ad.rank;
        for (int x = 0; x < splits; x += 4) {
          f32x4 lo[4], hi[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const float* at = p + min(x + y, splits - 1) * part;
            lo[y] = *reinterpret_cast<const f32x4*>(at);
            hi[y] = *reinterpret_cast<const f32x4*>(at + 4);
          }
#pragma unroll
          for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[i][e] += x + y < splits ? lo[y][e] : 0.0f;
              v[i][4 + e] += x + y < splits ? hi[y][e] : 0.0f;
            }
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (r + e >= rank) v[i][e] = 0.0f;
        const float size = fabsf(v[i][e]);
        if (size < __builtin_inff()) top = fmaxf(top, size);
      }
    }
    if (kHalf<T>) {
      // fp16: the row times a power of two, its largest finite value near 2^14.
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const int e = top > 0.0f ? 14 - (int)ilogbf(top) : 0;
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int x = 0; x < 8; ++x) v[i][x] = ldexpf(v[i][x], e);
      back = ldexpf(scale, -e);
    }
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        short t[3];
        split3<T>(v[i][e], t);
#pragma unroll
        for (int x = 0; x < 3; ++x) low[i][x][e] = t[x];
      }
  }

  const auto product = [&](s16x8* wf) {
    // Weights past the rank are not used, whatever they are.
    if (rank != 32 * RB) {
#pragma unroll
      for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (32 * i + 8 * quarter + e >= rank) wf[i][e] = 0;
    }
    f32x4 acc = {};
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int x = 0; x < 3; ++x) acc = mfma16<T>(wf[i], low[i][x], acc);
    return acc;
  };

  float by[CT];
#pragma unroll
  for (int i = 0; i < CT; ++i) by[i] = __shfl(back, 16 / CT * i + of_row);
  for (; n0 + COLS <= end; n0 += step) {
    loaded();
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      s16x8 wf[RB];
      const int r = 16 * t + col;
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const int c = 4 * i + quarter;
        wf[i] = lds_read<s16x8>(wl + (r * pieces + piece_of(pieces, r, c < pieces ? c : 0)) * 16);
      }
      const f32x4 acc = product(wf);
      *reinterpret_cast<f32x4*>(sums + col * (COLS + 4) + 16 * t + 4 * quarter) = acc;
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the weights are read
    F4 old[CT];
#pragma unroll
    for (int i = 0; i < CT; ++i) old[i] = v[i];
    if (n0 + step + COLS <= end) ask(n0 + step);
#pragma unroll
    for (int i = 0; i < CT; ++i) {
      const int m = 16 / CT * i + of_row;
      const f32x4 acc = *reinterpret_cast<const f32x4*>(sums + m * (COLS + 4) + of_col);
      f32x4 r;
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = fmaf(acc[e], by[i], old[i].v[e]);
      // Written once and not read again here: past the L2, which holds weights.
      if (tile * 16 + m < count) {
        typedef __attribute__((ext_vector_type(4), aligned(4))) float f32x4_4;
        __builtin_nontemporal_store(
            (f32x4_4)r, reinterpret_cast<f32x4_4*>(a.out + rows[i] * a.out_stride + n0 + of_col));
      }
    }
  }
  // What is left of the columns, a tile at a time.
  const float* y = a.y + row * a.y_stride;
  float* out = a.out + row * a.out_stride;
  for (const int stop = min(n0 + COLS, end); n0 < stop; n0 += 16) {
    s16x8 wf[RB];
    const int n = n0 + 4 * quarter;
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int r = 32 * i + 8 * quarter;
      wf[i] = *reinterpret_cast<const s16x8*>(w + (int64_t)min(n0 + col, N - 1) * a.ad.rank +
                                              (r < a.ad.rank ? r : 0));
    }
    const f32x4 acc = product(wf);
    if (real) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < end) out[n + e] = fmaf(acc[e], back, y[n + e]);
    }
  }
}

// How a call is cut.
struct Plan {
  int blocks, slots;  // blocks of rows, and distinct adapters of one at most
  int tiles;          // of 16 ranks, to a work-group of the first kernel
  int rank_groups, splits;
  int col_groups, cols;
};

Plan plan_of(const vqv_adapters& ad, int M) {
  Plan p;
  p.blocks = ceil_div(M, kBlock);
  p.slots = ad.n < kBlock ? ad.n : kBlock;
  if (p.slots > M) p.slots = M;
  p.tiles = ad.rank <= 16 ? 1 : ad.rank <= 32 ? 2 : 4;
  p.rank_groups = ceil_div(ad.rank, 16 * p.tiles);
  const int steps = ceil_div(ad.K, 32);
  int splits = ceil_div(256, p.blocks * p.rank_groups);
  if (splits > steps / 16) splits = steps / 16;
  if (splits > 8) splits = 8;
  p.splits = splits < 1 ? 1 : splits;
  // Columns of a work-group of the second kernel: 128 to a wave, 64 at a time (in one
  // run 2100 rows of rank 64: 115 us, with 64 120, with 256 132; 64 rows of 40 adapters of rank
  // 32: 19.3, 21.5, 23.7), or 16 where 64 leave fewer than one work-group to a CU if
  // an eighth of the slots are taken, or the weights of 64 would take all of a CU's LDS.
  const int64_t some = (int64_t)p.blocks * (p.slots / 8 > 1 ? p.slots / 8 : 1);
  const bool few = ad.rank > 128 || some * ceil_div(ad.N, 64 * kExpandWaves) < 256;
  p.cols = kExpandWaves * (few ? 16 : 128);
  p.col_groups = ceil_div(ad.N, p.cols);
  return p;
}

size_t slots_bytes(const Plan& p) { return (size_t)p.blocks * p.slots * sizeof(Slot); }

template <typename T, typename X, int RT>
hipError_t shrink(const LoraArgs& a, const Plan& p, hipStream_t stream) {
  const int64_t grid = (int64_t)p.blocks * p.slots * p.rank_groups * p.splits;
  hipLaunchKernelGGL((lora_shrink<T, X, RT>), dim3((unsigned)grid), dim3(kShrinkWaves * 64), 0,
                     stream, a, p.slots, p.splits, p.rank_groups);
  return hipGetLastError();
}

template <typename T, typename X>
hipError_t shrink_tiles(const LoraArgs& a, const Plan& p, hipStream_t stream) {
  if (p.tiles == 1) return shrink<T, X, 1>(a, p, stream);
  if (p.tiles == 2) return shrink<T, X, 2>(a, p, stream);
  return shrink<T, X, 4>(a, p, stream);
}

template <typename T, int RB, int CT>
hipError_t expand(const LoraArgs& a, const Plan& p, hipStream_t stream) {
  const int64_t grid = (int64_t)p.blocks * p.slots * ((p.col_groups + 7) / 8 * 8);
  hipLaunchKernelGGL((lora_expand<T, RB, CT>), dim3((unsigned)grid), dim3(kExpandWaves * 64), 0,
                     stream, a, p.slots, p.splits, p.col_groups, p.cols);
  return hipGetLastError();
}

template <typename T, int RB>
hipError_t expand_cols(const LoraArgs& a, const Plan& p, hipStream_t stream) {
  if constexpr (RB < 8) {
    if (p.cols == 128 * kExpandWaves) return expand<T, RB, 4>(a, p, stream);
  }
  return expand<T, RB, 1>(a, p, stream);
}

template <typename T>
hipError_t launch_type(LoraArgs a, bool wide, hipStream_t stream) {
  const Plan p = plan_of(a.ad, a.M);
  a.slots = static_cast<Slot*>(a.workspace);
  a.low = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + slots_bytes(p));
  const hipError_t e =
      wide ? shrink_tiles<T, float>(a, p, stream) : shrink_tiles<T, T>(a, p, stream);
  if (e != hipSuccess) return e;
  const int blocks = ceil_div(a.ad.rank, 32);
  if (blocks == 1) return expand_cols<T, 1>(a, p, stream);
  if (blocks == 2) return expand_cols<T, 2>(a, p, stream);
  if (blocks <= 4) return expand_cols<T, 4>(a, p, stream);
  return expand_cols<T, 8>(a, p, stream);
}

}  // namespace

bool lora_grids_fit(const vqv_adapters& ad, int M) {
  if (M < 1) return true;
  const Plan p = plan_of(ad, M);
  const int64_t groups = (int64_t)p.blocks * p.slots;
  return groups * p.rank_groups * p.splits < (1ll << 22) && groups * (p.col_groups + 7) < (1ll << 23);
}

size_t lora_workspace_bytes(const vqv_adapters& ad, int M) {
  if (M < 1) return 0;
  const Plan p = plan_of(ad, M);
  return slots_bytes(p) + (size_t)p.splits * M * ad.rank * sizeof(float);
}

hipError_t launch_lora_add(const LoraArgs& a, int act_dtype, hipStream_t stream) {
  const bool wide = act_dtype == VQV_FP32;
  return a.ad.dtype == VQV_BF16 ? launch_type<__bf16>(a, wide, stream)
                                : launch_type<_Float16>(a, wide, stream);
}

}  // namespace vqv
