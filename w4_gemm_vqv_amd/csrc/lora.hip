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

#include "serve_internal.h"

namespace vqv {
namespace {

typedef __attribute__((ext_vector_type(8))) short s16x8;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;

constexpr int kBlock = 64;       // rows that are looked at together
constexpr int kShrinkWaves = 8;
constexpr int kExpandWaves = 4;

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

  __device__ __forceinline__ void add(f32x4* acc) const {
#pragma unroll
    for (int t = 0; t < RT; ++t) {
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
// waits for a condition, and four steps' loads are in flight (chunks of 2100
// rows, rank 64: TIME_SHRINK us, one step at a time 33).
template <typename T, typename X, int RT>
__global__ __launch_bounds__(kShrinkWaves * 64) void lora_shrink(const LoraArgs a, int slots,
                                                                 int splits, int rank_groups) {
  __shared__ f32x4 sums[kShrinkWaves][RT][64];
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
  if (tile < tiles) {
    const int steps = (K + 31) / 32, whole = K / 32;
    const int u0 = (int)((int64_t)steps * part / parts);
    const int u1 = (int)((int64_t)steps * (part + 1) / parts);
    const X* x = static_cast<const X*>(a.x) + (int64_t)row * K;
    const uint16_t* w[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t)
      w[t] = static_cast<const uint16_t*>(a.ad.a) +
             ((int64_t)s.adapter * a.ad.rank + min(r0 + 16 * t + col, a.ad.rank - 1)) * K;
    int u = u0;
    for (; u + 4 <= min(u1, whole); u += 4) {
      Step<T, X, RT> step[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) step[e].template load<false>(w, x, 32 * (u + e) + 8 * quarter, K);
#pragma unroll
      for (int e = 0; e < 4; ++e) step[e].add(acc);
    }
    for (; u < u1; ++u) {
      Step<T, X, RT> step;
      step.template load<true>(w, x, 32 * u + 8 * quarter, K);
      step.add(acc);
    }
  }
#pragma unroll
  for (int t = 0; t < RT; ++t) sums[wave][t][lane] = acc[t];
  __syncthreads();
  if (tile >= tiles || wave % per_tile != 0 || !real) return;
  float* low = a.low + ((int64_t)split * a.M + row) * a.ad.rank + r0 + 4 * quarter;
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    for (int w = 1; w < per_tile; ++w) acc[t] += sums[wave + w][t][lane];
    if (r0 + 16 * t + 4 * quarter < a.ad.rank) *reinterpret_cast<f32x4*>(low + 16 * t) = acc[t];
  }
}

// x in three values of T, which hold all of its bits; an infinity or NaN in one.
template <typename T>
__device__ __forceinline__ void split3(float x, short* out) {
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    const T t = (T)x;
    out[i] = __builtin_bit_cast(short, t);
    const float rest = x - (float)t;
    x = fabsf(x) < __builtin_inff() ? rest : 0.0f;
  }
}

struct F4 {  // rows of any 4-byte alignment
  float v[4];
};

// RB blocks of 32 ranks. CT tiles of 16 columns are taken at a time, their
// loads before their products.
template <typename T, int RB>
__global__ __launch_bounds__(kExpandWaves * 64) void lora_expand(const LoraArgs a, int slots,
                                                                 int splits, int col_groups,
                                                                 int cols) {
  constexpr int CT = RB <= 2 ? 4 : RB == 4 ? 2 : 1;
  int id = blockIdx.x;
  const int c0 = id % col_groups * cols;
  id /= col_groups;
  const int slot = id % slots, block = id / slots;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quarter = lane >> 4;
  const int N = a.ad.N, end = min(c0 + cols, N);

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
        top = fmaxf(top, fabsf(v[i][e]));
      }
    }
    if (sizeof(T) == 2 && __builtin_bit_cast(unsigned short, (T)1.0f) == 0x3C00) {
      // fp16: the row times a power of two, its largest value near 2^14.
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const int e = top > 0.0f && top < __builtin_inff() ? 14 - (int)ilogbf(top) : 0;
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

  const uint16_t* w = static_cast<const uint16_t*>(a.ad.b) + (int64_t)s.adapter * N * a.ad.rank;
  const float* y = a.y + row * a.y_stride;
  float* out = a.out + row * a.out_stride;
  const auto tile_of = [&](int n0, const s16x8* wf, F4 before) {
    f32x4 acc = {};
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int x = 0; x < 3; ++x) acc = mfma16<T>(wf[i], low[i][x], acc);
#pragma unroll
    for (int e = 0; e < 4; ++e) before.v[e] = fmaf(acc[e], back, before.v[e]);
    return before;
  };
  // Weights of column n0 + col; those past the rank are zeros.
  const auto weights = [&](int n, s16x8* wf) {
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int r = 32 * i + 8 * quarter;
      wf[i] = *reinterpret_cast<const s16x8*>(w + (int64_t)n * a.ad.rank + (r < a.ad.rank ? r : 0));
    }
  };
  const auto cut = [&](s16x8* wf) {
    if (rank % 32 == 0 && rank == 32 * RB) return;
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (32 * i + 8 * quarter + e >= rank) wf[i][e] = 0;
  };
  const int step = tiles == 1 ? 16 * CT * kExpandWaves : 16 * CT;
  int n0 = c0 + (tiles == 1 ? 16 * CT * wave : 0);
  for (; n0 + 16 * CT <= end; n0 += step) {
    s16x8 wf[CT][RB];
    F4 v[CT];
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      weights(n0 + 16 * t + col, wf[t]);
      __builtin_memcpy(&v[t], y + n0 + 16 * t + 4 * quarter, 16);
    }
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      cut(wf[t]);
      v[t] = tile_of(n0 + 16 * t, wf[t], v[t]);
    }
    if (real) {
#pragma unroll
      for (int t = 0; t < CT; ++t) __builtin_memcpy(out + n0 + 16 * t + 4 * quarter, &v[t], 16);
    }
  }
  // What is left of the columns, a tile at a time.
  for (const int stop = min(n0 + 16 * CT, end); n0 < stop; n0 += 16) {
    s16x8 wf[RB];
    F4 v = {};
    const int n = n0 + 4 * quarter;
    weights(min(n0 + col, N - 1), wf);
    cut(wf);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < end) v.v[e] = y[n + e];
    v = tile_of(n0, wf, v);
    if (real) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < end) out[n + e] = v.v[e];
    }
  }
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

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
  // Columns of a work-group of the second kernel: while that leaves two
  // work-groups to a CU, if an eighth of the slots are taken.
  const int64_t some = (int64_t)p.blocks * (p.slots / 8 > 1 ? p.slots / 8 : 1);
  p.cols = 256;
  while (p.cols > 64 && some * ceil_div(ad.N, p.cols) < 512) p.cols /= 2;
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

template <typename T, int RB>
hipError_t expand(const LoraArgs& a, const Plan& p, hipStream_t stream) {
  const int64_t grid = (int64_t)p.blocks * p.slots * p.col_groups;
  hipLaunchKernelGGL((lora_expand<T, RB>), dim3((unsigned)grid), dim3(kExpandWaves * 64), 0,
                     stream, a, p.slots, p.splits, p.col_groups, p.cols);
  return hipGetLastError();
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
  if (blocks == 1) return expand<T, 1>(a, p, stream);
  if (blocks == 2) return expand<T, 2>(a, p, stream);
  if (blocks <= 4) return expand<T, 4>(a, p, stream);
  return expand<T, 8>(a, p, stream);
}

}  // namespace

bool lora_grids_fit(const vqv_adapters& ad, int M) {
  if (M < 1) return true;
  const Plan p = plan_of(ad, M);
  const int64_t groups = (int64_t)p.blocks * p.slots;
  return groups * p.rank_groups * p.splits < (1ll << 22) && groups * p.col_groups < (1ll << 23);
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
