// Verify of drafted tokens by sampling (vqv_verify_sampled).
//
// First kernel: one work-group per (row, chunk of 4096 logits), read once into
// registers: the chunk's largest value with its lowest index (argmax.h: NaN
// first), then sum exp((x - largest) / temperature) of the chunk.
// Second kernel: every work-group of a sequence joins the rows' chunks (largest
// value and sum of each row), takes the drafts in their order and so knows the
// row to draw from. After a rejection each then sums max(p - q, 0) over a chunk
// of that row, and the last to finish goes on; with all drafts accepted the
// chunks' sums are there, and the first goes on alone. It finds the chunk that
// the draw falls into, forms its probabilities once more and finds the token.
//
// Exponentials and sums are 64-bit: the draw's threshold is compared with sums
// over up to 10^5 tokens, and an error of fp32's size would pass a border
// between two tokens in a few of a hundred draws. Sums are taken in an order that
// does not depend on timing.
//
// What bounds it: the 64-bit exponentials beside the loads in the first kernel (64
// rows of 151936 logits: 13 us, 3 TB/s); the second is a chain of passes over a
// row's chunks, with a wait for the last work-group between, of 7 to 10 us.
// A call of 1 x 8 and 4 x 16 rows with draft probabilities and of 64 x 1: 14, 16 to 19
// (as blocks end) and 19 us. With sums by LDS atomics and 256 threads a draw they
// took 31, 37 and 35.

#include <limits.h>

#include "argmax.h"
#include "serve_internal.h"

namespace vqv {
namespace {

constexpr int kChunk = kVerifyChunk;
constexpr int kThreads = 256;          // of the first kernel
constexpr int kPer = kChunk / kThreads;
constexpr int kDraw = 1024;            // of the second: four tokens of a chunk each
constexpr int kDrawWaves = kDraw / 64;
static_assert(kChunk == 4 * kDraw, "");

// Of a row's chunk: sum of exp((x - top) / temperature), top as a key and its
// lowest index.
struct __align__(16) Part {
  double sum;
  unsigned key;
  int index;
};

struct Args {
  SampleArgs s;
  int chunks;
  Part* part;      // [B * T][chunks]
  double* rest;    // [B][chunks]: sums of what is left after a rejection
  unsigned* done;  // [B]
};

// 2^y of y <= 0: 2^n times the polynomial that is equal to 2^f at the ten
// Chebyshev points of [-1/2, 1/2] (relative error 1.9e-14).
__device__ __forceinline__ double exp2_of(double y) {
  y = fmax(y, -1100.0);
  const double n = rint(y), f = y - n;
  double r = 1.0205905320493103e-07;
  r = fma(r, f, 1.3259645243929057e-06);
  r = fma(r, f, 1.5252672925346873e-05);
  r = fma(r, f, 0.00015403433751254997);
  r = fma(r, f, 0.0013333558200793719);
  r = fma(r, f, 0.009618129193934304);
  r = fma(r, f, 0.05550410866465168);
  r = fma(r, f, 0.2402265069564034);
  r = fma(r, f, 0.6931471805599462);
  r = fma(r, f, 1.0000000000000135);
  return ldexp(r, (int)n);
}

// exp((x - top) / temperature) of x <= top, by = log2(e) / temperature. For
// -inf the product with by = 0 is NaN, which exp2_of's maximum drops.
__device__ __forceinline__ double exp_scaled(double x, double top, double by) {
  return exp2_of((x - top) * by);
}

__device__ __forceinline__ double by_of(float temperature) {
  return 1.4426950408889634074 / (double)temperature;
}

__device__ __forceinline__ float temperature_of(const SampleArgs& s, int b) {
  return s.temperature ? s.temperature[b] : 1.0f;
}

// Valid drafts of a sequence.
__device__ __forceinline__ int drafts_of(const SampleArgs& s, int b) {
  return s.draft_len ? min(max(s.draft_len[b], 0), s.T - 1) : s.T - 1;
}

// Whether p is 1 at the largest value: nothing else can be formed.
__device__ __forceinline__ bool one_hot(float temperature, unsigned key) {
  const float v = key_value(key);
  return !(temperature > 0.0f) || key == 0xFFFFFFFFu || v == __builtin_inff() ||
         v == -__builtin_inff();
}

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double moved(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const unsigned lo = __builtin_amdgcn_update_dpp(0, (int)u, CTRL, ROWS, 0xF, ROWS == 0xF);
  const unsigned hi = __builtin_amdgcn_update_dpp(0, (int)(u >> 32), CTRL, ROWS, 0xF, ROWS == 0xF);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// Inclusive sums over the lanes of a wave, in their order: within 16 lanes by
// steps of 1, 2, 4 and 8, then each row's and each half's sum to the next.
__device__ __forceinline__ double wave_scan(double x) {
  x += moved<0x111>(x);
  x += moved<0x112>(x);
  x += moved<0x114>(x);
  x += moved<0x118>(x);
  x += moved<0x142, 0xA>(x);
  x += moved<0x143, 0xC>(x);
  return x;
}

__device__ __forceinline__ double of_lane(double x, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const unsigned lo = __builtin_amdgcn_readlane((int)u, lane);
  const unsigned hi = __builtin_amdgcn_readlane((int)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double wave_sum(double x) { return of_lane(wave_scan(x), 63); }

// The better of all lanes' (key, index), the same in every lane.
__device__ __forceinline__ void wave_best(unsigned& key, int& index) {
  Top2 t{key, index, 0u};
  t = top2_best64(t);
  key = t.k1;
  index = t.i1;
}

// Sum over a work-group of WAVES waves, the same in every thread. `lds` is its own.
template <int WAVES>
__device__ __forceinline__ double group_sum(double x, double* lds) {
  x = wave_sum(x);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  double r = lds[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) r += lds[w];
  return r;
}

// Values c .. c+3 of a row of n.
__device__ __forceinline__ void load4(const float* row, int c, int n, float none, float* v) {
  if (c + 4 <= n) {
    __builtin_memcpy(v, row + c, 16);
  } else {
#pragma unroll
    for (int y = 0; y < 4; ++y) v[y] = c + y < n ? row[c + y] : none;
  }
}

__global__ __launch_bounds__(kThreads) void sample_parts(const Args a) {
  __shared__ unsigned keys[kThreads / 64];
  __shared__ int indices[kThreads / 64];
  __shared__ double sums[kThreads / 64];
  const int row = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks;
  const int b = row / a.s.T, i = row % a.s.T;
  if (chunk == 0 && i == 0 && threadIdx.x == 0) a.done[b] = 0u;
  if (i > drafts_of(a.s, b)) return;  // nothing is asked of it
  const int N = a.s.N, c0 = chunk * kChunk;
  float v[kPer / 4][4];
#pragma unroll
  for (int j = 0; j < kPer / 4; ++j)
    load4(a.s.logits + (int64_t)row * N, c0 + 4 * (threadIdx.x + kThreads * j), N,
          -__builtin_inff(), v[j]);
  const float t = temperature_of(a.s, b);
  const int wave = threadIdx.x >> 6;

  // The largest value, and whether there is a NaN.
  float best = v[0][0];
  bool nan = false;
#pragma unroll
  for (int j = 0; j < kPer / 4; ++j)
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      best = fmaxf(best, v[j][y]);
      nan |= v[j][y] != v[j][y];
    }
  unsigned key = nan ? 0xFFFFFFFFu : order_key(best);
  int index = 0;
  wave_best(key, index);
  if ((threadIdx.x & 63) == 0) keys[wave] = key;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) key = max(key, keys[w]);
  double sum = 0.0;
  index = 0;
  if (one_hot(t, key)) {
    // Its lowest place is what counts.
    index = INT_MAX;
#pragma unroll
    for (int j = kPer / 4 - 1; j >= 0; --j)
#pragma unroll
      for (int y = 3; y >= 0; --y) {
        const int c = c0 + 4 * (threadIdx.x + kThreads * j) + y;
        if (c < N && order_key(v[j][y]) == key) index = c;
      }
    unsigned same = key;
    if (index == INT_MAX) same = 0;
    wave_best(same, index);
    if ((threadIdx.x & 63) == 0) indices[wave] = index;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) index = min(index, indices[w]);
  } else {
    const double by = by_of(t), top = key_value(key);
#pragma unroll
    for (int j = 0; j < kPer / 4; ++j)
#pragma unroll
      for (int y = 0; y < 4; ++y) sum += exp_scaled((double)v[j][y], top, by);
    sum = group_sum<kThreads / 64>(sum, sums);
  }
  if (threadIdx.x == 0) a.part[(int64_t)row * a.chunks + chunk] = Part{sum, key, index};
}

// Of values that grow with the thread: the lowest `hit` (INT_MAX: none) and the
// highest `holds` (-1: none) of the waves before it and its own, for all threads.
// Lanes give theirs by ballots and waves by a place of their own in LDS: a
// thousand atomics on one word take 7 us.
struct Ends {
  int hit, holds;
};
template <int WAVES>
__device__ __forceinline__ Ends group_ends(int hit, int holds, Ends* lds) {
  const uint64_t hits = __ballot(hit != INT_MAX), held = __ballot(holds >= 0);
  Ends e{INT_MAX, -1};
  if (hits != 0) e.hit = __builtin_amdgcn_readlane(hit, __builtin_ctzll(hits));
  if (held != 0) e.holds = __builtin_amdgcn_readlane(holds, 63 - __builtin_clzll(held));
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = e;
  __syncthreads();
  e = lds[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) {
    e.hit = min(e.hit, lds[w].hit);
    e.holds = max(e.holds, lds[w].holds);
  }
  return e;
}

// A row's chunks joined, by one wave; uniform.
struct RowSum {
  double sum;
  unsigned key;
  int index;
};

__device__ __forceinline__ RowSum join_row(const Args& a, int row, float temperature) {
  const Part* part = a.part + (int64_t)row * a.chunks;
  const int lane = threadIdx.x & 63;
  const Part mine = lane < a.chunks ? part[lane] : Part{0.0, 0u, INT_MAX};
  unsigned key = mine.key;
  int index = mine.index;
  for (int c = lane + 64; c < a.chunks; c += 64) take_better(key, index, part[c].key, part[c].index);
  wave_best(key, index);
  double sum = 0.0;
  if (!one_hot(temperature, key)) {
    const double by = by_of(temperature), top = key_value(key);
    if (lane < a.chunks) sum = mine.sum * exp_scaled((double)key_value(mine.key), top, by);
    for (int c = lane + 64; c < a.chunks; c += 64)
      sum += part[c].sum * exp_scaled((double)key_value(part[c].key), top, by);
    sum = wave_sum(sum);
  }
  return RowSum{sum, key, index};
}

__global__ __launch_bounds__(kDraw) void sample_draw(const Args a) {
  __shared__ double sums[kDrawWaves], scans[2][kDrawWaves];
  __shared__ RowSum rows[64];
  __shared__ Ends ends[2][kDrawWaves];
  __shared__ int accepted, last_one;
  __shared__ double before;
  const SampleArgs& s = a.s;
  const int T = s.T, N = s.N;
  const int groups = gridDim.x / s.B;
  const int b = blockIdx.x / groups, group = blockIdx.x % groups;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float t = temperature_of(s, b);
  const int drafts = drafts_of(s, b);

  // What is asked of each draft, by the thread of its number.
  float x_of = 0.0f, q_of = 1.0f, u_of = 0.0f;
  int d_of = -1;
  if ((int)threadIdx.x < drafts) {
    const int64_t at = (int64_t)b * (T - 1) + threadIdx.x;
    d_of = s.draft[at];
    u_of = s.uniform[(int64_t)b * T + threadIdx.x];
    if ((unsigned)d_of < (unsigned)N) {
      x_of = s.logits[((int64_t)b * T + threadIdx.x) * N + d_of];
      if (s.probs) q_of = s.probs[at * N + d_of];
    }
  }
  const float u_draw = s.uniform[(int64_t)b * T + T - 1];
  for (int i = wave; i <= drafts; i += kDrawWaves) {
    const RowSum r = join_row(a, b * T + i, t);
    if (lane == 0) rows[i] = r;
  }
  __syncthreads();
  if (wave == 0) {
    bool ok = false;
    if (lane < drafts && (unsigned)d_of < (unsigned)N) {
      const RowSum r = rows[lane];
      const double p = one_hot(t, r.key)
                           ? (d_of == r.index ? 1.0 : 0.0)
                           : exp_scaled((double)x_of, (double)key_value(r.key), by_of(t)) / r.sum;
      ok = (double)u_of * (double)q_of < p;
    }
    const uint64_t good = __ballot(ok);
    if (lane == 0) accepted = ~good == 0 ? 64 : __builtin_ctzll(~good);
  }
  __syncthreads();
  const int accept = min(accepted, drafts);
  const RowSum r = rows[accept];
  const float* x = s.logits + ((int64_t)b * T + accept) * N;
  const bool hot = one_hot(t, r.key);
  const bool rejected = accept < drafts;
  const float* q = rejected && s.probs ? s.probs + ((int64_t)b * (T - 1) + accept) * N : nullptr;
  int d = rejected && !s.probs ? s.draft[(int64_t)b * (T - 1) + accept] : -1;
  const double by = hot ? 1.0 : by_of(t), top = key_value(r.key), inv = 1.0 / r.sum;
  double* rest = a.rest + (int64_t)b * a.chunks;
  // What the draw is from, at a thread's four tokens of a chunk: p, or what is
  // left of it after a rejection.
  double w[4];
  const auto form = [&](int chunk) {
    const int c = chunk * kChunk + 4 * (int)threadIdx.x;
    float v[4], take[4] = {};
    load4(x, c, N, -__builtin_inff(), v);
    if (q) load4(q, c, N, 0.0f, take);
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const double p = exp_scaled((double)v[y], top, by) * inv;
      w[y] = q ? (p > (double)take[y] ? p - (double)take[y] : 0.0) : c + y == d ? 0.0 : p;
    }
    return (w[0] + w[1]) + (w[2] + w[3]);
  };

  bool left = false;  // draws from what is left of p
  if (rejected && !hot) {
    for (int chunk = group; chunk < a.chunks; chunk += groups) {
      const double sum = group_sum<kDrawWaves>(form(chunk), sums);
      if (threadIdx.x == 0)
        __hip_atomic_store(rest + chunk, sum, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __syncthreads();  // `sums` is free again
    }
    // The last work-group of the sequence to come here goes on.
    if (threadIdx.x == 0)
      last_one = __hip_atomic_fetch_add(a.done + b, 1u, __ATOMIC_ACQ_REL,
                                        __HIP_MEMORY_SCOPE_AGENT) == (unsigned)groups - 1;
    __syncthreads();
    if (!last_one) return;
    left = true;
  } else if (group != 0) {
    return;
  }

  int token = r.index;
  if (!hot) {
    // Inclusive sums of the threads' values, in the threads' order, and all of them.
    struct Scan {
      double upto, total;
    };
    const auto inclusive = [&](double v, double* lds) {
      const double scan = wave_scan(v);
      if (lane == 63) lds[wave] = scan;
      __syncthreads();
      double lead = 0.0, total = 0.0;
#pragma unroll
      for (int i = 0; i < kDrawWaves; ++i) {
        if (i == wave) lead = total;
        total += lds[i];
      }
      return Scan{lead + scan, total};
    };
    // A chunk's share: of what is left, or of p. A thread has chunks first .. end - 1.
    const Part* part = a.part + ((int64_t)b * T + accept) * a.chunks;
    const int per = (a.chunks + kDraw - 1) / kDraw;
    const int first = min((int)threadIdx.x * per, a.chunks), end = min(first + per, a.chunks);
    const auto share = [&](int c) {
      if (left) return __hip_atomic_load(rest + c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      return part[c].sum * exp_scaled((double)key_value(part[c].key), top, by) * inv;
    };
    double mine = 0.0, one = 0.0;
    Scan all;
    for (;;) {
      mine = 0.0;
      for (int c = first; c < end; ++c) {
        one = share(c);
        mine += one;
      }
      all = inclusive(mine, scans[0]);
      if (!left || all.total > 0.0) break;
      left = false;  // nothing is left: draw from p
      q = nullptr;
      d = -1;
      __syncthreads();
    }
    const double goal = (double)u_draw * all.total;
    // The first chunk whose sum passes the goal, or the last that holds something.
    int hit = INT_MAX, holds = -1;
    double sum = all.upto - mine, lead = 0.0, lead_last = 0.0;
    for (int c = first; c < end; ++c) {
      const double share_of = per == 1 ? one : share(c);
      if (share_of > 0.0) {
        holds = c;
        lead_last = sum;
        if (hit == INT_MAX && sum + share_of > goal) {
          hit = c;
          lead = sum;
        }
      }
      sum += share_of;
    }
    const Ends at = group_ends<kDrawWaves>(hit, holds, ends[0]);
    const bool any = at.hit != INT_MAX;
    const int chunk = any ? at.hit : max(at.holds, 0);
    if (any ? hit == chunk : holds == chunk) before = any ? lead : lead_last;
    mine = form(chunk);
    sum = inclusive(mine, scans[1]).upto - mine;  // (and `before` is there for all)
    const double need = goal - before;
    const int c0 = chunk * kChunk + 4 * (int)threadIdx.x;
    hit = INT_MAX;
    holds = -1;
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      sum += w[y];
      if (w[y] > 0.0) {
        holds = c0 + y;
        if (hit == INT_MAX && sum > need) hit = c0 + y;
      }
    }
    const Ends in = group_ends<kDrawWaves>(any ? hit : INT_MAX, holds, ends[1]);
    token = in.hit != INT_MAX ? in.hit : in.holds >= 0 ? in.holds : r.index;
  }
  if (threadIdx.x == 0) {
    s.token[b] = token;
    s.accept_len[b] = accept;
  }
  if (s.logprob && threadIdx.x < (unsigned)T) {
    const int i = threadIdx.x;
    float out = 0.0f;
    if (i <= accept) {
      const RowSum m = rows[i];
      const int c = i < accept ? d_of : token;
      if (one_hot(t, m.key))
        out = c == m.index ? 0.0f : -__builtin_inff();
      else
        out = (float)(((double)(i < accept ? x_of : x[token]) - (double)key_value(m.key)) /
                          (double)t - log(m.sum));
    }
    s.logprob[(int64_t)b * T + i] = out;
  }
}

size_t padded(size_t n) { return (n + 15) / 16 * 16; }

}  // namespace

size_t sample_workspace_bytes(int B, int T, int N) {
  const size_t chunks = verify_chunks(N);
  return (size_t)B * T * chunks * sizeof(Part) + padded(B * chunks * sizeof(double)) +
         padded(B * sizeof(unsigned));
}

hipError_t launch_verify_sampled(const SampleArgs& s, hipStream_t stream) {
  Args a;
  a.s = s;
  a.chunks = verify_chunks(s.N);
  a.part = static_cast<Part*>(s.workspace);
  a.rest = reinterpret_cast<double*>(a.part + (size_t)s.B * s.T * a.chunks);
  a.done = reinterpret_cast<unsigned*>(reinterpret_cast<char*>(a.rest) +
                                       padded((size_t)s.B * a.chunks * sizeof(double)));
  hipLaunchKernelGGL(sample_parts, dim3((unsigned)(s.B * s.T * (int64_t)a.chunks)), dim3(kThreads),
                     0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int groups = s.T > 1 ? (a.chunks < 64 ? a.chunks : 64) : 1;
  hipLaunchKernelGGL(sample_draw, dim3((unsigned)(s.B * groups)), dim3(kDraw), 0, stream, a);
  return hipGetLastError();
}

}  // namespace vqv
