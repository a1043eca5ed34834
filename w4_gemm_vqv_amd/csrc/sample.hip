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
// between two tokens in a few of a hundred draws. exp is 2^n times a polynomial
// of degree 10 over half a binary step on each side (relative error 2e-13).
// Sums are taken in an order that does not depend on timing.

#include <limits.h>

#include "argmax.h"
#include "serve_internal.h"

namespace vqv {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = kVerifyChunk;
constexpr int kPer = kChunk / kThreads;

// Of a row's chunk: sum of exp((x - top) / temperature), top as a key and its
// lowest index.
struct __align__(16) Part {
  double sum;
  unsigned key;
  int index;
};

struct F4 {  // rows of any 4-byte alignment
  float v[4];
};

struct Args {
  SampleArgs s;
  int chunks;
  Part* part;      // [B * T][chunks]
  double* rest;    // [B][chunks]: sums of what is left after a rejection
  unsigned* done;  // [B]
};

// exp(x / temperature) of x <= 0, by = log2(e) / temperature.
__device__ __forceinline__ double exp_scaled(double x, double by) {
  const double y = fmax(x * by, -1100.0);
  const double n = rint(y);
  const double f = (y - n) * 0.69314718055994530942;
  double r = 1.0 / 3628800.0;
  r = fma(r, f, 1.0 / 362880.0);
  r = fma(r, f, 1.0 / 40320.0);
  r = fma(r, f, 1.0 / 5040.0);
  r = fma(r, f, 1.0 / 720.0);
  r = fma(r, f, 1.0 / 120.0);
  r = fma(r, f, 1.0 / 24.0);
  r = fma(r, f, 1.0 / 6.0);
  r = fma(r, f, 0.5);
  r = fma(r, f, 1.0);
  r = fma(r, f, 1.0);
  return ldexp(r, (int)n);
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

__device__ __forceinline__ double shuffle_xor(double x, int d) {
  return __shfl_xor(x, d);
}

// Sum over the work-group, the same in every thread.
__device__ __forceinline__ double group_sum(double x, double* lds) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x += shuffle_xor(x, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
  __syncthreads();
  double r = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) r += lds[w];
  return r;
}

// 16 values of a chunk per thread, runs of 4: element 4 (thread + 256 j) + y.
__device__ __forceinline__ void load_chunk(const float* row, int c0, int n, float none,
                                           float (*v)[4]) {
#pragma unroll
  for (int j = 0; j < kPer / 4; ++j) {
    const int c = c0 + 4 * (threadIdx.x + kThreads * j);
    if (c + 4 <= n) {
      __builtin_memcpy(v[j], row + c, 16);
    } else {
#pragma unroll
      for (int y = 0; y < 4; ++y) v[j][y] = c + y < n ? row[c + y] : none;
    }
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
  load_chunk(a.s.logits + (int64_t)row * N, c0, N, -__builtin_inff(), v);
  unsigned key = 0;
  int index = INT_MAX;
#pragma unroll
  for (int j = 0; j < kPer / 4; ++j)
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int c = c0 + 4 * (threadIdx.x + kThreads * j) + y;
      if (c < N) take_better(key, index, order_key(v[j][y]), c);
    }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    const unsigned k = __shfl_xor((int)key, d);
    const int x = __shfl_xor(index, d);
    take_better(key, index, k, x);
  }
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) {
    keys[wave] = key;
    indices[wave] = index;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) take_better(key, index, keys[w], indices[w]);
  const float t = temperature_of(a.s, b);
  double sum = 0.0;
  if (!one_hot(t, key)) {
    const double by = by_of(t), top = key_value(key);
#pragma unroll
    for (int j = 0; j < kPer / 4; ++j)
#pragma unroll
      for (int y = 0; y < 4; ++y) sum += exp_scaled((double)v[j][y] - top, by);
  }
  sum = group_sum(sum, sums);
  if (threadIdx.x == 0) a.part[(int64_t)row * a.chunks + chunk] = Part{sum, key, index};
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
  unsigned key = 0;
  int index = INT_MAX;
  for (int c = lane; c < a.chunks; c += 64) take_better(key, index, part[c].key, part[c].index);
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    const unsigned k = __shfl_xor((int)key, d);
    const int x = __shfl_xor(index, d);
    take_better(key, index, k, x);
  }
  double sum = 0.0;
  if (!one_hot(temperature, key)) {
    const double by = by_of(temperature), top = key_value(key);
    for (int c = lane; c < a.chunks; c += 64)
      sum += part[c].sum * exp_scaled((double)key_value(part[c].key) - top, by);
#pragma unroll
    for (int d = 32; d; d >>= 1) sum += shuffle_xor(sum, d);
  }
  return RowSum{sum, key, index};
}

__global__ __launch_bounds__(kThreads) void sample_draw(const Args a) {
  __shared__ double sums[kThreads / 64], scan[kThreads];
  __shared__ RowSum rows[64];
  __shared__ int good[64];
  __shared__ int last_one, found, at_chunk, top_index;
  __shared__ double before;
  const SampleArgs& s = a.s;
  const int T = s.T, N = s.N;
  const int groups = gridDim.x / s.B;
  const int b = blockIdx.x / groups, group = blockIdx.x % groups;
  const float t = temperature_of(s, b);
  const int drafts = drafts_of(s, b);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = wave; i <= drafts; i += kThreads / 64) {
    const RowSum r = join_row(a, b * T + i, t);
    if (lane == 0) {
      rows[i] = r;
      int ok = 0;
      if (i < drafts) {
        const int d = s.draft[(int64_t)b * (T - 1) + i];
        if ((unsigned)d < (unsigned)N) {
          double p;
          if (one_hot(t, r.key))
            p = d == r.index ? 1.0 : 0.0;
          else
            p = exp_scaled((double)s.logits[((int64_t)b * T + i) * N + d] -
                               (double)key_value(r.key), by_of(t)) / r.sum;
          const double q = s.probs ? s.probs[((int64_t)b * (T - 1) + i) * N + d] : 1.0;
          ok = (double)s.uniform[(int64_t)b * T + i] * q < p;
        }
      }
      good[i] = ok;
    }
  }
  __syncthreads();
  int accept = 0;
  while (accept < drafts && good[accept]) ++accept;
  const RowSum r = rows[accept];
  const float* x = s.logits + ((int64_t)b * T + accept) * N;
  const bool hot = one_hot(t, r.key);
  const bool rejected = accept < drafts;
  const float* q = rejected && s.probs ? s.probs + ((int64_t)b * (T - 1) + accept) * N : nullptr;
  const int d = rejected ? s.draft[(int64_t)b * (T - 1) + accept] : -1;
  const double by = hot ? 1.0 : by_of(t), top = key_value(r.key);
  const double* rest = a.rest + (int64_t)b * a.chunks;

  // Probabilities (times the row's sum, where nothing is taken from them) of a
  // thread's 16 consecutive tokens of a chunk.
  const auto weights = [&](int chunk, bool less, double* w) {
    const int c0 = chunk * kChunk + kPer * (int)threadIdx.x;
#pragma unroll
    for (int y = 0; y < kPer; ++y) {
      const int c = c0 + y;
      double p = 0.0;
      if (c < N) {
        p = exp_scaled((double)x[c] - top, by);
        if (less) {
          p /= r.sum;
          p = q ? (p > (double)q[c] ? p - (double)q[c] : 0.0) : c == d ? 0.0 : p;
        }
      }
      w[y] = p;
    }
  };

  bool left = false;  // draws from what is left of p
  if (rejected && !hot) {
    for (int chunk = group; chunk < a.chunks; chunk += groups) {
      float v[kPer / 4][4], u[kPer / 4][4] = {};
      load_chunk(x, chunk * kChunk, N, -__builtin_inff(), v);
      if (q) load_chunk(q, chunk * kChunk, N, 0.0f, u);
      double sum = 0.0;
#pragma unroll
      for (int j = 0; j < kPer / 4; ++j)
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int c = chunk * kChunk + 4 * (threadIdx.x + kThreads * j) + y;
          const double p = exp_scaled((double)v[j][y] - top, by) / r.sum;
          const double take = u[j][y];
          sum += q ? (p > take ? p - take : 0.0) : c == d ? 0.0 : p;
        }
      sum = group_sum(sum, sums);
      if (threadIdx.x == 0)
        __hip_atomic_store(const_cast<double*>(rest) + chunk, sum, __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
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
    // A chunk's share: of what is left, or of the row's sum.
    const Part* part = a.part + ((int64_t)b * T + accept) * a.chunks;
    const auto share = [&](int c) {
      if (left) return __hip_atomic_load(rest + c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      return part[c].sum * exp_scaled((double)key_value(part[c].key) - top, by);
    };
    const int per = (a.chunks + kThreads - 1) / kThreads;
    const int first = min((int)threadIdx.x * per, a.chunks), end = min(first + per, a.chunks);
    // Inclusive sums of the threads' values, in the threads' order.
    const auto inclusive = [&](double v) {
      __syncthreads();
      scan[threadIdx.x] = v;
      __syncthreads();
      for (int step = 1; step < kThreads; step <<= 1) {
        const double add = threadIdx.x >= (unsigned)step ? scan[threadIdx.x - step] : 0.0;
        __syncthreads();
        scan[threadIdx.x] += add;
        __syncthreads();
      }
      return scan[threadIdx.x];
    };
    double mine = 0.0, upto = 0.0, total = 0.0;
    for (int pass = 0; pass < 2; ++pass) {
      mine = 0.0;
      for (int c = first; c < end; ++c) mine += share(c);
      upto = inclusive(mine);
      total = scan[kThreads - 1];
      if (total > 0.0 || !left) break;
      left = false;  // nothing is left: draw from p
    }
    const double goal = (double)s.uniform[(int64_t)b * T + T - 1] * total;
    if (threadIdx.x == 0) {
      found = INT_MAX;
      at_chunk = -1;
      top_index = -1;
    }
    __syncthreads();
    // The first chunk whose sum passes the goal, or the last that holds something.
    int hit = INT_MAX, holds = -1;
    double sum = upto - mine, lead = 0.0, lead_last = 0.0;
    for (int c = first; c < end; ++c) {
      const double w = share(c);
      if (w > 0.0) {
        holds = c;
        lead_last = sum;
        if (hit == INT_MAX && sum + w > goal) {
          hit = c;
          lead = sum;
        }
      }
      sum += w;
    }
    if (hit != INT_MAX) atomicMin(&found, hit);
    if (holds >= 0) atomicMax(&at_chunk, holds);
    __syncthreads();
    const bool any = found != INT_MAX;
    const int chunk = any ? found : max(at_chunk, 0);
    if (any ? hit == chunk : holds == chunk) before = any ? lead : lead_last;
    __syncthreads();
    const double need = goal - before;
    if (threadIdx.x == 0) found = INT_MAX;
    double w[kPer];
    weights(chunk, left, w);
    mine = 0.0;
#pragma unroll
    for (int y = 0; y < kPer; ++y) mine += w[y];
    sum = inclusive(mine) - mine;
    hit = INT_MAX;
    holds = -1;
#pragma unroll
    for (int y = 0; y < kPer; ++y) {
      const int c = chunk * kChunk + kPer * (int)threadIdx.x + y;
      sum += w[y];
      if (w[y] > 0.0) {
        holds = c;
        if (hit == INT_MAX && sum > need) hit = c;
      }
    }
    if (any && hit != INT_MAX) atomicMin(&found, hit);
    if (holds >= 0) atomicMax(&top_index, holds);
    __syncthreads();
    token = found != INT_MAX ? found : top_index >= 0 ? top_index : r.index;
  }
  if (threadIdx.x == 0) {
    s.token[b] = token;
    s.accept_len[b] = accept;
  }
  if (s.logprob && threadIdx.x < (unsigned)T) {
    const int i = threadIdx.x;
    float out = 0.0f;
    if (i <= accept) {
      const RowSum& m = rows[i];
      const int c = i < accept ? s.draft[(int64_t)b * (T - 1) + i] : token;
      if (one_hot(t, m.key))
        out = c == m.index ? 0.0f : -__builtin_inff();
      else
        out = (float)(((double)s.logits[((int64_t)b * T + i) * N + c] -
                       (double)key_value(m.key)) / (double)t - log(m.sum));
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
  hipLaunchKernelGGL(sample_draw, dim3((unsigned)(s.B * groups)), dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace vqv
