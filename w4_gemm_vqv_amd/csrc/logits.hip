// Penalties, biases and grammar masks on logits (vqv_logits_edit), or fused
// with the greedy verify's first stage (vqv_logits_verify).
//
// One work-group takes 4096 tokens of a sequence and some of its rows. What
// the rows of a sequence share (counts, the set of seen tokens, biases) is
// read once into registers, and each row adds the draft that was fed at it to
// the counts on the way; the logits and the row's mask bits are read once.
// Bias entries may come in any order: each work-group looks through the
// sequence's entries and puts the numbers of those in its tokens into LDS (of
// entries with the same token the last one counts).
//
// Every step is one rounding in fp32 (no contraction to a fused
// multiply-add), so a token is chosen as the formulas choose it.
//
// The floor is memory: logits once (and once out), counts once per sequence.
// 64 rows over 151936 tokens with all edits and the verify take 30 us, 8.8 of
// them the floor: 39 vector instructions per token and row keep the vector
// units busy 35 % of the time, and the loads that follow one another at a
// work-group's start (biases, counts, the first row) take most of the rest.

#include "argmax.h"
#include "round_internal.h"

#pragma clang fp contract(off)

namespace vqv {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = kVerifyChunk;            // tokens of a work-group
constexpr int kQuads = kTile / (4 * kThreads);  // runs of 4 tokens of a thread

struct EditArgs {
  const float* logits;
  vqv_edits e;
  const int32_t* draft;
  const int32_t* mask;
  float* out;       // edit
  uint4* partials;  // verify
  int T, tiles, rows_per_group, words;
};

struct F4 {  // rows of any 4-byte alignment
  float v[4];
};

__device__ __forceinline__ unsigned bits4(const int32_t* __restrict__ words, int c) {
  return ((unsigned)words[c >> 5] >> (c & 31)) & 15u;
}

template <bool VERIFY>
__global__ __launch_bounds__(kThreads) void logits_edit(const EditArgs a) {
  __shared__ int entry[kTile];
  __shared__ uint4 sw[kThreads / 64];
  const int N = a.e.n, T = a.T;
  const int tile = blockIdx.x, b = blockIdx.z;
  const int c0 = tile * kTile;
  const int i0 = blockIdx.y * a.rows_per_group, i1 = min(i0 + a.rows_per_group, T);
  const bool penalties = a.e.repetition || a.e.frequency || a.e.presence;

  float bias[kQuads][4] = {};
  if (a.e.bias_start) {
#pragma unroll
    for (int j = 0; j < kQuads; ++j)
      *reinterpret_cast<int4*>(&entry[4 * (threadIdx.x + kThreads * j)]) =
          make_int4(-1, -1, -1, -1);
    __syncthreads();
    const int lo = max(a.e.bias_start[b], 0), hi = min(a.e.bias_start[b + 1], a.e.n_bias);
    for (int x = lo + threadIdx.x; x < hi; x += kThreads) {
      const int t = a.e.bias_token[x];
      if (t < N && (unsigned)(t - c0) < (unsigned)kTile) atomicMax(&entry[t - c0], x);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
      const int4 x = *reinterpret_cast<const int4*>(&entry[4 * (threadIdx.x + kThreads * j)]);
      if (x.x >= 0) bias[j][0] = a.e.bias_value[x.x];
      if (x.y >= 0) bias[j][1] = a.e.bias_value[x.y];
      if (x.z >= 0) bias[j][2] = a.e.bias_value[x.z];
      if (x.w >= 0) bias[j][3] = a.e.bias_value[x.w];
    }
  }

  int count[kQuads][4] = {};
  unsigned seen = 0;  // 4 bits per run
  float rep = 1.0f, freq = 0.0f, pres = 0.0f;
  if (penalties) {
    if (a.e.repetition) rep = a.e.repetition[b];
    if (a.e.frequency) freq = a.e.frequency[b];
    if (a.e.presence) pres = a.e.presence[b];
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
      const int c = c0 + 4 * (threadIdx.x + kThreads * j);
      if (a.e.counts) {
        const int32_t* p = a.e.counts + (int64_t)b * N + c;
        if (c + 4 <= N)
          __builtin_memcpy(count[j], p, 16);
        else
          for (int x = 0; x < 4; ++x)
            if (c + x < N) count[j][x] = p[x];
      }
      if (a.e.seen && c < N) seen |= bits4(a.e.seen + (int64_t)b * a.words, c) << (4 * j);
    }
  }
  const int32_t* draft = a.draft ? a.draft + (int64_t)b * (T - 1) : nullptr;

  // Draft number i - 1 is fed at row i: the rows from i on count it.
  const auto feed = [&](int i) {
    const unsigned t = (unsigned)(draft[i - 1] - c0);
    if (t < (unsigned)kTile) {
#pragma unroll
      for (int j = 0; j < kQuads; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          count[j][x] += t == 4 * (threadIdx.x + kThreads * j) + x;
    }
  };
  if (penalties && draft)
    for (int i = 1; i < i0; ++i) feed(i);

  for (int i = i0; i < i1; ++i) {
    if (penalties && draft && i) feed(i);
    const int64_t row = (int64_t)b * T + i;
    const float* x = a.logits + row * N;
    F4 v[kQuads];
    unsigned allowed = ~0u;
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
      const int c = c0 + 4 * (threadIdx.x + kThreads * j);
      if (c + 4 <= N) {
        __builtin_memcpy(&v[j], x + c, 16);
      } else {
        for (int y = 0; y < 4; ++y) v[j].v[y] = c + y < N ? x[c + y] : 0.0f;
      }
      if (a.mask && c < N) {
        const unsigned m = bits4(a.mask + row * a.words, c);
        allowed &= ~((~m & 15u) << (4 * j));
      }
    }
    Top2Scan best = top2_scan_none();
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
      const int c = c0 + 4 * (threadIdx.x + kThreads * j);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        float w = v[j].v[y];
        if (penalties) {
          const int n = count[j][y];
          if (n > 0 || (seen >> (4 * j + y) & 1u)) w = w > 0.0f ? w / rep : w * rep;
          w = w - freq * (float)n;
          if (n > 0) w = w - pres;
        }
        w = w + bias[j][y];
        if (!(allowed >> (4 * j + y) & 1u)) w = -__builtin_inff();
        v[j].v[y] = w;
        if (VERIFY && c + y < N) top2_scan(best, w, c + y, w == w);
      }
      if (!VERIFY) {
        float* o = a.out + row * N + c;
        if (c + 4 <= N)
          __builtin_memcpy(o, &v[j], 16);
        else
          for (int y = 0; y < 4; ++y)
            if (c + y < N) o[y] = v[j].v[y];
      }
    }
    if (VERIFY) {
      Top2 t = top2_best64(top2_of_scan(best));
      const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
      __syncthreads();  // the last row's partials have been read
      if (lane == 0) sw[wave] = top2_pack(t);
      __syncthreads();
      if (threadIdx.x == 0) {
        for (int w = 1; w < kThreads / 64; ++w) top2_merge(t, sw[w]);
        a.partials[row * a.tiles + tile] = top2_pack(t);
      }
    }
  }
}

// Rows of a work-group: all of a sequence's, so that its counts are read
// once, unless that leaves fewer than two work-groups for a CU (4 sequences of
// 16 rows: 4 rows, 30.1 us; 2 rows, 32.3).
int rows_per_group(int B, int T, int tiles) {
  int rows = T;
  while (rows > 1 && (int64_t)B * tiles * ((T + rows - 1) / rows) < 512) rows = (rows + 1) / 2;
  return rows;
}

template <bool VERIFY>
hipError_t launch(EditArgs a, hipStream_t stream) {
  a.tiles = verify_chunks(a.e.n);
  a.words = (a.e.n + 31) / 32;
  a.rows_per_group = rows_per_group(a.e.n_seqs, a.T, a.tiles);
  const dim3 grid(a.tiles, (a.T + a.rows_per_group - 1) / a.rows_per_group, a.e.n_seqs);
  hipLaunchKernelGGL(logits_edit<VERIFY>, grid, dim3(kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_logits_edit(const float* logits, const vqv_edits& edits, const int32_t* draft,
                              int T, const int32_t* mask, float* out, hipStream_t stream) {
  return launch<false>(EditArgs{logits, edits, draft, mask, out, nullptr, T, 0, 0, 0}, stream);
}

hipError_t launch_logits_verify(const float* logits, const vqv_edits& edits, const int32_t* mask,
                                const VerifyArgs& va, hipStream_t stream) {
  const hipError_t e = launch<true>(
      EditArgs{logits, edits, va.draft, mask, nullptr, va.partials, va.T, 0, 0, 0}, stream);
  if (e != hipSuccess) return e;
  VerifyArgs done = va;
  done.pgroups = verify_chunks(edits.n);
  return launch_verify_finish(done, stream);
}

}  // namespace vqv
