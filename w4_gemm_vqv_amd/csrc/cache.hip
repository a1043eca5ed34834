// Pages of a cache: copy, fork, trim, reserve, and the compaction of a
// block's confirmed rows.
//
// The book (which table holds which page) is small: one work-group or one
// wave per row does it. The moves of keys and values are spread over the
// whole GPU in 16-byte pieces; they are bound by memory. Sums of references
// are integer atomics, so their order does not matter, and free pages are
// given out by rank (prefix sums), so the result does not depend on timing. The
// end of a round of 32 blocks of 16 rows, 16 layers and 6000 pages takes 15 to
// 16 us: compact 5.4, trim 2.8, reserve 7.2, each bound by the latency of the
// few loads that follow one another.

#include <limits.h>

#include "round_common.h"
#include "round_internal.h"

namespace vqv {
namespace {

constexpr int kBook = 1024;           // threads of the book's work-group
constexpr int kPer = 16;              // pages per thread and step of its scan
constexpr int kStep = kBook * kPer;

struct Int4 {  // four references; rows of any 4-byte alignment
  int v[4];
};

// Inclusive scan over the kBook threads of the work-group; total in *all.
__device__ int scan_block(int x, int* waves, int* all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = x;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(s, d);
    if (lane >= d) s += o;
  }
  __syncthreads();  // `waves` may still be read from the last call
  if (lane == 63) waves[wave] = s;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < kBook / 64; ++w) {
    const int t = waves[w];
    before += w < wave ? t : 0;
    sum += t;
  }
  *all = sum;
  return before + s;
}

// Bits of the free pages among p0 .. p0 + kPer - 1.
__device__ unsigned free_bits(const int32_t* __restrict__ ref, int pages, int p0) {
  unsigned m = 0;
  if (p0 + kPer <= pages) {
#pragma unroll
    for (int q = 0; q < kPer / 4; ++q) {
      Int4 r;
      __builtin_memcpy(&r, ref + p0 + 4 * q, sizeof(r));
#pragma unroll
      for (int e = 0; e < 4; ++e) m |= (r.v[e] == 0 ? 1u : 0u) << (4 * q + e);
    }
  } else {
    for (int e = 0; e < kPer && p0 + e < pages; ++e) m |= (ref[p0 + e] == 0 ? 1u : 0u) << e;
  }
  return m;
}

// How many pages are free, counted only until `enough`. `first` are the free
// bits of this thread's pages of the first step.
__device__ int count_free(const int32_t* __restrict__ ref, int pages, int enough, unsigned first,
                          int* waves) {
  int found = 0;
  for (int base = 0; base < pages && found < enough; base += kStep) {
    const unsigned m = base ? free_bits(ref, pages, base + threadIdx.x * kPer) : first;
    int all;
    scan_block(__popc(m), waves, &all);
    found += all;
  }
  return found;
}

// Calls give(rank, page) for the `want` lowest free pages, and marks them
// with one reference.
template <typename F>
__device__ void give_free(int32_t* __restrict__ ref, int pages, int want, unsigned first,
                          int* waves, F give) {
  int found = 0;
  for (int base = 0; base < pages && found < want; base += kStep) {
    const int p0 = base + threadIdx.x * kPer;
    unsigned m = base ? free_bits(ref, pages, p0) : first;
    const int mine = __popc(m);
    int all;
    int rank = found + scan_block(mine, waves, &all) - mine;
    while (m && rank < want) {
      const int p = p0 + __ffs(m) - 1;
      m &= m - 1;
      ref[p] = 1;
      give(rank, p);
      ++rank;
    }
    found += all;
  }
}

// The last of n entries with off[i] <= rank.
__device__ int owner_of(const int32_t* off, int n, int rank) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= rank) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int pages_for(int tokens, int page_size) {
  return tokens <= 0 ? 0 : (tokens - 1) / page_size + 1;
}

__device__ __forceinline__ int clamp_int(int x, int lo, int hi) {
  return x < lo ? lo : x > hi ? hi : x;
}

// One wave per entry. A row may be named several times, with lengths of its
// own: a page leaves the table by an exchange, so that it is given back once,
// and held and length come to the shortest by atomic minima, in any order.
__global__ __launch_bounds__(64) void cache_trim(const vqv_pages pg,
                                                 const int32_t* __restrict__ keep_len,
                                                 const int32_t* __restrict__ rows) {
  const int i = blockIdx.x;
  const int row = rows ? rows[i] : i;
  if ((unsigned)row >= (unsigned)pg.rows) return;
  const int keep = max(keep_len[i], 0);
  const int held = clamp_int(pg.held[row], 0, pg.width);
  const int length = pg.length[row];
  const int stay = pages_for(keep, pg.page_size);
  int32_t* t = pg.table + (int64_t)row * pg.width;
  for (int j = stay + (int)threadIdx.x; j < held; j += 64) {
    const int p = atomicExch(&t[j], -1);
    if ((unsigned)p < (unsigned)pg.pages) atomicSub(&pg.ref[p], 1);
  }
  if (threadIdx.x == 0) {
    if (stay < held) atomicMin(&pg.held[row], stay);
    if (keep < length) atomicMin(&pg.length[row], keep);
  }
}

// Whether the next token of row i would be written to a page that other rows
// hold too: a row that was cut inside the pages that it shares.
__device__ __forceinline__ bool ends_in_shared_page(const vqv_pages& pg, int i, int held,
                                                    int length, int goal_len) {
  const int j = length / pg.page_size;
  if (goal_len <= length || j >= held) return false;
  const int p = pg.table[(int64_t)i * pg.width + j];
  return (unsigned)p < (unsigned)pg.pages && pg.ref[p] > 1;
}

// One work-group. off[]: the rank of each row's first new page, in LDS while
// the rows fit there. Loads that do not depend on each other go out together,
// and what a thread has read it keeps, as their latency is all the time there
// is (32 rows and 6000 pages: 8.5 us before, 7.2 so; the look at each row's last
// page does not show in the end of a round, 15.1 us with and without).
__global__ __launch_bounds__(kBook) void cache_reserve(const vqv_pages pg,
                                                       const int32_t* __restrict__ goal_len,
                                                       int n, int32_t* __restrict__ ok,
                                                       int32_t* __restrict__ scratch) {
  __shared__ int waves[kBook / 64];
  __shared__ int held_of[kBook], off_of[kBook];
  __shared__ int granted;
  const bool few = n <= kBook;
  int32_t* off = few ? off_of : scratch;
  const unsigned first = free_bits(pg.ref, pg.pages, threadIdx.x * kPer);
  if (threadIdx.x == 0) granted = 0;
  int total = 0, goal = 0, held = 0, need = 0;
  bool good = false;
  for (int base = 0; base < n; base += kBook) {
    const int i = base + threadIdx.x;
    need = 0;
    if (i < n) {
      const int tokens = goal_len[i], length = max(pg.length[i], 0);
      goal = pages_for(tokens, pg.page_size);
      held = clamp_int(pg.held[i], 0, pg.width);
      good = goal <= pg.width && !ends_in_shared_page(pg, i, held, length, tokens);
      need = good ? max(goal - held, 0) : 0;
      if (!few) ok[i] = good;
    }
    int all;
    const int end = scan_block(need, waves, &all);
    if (i < n) off[i] = total + end - need;
    total = min(total + all, INT_MAX / 2);
  }
  held_of[threadIdx.x] = held;  // of the only step where the rows are few
  const int found = total ? count_free(pg.ref, pg.pages, total, first, waves) : 0;
  for (int i = threadIdx.x; i < n; i += kBook) {
    if (!few) {
      goal = pages_for(goal_len[i], pg.page_size);
      held = clamp_int(pg.held[i], 0, pg.width);
      good = ok[i] != 0;
      need = good ? max(goal - held, 0) : 0;
    }
    good = good && (need == 0 || off[i] + need <= found);
    ok[i] = good;
    if (good && need) atomicMax(&granted, off[i] + need);
  }
  __syncthreads();
  const int want = granted;
  give_free(pg.ref, pg.pages, want, first, waves, [&](int rank, int p) {
    const int i = owner_of(off, n, rank);
    const int h = few ? held_of[i] : clamp_int(pg.held[i], 0, pg.width);
    pg.table[(int64_t)i * pg.width + h + rank - off[i]] = p;
  });
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kBook)
    if (ok[i]) {
      if (!few) goal = pages_for(goal_len[i], pg.page_size);
      if (goal > pg.held[i]) pg.held[i] = goal;
    }
}

// The book of a fork, one work-group: which pairs are good, and their new
// pages; from[i] and to[i] are the pages to copy, or -1. The children's tables
// are written next to the copies, where the whole GPU is at hand.
__global__ __launch_bounds__(kBook) void cache_fork_book(
    const vqv_pages pg, const int32_t* __restrict__ parent, const int32_t* __restrict__ child,
    int n, int32_t* __restrict__ ok, int32_t* __restrict__ named, int32_t* __restrict__ parents,
    int32_t* __restrict__ scratch, int32_t* __restrict__ from, int32_t* __restrict__ to) {
  __shared__ int waves[kBook / 64];
  __shared__ int off_of[kBook];
  int32_t* off = n <= kBook ? off_of : scratch;
  const unsigned first = free_bits(pg.ref, pg.pages, threadIdx.x * kPer);
  for (int i = threadIdx.x; i < pg.rows; i += kBook) {
    named[i] = INT_MAX;
    parents[i] = 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kBook) {
    if ((unsigned)child[i] < (unsigned)pg.rows) atomicMin(&named[child[i]], i);
    if ((unsigned)parent[i] < (unsigned)pg.rows) atomicOr(&parents[parent[i]], 1);
  }
  __syncthreads();
  int total = 0;
  for (int base = 0; base < n; base += kBook) {
    const int i = base + threadIdx.x;
    int need = 0;
    if (i < n) {
      const int c = child[i], p = parent[i];
      bool good = (unsigned)c < (unsigned)pg.rows && (unsigned)p < (unsigned)pg.rows;
      good = good && named[c] == i && !parents[c] && pg.held[c] <= 0;
      int old = -1;
      if (good) {
        const int held = clamp_int(pg.held[p], 0, pg.width);
        const int length = max(pg.length[p], 0);
        const int full = length / pg.page_size;
        if (length % pg.page_size && full < held) {
          old = pg.table[(int64_t)p * pg.width + full];
          good = (unsigned)old < (unsigned)pg.pages;
          need = good;
          if (!good) old = -1;
        }
      }
      ok[i] = good;
      from[i] = old;
      to[i] = need ? 0 : -1;
    }
    int all;
    const int end = scan_block(need, waves, &all);
    if (i < n) off[i] = total + end - need;
    total += all;
  }
  const int found = total ? min(count_free(pg.ref, pg.pages, total, first, waves), total) : 0;
  __syncthreads();
  give_free(pg.ref, pg.pages, found, first, waves, [&](int rank, int p) {
    to[owner_of(off, n, rank)] = p;
  });
  for (int i = threadIdx.x; i < n; i += kBook)
    if (to[i] >= 0 && off[i] >= found) {  // no page left for it
      ok[i] = 0;
      to[i] = -1;
    }
}

// What a fork's copies write of its book.
struct Branches {
  vqv_pages pages;
  const int32_t* parent;
  const int32_t* child;
  const int32_t* ok;
};

// The table, held and length of branch i (new page `own`, or -1), by a
// work-group of 256. Parents are no children, so nothing read here changes.
__device__ __forceinline__ void write_branch(const Branches& f, int i, int own) {
  const vqv_pages& pg = f.pages;
  if (!f.ok[i]) return;
  const int p = f.parent[i], c = f.child[i];
  const int held = clamp_int(pg.held[p], 0, pg.width);
  const int length = max(pg.length[p], 0);
  const int full = min(length / pg.page_size, held);
  const int32_t* tp = pg.table + (int64_t)p * pg.width;
  int32_t* tc = pg.table + (int64_t)c * pg.width;
  for (int j = threadIdx.x; j < full; j += 256) {
    const int page = tp[j];
    tc[j] = page;
    if ((unsigned)page < (unsigned)pg.pages) atomicAdd(&pg.ref[page], 1);
  }
  if (threadIdx.x == 0) {
    if (own >= 0) tc[full] = own;
    pg.held[c] = full + (own >= 0);
    pg.length[c] = own >= 0 ? length : full * pg.page_size;
  }
}

// The strided places of one page's 16-byte pieces.
struct PageShape {
  int64_t layer_stride, page_stride;
  int64_t outer_stride, inner_stride;  // of the two of slots and heads
  int inner, per;                      // inner count; pieces per head and slot
  int pieces;                          // of a page
  int pages, layers;
};

typedef __attribute__((ext_vector_type(4))) unsigned u32x4;

// One work-group per kCopy pieces of a page, layer and tensor, in the order of
// their places (3000 pages of 32 KB on 4 layers: 306 us, 5.1 TB/s, and no less
// where dense pages are copied as runs of bytes). FORK: the first work-group of
// a pair writes the branch.
constexpr int kCopyPer = 4;
constexpr int kCopy = 256 * kCopyPer;

template <bool FORK>
__global__ __launch_bounds__(256) void cache_copy(uint16_t* __restrict__ k,
                                                  uint16_t* __restrict__ v, const PageShape s,
                                                  const int32_t* __restrict__ src,
                                                  const int32_t* __restrict__ dst,
                                                  const Branches f) {
  const int i = blockIdx.y;
  const int from = src[i], to = dst[i];
  if (FORK && blockIdx.x == 0 && blockIdx.z == 0) write_branch(f, i, to);
  if ((unsigned)from >= (unsigned)s.pages || (unsigned)to >= (unsigned)s.pages || from == to)
    return;
  uint16_t* base = (blockIdx.z & 1 ? v : k) + (int64_t)(blockIdx.z >> 1) * s.layer_stride;
  const uint16_t* a = base + (int64_t)from * s.page_stride;
  uint16_t* b = base + (int64_t)to * s.page_stride;
  const int p0 = blockIdx.x * kCopy + threadIdx.x;
  u32x4 r[kCopyPer];
  int64_t at[kCopyPer];
#pragma unroll
  for (int j = 0; j < kCopyPer; ++j) {
    const int p = p0 + j * 256;
    const int c = p % s.per, t = p / s.per;
    at[j] = (int64_t)(t / s.inner) * s.outer_stride + (int64_t)(t % s.inner) * s.inner_stride +
            c * 8;
    if (p < s.pieces) r[j] = *reinterpret_cast<const u32x4*>(a + at[j]);
  }
#pragma unroll
  for (int j = 0; j < kCopyPer; ++j)
    if (p0 + j * 256 < s.pieces) *reinterpret_cast<u32x4*>(b + at[j]) = r[j];
}

// One work-group per sequence and 256 of the columns (layer, tensor, head,
// 16-byte piece); each thread walks its column's kept rows upwards. The r-th
// kept row moves to place r, at or below its own, so a run of rows that is
// read before it is written never loses a later row.
constexpr int kRun = 8;

__global__ __launch_bounds__(256) void cache_compact(const vqv_cache c, const vqv_seqs s,
                                                     const int32_t* __restrict__ keep,
                                                     int32_t* __restrict__ new_len) {
  __shared__ int64_t from[256], to[256];
  __shared__ int waves[4];
  const int b = blockIdx.y;
  const int first = max(s.row_start[b], 0), next = min(s.row_start[b + 1], s.n_rows);
  const int n = max(next - first, 0);
  const int64_t p0 = (int64_t)s.kv_len[b] - n;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;

  const int per = c.dim >> 3;
  const int cols = c.layers * 2 * c.kv_heads * per;
  const int col = blockIdx.x * 256 + threadIdx.x;
  const int piece = col % per, head = col / per % c.kv_heads;
  const int plane = col / per / c.kv_heads;
  uint16_t* base = static_cast<uint16_t*>(plane & 1 ? c.v : c.k) +
                   (int64_t)(plane >> 1) * c.layer_stride + (int64_t)head * c.head_stride +
                   piece * 8;

  int done = 0;  // kept rows of earlier runs of 256
  for (int i0 = 0; i0 < n; i0 += 256) {
    const int i = i0 + threadIdx.x;
    const bool kept = i < n && keep[first + i] != 0;
    const unsigned long long m = __ballot(kept);
    __syncthreads();
    if (lane == 0) waves[wave] = __popcll(m);
    __syncthreads();
    int rank = __popcll(m & ((1ull << lane) - 1)), all = 0;
    for (int w = 0; w < 4; ++w) {
      rank += w < wave ? waves[w] : 0;
      all += waves[w];
    }
    if (kept) {
      // -1: before the first token
      const int t = (int)max(p0 + i, (int64_t)-1), d = (int)max(p0 + done + rank, (int64_t)-1);
      const int tp = page_of(s, b, t, c.page_size, c.pages);
      const int dp = page_of(s, b, d, c.page_size, c.pages);
      const bool move = t != d && tp >= 0 && dp >= 0;
      from[rank] = move ? (int64_t)tp * c.page_stride + (int64_t)(t % c.page_size) * c.slot_stride
                        : -1;
      to[rank] = move ? (int64_t)dp * c.page_stride + (int64_t)(d % c.page_size) * c.slot_stride
                      : -1;
    }
    __syncthreads();
    if (col < cols) {
      for (int r0 = 0; r0 < all; r0 += kRun) {
        u32x4 x[kRun];
#pragma unroll
        for (int j = 0; j < kRun; ++j)
          if (r0 + j < all && from[r0 + j] >= 0)
            x[j] = *reinterpret_cast<const u32x4*>(base + from[r0 + j]);
#pragma unroll
        for (int j = 0; j < kRun; ++j)
          if (r0 + j < all && from[r0 + j] >= 0)
            *reinterpret_cast<u32x4*>(base + to[r0 + j]) = x[j];
      }
    }
    done += all;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) new_len[b] = (int)max(p0 + done, (int64_t)INT_MIN);
}

template <bool FORK>
hipError_t launch_copy(const vqv_cache& c, const int32_t* src, const int32_t* dst, int n,
                       Branches f, hipStream_t stream) {
  PageShape s{};
  s.layer_stride = c.layer_stride;
  s.page_stride = c.page_stride;
  const bool slots_inner = c.slot_stride <= c.head_stride;
  s.inner = slots_inner ? c.page_size : c.kv_heads;
  s.inner_stride = slots_inner ? c.slot_stride : c.head_stride;
  s.outer_stride = slots_inner ? c.head_stride : c.slot_stride;
  const int outer = slots_inner ? c.kv_heads : c.page_size;
  s.per = c.dim >> 3;
  s.pieces = outer * s.inner * s.per;
  s.pages = c.pages;
  s.layers = c.layers;
  // The grid's y holds 65535 pairs at a time.
  for (int i = 0; i < n; i += 65535) {
    const dim3 grid((s.pieces + kCopy - 1) / kCopy, n - i < 65535 ? n - i : 65535, c.layers * 2);
    hipLaunchKernelGGL(cache_copy<FORK>, grid, dim3(256), 0, stream, static_cast<uint16_t*>(c.k),
                       static_cast<uint16_t*>(c.v), s, src + i, dst + i, f);
    if (FORK) {
      f.parent += 65535;
      f.child += 65535;
      f.ok += 65535;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_cache_copy(const vqv_cache& cache, const int32_t* src, const int32_t* dst,
                             int n, hipStream_t stream) {
  return launch_copy<false>(cache, src, dst, n, Branches{}, stream);
}

hipError_t launch_cache_trim(const vqv_pages& pages, const int32_t* keep_len, const int32_t* rows,
                             int n, hipStream_t stream) {
  hipLaunchKernelGGL(cache_trim, dim3(n), dim3(64), 0, stream, pages, keep_len, rows);
  return hipGetLastError();
}

hipError_t launch_cache_reserve(const vqv_pages& pages, const int32_t* goal_len, int n,
                                int32_t* ok, int32_t* scratch, hipStream_t stream) {
  hipLaunchKernelGGL(cache_reserve, dim3(1), dim3(kBook), 0, stream, pages, goal_len, n, ok,
                     scratch);
  return hipGetLastError();
}

hipError_t launch_cache_fork(const vqv_cache& cache, const vqv_pages& pages,
                             const int32_t* parent, const int32_t* child, int n, int32_t* ok,
                             int32_t* scratch, hipStream_t stream) {
  const int64_t r = pages.rows;
  int32_t *named = scratch, *parents = scratch + r, *off = scratch + 2 * r;
  int32_t *from = scratch + 3 * r, *to = scratch + 4 * r;
  hipLaunchKernelGGL(cache_fork_book, dim3(1), dim3(kBook), 0, stream, pages, parent, child, n,
                     ok, named, parents, off, from, to);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  return launch_copy<true>(cache, from, to, n, Branches{pages, parent, child, ok}, stream);
}

hipError_t launch_cache_compact(const vqv_cache& cache, const vqv_seqs& seqs, const int32_t* keep,
                                int32_t* new_len, hipStream_t stream) {
  const int cols = cache.layers * 2 * cache.kv_heads * (cache.dim >> 3);
  hipLaunchKernelGGL(cache_compact, dim3((cols + 255) / 256, seqs.n_seqs), dim3(256), 0, stream,
                     cache, seqs, keep, new_len);
  return hipGetLastError();
}

}  // namespace vqv
