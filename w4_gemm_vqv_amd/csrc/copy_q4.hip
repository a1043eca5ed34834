// A 4-bit cache's tokens as fp16, for calls of many query rows a sequence
// (vqv_paged_attn_q4).
//
// Attention over the records forms every key and value from its code once per
// tile of 32 (row, head) pairs. From kCopiedPairs pairs on it costs less to form
// them once, into the workspace, and let the 16-bit cache's attention read them,
// whose tiles have 256 pairs: 2048 rows over 10240 tokens, 32 heads of 128 on 8, take
// 393 to 414 us, from the records 730 (heads of 256 1245 and 1980).
// The copy has pages of the cache's size, [page][head][slot][dim], and a table of
// its own; a page that is not there is not there in the copy either. Sequences of
// fewer rows, or longer than max_kv says, are read from the records.
//
// A sequence's place in the copy is its number or, where rows leave fewer that can
// be copied, floor(first pair / kCopiedPairs): those that are copied have
// kCopiedPairs or more each, so no two get the same one. Where not all of them fit
// kMostBytes, the copy has that size, whatever else the call grows by: it holds the
// sequences of the first places that do, each up to as many pages as fit alone, and
// the others are read from the records.

#include "attn_common.h"
#include "round_common.h"
#include "serve_internal.h"

namespace vqv {
namespace {

constexpr int kTokens = 16;              // of a work-group
constexpr size_t kMostBytes = 1u << 30;  // of a copy

// Scores (rows * heads * tokens of the longest sequence) from which the copy pays
// for itself and two more launches, with 32 heads of 128 on 8: at 2^27 117 us become
// 85 (2048 rows of as many tokens), 177 140 (512 of 8192), 230 168 (128 of 32768) and
// 165 163 (1024 of 4096); at 2^26 84 would become 123 (1024 of 2048), 97 97 (512 of
// 4096), but 125 101 (128 of 16384).
constexpr double kLeastScores = 1 << 27;

struct CopyArgs {
  const char* k;  // of the layer
  const char* v;
  int64_t page_stride, slot_stride, head_stride;
  int pages, page_size, kv_heads, group;
  vqv_seqs seqs;
  Copied copied;
  int width, chunks;
  uint16_t* kc;
  uint16_t* vc;
  int32_t* table;
};

constexpr int threads(int dim) { return (kTokens * dim / 8 + 63) / 64 * 64; }  // whole waves

// One thread per 8 values of a token's key and value head, a work-group per head:
// 10240 tokens of 8 heads of 128 in 12 to 14 us, 55 MB at 4.2 TB/s (with two heads to
// a work-group it took 14.5 where this took 12.5, with all eight 21).
template <int D>
__global__ __launch_bounds__(threads(D)) void copy_q4(const CopyArgs a) {
  constexpr int PER = D / 8;
  typedef __attribute__((ext_vector_type(2))) _Float16 h2;
  const int part = blockIdx.x / a.kv_heads, h = blockIdx.x % a.kv_heads;
  const int slot = part / a.chunks;
  int b = slot;
  if (!a.copied.by_number) {
    // A copied sequence whose first pair is in the slot's range has the range's
    // last row too.
    const int row = ((slot + 1) * kCopiedPairs + a.group - 1) / a.group - 1;
    b = seq_of_row(a.seqs.row_start, a.seqs.n_seqs, row);
    if (b >= a.seqs.n_seqs || max(a.seqs.row_start[b], 0) * a.group / kCopiedPairs != slot) return;
  }
  if (!is_copied(a.seqs, b, a.group, a.copied)) return;

  const int t = part % a.chunks * kTokens + threadIdx.x / PER, piece = threadIdx.x % PER;
  const int i = t / a.page_size, s = t % a.page_size;
  if (threadIdx.x >= kTokens * PER || i >= a.width) return;
  const int entry = a.seqs.table[b * a.seqs.table_stride + i];
  const bool there = entry >= 0 && entry < a.pages;
  if (s == 0 && piece == 0 && h == 0)
    a.table[(int64_t)b * a.width + i] = there ? slot * a.width + i : -1;
  if (!there || t >= a.seqs.kv_len[b]) return;

  const int64_t from = entry * a.page_stride + s * a.slot_stride + h * a.head_stride;
  const int64_t to =
      (((int64_t)(slot * a.width + i) * a.kv_heads + h) * a.page_size + s) * D + 8 * piece;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const char* rec = (x == 0 ? a.k : a.v) + from;
    const unsigned codes = *reinterpret_cast<const unsigned*>(rec + 4 * piece);
    const h2 sb = *reinterpret_cast<const h2*>(rec + D / 2 + piece / 4 * 4);
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] =
          pack2<_Float16>(fmaf((float)(codes >> (4 * e) & 15u), (float)sb[0], (float)sb[1]),
                          fmaf((float)(codes >> (16 + 4 * e) & 15u), (float)sb[0], (float)sb[1]));
    *reinterpret_cast<u32x4*>((x == 0 ? a.kc : a.vc) + to) = w;
  }
}

template <int D>
hipError_t launch_dim(const CopyArgs& a, int slots, hipStream_t stream) {
  hipLaunchKernelGGL((copy_q4<D>), dim3((unsigned)(slots * a.chunks * a.kv_heads)), dim3(threads(D)), 0,
                     stream, a);
  return hipGetLastError();
}

}  // namespace

CopyPlan copy_plan(const vqv_cache_q4& c, const vqv_seqs& s, int heads, int window) {
  CopyPlan p = {};
  const int group = heads / c.kv_heads;
  const int rows = s.max_rows < s.n_rows ? s.max_rows : s.n_rows;
  if (window > 0 || (int64_t)rows * group < kCopiedPairs) return p;
  if ((double)rows * heads * s.max_kv < kLeastScores || s.table_width < 1) return p;
  const int64_t most = (int64_t)s.n_rows * group / kCopiedPairs;
  int64_t slots = most < s.n_seqs ? most : s.n_seqs;
  p.copied.by_number = slots == s.n_seqs;
  int64_t width = ((int64_t)s.max_kv + c.page_size - 1) / c.page_size;
  if (width > s.table_width) width = s.table_width;
  // Of a page's keys (values), and of an entry of each sequence's table.
  const double page = (double)c.page_size * c.kv_heads * c.dim * 2, entries = 4.0 * s.n_seqs;
  const bool all = (2 * slots * page + entries) * width + 16 <= (double)kMostBytes;
  if (!all) {
    const int64_t fit = (int64_t)((kMostBytes - 16) / (2 * page + entries));
    if (fit < 1) return p;
    if (width > fit) width = fit;
    const int64_t held = (int64_t)((kMostBytes - 16 - entries * width) / (2 * page * width));
    if (slots > held) slots = held;
  }
  const int64_t tokens = width * c.page_size;
  p.copied.len = tokens < s.max_kv && width < s.table_width ? (int)tokens : s.max_kv;
  p.copied.slots = (int)slots;
  p.width = (int)width;
  p.values = (size_t)(slots * width) * (size_t)page;
  p.bytes = all ? (2 * p.values + (size_t)(entries * width) + 15) / 16 * 16 : kMostBytes;
  p.attn = attn_plan(copy_cache(c, p, nullptr), copy_seqs(s, p, nullptr), heads, 0, 0);
  if ((int64_t)c.kv_heads * s.n_seqs * p.attn.groups * p.attn.splits >= (1ll << 23) ||
      (p.attn.splits > 1 && (int64_t)s.n_rows * heads >= (1ll << 24)))
    return CopyPlan{};
  return p;
}

vqv_cache copy_cache(const vqv_cache_q4& c, const CopyPlan& p, void* workspace) {
  vqv_cache r = {};
  r.k = workspace;
  r.v = static_cast<char*>(workspace) + p.values;
  r.dtype = VQV_FP16;
  r.layers = 1;
  r.pages = p.copied.slots * p.width;
  r.page_size = c.page_size;
  r.kv_heads = c.kv_heads;
  r.dim = c.dim;
  r.slot_stride = c.dim;
  r.head_stride = (int64_t)c.page_size * c.dim;
  r.page_stride = c.kv_heads * r.head_stride;
  r.layer_stride = r.pages * r.page_stride;
  return r;
}

vqv_seqs copy_seqs(const vqv_seqs& s, const CopyPlan& p, void* workspace) {
  vqv_seqs r = s;
  r.table = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + 2 * p.values);
  r.table_stride = p.width;
  r.table_width = p.width;
  return r;
}

hipError_t launch_copy_q4(const vqv_cache_q4& c, int layer, const vqv_seqs& s, int heads,
                          const CopyPlan& p, void* workspace, hipStream_t stream) {
  const int64_t tokens = (int64_t)p.width * c.page_size;
  const CopyArgs a{static_cast<const char*>(c.k) + layer * c.layer_stride,
                   static_cast<const char*>(c.v) + layer * c.layer_stride,
                   c.page_stride,
                   c.slot_stride,
                   c.head_stride,
                   c.pages,
                   c.page_size,
                   c.kv_heads,
                   heads / c.kv_heads,
                   s,
                   p.copied,
                   p.width,
                   ceil_div(tokens < p.copied.len ? tokens : p.copied.len, kTokens),
                   static_cast<uint16_t*>(workspace),
                   reinterpret_cast<uint16_t*>(static_cast<char*>(workspace) + p.values),
                   reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + 2 * p.values)};
  switch (c.dim) {
    case 64: return launch_dim<64>(a, p.copied.slots, stream);
    case 80: return launch_dim<80>(a, p.copied.slots, stream);
    case 96: return launch_dim<96>(a, p.copied.slots, stream);
    case 128: return launch_dim<128>(a, p.copied.slots, stream);
    case 192: return launch_dim<192>(a, p.copied.slots, stream);
    default: return launch_dim<256>(a, p.copied.slots, stream);
  }
}

}  // namespace vqv
