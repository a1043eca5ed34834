// Entry points of include/vqv_round.h: argument checks on the host, then the
// launches on the caller's stream.

#include <math.h>
#include <stdint.h>

#include "round_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Whether every non-NULL pointer of the list can hold int32 or fp32 values.
template <typename... P>
bool words_aligned(const P*... p) {
  return (... && aligned(p, 4));
}

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a && b && na && nb && a0 < b0 + nb && b0 < a0 + na;
}

vqv_status check_cache(const vqv_cache* c) {
  if (!c || !c->k || !c->v) return VQV_ERR_ARG;
  if (c->layers < 1 || c->pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->dim < 1)
    return VQV_ERR_ARG;
  if (c->layer_stride < 0 || c->page_stride < 0 || c->slot_stride < 0 || c->head_stride < 0)
    return VQV_ERR_ARG;
  if (c->dtype == VQV_FP32) return VQV_ERR_UNSUPPORTED;
  if (c->dtype != VQV_BF16 && c->dtype != VQV_FP16) return VQV_ERR_ARG;
  if (c->dim % 8 || c->dim > 256 || c->kv_heads > 65535 || c->layers > 32767)
    return VQV_ERR_UNSUPPORTED;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->layer_stride % 8 || c->page_stride % 8 ||
      c->slot_stride % 8 || c->head_stride % 8)
    return VQV_ERR_ALIGN;
  // Places in a layer are counted in 32-bit units of 8 values.
  const double units = ((double)(c->pages - 1) * c->page_stride +
                        (double)(c->page_size - 1) * c->slot_stride +
                        (double)(c->kv_heads - 1) * c->head_stride + c->dim) / 8;
  if (units >= 4294967296.0) return VQV_ERR_UNSUPPORTED;
  if ((int64_t)c->page_size * c->kv_heads * (c->dim / 8) >= (1ll << 31) ||
      (int64_t)c->layers * 2 * c->kv_heads * (c->dim / 8) >= (1ll << 31))
    return VQV_ERR_UNSUPPORTED;
  return VQV_OK;
}

vqv_status check_seqs(const vqv_seqs* s) {
  if (!s || !s->row_start || !s->kv_len || !s->table) return VQV_ERR_ARG;
  if (s->n_seqs < 1 || s->table_width < 1 || s->n_rows < 0 || s->max_rows < 0 || s->max_kv < 0 ||
      s->table_stride < s->table_width)
    return VQV_ERR_ARG;
  if (s->n_seqs > 65535) return VQV_ERR_UNSUPPORTED;
  if (!words_aligned(s->row_start, s->kv_len, s->table)) return VQV_ERR_ALIGN;
  return VQV_OK;
}

vqv_status check_pages(const vqv_pages* p) {
  if (!p || !p->ref || !p->table || !p->held || !p->length) return VQV_ERR_ARG;
  if (p->pages < 1 || p->rows < 1 || p->width < 1 || p->page_size < 1) return VQV_ERR_ARG;
  if ((int64_t)p->rows * p->width >= (1ll << 31) || p->pages > (1 << 30))
    return VQV_ERR_UNSUPPORTED;
  if (!words_aligned(p->ref, p->table, p->held, p->length)) return VQV_ERR_ALIGN;
  return VQV_OK;
}

vqv_status check_edits(const vqv_edits* e, int T) {
  if (!e || e->n_seqs < 1 || e->n < 1 || T < 1 || T > 64 || e->n_bias < 0) return VQV_ERR_ARG;
  if ((double)e->n_seqs * T * e->n >= 2147483648.0) return VQV_ERR_ARG;
  if (e->bias_start && e->n_bias && (!e->bias_token || !e->bias_value)) return VQV_ERR_ARG;
  // The last tile's tokens are counted in 32 bits.
  if (e->n_seqs > 65535 || e->n > INT32_MAX - (vqv::kVerifyChunk - 1)) return VQV_ERR_UNSUPPORTED;
  if (!words_aligned(e->counts, e->seen, e->repetition, e->frequency, e->presence, e->bias_start,
                     e->bias_token, e->bias_value))
    return VQV_ERR_ALIGN;
  return VQV_OK;
}

// The inputs of an edit, for overlap checks.
struct Span {
  const void* p;
  size_t n;
};
struct EditSpans {
  Span in[10];
};

EditSpans edit_spans(const vqv_edits& e, const int32_t* draft, int T, const int32_t* mask) {
  const size_t b = e.n_seqs, n = e.n, words = (n + 31) / 32;
  return EditSpans{{{e.counts, b * n * 4},
                    {e.seen, b * words * 4},
                    {e.repetition, b * 4},
                    {e.frequency, b * 4},
                    {e.presence, b * 4},
                    {e.bias_start, (b + 1) * 4},
                    {e.bias_token, (size_t)e.n_bias * 4},
                    {e.bias_value, (size_t)e.n_bias * 4},
                    {draft, b * (T - 1) * 4},
                    {mask, b * T * words * 4}}};
}

bool any_overlap(const void* p, size_t n, const EditSpans& s) {
  for (const Span& x : s.in)
    if (overlaps(p, n, x.p, x.n)) return true;
  return false;
}

vqv_status status_of(hipError_t e) { return e == hipSuccess ? VQV_OK : VQV_ERR_HIP; }

}  // namespace

extern "C" {

vqv_status vqv_rope_plan(vqv_rope* plan, int rot, double base, int interleaved, int scaling,
                         double factor, int original_len) {
  if (!plan || rot < 2 || rot % 2 || !(base > 0.0) || !isfinite(base)) return VQV_ERR_ARG;
  if (rot > 256) return VQV_ERR_UNSUPPORTED;
  if (scaling < VQV_ROPE_NONE || scaling > VQV_ROPE_SMOOTH) return VQV_ERR_ARG;
  if (scaling != VQV_ROPE_NONE && (!(factor > 0.0) || !isfinite(factor))) return VQV_ERR_ARG;
  if ((scaling == VQV_ROPE_YARN || scaling == VQV_ROPE_SMOOTH) && original_len < 1)
    return VQV_ERR_ARG;
  if (scaling == VQV_ROPE_YARN && !(base > 1.0)) return VQV_ERR_ARG;
  const double tau = 6.283185307179586476925287;
  plan->rot = rot;
  plan->interleaved = interleaved != 0;
  plan->mscale = 1.0f;
  plan->reserved = 0;
  double b = base;
  if (scaling == VQV_ROPE_NTK && rot > 2) b *= pow(factor, (double)rot / (rot - 2));
  double lo = 0.0, hi = 0.0;
  if (scaling == VQV_ROPE_YARN) {
    // The pair that makes `turns` turns in original_len positions.
    const auto pair = [&](double turns) {
      return rot * log(original_len / (turns * tau)) / (2.0 * log(base));
    };
    lo = fmax(floor(pair(32.0)), 0.0);
    hi = fmin(ceil(pair(1.0)), rot - 1.0);
    if (factor > 1.0) plan->mscale = (float)(0.1 * log(factor) + 1.0);
  }
  for (int i = 0; i < 128; ++i) plan->turns[i] = 0.0;
  for (int i = 0; i < rot / 2; ++i) {
    double f = pow(b, -2.0 * i / rot);
    double part = 0.0;  // of f / factor
    if (scaling == VQV_ROPE_LINEAR) part = 1.0;
    if (scaling == VQV_ROPE_YARN) part = fmin(fmax((i - lo) / fmax(hi - lo, 0.001), 0.0), 1.0);
    if (scaling == VQV_ROPE_SMOOTH)
      part = 1.0 - fmin(fmax((original_len * f / tau - 1.0) / 3.0, 0.0), 1.0);
    if (part > 0.0) f = f / factor * part + f * (1.0 - part);
    plan->turns[i] = f / tau;
  }
  return VQV_OK;
}

vqv_status vqv_rope_append(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                           const void* k, int64_t k_row_stride, int64_t k_head_stride,
                           const void* v, int64_t v_row_stride, int64_t v_head_stride,
                           vqv_dtype in_dtype, int heads, const vqv_cache* cache, int layer,
                           const vqv_seqs* seqs, const vqv_rope* rope, void* q_out,
                           void* hip_stream) {
  vqv_status st = check_cache(cache);
  if (st != VQV_OK) return st;
  if ((st = check_seqs(seqs)) != VQV_OK) return st;
  // The rows of an empty call may have no memory at all.
  if (!rope || (seqs->n_rows && (!q || !k || !v || !q_out))) return VQV_ERR_ARG;
  if (in_dtype != VQV_BF16 && in_dtype != VQV_FP16 && in_dtype != VQV_FP32) return VQV_ERR_ARG;
  if (heads < 1 || layer < 0 || layer >= cache->layers) return VQV_ERR_ARG;
  if (rope->rot < 2 || rope->rot % 2 || rope->rot > 256 || rope->rot > cache->dim)
    return VQV_ERR_ARG;
  const int esz = in_dtype == VQV_FP32 ? 4 : 2;
  const int64_t strides[6] = {q_row_stride, q_head_stride, k_row_stride,
                              k_head_stride, v_row_stride, v_head_stride};
  for (const int64_t x : strides) {
    if (x < 0) return VQV_ERR_ARG;
    if (x * esz % 16) return VQV_ERR_ALIGN;
  }
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16))
    return VQV_ERR_ALIGN;
  if (heads > 65535 || (int64_t)heads * cache->dim >= (1ll << 31) || seqs->n_rows >= (1 << 23))
    return VQV_ERR_UNSUPPORTED;
  if (seqs->n_rows == 0) return VQV_OK;
  const auto span = [&](int64_t rs, int64_t hs, int h) {
    return (size_t)((seqs->n_rows - 1) * rs + (h - 1) * hs + cache->dim) * esz;
  };
  const size_t out = (size_t)seqs->n_rows * heads * cache->dim * 2;
  if (overlaps(q_out, out, q, span(q_row_stride, q_head_stride, heads)) ||
      overlaps(q_out, out, k, span(k_row_stride, k_head_stride, cache->kv_heads)) ||
      overlaps(q_out, out, v, span(v_row_stride, v_head_stride, cache->kv_heads)))
    return VQV_ERR_ARG;
  (void)hipGetLastError();
  return status_of(vqv::launch_rope_append(
      {q, q_row_stride, q_head_stride}, {k, k_row_stride, k_head_stride},
      {v, v_row_stride, v_head_stride}, (int)in_dtype, heads, *cache, layer, *seqs, *rope, q_out,
      static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"

namespace {

// What vqv_paged_attn checks of its sizes, and the plan.
vqv_status plan_attn(const vqv_cache* cache, const vqv_seqs* seqs, int heads, int window,
                     int sinks, vqv::AttnPlan* plan) {
  vqv_status st = check_cache(cache);
  if (st != VQV_OK) return st;
  if ((st = check_seqs(seqs)) != VQV_OK) return st;
  if (heads < 1 || heads % cache->kv_heads || window < 0 || sinks < 0) return VQV_ERR_ARG;
  if (!vqv::attn_dim_supported(cache->dim) || heads / cache->kv_heads > 1024)
    return VQV_ERR_UNSUPPORTED;
  if ((int64_t)seqs->max_rows * heads >= (1ll << 30) ||
      (int64_t)seqs->n_rows * heads >= (1ll << 30))
    return VQV_ERR_UNSUPPORTED;
  *plan = vqv::attn_plan(*cache, *seqs, heads, window, sinks);
  if ((int64_t)cache->kv_heads * seqs->n_seqs * plan->groups * plan->splits >= (1ll << 23))
    return VQV_ERR_UNSUPPORTED;  // threads of a grid are counted in 32 bits
  if (plan->splits > 1 && (int64_t)seqs->n_rows * heads >= (1ll << 24)) return VQV_ERR_UNSUPPORTED;
  return VQV_OK;
}

}  // namespace

extern "C" {

size_t vqv_paged_attn_workspace_bytes(const vqv_cache* cache, const vqv_seqs* seqs, int heads,
                                      int window, int sinks) {
  vqv::AttnPlan plan;
  if (plan_attn(cache, seqs, heads, window, sinks, &plan) != VQV_OK) return 0;
  return vqv::attn_partial_bytes(*cache, *seqs, heads, plan);
}

vqv_status vqv_paged_attn(const void* q, const vqv_cache* cache, int layer, const vqv_seqs* seqs,
                          int heads, float scale, int window, int sinks, void* out,
                          void* workspace, size_t workspace_bytes, void* hip_stream) {
  vqv::AttnPlan plan;
  const vqv_status st = plan_attn(cache, seqs, heads, window, sinks, &plan);
  if (st != VQV_OK) return st;
  if ((seqs->n_rows && (!q || !out)) || layer < 0 || layer >= cache->layers) return VQV_ERR_ARG;
  if (!(scale > 0.0f) || !isfinite(scale)) return VQV_ERR_ARG;
  if (!aligned(q, 16) || !aligned(out, 16)) return VQV_ERR_ALIGN;
  const size_t bytes = (size_t)seqs->n_rows * heads * cache->dim * 2;
  const size_t need = vqv::attn_partial_bytes(*cache, *seqs, heads, plan);
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
    return VQV_ERR_WORKSPACE;
  if (overlaps(out, bytes, q, bytes) || overlaps(workspace, need, q, bytes) ||
      overlaps(workspace, need, out, bytes))
    return VQV_ERR_ARG;
  if (seqs->n_rows == 0 || seqs->max_rows == 0) return VQV_OK;
  (void)hipGetLastError();
  return status_of(vqv::launch_paged_attn(q, *cache, layer, *seqs, heads, scale, window, sinks,
                                          out, workspace, plan,
                                          static_cast<hipStream_t>(hip_stream)));
}

size_t vqv_cache_workspace_bytes(const vqv_pages* pages) {
  if (check_pages(pages) != VQV_OK) return 0;
  return (size_t)pages->rows * vqv::kCacheScratchPerRow * sizeof(int32_t);
}

vqv_status vqv_cache_copy(const vqv_cache* cache, const int32_t* src, const int32_t* dst, int n,
                          void* hip_stream) {
  const vqv_status st = check_cache(cache);
  if (st != VQV_OK) return st;
  if (n < 0 || (n && (!src || !dst))) return VQV_ERR_ARG;
  if (!words_aligned(src, dst)) return VQV_ERR_ALIGN;
  if (n == 0) return VQV_OK;
  (void)hipGetLastError();
  return status_of(
      vqv::launch_cache_copy(*cache, src, dst, n, static_cast<hipStream_t>(hip_stream)));
}

vqv_status vqv_cache_trim(const vqv_pages* pages, const int32_t* keep_len, const int32_t* rows,
                          int n, void* hip_stream) {
  const vqv_status st = check_pages(pages);
  if (st != VQV_OK) return st;
  if (n < 0 || (n && !keep_len) || (!rows && n > pages->rows)) return VQV_ERR_ARG;
  if (!words_aligned(keep_len, rows)) return VQV_ERR_ALIGN;
  if (n > (1 << 24)) return VQV_ERR_UNSUPPORTED;
  if (n == 0) return VQV_OK;
  (void)hipGetLastError();
  return status_of(
      vqv::launch_cache_trim(*pages, keep_len, rows, n, static_cast<hipStream_t>(hip_stream)));
}

vqv_status vqv_cache_reserve(const vqv_pages* pages, const int32_t* goal_len, int n, int32_t* ok,
                             void* workspace, size_t workspace_bytes, void* hip_stream) {
  const vqv_status st = check_pages(pages);
  if (st != VQV_OK) return st;
  if (n < 0 || n > pages->rows || (n && (!goal_len || !ok))) return VQV_ERR_ARG;
  if (!words_aligned(goal_len, ok)) return VQV_ERR_ALIGN;
  const size_t need = vqv_cache_workspace_bytes(pages);
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return VQV_ERR_WORKSPACE;
  if (overlaps(ok, (size_t)n * 4, goal_len, (size_t)n * 4) ||
      overlaps(workspace, need, goal_len, (size_t)n * 4) ||
      overlaps(workspace, need, ok, (size_t)n * 4))
    return VQV_ERR_ARG;
  if (n == 0) return VQV_OK;
  (void)hipGetLastError();
  return status_of(vqv::launch_cache_reserve(*pages, goal_len, n, ok,
                                             static_cast<int32_t*>(workspace),
                                             static_cast<hipStream_t>(hip_stream)));
}

vqv_status vqv_cache_fork(const vqv_cache* cache, const vqv_pages* pages, const int32_t* parent,
                          const int32_t* child, int n, int32_t* ok, void* workspace,
                          size_t workspace_bytes, void* hip_stream) {
  vqv_status st = check_cache(cache);
  if (st != VQV_OK) return st;
  if ((st = check_pages(pages)) != VQV_OK) return st;
  if (pages->pages != cache->pages || pages->page_size != cache->page_size) return VQV_ERR_ARG;
  if (n < 0 || n > pages->rows || (n && (!parent || !child || !ok))) return VQV_ERR_ARG;
  if (!words_aligned(parent, child, ok)) return VQV_ERR_ALIGN;
  const size_t need = vqv_cache_workspace_bytes(pages), list = (size_t)n * 4;
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return VQV_ERR_WORKSPACE;
  if (overlaps(ok, list, parent, list) || overlaps(ok, list, child, list) ||
      overlaps(workspace, need, parent, list) || overlaps(workspace, need, child, list) ||
      overlaps(workspace, need, ok, list))
    return VQV_ERR_ARG;
  if (n == 0) return VQV_OK;
  (void)hipGetLastError();
  return status_of(vqv::launch_cache_fork(*cache, *pages, parent, child, n, ok,
                                          static_cast<int32_t*>(workspace),
                                          static_cast<hipStream_t>(hip_stream)));
}

vqv_status vqv_cache_compact(const vqv_cache* cache, const vqv_seqs* seqs, const int32_t* keep,
                             int32_t* new_len, void* hip_stream) {
  vqv_status st = check_cache(cache);
  if (st != VQV_OK) return st;
  if ((st = check_seqs(seqs)) != VQV_OK) return st;
  if (!new_len || (seqs->n_rows && !keep)) return VQV_ERR_ARG;
  if (!words_aligned(keep, new_len)) return VQV_ERR_ALIGN;
  const size_t nb = (size_t)seqs->n_seqs * 4;
  if (overlaps(new_len, nb, keep, (size_t)seqs->n_rows * 4) ||
      overlaps(new_len, nb, seqs->kv_len, nb) || overlaps(new_len, nb, seqs->row_start, nb + 4))
    return VQV_ERR_ARG;
  (void)hipGetLastError();
  return status_of(vqv::launch_cache_compact(*cache, *seqs, keep, new_len,
                                             static_cast<hipStream_t>(hip_stream)));
}

vqv_status vqv_logits_edit(const float* logits, const vqv_edits* edits, const int32_t* draft,
                           int T, const int32_t* mask, float* out, void* hip_stream) {
  const vqv_status st = check_edits(edits, T);
  if (st != VQV_OK) return st;
  if (!logits || !out) return VQV_ERR_ARG;
  if (!aligned(logits, 16) || !aligned(out, 16) || !words_aligned(draft, mask))
    return VQV_ERR_ALIGN;
  const size_t bytes = (size_t)edits->n_seqs * T * edits->n * 4;
  if (out != logits && overlaps(out, bytes, logits, bytes)) return VQV_ERR_ARG;
  if (any_overlap(out, bytes, edit_spans(*edits, draft, T, mask))) return VQV_ERR_ARG;
  (void)hipGetLastError();
  return status_of(vqv::launch_logits_edit(logits, *edits, draft, T, mask, out,
                                           static_cast<hipStream_t>(hip_stream)));
}

vqv_status vqv_logits_verify(const float* logits, const vqv_edits* edits, const int32_t* draft,
                             const int32_t* draft_len, int T, const int32_t* mask,
                             int32_t* argmax, int32_t* accept_len, float* margin,
                             void* workspace, size_t workspace_bytes, void* hip_stream) {
  const vqv_status st = check_edits(edits, T);
  if (st != VQV_OK) return st;
  if (!logits || !argmax || !accept_len || (T > 1 && !draft)) return VQV_ERR_ARG;
  if (!aligned(logits, 16) ||
      !words_aligned(draft, draft_len, mask, argmax, accept_len) || !aligned(margin, 4))
    return VQV_ERR_ALIGN;
  const int B = edits->n_seqs;
  const size_t need = vqv_verify_workspace_bytes(B, T, edits->n), rows = (size_t)B * T;
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return VQV_ERR_WORKSPACE;
  const EditSpans in = edit_spans(*edits, draft, T, mask);
  const Span outs[4] = {{argmax, rows * 4}, {accept_len, (size_t)B * 4}, {margin, rows * 4},
                        {workspace, need}};
  for (int o = 0; o < 4; ++o) {
    if (any_overlap(outs[o].p, outs[o].n, in) ||
        overlaps(outs[o].p, outs[o].n, logits, rows * edits->n * 4) ||
        overlaps(outs[o].p, outs[o].n, draft_len, (size_t)B * 4))
      return VQV_ERR_ARG;
    for (int o2 = o + 1; o2 < 4; ++o2)
      if (overlaps(outs[o].p, outs[o].n, outs[o2].p, outs[o2].n)) return VQV_ERR_ARG;
  }
  (void)hipGetLastError();
  const vqv::VerifyArgs va{draft, draft_len, B, T, argmax, accept_len, margin,
                           static_cast<uint4*>(workspace), 0};
  return status_of(vqv::launch_logits_verify(logits, *edits, mask, va,
                                             static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
