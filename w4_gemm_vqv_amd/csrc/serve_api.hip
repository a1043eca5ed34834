// Entry points of include/vqv_serve.h: argument checks on the host, then the
// launches on the caller's stream.

#include "api_checks.h"
#include "serve_internal.h"

namespace {

vqv_status check_cache_q4(const vqv_cache_q4* c) {
  if (!c || !c->k || !c->v) return VQV_ERR_ARG;
  if (c->layers < 1 || c->pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->dim < 1)
    return VQV_ERR_ARG;
  if (c->layer_stride < 0 || c->page_stride < 0 || c->slot_stride < 0 || c->head_stride < 0)
    return VQV_ERR_ARG;
  if (!vqv::attn_dim_supported(c->dim) || c->kv_heads > 65535 || c->layers > 32767)
    return VQV_ERR_UNSUPPORTED;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->layer_stride % 16 || c->page_stride % 16 ||
      c->slot_stride % 16 || c->head_stride % 16)
    return VQV_ERR_ALIGN;
  // Places in a layer are counted in 32-bit units of 16 bytes.
  const double units = ((double)(c->pages - 1) * c->page_stride +
                        (double)(c->page_size - 1) * c->slot_stride +
                        (double)(c->kv_heads - 1) * c->head_stride +
                        vqv::q4_record_bytes(c->dim)) / 16;
  if (units >= 4294967296.0) return VQV_ERR_UNSUPPORTED;
  return VQV_OK;
}

// Bytes of a layer's keys or values.
size_t layer_span(const vqv_cache_q4& c) {
  return (size_t)(c.pages - 1) * c.page_stride + (size_t)(c.page_size - 1) * c.slot_stride +
         (size_t)(c.kv_heads - 1) * c.head_stride + vqv::q4_record_bytes(c.dim);
}

bool half_type(int t) { return t == VQV_BF16 || t == VQV_FP16; }

}  // namespace

extern "C" {

size_t vqv_q4_record_bytes(int dim) {
  return vqv::attn_dim_supported(dim) ? (size_t)vqv::q4_record_bytes(dim) : 0;
}

vqv_status vqv_rope_append_q4(const void* q, int64_t q_row_stride, int64_t q_head_stride,
                              const void* k, int64_t k_row_stride, int64_t k_head_stride,
                              const void* v, int64_t v_row_stride, int64_t v_head_stride,
                              vqv_dtype in_dtype, int heads, const vqv_cache_q4* cache, int layer,
                              const vqv_seqs* seqs, const vqv_rope* rope, void* q_out,
                              vqv_dtype q_dtype, void* hip_stream) {
  vqv_status st = check_cache_q4(cache);
  if (st != VQV_OK) return st;
  if ((st = check_seqs(seqs)) != VQV_OK) return st;
  // The rows of an empty call may have no memory at all.
  if (!rope || (seqs->n_rows && (!q || !k || !v || !q_out))) return VQV_ERR_ARG;
  if (!half_type(in_dtype) && in_dtype != VQV_FP32) return VQV_ERR_ARG;
  if (q_dtype == VQV_FP32) return VQV_ERR_UNSUPPORTED;
  if (!half_type(q_dtype)) return VQV_ERR_ARG;
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
  if (heads > 65535 || (int64_t)heads * cache->dim >= (1ll << 31) ||
      (int64_t)cache->kv_heads * cache->dim >= (1ll << 29) || seqs->n_rows >= (1 << 23))
    return VQV_ERR_UNSUPPORTED;
  if (seqs->n_rows == 0) return VQV_OK;
  const auto span = [&](int64_t rs, int64_t hs, int h) {
    return rows_span(seqs->n_rows, rs, hs, h, cache->dim, esz);
  };
  const size_t out = (size_t)seqs->n_rows * heads * cache->dim * 2;
  if (overlaps(q_out, out, q, span(q_row_stride, q_head_stride, heads)) ||
      overlaps(q_out, out, k, span(k_row_stride, k_head_stride, cache->kv_heads)) ||
      overlaps(q_out, out, v, span(v_row_stride, v_head_stride, cache->kv_heads)))
    return VQV_ERR_ARG;
  (void)hipGetLastError();
  return status_of(vqv::launch_rope_append_q4(
      {q, q_row_stride, q_head_stride}, {k, k_row_stride, k_head_stride},
      {v, v_row_stride, v_head_stride}, (int)in_dtype, heads, *cache, layer, *seqs, *rope, q_out,
      (int)q_dtype, static_cast<hipStream_t>(hip_stream)));
}

vqv_status vqv_cache_q4_read(const vqv_cache_q4* cache, int layer, const vqv_seqs* seqs,
                             void* k_out, void* v_out, vqv_dtype out_dtype, void* hip_stream) {
  vqv_status st = check_cache_q4(cache);
  if (st != VQV_OK) return st;
  if ((st = check_seqs(seqs)) != VQV_OK) return st;
  if (layer < 0 || layer >= cache->layers) return VQV_ERR_ARG;
  if (!half_type(out_dtype) && out_dtype != VQV_FP32) return VQV_ERR_ARG;
  if (!aligned(k_out, 16) || !aligned(v_out, 16)) return VQV_ERR_ALIGN;
  if (seqs->n_rows >= (1 << 23) || (int64_t)cache->kv_heads * cache->dim >= (1ll << 29))
    return VQV_ERR_UNSUPPORTED;
  const size_t bytes = (size_t)seqs->n_rows * cache->kv_heads * cache->dim *
                       (out_dtype == VQV_FP32 ? 4 : 2);
  const size_t held = layer_span(*cache);
  const char* k = static_cast<const char*>(cache->k) + layer * cache->layer_stride;
  const char* v = static_cast<const char*>(cache->v) + layer * cache->layer_stride;
  for (const void* o : {k_out, v_out})
    if (overlaps(o, bytes, k, held) || overlaps(o, bytes, v, held)) return VQV_ERR_ARG;
  if (overlaps(k_out, bytes, v_out, bytes)) return VQV_ERR_ARG;
  if (seqs->n_rows == 0 || (!k_out && !v_out)) return VQV_OK;
  (void)hipGetLastError();
  return status_of(vqv::launch_cache_q4_read(*cache, layer, *seqs, k_out, v_out, (int)out_dtype,
                                             static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"

namespace {

// What vqv_paged_attn_q4 checks of its sizes, and the plan.
vqv_status plan_attn_q4(const vqv_cache_q4* cache, const vqv_seqs* seqs, int heads, int window,
                        int sinks, vqv_dtype dtype, vqv::AttnPlan* plan, vqv::CopyPlan* copy) {
  vqv_status st = check_cache_q4(cache);
  if (st != VQV_OK) return st;
  if ((st = check_seqs(seqs)) != VQV_OK) return st;
  if (heads < 1 || heads % cache->kv_heads || window < 0 || sinks < 0) return VQV_ERR_ARG;
  if (heads / cache->kv_heads > 1024) return VQV_ERR_UNSUPPORTED;
  if ((int64_t)seqs->max_rows * heads >= (1ll << 30) ||
      (int64_t)seqs->n_rows * heads >= (1ll << 30))
    return VQV_ERR_UNSUPPORTED;
  *plan = vqv::attn_q4_plan(*cache, *seqs, heads, window, sinks);
  if ((int64_t)cache->kv_heads * seqs->n_seqs * plan->groups * plan->splits >= (1ll << 23))
    return VQV_ERR_UNSUPPORTED;  // threads of a grid are counted in 32 bits
  if (plan->splits > 1 && (int64_t)seqs->n_rows * heads >= (1ll << 24)) return VQV_ERR_UNSUPPORTED;
  // fp16 keys as one value each would be the larger part of fp16 outputs' error.
  *copy = dtype == VQV_BF16 ? vqv::copy_plan(*cache, *seqs, heads, window) : vqv::CopyPlan{};
  return VQV_OK;
}

// Of the partial sums over the records, and, where tokens are copied, of the copy
// and the sums over it (at the workspace's start, in turn).
size_t attn_q4_bytes(const vqv_cache_q4& cache, const vqv_seqs& seqs, int heads,
                     const vqv::AttnPlan& plan, const vqv::CopyPlan& copy) {
  size_t part = vqv::attn_partial_bytes(cache.dim, seqs, heads, plan);
  if (copy.copied.slots == 0) return part;
  const size_t wide = vqv::attn_partial_bytes(cache.dim, seqs, heads, copy.attn);
  if (wide > part) part = wide;
  return (part + 15) / 16 * 16 + copy.bytes;
}

}  // namespace

extern "C" {

size_t vqv_paged_attn_q4_workspace_bytes(const vqv_cache_q4* cache, const vqv_seqs* seqs,
                                         int heads, int window, int sinks) {
  vqv::AttnPlan plan;
  vqv::CopyPlan copy;
  if (plan_attn_q4(cache, seqs, heads, window, sinks, VQV_BF16, &plan, &copy) != VQV_OK) return 0;
  return attn_q4_bytes(*cache, *seqs, heads, plan, copy);
}

size_t vqv_paged_attn_q4_type_workspace_bytes(const vqv_cache_q4* cache, const vqv_seqs* seqs,
                                              vqv_dtype dtype, int heads, int window, int sinks) {
  vqv::AttnPlan plan;
  vqv::CopyPlan copy;
  if (!half_type(dtype) ||
      plan_attn_q4(cache, seqs, heads, window, sinks, dtype, &plan, &copy) != VQV_OK)
    return 0;
  return attn_q4_bytes(*cache, *seqs, heads, plan, copy);
}

vqv_status vqv_paged_attn_q4(const void* q, vqv_dtype dtype, const vqv_cache_q4* cache, int layer,
                             const vqv_seqs* seqs, int heads, float scale, int window, int sinks,
                             void* out, void* workspace, size_t workspace_bytes,
                             void* hip_stream) {
  vqv::AttnPlan plan;
  vqv::CopyPlan copy;
  const vqv_status st = plan_attn_q4(cache, seqs, heads, window, sinks, dtype, &plan, &copy);
  if (st != VQV_OK) return st;
  if ((seqs->n_rows && (!q || !out)) || layer < 0 || layer >= cache->layers) return VQV_ERR_ARG;
  if (dtype == VQV_FP32) return VQV_ERR_UNSUPPORTED;
  if (!half_type(dtype)) return VQV_ERR_ARG;
  if (!(scale > 0.0f) || !isfinite(scale)) return VQV_ERR_ARG;
  if (!aligned(q, 16) || !aligned(out, 16)) return VQV_ERR_ALIGN;
  const size_t bytes = (size_t)seqs->n_rows * heads * cache->dim * 2;
  const size_t need = attn_q4_bytes(*cache, *seqs, heads, plan, copy);
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
    return VQV_ERR_WORKSPACE;
  if (overlaps(out, bytes, q, bytes) || overlaps(workspace, need, q, bytes) ||
      overlaps(workspace, need, out, bytes))
    return VQV_ERR_ARG;
  if (seqs->n_rows == 0 || seqs->max_rows == 0) return VQV_OK;
  (void)hipGetLastError();
  const auto stream = static_cast<hipStream_t>(hip_stream);
  if (copy.copied.slots) {
    void* held = static_cast<char*>(workspace) + (need - copy.bytes);
    hipError_t e = vqv::launch_copy_q4(*cache, layer, *seqs, heads, copy, held, stream);
    if (e == hipSuccess)
      e = vqv::launch_paged_attn_copied(q, vqv::copy_cache(*cache, copy, held),
                                        vqv::copy_seqs(*seqs, copy, held), heads, scale,
                                        copy.copied, out, workspace, copy.attn, stream);
    if (e != hipSuccess) return status_of(e);
  }
  return status_of(vqv::launch_paged_attn_q4(q, (int)dtype, *cache, layer, *seqs, heads, scale,
                                             window, sinks, copy.copied, out, workspace, plan,
                                             stream));
}

}  // extern "C"

namespace {

vqv_status check_sample(int B, int T, int N) {
  if (B < 1 || T < 1 || T > 64 || N < 1) return VQV_ERR_ARG;
  if ((double)B * T * N >= 2147483648.0) return VQV_ERR_ARG;
  // The last chunk's tokens are counted in 32 bits, a grid's threads too.
  if (B > 65535 || N > INT32_MAX - (vqv::kVerifyChunk - 1) ||
      (int64_t)B * T * vqv::verify_chunks(N) >= (1ll << 23))
    return VQV_ERR_UNSUPPORTED;
  return VQV_OK;
}

vqv_status check_adapters(const vqv_adapters* a) {
  if (!a || !a->a || !a->b || !a->scale) return VQV_ERR_ARG;
  if (a->n < 1 || a->N < 1 || a->rank < 8 || a->rank % 8 || a->K < 8 || a->K % 8)
    return VQV_ERR_ARG;
  if (a->dtype == VQV_FP32) return VQV_ERR_UNSUPPORTED;
  if (!half_type(a->dtype)) return VQV_ERR_ARG;
  // Columns past the last, up to the end of its work-group and of the 8 groups that go to the
  // XCDs together (lora.hip), are counted in 32 bits.
  if (a->rank > 256 || a->K > 32768 || a->N > INT32_MAX - 8 * 512) return VQV_ERR_UNSUPPORTED;
  if (!aligned(a->a, 16) || !aligned(a->b, 16) || !words_aligned(a->scale, a->ranks))
    return VQV_ERR_ALIGN;
  return VQV_OK;
}

vqv_status check_rows(const vqv_adapters& a, int M) {
  if (M < 0) return VQV_ERR_ARG;
  if (M >= (1 << 22) || (double)M * a.N >= 1099511627776.0 || (double)M * a.K >= 1099511627776.0)
    return VQV_ERR_UNSUPPORTED;
  return vqv::lora_grids_fit(a, M) ? VQV_OK : VQV_ERR_UNSUPPORTED;
}

// Whether y and out are different columns of rows of one length.
bool columns_apart(const float* y, const float* out, int N, int64_t y_stride, int64_t out_stride) {
  if (y_stride != out_stride) return false;
  int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(out) - reinterpret_cast<uintptr_t>(y)) / 4 % y_stride;
  if (d < 0) d += y_stride;
  return d >= N && y_stride - d >= N;
}

}  // namespace

extern "C" {

size_t vqv_verify_sampled_workspace_bytes(int B, int T, int N) {
  return check_sample(B, T, N) == VQV_OK ? vqv::sample_workspace_bytes(B, T, N) : 0;
}

vqv_status vqv_verify_sampled(const float* logits, const int32_t* draft, const float* draft_probs,
                              const int32_t* draft_len, const float* temperature,
                              const float* uniform, int B, int T, int N, int32_t* token,
                              int32_t* accept_len, float* logprob, void* workspace,
                              size_t workspace_bytes, void* hip_stream) {
  const vqv_status st = check_sample(B, T, N);
  if (st != VQV_OK) return st;
  if (!logits || !uniform || !token || !accept_len || (T > 1 && !draft)) return VQV_ERR_ARG;
  if (!aligned(logits, 16) || !aligned(draft_probs, 16) ||
      !words_aligned(draft, draft_len, token, accept_len) ||
      !words_aligned(temperature, uniform, logprob))
    return VQV_ERR_ALIGN;
  const size_t need = vqv::sample_workspace_bytes(B, T, N), rows = (size_t)B * T;
  if (!workspace || workspace_bytes < need || !aligned(workspace, 16)) return VQV_ERR_WORKSPACE;
  struct Span {
    const void* p;
    size_t n;
  };
  const size_t drafts = (size_t)B * (T - 1);
  const Span in[6] = {{logits, rows * N * 4},  {draft, drafts * 4},
                      {draft_probs, drafts * N * 4}, {draft_len, (size_t)B * 4},
                      {temperature, (size_t)B * 4}, {uniform, rows * 4}};
  const Span out[4] = {{token, (size_t)B * 4}, {accept_len, (size_t)B * 4},
                       {logprob, rows * 4}, {workspace, need}};
  for (int o = 0; o < 4; ++o) {
    for (const Span& i : in)
      if (overlaps(out[o].p, out[o].n, i.p, i.n)) return VQV_ERR_ARG;
    for (int x = o + 1; x < 4; ++x)
      if (overlaps(out[o].p, out[o].n, out[x].p, out[x].n)) return VQV_ERR_ARG;
  }
  (void)hipGetLastError();
  return status_of(vqv::launch_verify_sampled(
      vqv::SampleArgs{logits, T > 1 ? draft : nullptr, T > 1 ? draft_probs : nullptr, draft_len,
                      temperature, uniform, B, T, N, token, accept_len, logprob, workspace},
      static_cast<hipStream_t>(hip_stream)));
}

size_t vqv_lora_add_workspace_bytes(const vqv_adapters* adapters, int M) {
  if (check_adapters(adapters) != VQV_OK || check_rows(*adapters, M) != VQV_OK) return 0;
  return vqv::lora_workspace_bytes(*adapters, M);
}

vqv_status vqv_lora_add(const void* x, vqv_dtype act_dtype, const vqv_adapters* adapters,
                        const int32_t* which, int M, const float* y, int64_t y_stride, float* out,
                        int64_t out_stride, void* workspace, size_t workspace_bytes,
                        void* hip_stream) {
  vqv_status st = check_adapters(adapters);
  if (st != VQV_OK) return st;
  if ((st = check_rows(*adapters, M)) != VQV_OK) return st;
  const vqv_adapters& a = *adapters;
  if (M && (!x || !which || !y || !out)) return VQV_ERR_ARG;
  if (!half_type(act_dtype) && act_dtype != VQV_FP32) return VQV_ERR_ARG;
  if (act_dtype != VQV_FP32 && (int)act_dtype != a.dtype) return VQV_ERR_UNSUPPORTED;
  if (y_stride < a.N || out_stride < a.N) return VQV_ERR_ARG;
  if ((double)M * y_stride >= 1152921504606846976.0 ||
      (double)M * out_stride >= 1152921504606846976.0)
    return VQV_ERR_UNSUPPORTED;
  if (!aligned(x, 16) || !words_aligned(which, y, out)) return VQV_ERR_ALIGN;
  if (M == 0) return VQV_OK;
  const size_t need = vqv::lora_workspace_bytes(a, M);
  if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
    return VQV_ERR_WORKSPACE;
  struct Span {
    const void* p;
    size_t n;
  };
  const size_t yb = ((size_t)(M - 1) * y_stride + a.N) * 4;
  const size_t ob = ((size_t)(M - 1) * out_stride + a.N) * 4;
  const Span in[6] = {{x, (size_t)M * a.K * (act_dtype == VQV_FP32 ? 4 : 2)},
                      {a.a, (size_t)a.n * a.rank * a.K * 2},
                      {a.b, (size_t)a.n * a.rank * a.N * 2},
                      {a.scale, (size_t)a.n * 4},
                      {a.ranks, (size_t)a.n * 4},
                      {which, (size_t)M * 4}};
  for (const Span& i : in)
    if (overlaps(out, ob, i.p, i.n) || overlaps(workspace, need, i.p, i.n)) return VQV_ERR_ARG;
  if (overlaps(workspace, need, y, yb) || overlaps(workspace, need, out, ob)) return VQV_ERR_ARG;
  if (out == y ? out_stride != y_stride
               : overlaps(out, ob, y, yb) && !columns_apart(y, out, a.N, y_stride, out_stride))
    return VQV_ERR_ARG;
  (void)hipGetLastError();
  return status_of(vqv::launch_lora_add(
      vqv::LoraArgs{x, a, which, M, y, y_stride, out, out_stride, workspace, nullptr, nullptr},
      (int)act_dtype, static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
