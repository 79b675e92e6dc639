// C ABI of the serving operators: argument checks, work split and dispatch.
#include <hip/hip_runtime.h>

#include <cmath>
#include <iterator>

#include "host_util.h"
#include "kernels.h"
#include "swm.h"

namespace {

using swm::swm_log;

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

// The sizes of a cache.
swm_status check_sizes(const swm_kv_cache* c) {
  if (!c || c->batch < 0 || c->pages_per_seq < 0 || c->pages < 1 || c->page_size < 1 || c->heads < 1 || c->dim < 1)
    return SWM_ERR_INVALID_ARG;
  if (c->dim % 8 || c->dim > 256 || c->batch > 65535 || c->heads > 65535) return SWM_ERR_UNSUPPORTED;
  const int64_t most = (int64_t(1) << 31) - 65536;
  if (c->pages >= most || c->page_size >= most || c->pages_per_seq >= most ||
      c->pages_per_seq * c->page_size >= most)
    return SWM_ERR_UNSUPPORTED;
  return SWM_OK;
}

swm_status check_cache(const swm_kv_cache* c, swm::KvView* v) {
  swm_status st = check_sizes(c);
  if (st != SWM_OK) return st;
  if (c->batch > 0 && (!c->k || !c->v || !c->lengths || (!c->table && c->pages_per_seq > 0)))
    return SWM_ERR_INVALID_ARG;
  if (c->k_page < 0 || c->k_slot < 0 || c->k_head < 0 || c->v_page < 0 || c->v_slot < 0 || c->v_head < 0 ||
      c->table_ld < 0)
    return SWM_ERR_INVALID_ARG;
  if (c->k_page % 8 || c->k_slot % 8 || c->k_head % 8 || c->v_page % 8 || c->v_slot % 8 || c->v_head % 8 ||
      misaligned(c->k) || misaligned(c->v))
    return SWM_ERR_ALIGN;
  v->k = static_cast<uint16_t*>(c->k);
  v->v = static_cast<uint16_t*>(c->v);
  v->table = c->table;
  v->lengths = c->lengths;
  v->k_p = c->k_page;
  v->k_s = c->k_slot;
  v->k_h = c->k_head;
  v->v_p = c->v_page;
  v->v_s = c->v_slot;
  v->v_h = c->v_head;
  v->table_b = c->table_ld;
  v->pages = c->pages;
  v->S = c->page_size;
  v->Hkv = c->heads;
  v->D = c->dim;
  v->B = c->batch;
  v->per_seq = c->pages_per_seq;
  return SWM_OK;
}

swm_status plan_for(const swm_kv_cache* c, int64_t q_heads, bool weights, swm::AttnPlan* p) {
  int dev = 0;
  SWM_HIP(hipGetDevice(&dev));
  *p = swm::plan_attention(c->batch, q_heads, c->heads, c->dim, c->pages_per_seq * c->page_size, weights,
                           swm::num_cus(dev));
  return SWM_OK;
}

// Whether rows of `len` entries, n0 at one stride by n1 at another, surely share memory.
bool rows_overlap(int64_t len, int64_t n0, int64_t stride0, int64_t n1, int64_t stride1) {
  return (n0 > 1 && stride0 < len) || (n1 > 1 && stride1 < len) || (n0 > 1 && n1 > 1 && stride0 == stride1);
}

// Whether rows of a cache's pools surely share memory.
bool cache_rows_overlap(const swm_kv_cache* c) {
  return rows_overlap(c->dim, c->pages, c->k_page, c->heads, c->k_head) ||
         rows_overlap(c->dim, c->pages, c->v_page, c->heads, c->v_head) ||
         rows_overlap(c->dim, c->page_size, c->k_slot, c->heads, c->k_head) ||
         rows_overlap(c->dim, c->page_size, c->v_slot, c->heads, c->v_head);
}

// Memory of an argument: rows of `bytes`, `step` bytes apart.
struct Span {
  uintptr_t at;
  int64_t rows, bytes, step;
};
template <typename T>
Span span_of(const T* p, int64_t rows, int64_t len, int64_t ld) {
  return {reinterpret_cast<uintptr_t>(p), len > 0 ? rows : 0, len * int64_t(sizeof(T)), ld * int64_t(sizeof(T))};
}
template <typename T>
Span span_of(const T* p, int64_t n) {
  return span_of(p, n > 0, n, n);
}

// Whether two have a byte in common; b is one row.
bool spans_meet(const Span& a, const Span& b) {
  if (a.rows < 1 || b.rows < 1) return false;
  const int64_t from = int64_t(b.at - a.at), to = from + b.bytes;  // in bytes from a's first
  // the first row of a that ends behind b's start
  const int64_t r = from < a.bytes ? 0 : a.rows > 1 ? (from - a.bytes) / a.step + 1 : a.rows;
  return r < a.rows && r * a.step < to;
}

bool heads_fit(const swm_kv_cache* c, int64_t q_heads) {
  return q_heads >= 1 && q_heads % c->heads == 0;
}

}  // namespace

extern "C" {

size_t swm_paged_attention_workspace_bytes(const swm_kv_cache* c, int64_t q_heads, int32_t weights) {
  swm::AttnPlan p;
  if (check_sizes(c) != SWM_OK || !heads_fit(c, q_heads) || q_heads > 65535 || c->batch == 0) return 0;
  return plan_for(c, q_heads, weights != 0, &p) == SWM_OK ? p.bytes : 0;
}

swm_status swm_paged_attention(const swm_kv_cache* c, const void* q, int64_t q_batch, int64_t q_head,
                               int64_t q_heads, float scale, const uint8_t* mask, int64_t mask_ld, float* weights,
                               int64_t w_page, int64_t w_head, void* out, int64_t out_batch, int64_t out_head,
                               void* workspace, size_t ws_bytes, void* stream) {
  swm::KvView v;
  swm_status st = check_cache(c, &v);
  if (st != SWM_OK) return st;
  if (!heads_fit(c, q_heads) || !std::isfinite(scale)) return SWM_ERR_INVALID_ARG;
  if (q_heads > 65535) return SWM_ERR_UNSUPPORTED;
  if (c->batch == 0) return SWM_OK;
  const int64_t cap = c->pages_per_seq * c->page_size;
  if (!q || !out || q_batch < 0 || q_head < 0 || out_batch < 0 || out_head < 0) return SWM_ERR_INVALID_ARG;
  if ((mask && mask_ld < cap) || (weights && (w_page < 0 || w_head < 0))) return SWM_ERR_INVALID_ARG;
  if (rows_overlap(c->dim, c->batch, out_batch, q_heads, out_head)) return SWM_ERR_INVALID_ARG;
  if (q_batch % 8 || q_head % 8 || misaligned(q)) return SWM_ERR_ALIGN;
  swm::AttnPlan p;
  st = plan_for(c, q_heads, weights != nullptr, &p);
  if (st != SWM_OK) return st;
  // either launch: at most 2^24 - 1 workgroups of 256 threads
  if (c->batch * q_heads + c->batch * c->heads * p.adds >= (int64_t(1) << 24) ||
      p.grid >= (int64_t(1) << 24))
    return SWM_ERR_UNSUPPORTED;
  if (p.bytes > 0) {
    if (!workspace || ws_bytes < p.bytes) return SWM_ERR_INVALID_ARG;
    if (misaligned(workspace)) return SWM_ERR_ALIGN;
  }
  swm_log("paged_attention B=%lld heads=%lld/%lld D=%lld capacity=%lld: %lld workgroups%s%s", (long long)c->batch,
          (long long)q_heads, (long long)c->heads, (long long)c->dim, (long long)cap, (long long)p.grid,
          p.room > 0  ? ", split by length" : p.order ? ", sorted by length" : "", weights ? ", weights added" : "");
  swm::AttnCall r;
  r.q = static_cast<const uint16_t*>(q);
  r.out = static_cast<uint16_t*>(out);
  r.mask = mask;
  r.weights = weights;
  r.q_b = q_batch;
  r.q_h = q_head;
  r.o_b = out_batch;
  r.o_h = out_head;
  r.mask_b = mask_ld;
  r.w_p = w_page;
  r.w_h = w_head;
  r.Hq = q_heads;
  r.scale = scale;
  SWM_HIP(swm::launch_attention(v, r, p, workspace, static_cast<hipStream_t>(stream)));
  return SWM_OK;
}

swm_status swm_kv_evict(const swm_kv_cache* c, const float* weights, int64_t w_page, int64_t w_head,
                        const int32_t* positions, int64_t p_page, int64_t p_head, int64_t budget, int64_t recent,
                        float* weights_out, int64_t wo_page, int64_t wo_head, int32_t* positions_out,
                        int64_t po_page, int64_t po_head, int32_t* lengths_out, int32_t* kept, void* stream) {
  swm::KvView v;
  swm_status st = check_cache(c, &v);
  if (st != SWM_OK) return st;
  if (budget < 0 || recent < 0 || budget >= (int64_t(1) << 31) || recent >= (int64_t(1) << 31))
    return SWM_ERR_INVALID_ARG;
  if (w_page < 0 || w_head < 0 || p_page < 0 || p_head < 0 || wo_page < 0 || wo_head < 0 || po_page < 0 ||
      po_head < 0)
    return SWM_ERR_INVALID_ARG;
  if (c->batch == 0) return SWM_OK;
  if (!weights || !positions || !weights_out || !positions_out || !lengths_out || (!kept && budget > 0))
    return SWM_ERR_INVALID_ARG;
  if (lengths_out == c->lengths || (weights_out == weights && (wo_page != w_page || wo_head != w_head)) ||
      (positions_out == positions && (po_page != p_page || po_head != p_head)))
    return SWM_ERR_INVALID_ARG;
  // rows move within a head, so heads own theirs
  if (rows_overlap(c->dim, c->pages, c->k_page, c->heads, c->k_head) ||
      rows_overlap(c->dim, c->pages, c->v_page, c->heads, c->v_head))
    return SWM_ERR_INVALID_ARG;
  if (rows_overlap(c->page_size, c->pages, wo_page, c->heads, wo_head) ||
      rows_overlap(c->page_size, c->pages, po_page, c->heads, po_head))
    return SWM_ERR_INVALID_ARG;
  swm_log("kv_evict B=%lld heads=%lld D=%lld capacity=%lld: budget %lld, recent %lld", (long long)c->batch,
          (long long)c->heads, (long long)c->dim, (long long)(c->pages_per_seq * c->page_size), (long long)budget,
          (long long)recent);
  swm::EvictCall r;
  r.weights = weights;
  r.positions = positions;
  r.weights_out = weights_out;
  r.positions_out = positions_out;
  r.lengths_out = lengths_out;
  r.kept = kept;
  r.w_p = w_page;
  r.w_h = w_head;
  r.p_p = p_page;
  r.p_h = p_head;
  r.wo_p = wo_page;
  r.wo_h = wo_head;
  r.po_p = po_page;
  r.po_h = po_head;
  r.budget = budget;
  r.recent = recent;
  int dev = 0;
  SWM_HIP(hipGetDevice(&dev));
  SWM_HIP(swm::launch_evict(v, r, swm::num_cus(dev), static_cast<hipStream_t>(stream)));
  return SWM_OK;
}

swm_status swm_token_logprobs(const void* logits, int32_t fp32, int64_t N, int64_t V, int64_t ld,
                              const void* targets, int32_t wide, float* logp, float* entropy, int32_t top,
                              int64_t* top_ids, float* top_logp, void* stream) {
  if (N < 0 || V < 1 || ld < V || top < 0 || (targets && !logp)) return SWM_ERR_INVALID_ARG;
  if (top > swm::kLogprobMaxTop || V >= (int64_t(1) << 31) - 65536 || N >= (int64_t(1) << 22))
    return SWM_ERR_UNSUPPORTED;
  if (N == 0) return SWM_OK;
  if (!logits || (top > 0 && (!top_ids || !top_logp))) return SWM_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(logits) % (fp32 ? 4 : 2)) return SWM_ERR_ALIGN;
  swm::LogprobCall r;
  r.logits = logits;
  r.targets = targets;
  r.logp = logp;
  r.entropy = entropy;
  r.top_logp = top_logp;
  r.top_ids = top_ids;
  r.N = N;
  r.V = V;
  r.ld = ld;
  r.top = top;
  r.fp32 = fp32 != 0;
  r.wide = wide != 0;
  swm_log("token_logprobs N=%lld V=%lld top=%d, %s logits", (long long)N, (long long)V, top, fp32 ? "fp32" : "fp16");
  int dev = 0;
  SWM_HIP(hipGetDevice(&dev));
  SWM_HIP(swm::launch_logprobs(r, swm::num_cus(dev), static_cast<hipStream_t>(stream)));
  return SWM_OK;
}

swm_status swm_prompt_attention(const void* q, int64_t q_token, int64_t q_head, const void* k, int64_t k_token,
                                int64_t k_head, const void* v, int64_t v_token, int64_t v_head, int64_t tokens,
                                int64_t q_heads, int64_t heads, int64_t dim, const int32_t* starts, int64_t batch,
                                float scale, int32_t causal, void* out, int64_t out_token, int64_t out_head,
                                void* stream) {
  if (tokens < 0 || batch < 0 || heads < 1 || q_heads < 1 || q_heads % heads || dim < 1 || !std::isfinite(scale))
    return SWM_ERR_INVALID_ARG;
  if (dim % 8 || dim > 256 || batch > 65535 || q_heads > 65535 || tokens >= (int64_t(1) << 31) - 65536)
    return SWM_ERR_UNSUPPORTED;
  if (tokens == 0 || batch == 0) return SWM_OK;
  if (!q || !k || !v || !out || !starts) return SWM_ERR_INVALID_ARG;
  if (q_token < 0 || q_head < 0 || k_head < 0 || v_head < 0 || out_token < 0 || out_head < 0) return SWM_ERR_INVALID_ARG;
  if (k_token < dim || v_token < dim) return SWM_ERR_INVALID_ARG;
  if (rows_overlap(dim, tokens, out_token, q_heads, out_head)) return SWM_ERR_INVALID_ARG;
  if (q_token % 8 || q_head % 8 || k_token % 8 || k_head % 8 || v_token % 8 || v_head % 8 || misaligned(q) ||
      misaligned(k) || misaligned(v))
    return SWM_ERR_ALIGN;
  // a tile's rows are addressed with 32-bit byte offsets
  const int64_t most = int64_t(1) << 23;
  if (k_token >= most || v_token >= most || swm::prompt_grid(tokens, batch, q_heads) >= (int64_t(1) << 24))
    return SWM_ERR_UNSUPPORTED;
  swm_log("prompt_attention tokens=%lld sequences=%lld heads=%lld/%lld D=%lld%s", (long long)tokens,
          (long long)batch, (long long)q_heads, (long long)heads, (long long)dim, causal ? ", causal" : "");
  swm::PromptCall r;
  r.q = static_cast<const uint16_t*>(q);
  r.k = static_cast<const uint16_t*>(k);
  r.v = static_cast<const uint16_t*>(v);
  r.out = static_cast<uint16_t*>(out);
  r.starts = starts;
  r.q_t = q_token;
  r.q_h = q_head;
  r.k_t = k_token;
  r.k_h = k_head;
  r.v_t = v_token;
  r.v_h = v_head;
  r.o_t = out_token;
  r.o_h = out_head;
  r.B = batch;
  r.T = tokens;
  r.Hq = q_heads;
  r.Hkv = heads;
  r.D = dim;
  r.scale = scale;
  r.causal = causal != 0;
  int dev = 0;
  SWM_HIP(hipGetDevice(&dev));
  SWM_HIP(swm::launch_prompt(r, swm::num_cus(dev), static_cast<hipStream_t>(stream)));
  return SWM_OK;
}

swm_status swm_kv_reserve(const swm_kv_cache* c, const int32_t* counts, int32_t* free_pages, int64_t free_size,
                          int32_t* free_count, int64_t tokens, int32_t* starts, int64_t* slots, int32_t* granted,
                          void* stream) {
  swm::KvView v;
  swm_status st = check_cache(c, &v);
  if (st != SWM_OK) return st;
  if (free_size < 0 || tokens < 0) return SWM_ERR_INVALID_ARG;
  if (free_size >= (int64_t(1) << 31) - 65536 || tokens >= (int64_t(1) << 31) - 65536) return SWM_ERR_UNSUPPORTED;
  if (!starts || !free_count || (!free_pages && free_size > 0) || (!slots && tokens > 0)) return SWM_ERR_INVALID_ARG;
  if (c->batch > 0 && (!counts || !granted)) return SWM_ERR_INVALID_ARG;
  if (free_size < c->pages) return SWM_ERR_SHAPE;
  if (c->batch > 1 && c->table_ld < c->pages_per_seq) return SWM_ERR_INVALID_ARG;
  // What is written is nobody else's; of these only counts is not.
  const Span spans[] = {span_of(c->table, c->batch, c->pages_per_seq, c->table_ld), span_of(c->lengths, c->batch),
                        span_of(counts, c->batch),    span_of(free_pages, free_size),
                        span_of(free_count, 1),       span_of(starts, c->batch + 1),
                        span_of(slots, tokens),       span_of(granted, c->batch)};
  for (const Span* a = spans; a != std::end(spans); ++a)
    for (const Span* b = a + 1; b != std::end(spans); ++b)
      if (spans_meet(*a, *b)) return SWM_ERR_INVALID_ARG;
  swm_log("kv_reserve B=%lld capacity=%lld: %lld tokens, %lld free pages at most", (long long)c->batch,
          (long long)(c->pages_per_seq * c->page_size), (long long)tokens, (long long)free_size);
  swm::ReserveCall r;
  r.counts = counts;
  r.free_pages = free_pages;
  r.free_size = free_size;
  r.free_count = free_count;
  r.tokens = tokens;
  r.starts = starts;
  r.slots = slots;
  r.granted = granted;
  SWM_HIP(swm::launch_reserve(v, r, static_cast<hipStream_t>(stream)));
  return SWM_OK;
}

swm_status swm_kv_append(const swm_kv_cache* c, const void* k, int64_t k_token, int64_t k_head, const void* v,
                         int64_t v_token, int64_t v_head, int64_t tokens, const int64_t* slots, float* weights,
                         int64_t w_page, int64_t w_head, int32_t* positions, int64_t p_page, int64_t p_head,
                         const int32_t* at, void* stream) {
  swm::KvView w;
  swm_status st = check_cache(c, &w);
  if (st != SWM_OK) return st;
  if (tokens < 0 || k_token < 0 || k_head < 0 || v_token < 0 || v_head < 0) return SWM_ERR_INVALID_ARG;
  if ((weights && (w_page < 0 || w_head < 0)) || (positions && (p_page < 0 || p_head < 0 || (!at && tokens > 0))))
    return SWM_ERR_INVALID_ARG;
  if (tokens == 0) return SWM_OK;
  if (!c->k || !c->v || !k || !v || !slots) return SWM_ERR_INVALID_ARG;
  if (k_token % 8 || k_head % 8 || v_token % 8 || v_head % 8 || misaligned(k) || misaligned(v)) return SWM_ERR_ALIGN;
  if (cache_rows_overlap(c)) return SWM_ERR_INVALID_ARG;
  if ((weights && rows_overlap(c->page_size, c->pages, w_page, c->heads, w_head)) ||
      (positions && rows_overlap(c->page_size, c->pages, p_page, c->heads, p_head)))
    return SWM_ERR_INVALID_ARG;
  const int64_t most = (int64_t(1) << 31) - 65536;
  if (tokens >= most || tokens * (c->heads * (c->dim / 8)) / 1024 >= (int64_t(1) << 24) - 1)
    return SWM_ERR_UNSUPPORTED;
  swm_log("kv_append tokens=%lld heads=%lld D=%lld%s%s", (long long)tokens, (long long)c->heads, (long long)c->dim,
          weights ? ", weights" : "", positions ? ", positions" : "");
  swm::AppendCall r;
  r.k = static_cast<const uint16_t*>(k);
  r.v = static_cast<const uint16_t*>(v);
  r.k_t = k_token;
  r.k_h = k_head;
  r.v_t = v_token;
  r.v_h = v_head;
  r.T = tokens;
  r.slots = slots;
  r.weights = weights;
  r.w_p = w_page;
  r.w_h = w_head;
  r.positions = positions;
  r.p_p = p_page;
  r.p_h = p_head;
  r.at = at;
  SWM_HIP(swm::launch_append(w, r, static_cast<hipStream_t>(stream)));
  return SWM_OK;
}

size_t swm_tree_attention_workspace_bytes(const swm_kv_cache* c, int64_t q_heads, int64_t max_tokens) {
  if (check_sizes(c) != SWM_OK || !heads_fit(c, q_heads) || q_heads > 65535 || c->batch == 0 || max_tokens < 1 ||
      max_tokens > swm::kTreeMost)
    return 0;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 0;
  return swm::plan_tree(c->batch, q_heads, c->heads, c->dim, c->pages_per_seq * c->page_size, max_tokens,
                        swm::num_cus(dev)).bytes;
}

swm_status swm_tree_attention(const swm_kv_cache* c, const void* q, int64_t q_token, int64_t q_head, int64_t q_heads,
                              int64_t tokens, const int32_t* starts, const int32_t* parents, int64_t max_tokens,
                              float scale, const uint8_t* mask, int64_t mask_ld, void* out, int64_t out_token,
                              int64_t out_head, void* workspace, size_t ws_bytes, void* stream) {
  swm::KvView v;
  swm_status st = check_cache(c, &v);
  if (st != SWM_OK) return st;
  if (!heads_fit(c, q_heads) || !std::isfinite(scale) || tokens < 0 || max_tokens < 0) return SWM_ERR_INVALID_ARG;
  if (q_heads > 65535 || max_tokens > swm::kTreeMost || tokens >= (int64_t(1) << 31) - 65536)
    return SWM_ERR_UNSUPPORTED;
  // a load's rows are addressed from its first with 32-bit byte offsets
  if (c->k_slot >= (int64_t(1) << 26) || c->v_slot >= (int64_t(1) << 26)) return SWM_ERR_UNSUPPORTED;
  if (c->batch == 0 || tokens == 0 || max_tokens == 0) return SWM_OK;
  const int64_t cap = c->pages_per_seq * c->page_size;
  if (!q || !out || !starts || q_token < 0 || q_head < 0 || out_token < 0 || out_head < 0) return SWM_ERR_INVALID_ARG;
  if (mask && mask_ld < cap) return SWM_ERR_INVALID_ARG;
  if (rows_overlap(c->dim, tokens, out_token, q_heads, out_head)) return SWM_ERR_INVALID_ARG;
  if (q_token % 8 || q_head % 8 || misaligned(q)) return SWM_ERR_ALIGN;
  int dev = 0;
  SWM_HIP(hipGetDevice(&dev));
  const swm::TreePlan p = swm::plan_tree(c->batch, q_heads, c->heads, c->dim, cap, max_tokens, swm::num_cus(dev));
  // at most 2^23 - 1 workgroups of 512 threads, 2^24 - 1 of 256 in the second launch
  if (p.grid >= (int64_t(1) << 23) || tokens * q_heads >= (int64_t(1) << 26) - 4) return SWM_ERR_UNSUPPORTED;
  if (p.bytes > 0) {
    if (!workspace || ws_bytes < p.bytes) return SWM_ERR_INVALID_ARG;
    if (misaligned(workspace)) return SWM_ERR_ALIGN;
  }
  swm_log("tree_attention B=%lld tokens=%lld heads=%lld/%lld D=%lld capacity=%lld: %lld workgroups, %d pieces at most",
          (long long)c->batch, (long long)tokens, (long long)q_heads, (long long)c->heads, (long long)c->dim,
          (long long)cap, (long long)p.grid, p.room);
  swm::TreeCall r;
  r.q = static_cast<const uint16_t*>(q);
  r.out = static_cast<uint16_t*>(out);
  r.starts = starts;
  r.parents = parents;
  r.mask = mask;
  r.q_t = q_token;
  r.q_h = q_head;
  r.o_t = out_token;
  r.o_h = out_head;
  r.mask_b = mask_ld;
  r.T = tokens;
  r.Hq = q_heads;
  r.most = max_tokens;
  r.scale = scale;
  SWM_HIP(swm::launch_tree(v, r, p, workspace, static_cast<hipStream_t>(stream)));
  return SWM_OK;
}

}  // extern "C"
