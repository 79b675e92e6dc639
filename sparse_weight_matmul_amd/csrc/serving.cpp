// C ABI of the serving operators: argument checks, work split and dispatch.
#include <hip/hip_runtime.h>

#include <cmath>

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

}  // extern "C"
