// C ABI of the attention, cache and norm entry points: argument validation and dispatch.  Every rejection
// happens here, before anything is launched.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "spa.h"
#include "spa_check_layer.h"
#include "spa_layer.h"

namespace {

using namespace spa_check;

spa_status hip_status(hipError_t e) { return e == hipSuccess ? SPA_OK : SPA_ERR_HIP; }
hipStream_t stream_of(void* s) { return static_cast<hipStream_t>(s); }

}  // namespace

extern "C" {

spa_status spa_kv_write(const spa_heads* k, const spa_heads* v, int32_t t, const int32_t* slots,
                        const spa_kv_cache* cache, void* stream) {
  if (spa_status s = check_kv_write(k, v, t, slots, cache)) return s;
  if (t == 0) return SPA_OK;
  return hip_status(spa::launch_kv_write(*k, *v, t, slots, *cache, stream_of(stream)));
}

spa_status spa_kv_read(const spa_kv_cache* cache, const int32_t* page_table, int32_t n_seqs, int32_t max_pages,
                       const int32_t* cu_seqlens, int32_t total, void* k_out, void* v_out, void* stream) {
  if (spa_status s = check_kv_read(cache, page_table, n_seqs, max_pages, cu_seqlens, total, k_out, v_out)) return s;
  if (n_seqs == 0 || total == 0) return SPA_OK;
  return hip_status(spa::launch_kv_read(*cache, page_table, n_seqs, max_pages, cu_seqlens, total, k_out, v_out,
                                        stream_of(stream)));
}

spa_status spa_kv_plan(const int32_t* lens, const int32_t* fresh, const int32_t* done, int32_t n_seqs, int32_t* page_table,
                       int32_t max_pages, int32_t page_size, const spa_page_pool* pool, int32_t t, int32_t* slots,
                       int32_t* positions, int32_t* cu_q, int32_t* cu_k, int32_t* lens_out, void* stream) {
  if (spa_status s = check_kv_plan(lens, fresh, done, n_seqs, page_table, max_pages, page_size, pool, t, slots, positions, cu_q, cu_k,
                                   lens_out))
    return s;
  spa::PlanArgs a{};
  a.lens = lens; a.fresh = fresh; a.done = n_seqs ? done : nullptr;
  a.table = page_table;
  a.stack = pool->pages; a.count = pool->count; a.count_out = pool->count_out;
  a.slots = slots; a.positions = positions; a.cu_q = cu_q; a.cu_k = cu_k; a.lens_out = lens_out;
  a.n_seqs = n_seqs; a.max_pages = max_pages; a.n_pages = pool->n_pages; a.t = t;
  a.page = spa::FastDiv((uint32_t)page_size);
  return hip_status(spa::launch_kv_plan(a, stream_of(stream)));
}

size_t spa_attention_decode_workspace_bytes(int32_t n_seqs, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim) {
  if (n_seqs < 1 || n_seqs > kMaxSeqs || n_q_heads < 1 || n_q_heads > kMaxHeads || n_kv_heads < 1 ||
      n_q_heads % n_kv_heads || head_dim < 1 || !built_head_dim(head_dim))
    return 0;
  return decode_attn_plan(n_seqs, n_q_heads, n_kv_heads, head_dim).bytes;
}

spa_status attention_decode(const spa_heads* q, int32_t n_seqs, int32_t n_q_heads, const spa_kv_cache* cache,
                            const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens, float scale,
                            void* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (spa_status s = check_attention_decode(q, n_seqs, n_q_heads, cache, page_table, max_pages, seq_lens, scale, out))
    return s;
  if (n_seqs == 0) return SPA_OK;
  const DecodeAttnPlan p = decode_attn_plan(n_seqs, n_q_heads, cache->n_heads, cache->head_dim);
  if (!workspace || workspace_bytes < p.bytes || !aligned16(workspace)) return SPA_ERR_INVALID;
  char* base = static_cast<char*>(workspace);
  return hip_status(spa::launch_attention_decode(*q, n_seqs, n_q_heads, *cache, page_table, max_pages, seq_lens, scale,
                                                 out, lse, reinterpret_cast<float*>(base + p.o),
                                                 reinterpret_cast<float*>(base + p.ml), reinterpret_cast<int32_t*>(base + p.of),
                                                 stream_of(stream)));
}

size_t spa_attention_prefill_workspace_bytes(int32_t tq, int32_t tk, int32_t n_seqs, int32_t n_q_heads,
                                             int32_t head_dim) {
  if (tq < 1 || tq > kMaxRows || tk < 0 || tk > kMaxRows || n_seqs < 1 || n_seqs > kMaxSeqs || n_q_heads < 1 ||
      n_q_heads > kMaxHeads || head_dim < 1 || !built_head_dim(head_dim))
    return 0;
  return prefill_attn_plan(tq, tk, n_seqs, n_q_heads, head_dim).bytes;
}

spa_status attention_prefill(const spa_heads* q, const spa_heads* k, const spa_heads* v, int32_t dtype, int32_t tq,
                             int32_t tk, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, const int32_t* cu_q,
                             const int32_t* cu_k, int32_t n_seqs, int32_t causal, float scale, void* out, float* lse,
                             void* workspace, size_t workspace_bytes, void* stream) {
  if (spa_status s = check_attention_prefill(q, k, v, dtype, tq, tk, n_q_heads, n_kv_heads, head_dim, cu_q, cu_k, n_seqs,
                                             scale, out))
    return s;
  if (tq == 0 || n_seqs == 0) return SPA_OK;
  const PrefillAttnPlan p = prefill_attn_plan(tq, tk, n_seqs, n_q_heads, head_dim);
  if (p.bytes && (!workspace || workspace_bytes < p.bytes || !aligned16(workspace))) return SPA_ERR_INVALID;
  char* base = static_cast<char*>(workspace);
  const spa_heads none{q->data, 0, 0};   // no keys at all: nothing is read through these
  return hip_status(spa::launch_attention_prefill(*q, tk ? *k : none, tk ? *v : none, dtype, tq, tk, n_q_heads,
                                                  n_kv_heads, head_dim, cu_q, cu_k, n_seqs, causal != 0, scale, out, lse,
                                                  p.splits, p.bytes ? reinterpret_cast<float*>(base + p.o) : nullptr,
                                                  p.bytes ? reinterpret_cast<float*>(base + p.ml) : nullptr,
                                                  stream_of(stream)));
}

spa_status qk_norm_rope(const spa_heads* q, const spa_heads* k, const spa_heads* v, int32_t dtype, int32_t t,
                        int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, const int32_t* positions,
                        const spa_rope* rope, const spa_norm* q_norm, const spa_norm* k_norm, float eps,
                        const spa_heads* q_out, const spa_heads* k_out, const int32_t* slots, const spa_kv_cache* cache,
                        void* stream) {
  if (spa_status s = check_qk_norm_rope(q, k, v, dtype, t, n_q_heads, n_kv_heads, head_dim, positions, rope, q_norm, k_norm,
                                        eps, q_out, k_out, slots, cache))
    return s;
  if (t == 0) return SPA_OK;
  const spa_norm none{SPA_NORM_NONE, nullptr, nullptr};
  spa::RopeArgs a{};
  const spa_heads* src[3] = {q, k, v};
  for (int i = 0; i < 3; ++i) {
    if (!src[i]) continue;
    a.src[i] = static_cast<const uint16_t*>(src[i]->data);
    a.row[i] = src[i]->row_stride;
    a.head[i] = src[i]->head_stride;
  }
  const spa_heads* dst[2] = {q_out, k_out};
  for (int i = 0; i < 2; ++i) {
    if (!dst[i]) continue;
    a.dst[i] = static_cast<uint16_t*>(const_cast<void*>(dst[i]->data));
    a.drow[i] = dst[i]->row_stride;
    a.dhead[i] = dst[i]->head_stride;
  }
  a.pos = positions;
  a.norm[0] = q_norm ? *q_norm : none;
  a.norm[1] = k_norm ? *k_norm : none;
  a.eps = eps;
  a.t = t; a.hq = n_q_heads; a.hkv = n_kv_heads; a.d = head_dim;
  if (rope) {
    a.freq = rope->inv_freq;
    a.rot = rope->rotary_dim;
    a.neighbours = rope->interleaved != 0;
  }
  a.slots = slots;
  return hip_status(spa::launch_qk_norm_rope(dtype, cache, a, stream_of(stream)));
}

spa_status gated_residual_norm(const void* x, int32_t dtype, int32_t t, int32_t c, const void* residual,
                               int32_t stream_dtype, const spa_norm* post, const void* gate, int32_t gate_rows,
                               float scale, const spa_norm* pre, float eps, void* h, void* y, void* stream) {
  if (spa_status s = check_norm(x, dtype, t, c, residual, stream_dtype, post, gate, gate_rows, scale, pre, eps, h, y))
    return s;
  if (t == 0) return SPA_OK;
  const spa_norm none{SPA_NORM_NONE, nullptr, nullptr};
  spa::NormArgs a{};
  a.x = x; a.residual = residual; a.gate = gate; a.h = h; a.y = y;
  a.t = t; a.c = c;
  a.gate_per_token = gate && gate_rows == t && t != 1;
  a.scale = scale; a.eps = eps;
  a.post = post ? *post : none;
  a.pre = pre ? *pre : none;
  return hip_status(spa::launch_norm(dtype, stream_dtype, a, stream_of(stream)));
}

}  // extern "C"
