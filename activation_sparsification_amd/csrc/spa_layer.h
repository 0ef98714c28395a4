// Host-side launchers of the attention, cache and norm kernels (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "spa.h"
#include "spa_div.h"

namespace spa {

hipError_t launch_kv_write(const spa_heads& k, const spa_heads& v, int t, const int32_t* slots, const spa_kv_cache& c,
                           hipStream_t st);
hipError_t launch_kv_read(const spa_kv_cache& c, const int32_t* table, int n_seqs, int max_pages, const int32_t* cu,
                          int total, void* k_out, void* v_out, hipStream_t st);

struct PlanArgs {
  const int32_t* lens;       // [n_seqs]
  const int32_t* fresh;      // [n_seqs]: new tokens
  const int32_t* done;       // [n_seqs] or NULL
  int32_t* table;            // [n_seqs][max_pages]
  int32_t* stack;            // [n_pages]: the free pages
  const int32_t* count;      // how many
  int32_t* count_out;        // [2]: how many are left, and how many there were too few
  int32_t* slots;            // [t]
  int32_t* positions;        // [t]
  int32_t* cu_q;             // [n_seqs + 1]
  int32_t* cu_k;             // [n_seqs + 1]
  int32_t* lens_out;         // [n_seqs]
  int n_seqs, max_pages, n_pages, t;
  FastDiv page;
};
hipError_t launch_kv_plan(PlanArgs a, hipStream_t st);

hipError_t launch_attention_decode(const spa_heads& q, int n_seqs, int n_q_heads, const spa_kv_cache& c,
                                   const int32_t* table, int max_pages, const int32_t* lens, float scale, void* out,
                                   float* lse, float* part_o, float* part_ml, int32_t* part_of, hipStream_t st);

// The same over a SPA_KV_MXFP4 cache.
hipError_t launch_attention_decode_mx(const spa_heads& q, int n_seqs, int n_q_heads, const spa_kv_cache& c,
                                      const int32_t* table, int max_pages, const int32_t* lens, float scale, void* out,
                                      float* lse, float* part_o, float* part_ml, int32_t* part_of, hipStream_t st);

hipError_t launch_attention_prefill(const spa_heads& q, const spa_heads& k, const spa_heads& v, int dtype, int tq,
                                    int tk, int n_q_heads, int n_kv_heads, int head_dim, const int32_t* cu_q,
                                    const int32_t* cu_k, int n_seqs, bool causal, float scale, void* out, float* lse,
                                    int splits, float* part_o, float* part_ml, hipStream_t st);

struct NormArgs {
  const void* x;
  const void* residual;      // or NULL
  const void* gate;          // or NULL
  void* h;                   // or NULL
  void* y;                   // or NULL
  int t, c;
  int gate_per_token;        // gate is [t][c], not [c]
  float scale, eps;
  spa_norm post, pre;
};
struct RopeArgs {
  const uint16_t* src[3];    // queries, keys, values (with a cache)
  int64_t row[3], head[3];   // strides
  uint16_t* dst[2];          // queries, keys (or NULL)
  int64_t drow[2], dhead[2];
  const int32_t* pos;        // [t]; NULL without rotation
  const float* freq;         // [rot / 2]
  spa_norm norm[2];          // of queries and keys
  float eps;
  int t, hq, hkv, d, rot, neighbours;
  const int32_t* slots;      // [t], with a cache
  void* pages[2];            // launch_qk_norm_rope fills in the cache's
  void* scale[2];
  int n_pages;
  FastDiv page;
};
hipError_t launch_qk_norm_rope(int dtype, const spa_kv_cache* cache, RopeArgs a, hipStream_t st);

hipError_t launch_norm(int dtype, int stream_dtype, const NormArgs& a, hipStream_t st);

}  // namespace spa
