// Host-side launchers of the attention, cache and norm kernels (internal to the library).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "spa.h"

namespace spa {

hipError_t launch_kv_write(const spa_heads& k, const spa_heads& v, int t, const int32_t* slots, const spa_kv_cache& c,
                           hipStream_t st);
hipError_t launch_kv_read(const spa_kv_cache& c, const int32_t* table, int n_seqs, int max_pages, const int32_t* cu,
                          int total, void* k_out, void* v_out, hipStream_t st);

hipError_t launch_attention_decode(const spa_heads& q, int n_seqs, int n_q_heads, const spa_kv_cache& c,
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
hipError_t launch_norm(int dtype, int stream_dtype, const NormArgs& a, hipStream_t st);

}  // namespace spa
