// Argument checks of the attention, cache and norm entry points, and the decode attention's workspace
// layout, in plain C++ (no HIP types), so that the library and a host-only sanitizer build run the same
// code.  The entry points call these before anything is launched.
#pragma once

#include <math.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "spa.h"
#include "spa_check.h"

namespace spa_check {

constexpr int32_t kMaxHeads = 1 << 12;
constexpr int32_t kMaxHeadDim = 256;
constexpr int32_t kMaxRows = 1 << 30;             // packed rows of a call
constexpr int64_t kMaxVectors = int64_t(1) << 26;  // (token, head) pairs of a cache call: the launch counts threads in 32 bits
constexpr int32_t kMaxSeqs = 1 << 20;
constexpr int64_t kMaxStride = int64_t(1) << 23;  // elements between rows: 64 rows of it stay below 2^31 bytes
constexpr int64_t kMaxPositions = int64_t(1) << 29;    // of one sequence's table: 64 sequences' tiles add up in 31 bits
constexpr int64_t kMaxDecodeRows = int64_t(1) << 23;   // (sequence, query head) pairs of a call
constexpr int32_t kMaxNormC = 1 << 16;            // channels a workgroup holds in registers

inline bool valid_heads(const spa_heads* h) { return h && h->data; }
// Built: every vector starts on 16 bytes, and a tile of rows is addressed with 32-bit offsets.
inline bool built_heads(const spa_heads* h) {
  return aligned16(h->data) && h->row_stride % 8 == 0 && h->head_stride % 8 == 0;
}
inline bool valid_strides(const spa_heads* h) {
  return h->row_stride >= 0 && h->row_stride <= kMaxStride && h->head_stride >= 0 && h->head_stride <= kMaxStride;
}
inline bool dtype16(int dt) { return dt == SPA_F16 || dt == SPA_BF16; }
inline bool valid_head_dim(int32_t d) { return d >= 1 && d <= kMaxDim; }
inline bool built_head_dim(int32_t d) { return d % 8 == 0 && d <= kMaxHeadDim; }
inline int kv_bytes(const spa_kv_cache* c) { return c->format == SPA_KV_NATIVE ? 2 : 1; }

inline spa_status check_cache(const spa_kv_cache* c) {
  if (!c || !valid_dtype(c->dtype)) return SPA_ERR_INVALID;
  if (c->format < SPA_KV_NATIVE || c->format > SPA_KV_INT8) return SPA_ERR_INVALID;
  if (c->n_pages < 1 || c->page_size < 1 || c->n_heads < 1 || c->n_heads > kMaxHeads) return SPA_ERR_INVALID;
  if (!valid_head_dim(c->head_dim)) return SPA_ERR_INVALID;
  if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return SPA_ERR_INVALID;
  if (c->format != SPA_KV_NATIVE && (!c->k_scale || !c->v_scale || !aligned16(c->k_scale) || !aligned16(c->v_scale)))
    return SPA_ERR_INVALID;
  if (c->dtype == SPA_F32 || !built_head_dim(c->head_dim)) return SPA_ERR_UNSUPPORTED;
  // slots and cached vectors are numbered in 31 bits (their bytes are not)
  if ((int64_t)c->n_pages * c->page_size > INT32_MAX / c->n_heads) return SPA_ERR_UNSUPPORTED;
  return SPA_OK;
}

inline spa_status check_kv_write(const spa_heads* k, const spa_heads* v, int32_t t, const int32_t* slots,
                                 const spa_kv_cache* c) {
  if (t < 0 || t > kMaxRows) return SPA_ERR_INVALID;
  const spa_status s = check_cache(c);
  if (s == SPA_ERR_INVALID) return s;
  if (t == 0) return s;
  if (!valid_heads(k) || !valid_heads(v) || !slots || !valid_strides(k) || !valid_strides(v)) return SPA_ERR_INVALID;
  if (s != SPA_OK) return s;
  if ((int64_t)t * c->n_heads > kMaxVectors) return SPA_ERR_UNSUPPORTED;
  return built_heads(k) && built_heads(v) ? SPA_OK : SPA_ERR_UNSUPPORTED;
}

inline spa_status check_kv_read(const spa_kv_cache* c, const int32_t* table, int32_t n_seqs, int32_t max_pages,
                                const int32_t* cu, int32_t total, const void* k_out, const void* v_out) {
  if (n_seqs < 0 || n_seqs > kMaxSeqs || max_pages < 0 || total < 0 || total > kMaxRows) return SPA_ERR_INVALID;
  const spa_status s = check_cache(c);
  if (s == SPA_ERR_INVALID) return s;
  if (n_seqs == 0 || total == 0) return s;
  if (max_pages < 1 || !table || !cu || !k_out || !v_out || !aligned16(k_out) || !aligned16(v_out)) return SPA_ERR_INVALID;
  if (s == SPA_OK && (int64_t)total * c->n_heads > kMaxVectors) return SPA_ERR_UNSUPPORTED;
  return s;
}

inline bool valid_scale(float s) { return s > 0.f && s <= 1e30f; }   // false for NaN

// ---- decode attention ----
inline spa_status check_attention_decode(const spa_heads* q, int32_t n_seqs, int32_t n_q_heads, const spa_kv_cache* c,
                                         const int32_t* table, int32_t max_pages, const int32_t* lens, float scale,
                                         const void* out) {
  if (n_seqs < 0 || n_seqs > kMaxSeqs || n_q_heads < 1 || n_q_heads > kMaxHeads || max_pages < 0) return SPA_ERR_INVALID;
  if (!valid_scale(scale)) return SPA_ERR_INVALID;
  const spa_status s = check_cache(c);
  if (s == SPA_ERR_INVALID) return s;
  if (n_q_heads % c->n_heads) return SPA_ERR_INVALID;
  if (n_seqs == 0) return s;
  if (!valid_heads(q) || !valid_strides(q) || !lens || !out || !aligned16(out)) return SPA_ERR_INVALID;
  if (max_pages > 0 && !table) return SPA_ERR_INVALID;
  if (s != SPA_OK) return s;
  if ((int64_t)max_pages * c->page_size > kMaxPositions) return SPA_ERR_UNSUPPORTED;
  if ((int64_t)n_seqs * n_q_heads > kMaxDecodeRows) return SPA_ERR_UNSUPPORTED;
  return built_heads(q) ? SPA_OK : SPA_ERR_UNSUPPORTED;
}

// Query heads of one key-value head are worked on 16 at a time (the matrix instruction's columns).
inline int head_tiles(int n_q_heads, int n_kv_heads) { return (n_q_heads / n_kv_heads + 15) / 16; }
// Workgroups that share the cache of one key-value head and head tile: as many as the chip holds at a time over all
// heads, 3, 2 or 1 to a compute unit as the registers for the head's dimensions allow.  Rounded up: heads that do not
// divide the places get a few more workgroups than the chip holds (20 heads of 128: 520 on 512).
inline int decode_groups(int n_q_heads, int n_kv_heads, int head_dim) {
  const int places = head_dim <= 64 ? 768 : head_dim <= 128 ? 512 : 256;
  const int per_unit = n_kv_heads * head_tiles(n_q_heads, n_kv_heads);
  return (places + per_unit - 1) / per_unit;
}
struct DecodeAttnPlan {
  // [2 groups][heads][head_dim] float32 partial outputs, [2 groups][heads][2] maximum and sum, [n_seqs][2] first slot
  // and number of pieces
  size_t o, ml, of, bytes;
};
inline DecodeAttnPlan decode_attn_plan(int n_seqs, int n_q_heads, int n_kv_heads, int head_dim) {
  DecodeAttnPlan p{};
  const size_t rows = (size_t)2 * decode_groups(n_q_heads, n_kv_heads, head_dim) * n_q_heads;
  p.o = 0;
  p.ml = round256(rows * head_dim * 4);
  p.of = p.ml + round256(rows * 8);
  p.bytes = p.of + round256((size_t)n_seqs * 8);
  return p;
}

// ---- prompt attention ----
inline spa_status check_attention_prefill(const spa_heads* q, const spa_heads* k, const spa_heads* v, int32_t dtype,
                                          int32_t tq, int32_t tk, int32_t n_q_heads, int32_t n_kv_heads,
                                          int32_t head_dim, const int32_t* cu_q, const int32_t* cu_k, int32_t n_seqs,
                                          float scale, const void* out) {
  if (!valid_dtype(dtype) || tq < 0 || tq > kMaxRows || tk < 0 || tk > kMaxRows || n_seqs < 0 || n_seqs > kMaxSeqs)
    return SPA_ERR_INVALID;
  if (n_q_heads < 1 || n_q_heads > kMaxHeads || n_kv_heads < 1 || n_q_heads % n_kv_heads) return SPA_ERR_INVALID;
  if (!valid_head_dim(head_dim) || !valid_scale(scale)) return SPA_ERR_INVALID;
  const bool built = dtype != SPA_F32 && built_head_dim(head_dim);
  if (tq == 0 || n_seqs == 0) return built ? SPA_OK : SPA_ERR_UNSUPPORTED;
  if (!valid_heads(q) || !valid_strides(q) || !cu_q || !cu_k || !out || !aligned16(out)) return SPA_ERR_INVALID;
  if (tk > 0 && (!valid_heads(k) || !valid_heads(v) || !valid_strides(k) || !valid_strides(v))) return SPA_ERR_INVALID;
  if (!built || !built_heads(q)) return SPA_ERR_UNSUPPORTED;
  if (tk > 0 && (!built_heads(k) || !built_heads(v))) return SPA_ERR_UNSUPPORTED;
  if (((int64_t)tq / 128 + n_seqs) * n_q_heads > (int64_t(1) << 23)) return SPA_ERR_UNSUPPORTED;   // workgroups
  return SPA_OK;
}

// Pieces that the keys of a tile of 128 query rows are divided into when the call's tiles alone leave most of the
// chip idle: up to 8, and no more than fill two workgroups on each of 256 compute units.  The number of tiles is
// estimated (every sequence ends with half a tile); sequences' keys stay on the device, where a piece is at least 4
// key steps, so a call whose keys altogether are no more than that is not divided.  Of those the number is taken that
// ends soonest by what was measured: a tile walks its keys at 400 + 6 head_dim ns per 64, whether one workgroup or
// two stand on its unit (the longest of n sequences is taken as 2n / (n + 1) times their mean, which is too short for one
// long sequence among many short ones: such a call is divided little or not at all); a join costs 5 us, and each piece
// 4 bytes per output element written and read at 4 TB/s.  Against pieces up to two workgroups on each unit
// (us): a prompt of 700 by 32 heads of 128 26.4 -> 18.7, six of up to 300 by 16 19.2 -> 12.3, four of 300 18.3 ->
// 12.4; worst 2000 by 8 heads 29.6 -> 31.5.  One workgroup to a unit takes 75 us for 4000 by 8 heads, this 59.
constexpr int kPrefillTarget = 512, kMaxSplits = 8;
inline int prefill_splits(int tq, int tk, int n_seqs, int n_q_heads, int head_dim) {
  const int64_t groups = ((int64_t)tq / 128 + (n_seqs + 1) / 2) * n_q_heads;
  int64_t most = kPrefillTarget / (groups > 0 ? groups : 1);
  most = most < tk / 256 ? most : tk / 256;
  most = most < kMaxSplits ? most : kMaxSplits;
  const double longest = 2.0 * tk / (n_seqs + 1);
  const double walk = longest / 64 * (400 + 6 * head_dim);      // ns
  const double piece = double(tq) * n_q_heads * head_dim * 8 / 4000;
  int best = 1;
  double least = walk;
  for (int s = 2; s <= most; ++s) {
    const double t = walk / s + 5000 + piece * s;
    if (t < least) {
      least = t;
      best = s;
    }
  }
  return best;
}
struct PrefillAttnPlan {
  int splits;
  size_t o, ml, bytes;    // [splits][tq][heads][head_dim] float32 partial outputs, [splits][tq][heads][2] maximum and sum
};
inline PrefillAttnPlan prefill_attn_plan(int tq, int tk, int n_seqs, int n_q_heads, int head_dim) {
  PrefillAttnPlan p{};
  p.splits = prefill_splits(tq, tk, n_seqs, n_q_heads, head_dim);
  if (p.splits == 1) return p;
  const size_t rows = (size_t)p.splits * tq * n_q_heads;
  p.ml = round256(rows * head_dim * 4);
  p.bytes = p.ml + round256(rows * 8);
  return p;
}

// ---- norms ----
inline bool valid_norm(const spa_norm* n) {
  return !n || (n->kind >= SPA_NORM_NONE && n->kind <= SPA_NORM_LAYER);
}
inline spa_status check_norm(const void* x, int32_t dtype, int32_t t, int32_t c, const void* residual,
                             int32_t stream_dtype, const spa_norm* post, const void* gate, int32_t gate_rows,
                             float scale, const spa_norm* pre, float eps, const void* h, const void* y) {
  if (!valid_dtype(dtype) || !valid_dtype(stream_dtype) || t < 0 || t > kMaxRows || c < 1 || c > kMaxDim)
    return SPA_ERR_INVALID;
  if (!valid_norm(post) || !valid_norm(pre) || !(eps >= 0.f && eps <= 1e30f)) return SPA_ERR_INVALID;
  if (!(scale >= -1e30f && scale <= 1e30f)) return SPA_ERR_INVALID;
  if (gate_rows != 0 && gate_rows != 1 && gate_rows != t) return SPA_ERR_INVALID;
  if (t == 0) return SPA_OK;
  if ((gate_rows != 0) != (gate != nullptr)) return SPA_ERR_INVALID;
  if (!x || (!h && !y) || h == y) return SPA_ERR_INVALID;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(gate) || !aligned16(h) || !aligned16(y)) return SPA_ERR_INVALID;
  for (const spa_norm* n : {post, pre})
    if (n && (!aligned16(n->weight) || !aligned16(n->bias))) return SPA_ERR_INVALID;
  // the residual stream is in the block's type or in float32
  if (stream_dtype != dtype && stream_dtype != SPA_F32) return SPA_ERR_UNSUPPORTED;
  return c <= kMaxNormC ? SPA_OK : SPA_ERR_UNSUPPORTED;
}

}  // namespace spa_check
