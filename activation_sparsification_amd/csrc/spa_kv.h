// A vector's way into the paged cache (device code shared by the calls that write one).
#pragma once

#include "spa_common.h"

namespace spa {

// 4-byte words of 8 elements as stored.
template <int FMT> constexpr int kWords = FMT == SPA_KV_NATIVE ? 4 : FMT == SPA_KV_MXFP4 ? 1 : 2;

template <int LG>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
#pragma unroll
  for (int off = LG / 2; off >= 1; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, kWave));
  return v;
}

// Codes of 8 values and their vector's scale: the definition's float32 operations in its order.  The largest magnitude
// is found on the bit patterns, which order like the numbers with infinity and NaN at the top: no such value is passed
// over.
template <int FMT, int LG>
__device__ __forceinline__ uint2 quantise(const float (&x)[8], float& scale) {
#pragma clang fp contract(off)
  constexpr float top = FMT == SPA_KV_FP8 ? 448.f : 127.f;
  uint32_t bits = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) bits = max(bits, __float_as_uint(x[e]) & 0x7FFFFFFFu);
  const float a = __uint_as_float(group_max<LG>(bits));
  const bool finite = a < INFINITY, live = finite && a >= 0x1p-100f;
  scale = live ? __fdiv_rn(a, top) : finite ? 0.f : NAN;
  const float inv = live ? __fdiv_rn(top, a) : 0.f;
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = finite ? x[4 * h + e] * inv : 0.f;
    if constexpr (FMT == SPA_KV_FP8) {
      w[h] = fp8_pair(q[0], q[1]) | (fp8_pair(q[2], q[3]) << 16);
    } else {
      w[h] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[h] |= ((uint32_t)(int)rintf(q[e]) & 0xFFu) << (8 * e);
    }
  }
  return make_uint2(w[0], w[1]);
}

// Codes of 8 of 32 elements that four lanes hold, and the exponent byte of the 32: from the largest magnitude's own exponent
// field E and significand, 2^(E - 129), or twice that where the significand is above 1.75 (the magnitude above 7 * 2^(E - 129)).
// The conversion divides by the scale and rounds once, to nearest even, 6 at the most.
template <int DT>
__device__ __forceinline__ uint32_t quantise_mx(const float (&x)[8], uint32_t& scale) {
  uint32_t a = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) a = max(a, __float_as_uint(x[e]) & 0x7FFFFFFFu);
  a = group_max<4>(a);
  const bool finite = a < 0x7F800000u, live = finite && __uint_as_float(a) >= 0x1p-100f;
  constexpr uint32_t kTop = 127 + (DT == SPA_F16 ? 13 : 125);
  scale = live ? min((a >> 23) - 2 + ((a & 0x7FFFFFu) > 0x600000u), kTop) : finite ? 0u : 255u;
  const float unit = __uint_as_float(scale << 23);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], unit, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], unit, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], unit, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], unit, 3);
  return live ? w : 0u;
}

// Stores one vector at place `off` of page and head `block`: lane i of the LG that hold it has the elements 8 i .. 8 i + 7 in
// raw.  Every lane of the vector calls this; live: the place exists and the lane's elements are within head_dim.
template <int DT, int FMT, int LG>
__device__ __forceinline__ void store_vector(void* pages, void* scales, size_t block, int off, int page_size, int d, int lane,
                                             bool live, const uint4& raw) {
  const size_t cell = block * page_size + off;
  if constexpr (FMT == SPA_KV_NATIVE) {
    if (live) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(pages) + cell * d + lane * 8) = raw;
  } else {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = elem16<DT>(raw, e);
    if constexpr (FMT == SPA_KV_MXFP4) {
      uint32_t scale;
      const uint32_t codes = quantise_mx<DT>(x, scale);
      if (live) static_cast<uint32_t*>(pages)[cell * (d / 8) + lane] = codes;
      if (live && lane % 4 == 0)
        static_cast<uint8_t*>(scales)[(block * ((d + 31) / 32) + lane / 4) * page_size + off] = (uint8_t)scale;
    } else {
      float scale;
      const uint2 codes = quantise<FMT, LG>(x, scale);
      if (live) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pages) + cell * d + lane * 8) = codes;
      if (live && lane == 0) static_cast<float*>(scales)[cell] = scale;
    }
  }
}

}  // namespace spa
