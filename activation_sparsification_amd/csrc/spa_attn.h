// Device helpers shared by the cache and attention kernels (gfx950).
#pragma once

#include "spa_common.h"
#include "spa_div.h"

namespace spa {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Four 8-bit codes as float32.
template <int FMT>
__device__ __forceinline__ void codes_to_f32(uint32_t w, float* out) {
  if constexpr (FMT == SPA_KV_FP8) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    out[0] = lo[0]; out[1] = lo[1]; out[2] = hi[0]; out[3] = hi[1];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = (float)((int)(w << (24 - 8 * e)) >> 24);
  }
}

template <int DT> struct Vec8;
template <> struct Vec8<SPA_BF16> { using T = bf16x8; };
template <> struct Vec8<SPA_F16> { using T = f16x8; };

template <int DT>
__device__ __forceinline__ f32x4 mfma16(const uint4& a, const uint4& b, f32x4 c) {
  using V = typename Vec8<DT>::T;
  if constexpr (DT == SPA_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b), c, 0, 0, 0);
}
template <int DT>
__device__ __forceinline__ f32x16 mfma32(const uint4& a, const uint4& b, f32x16 c) {
  using V = typename Vec8<DT>::T;
  if constexpr (DT == SPA_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b), c, 0, 0, 0);
}

// 2^x and log2 x on the transcendental unit.  The arguments that occur are 0, finite numbers of ordinary size
// and -inf (2^-inf = 0); results below 2^-126 may flush to 0.
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_hw(float x) { return __builtin_amdgcn_logf(x); }
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Inclusive sum over the lanes of a wave, by DPP: shifts within rows of 16, then the rows before.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ int dpp_i(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROW_MASK, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int v) {
  v += dpp_i<0x111, 0xF>(v);   // row_shr 1
  v += dpp_i<0x112, 0xF>(v);   // row_shr 2
  v += dpp_i<0x114, 0xF>(v);   // row_shr 4
  v += dpp_i<0x118, 0xF>(v);   // row_shr 8
  v += dpp_i<0x142, 0xA>(v);   // row_bcast15 -> rows 1, 3
  v += dpp_i<0x143, 0xC>(v);   // row_bcast31 -> rows 2, 3
  return v;
}

// The item with this index when sequence s contributes count(s) of them: its sequence and its number within
// it.  Every wave finds it by itself; seq = n when there is none.
template <typename Count>
__device__ __forceinline__ void locate(int index, int n, Count count, int& seq, int& local) {
  const int lane = threadIdx.x & (kWave - 1);
  int before = 0;
  for (int base = 0; base < n; base += kWave) {
    const int c = base + lane < n ? count(base + lane) : 0;
    const int incl = wave_scan(c) + before;
    const uint64_t past = __ballot(incl > index);
    if (past) {
      const int at = __ffsll((unsigned long long)past) - 1;
      seq = base + at;
      local = index - __shfl(incl - c, at, kWave);
      return;
    }
    before = __shfl(incl, kWave - 1, kWave);
  }
  seq = n;
  local = 0;
}

}  // namespace spa
