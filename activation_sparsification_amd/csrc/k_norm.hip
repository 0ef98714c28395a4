// Norms after one block and before the next, with the block's gate and residual scale:
//   u = N_post(x),  h = residual + scale * gate * u,  y = N_pre(h).
//
// Bound by HBM for many rows, by latency for one.  A workgroup holds a row in registers from its one read to its
// one write, so the traffic is the inputs once and the outputs once; it walks over rows with the next row's loads
// in flight while this one is reduced, and keeps the weights.  Sums go DPP adds -> LDS -> every thread.  The layer
// norm's variance is taken about the mean in a second pass over the registers (no cancellation).
//
// 4096 x 4096 float16, layer norms and a gate for each token: 36 us, 4.7 TB/s (51 us with one workgroup to a row); one
// bfloat16 token of 4096: 3 us.
#include <algorithm>

#include "spa_common.h"
#include "spa_layer.h"

namespace spa {

namespace {

// VEC consecutive elements as stored (VEC == 8: 16-byte loads; VEC == 1: any alignment).
template <int DT, int VEC>
struct Stored {
  static constexpr int kBytes = VEC * Dt<DT>::bytes, kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const void* p, size_t i) {
    using T = typename Dt<DT>::T;
    const T* s = static_cast<const T*>(p) + i;
    if constexpr (VEC == 1) {
      if constexpr (DT == SPA_F32) w[0] = __float_as_uint(s[0]);
      else w[0] = s[0];
    } else {
#pragma unroll
      for (int k = 0; k < kWords; k += 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(s) + 4 * k);
        w[k] = v.x; w[k + 1] = v.y; w[k + 2] = v.z; w[k + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ float at(int e) const {
    if constexpr (DT == SPA_F32) return __uint_as_float(w[e]);
    else {
      const uint32_t h = e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xFFFFu;
      return DT == SPA_BF16 ? bf16_to_f32(h) : f16_to_f32(h);
    }
  }
};
template <int DT, int VEC>
__device__ __forceinline__ void store_vec(void* p, size_t i, const float (&v)[VEC]) {
  using T = typename Dt<DT>::T;
  T* d = static_cast<T*>(p) + i;
  if constexpr (VEC == 1) {
    if constexpr (DT == SPA_F32) d[0] = v[0];
    else d[0] = (uint16_t)pack2<DT>(v[0], 0.f);
  } else if constexpr (DT == SPA_F32) {
    reinterpret_cast<float4*>(d)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(d)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(d) =
        make_uint4(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7]));
  }
}

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ float dpp_f(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, ROW_MASK, 0xF, false));
}
// Sum over the wave in a fixed order, the same on every lane (pairs, quads, 8, 16, then the four rows).
__device__ __forceinline__ float wave_sum_f(float v) {
  v += dpp_f<0xB1, 0xF>(v);
  v += dpp_f<0x4E, 0xF>(v);
  v += dpp_f<0x141, 0xF>(v);
  v += dpp_f<0x140, 0xF>(v);
  v += dpp_f<0x142, 0xA>(v);
  v += dpp_f<0x143, 0xC>(v);
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// Sum over the workgroup, the same on every thread.  Two buffers of 16 floats in turn, so that one barrier per
// sum is enough (a buffer is written again only after the barrier of the sum between).
__device__ __forceinline__ float group_sum(float v, float (&s_buf)[2][16], int& flip) {
  v = wave_sum_f(v);
  const int waves = blockDim.x / kWave;
  if (waves == 1) return v;
  float* s = s_buf[flip];
  flip ^= 1;
  if ((threadIdx.x & (kWave - 1)) == 0) s[threadIdx.x / kWave] = v;
  __syncthreads();
  // every row of 16 lanes adds the waves' sums the same way
  const int w = threadIdx.x & 15;
  v = w < waves ? s[w] : 0.f;
  v += dpp_f<0xB1, 0xF>(v);
  v += dpp_f<0x4E, 0xF>(v);
  v += dpp_f<0x141, 0xF>(v);
  return v + dpp_f<0x140, 0xF>(v);
}

// v <- N(v); elements past the row (live false) hold anything and are not counted.  The weights are in w and b, or,
// with kLate, read here.
template <int DT, int VEC, int U, bool kLate>
__device__ __forceinline__ void norm_row(float (&v)[U][VEC], const bool (&live)[U], const int (&at)[U], const spa_norm& n,
                                         float inv_c, float eps, const Stored<DT, VEC> (&w)[U],
                                         const Stored<DT, VEC> (&b)[U], float (&s_buf)[2][16], int& flip) {
  if (n.kind == SPA_NORM_NONE) return;
  if (n.kind == SPA_NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (live[u])
#pragma unroll
        for (int e = 0; e < VEC; ++e) s += v[u][e];
    const float mean = group_sum(s, s_buf, flip) * inv_c;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[u][e] -= mean;
  }
  float q = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (live[u])
#pragma unroll
      for (int e = 0; e < VEC; ++e) q += v[u][e] * v[u][e];
  const float r = 1.f / sqrtf(group_sum(q, s_buf, flip) * inv_c + eps);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    Stored<DT, VEC> lw = w[u], lb = b[u];
    if constexpr (kLate) {
      if (live[u] && n.weight) lw.load(n.weight, at[u]);
      if (live[u] && n.bias) lb.load(n.bias, at[u]);
    }
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float x = v[u][e] * r;
      if (n.weight) x *= lw.at(e);
      if (n.bias) x += lb.at(e);
      v[u][e] = x;
    }
  }
}

// kAhead: the weights stay in registers and the next row is read while this one is worked on.  Rows that need more
// than 8 elements of a thread have no registers for that; there a workgroup takes one row (up to 2^20 of them) and
// reads the gate and the weights (from L2) where they are used.
template <int DT, int ST, int VEC, int U>
__global__ void __launch_bounds__(1024) k_gated_norm(NormArgs a) {
  constexpr bool kAhead = U * VEC <= 8;
  __shared__ float s_buf[2][16];
  int flip = 0;
  int at[U];
  bool live[U];
  Stored<DT, VEC> pw[U], pb[U], nw[U], nb[U], x[U], gate[U];
  Stored<ST, VEC> res[U];
  auto fetch = [&](int row) {
    const size_t base = (size_t)row * a.c;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!live[u]) continue;
      x[u].load(a.x, base + at[u]);
      if (a.residual) res[u].load(a.residual, base + at[u]);
      if (kAhead && a.gate_per_token) gate[u].load(a.gate, base + at[u]);
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) {
    at[u] = (u * (int)blockDim.x + (int)threadIdx.x) * VEC;
    live[u] = at[u] < a.c;
  }
  int row = blockIdx.x;
  if constexpr (kAhead) {
    fetch(row);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!live[u]) continue;
      if (a.gate && !a.gate_per_token) gate[u].load(a.gate, at[u]);
      if (a.post.weight) pw[u].load(a.post.weight, at[u]);
      if (a.post.bias) pb[u].load(a.post.bias, at[u]);
      if (a.pre.weight) nw[u].load(a.pre.weight, at[u]);
      if (a.pre.bias) nb[u].load(a.pre.bias, at[u]);
    }
  }
  const float inv_c = 1.f / (float)a.c;
  for (; row < a.t; row += gridDim.x) {
    if constexpr (!kAhead) fetch(row);
    const size_t base = (size_t)row * a.c;
    float v[U][VEC];
    Stored<DT, VEC> g[U];
    Stored<ST, VEC> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[u][e] = x[u].at(e);
      r[u] = res[u];
      g[u] = gate[u];
      if (!kAhead && a.gate && live[u]) g[u].load(a.gate, (a.gate_per_token ? base : 0) + at[u]);
    }
    // the rows of this workgroup are its own: the next one is read before this one's outputs are written
    if (kAhead && row + (int)gridDim.x < a.t) fetch(row + gridDim.x);
    norm_row<DT, VEC, U, !kAhead>(v, live, at, a.post, inv_c, a.eps, pw, pb, s_buf, flip);
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float k = a.gate ? a.scale * g[u].at(e) : a.scale;
        v[u][e] = (a.residual ? r[u].at(e) : 0.f) + k * v[u][e];
      }
      if (a.h && live[u]) store_vec<ST, VEC>(a.h, base + at[u], v[u]);
    }
    if (!a.y) continue;
    norm_row<DT, VEC, U, !kAhead>(v, live, at, a.pre, inv_c, a.eps, nw, nb, s_buf, flip);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (live[u]) store_vec<DT, VEC>(a.y, base + at[u], v[u]);
  }
}

constexpr int kUnits = 256;              // compute units
constexpr int kResident = 1024;          // threads of a unit that walk over rows

template <int DT, int ST, int VEC, int U>
hipError_t go(const NormArgs& a, hipStream_t st) {
  const int per = VEC * U;
  const int threads = ((a.c + per - 1) / per + kWave - 1) / kWave * kWave;
  // one workgroup to a row, or as many as the chip holds where they walk over rows
  const int places = U * VEC <= 8 ? kUnits * std::max(1, kResident / threads) : 1 << 20;
  hipLaunchKernelGGL((k_gated_norm<DT, ST, VEC, U>), dim3(std::min(a.t, places)), dim3(threads), 0, st, a);
  return hipGetLastError();
}

template <int DT, int ST>
hipError_t pick(const NormArgs& a, hipStream_t st) {
  if (a.c % 8 == 0) {
    if (a.c <= 8192) return go<DT, ST, 8, 1>(a, st);
    if (a.c <= 16384) return go<DT, ST, 8, 2>(a, st);
    if (a.c <= 32768) return go<DT, ST, 8, 4>(a, st);
    return go<DT, ST, 8, 8>(a, st);
  }
  if (a.c <= 4096) return go<DT, ST, 1, 4>(a, st);
  if (a.c <= 16384) return go<DT, ST, 1, 16>(a, st);
  return go<DT, ST, 1, 64>(a, st);
}

}  // namespace

hipError_t launch_norm(int dtype, int stream_dtype, const NormArgs& a, hipStream_t st) {
  if (dtype == SPA_F32) return pick<SPA_F32, SPA_F32>(a, st);
  if (dtype == SPA_F16) return stream_dtype == SPA_F32 ? pick<SPA_F16, SPA_F32>(a, st) : pick<SPA_F16, SPA_F16>(a, st);
  return stream_dtype == SPA_F32 ? pick<SPA_BF16, SPA_F32>(a, st) : pick<SPA_BF16, SPA_BF16>(a, st);
}

}  // namespace spa
