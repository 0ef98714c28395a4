// Norms after one block and before the next, with the block's gate and residual scale:
//   u = N_post(x),  h = residual + scale * gate * u,  y = N_pre(h).
//
// One workgroup per row.  The row stays in registers as float32 from its one read to its one write, so the
// HBM traffic is the inputs once and the outputs once; the reductions go wave butterfly -> LDS -> every thread.
// The layer norm's variance is taken about the mean in a second pass over the registers (no cancellation).
// Every load of the row, its residual, gate and weights is issued before the first reduction.
#include "spa_common.h"
#include "spa_layer.h"

namespace spa {

namespace {

// VEC consecutive elements of DT at index i (VEC == 8: 16-byte loads; VEC == 1: any alignment).
template <int DT, int VEC>
__device__ __forceinline__ void load_vec(const void* p, size_t i, float (&out)[VEC]) {
  using T = typename Dt<DT>::T;
  const T* s = static_cast<const T*>(p) + i;
  if constexpr (VEC == 1) {
    out[0] = to_f32<DT>(s[0]);
  } else if constexpr (DT == SPA_F32) {
    const float4 a = reinterpret_cast<const float4*>(s)[0], b = reinterpret_cast<const float4*>(s)[1];
    out[0] = a.x; out[1] = a.y; out[2] = a.z; out[3] = a.w;
    out[4] = b.x; out[5] = b.y; out[6] = b.z; out[7] = b.w;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(s);
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = elem16<DT>(v, e);
  }
}
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

// Sum over the workgroup, the same bits on every thread.  s_tmp: 16 floats; `flip` alternates the halves of a
// 32-float buffer so that one barrier per reduction is enough.
__device__ __forceinline__ float group_sum(float v, float* s_buf, int& flip) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, kWave);
  const int waves = blockDim.x / kWave;
  if (waves == 1) return v;
  float* s = s_buf + 16 * flip;
  flip ^= 1;
  if ((threadIdx.x & (kWave - 1)) == 0) s[threadIdx.x / kWave] = v;
  __syncthreads();
  float total = 0.f;
  for (int w = 0; w < waves; ++w) total += s[w];
  return total;
}

// v[U][VEC] <- N(v); elements past the row (live[u] false) hold anything and are not counted.
template <int DT, int VEC, int U>
__device__ __forceinline__ void norm_row(float (&v)[U][VEC], const bool (&live)[U], const spa_norm& n, int c, float eps,
                                         const float (&w)[U][VEC], const float (&b)[U][VEC], float* s_buf, int& flip) {
  if (n.kind == SPA_NORM_NONE) return;
  const float inv_c = 1.f / (float)c;
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
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[u][e] = v[u][e] * r * w[u][e] + b[u][e];
}

template <int DT, int ST, int VEC, int U>
__global__ void __launch_bounds__(1024) k_gated_norm(NormArgs a) {
  __shared__ float s_buf[32];
  const size_t row = (size_t)blockIdx.x * a.c;
  int flip = 0;
  float v[U][VEC], res[U][VEC], gate[U][VEC], pw[U][VEC], pb[U][VEC], nw[U][VEC], nb[U][VEC];
  bool live[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = (u * (int)blockDim.x + (int)threadIdx.x) * VEC;
    live[u] = i < a.c;
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[u][e] = res[u][e] = pb[u][e] = nb[u][e] = 0.f, gate[u][e] = pw[u][e] = nw[u][e] = 1.f;
    if (!live[u]) continue;
    load_vec<DT, VEC>(a.x, row + i, v[u]);
    if (a.residual) load_vec<ST, VEC>(a.residual, row + i, res[u]);
    if (a.gate) load_vec<DT, VEC>(a.gate, (a.gate_per_token ? row : 0) + i, gate[u]);
    if (a.post.weight) load_vec<DT, VEC>(a.post.weight, i, pw[u]);
    if (a.post.bias) load_vec<DT, VEC>(a.post.bias, i, pb[u]);
    if (a.pre.weight) load_vec<DT, VEC>(a.pre.weight, i, nw[u]);
    if (a.pre.bias) load_vec<DT, VEC>(a.pre.bias, i, nb[u]);
  }
  norm_row<DT, VEC, U>(v, live, a.post, a.c, a.eps, pw, pb, s_buf, flip);
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[u][e] = res[u][e] + a.scale * (gate[u][e] * v[u][e]);
    if (a.h && live[u]) store_vec<ST, VEC>(a.h, row + (u * (int)blockDim.x + (int)threadIdx.x) * VEC, v[u]);
  }
  if (!a.y) return;
  norm_row<DT, VEC, U>(v, live, a.pre, a.c, a.eps, nw, nb, s_buf, flip);
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (live[u]) store_vec<DT, VEC>(a.y, row + (u * (int)blockDim.x + (int)threadIdx.x) * VEC, v[u]);
}

template <int DT, int ST, int VEC, int U>
hipError_t go(const NormArgs& a, hipStream_t st) {
  const int per = VEC * U;
  const int threads = ((a.c + per - 1) / per + kWave - 1) / kWave * kWave;
  hipLaunchKernelGGL((k_gated_norm<DT, ST, VEC, U>), dim3(a.t), dim3(threads), 0, st, a);
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
