// Norm of each query and key head and its rotation by position in one pass, with the keys and values of a call put into the
// paged cache on the way:
//   u = N(x) over the head's d elements;  y_a = u_a cos - u_b sin,  y_b = u_a sin + u_b cos  for the pairs (a, b) of the first
//   r elements, at the angle position * inv_freq[i] of pair i;  the others are y = u.
//
// Bound by HBM for many rows, by latency for few.  A head is held by LG lanes, 8 elements each, taken so that both elements of
// a pair are in one lane: two runs of 4 elements, 4 i and r / 2 + 4 i (neighbours: 8 i and 8 i + 4).  Every byte moves once.
// Angles are turns: position * (inv_freq / 2 pi) in float64 is off by at most 2^-51 of itself, 2^-22 of a turn at any 32-bit
// position and frequency of one, where float32 would keep none at far ones; the whole turns go, and the sine and cosine of the
// rest are float32.  A workgroup forms them once for its tokens, in LDS, while its first rows are on their way.  8191 tokens of
// 32 + 8 heads of 128: 31 to 32 us a call among others, 5.3 TB/s, where a copy of as many bytes takes 29.7; 48 of them, with the
// values into the cache, 3.6 us on the GPU.
#include <algorithm>

#include "spa_attn.h"
#include "spa_kv.h"
#include "spa_layer.h"

namespace spa {

namespace {

constexpr int kThreads = 256;
// Up to kFewTokens a workgroup takes one token and as many heads as it has lane groups, above them kTokens tokens and all heads.
// 32 + 8 heads of 128, one token to a workgroup and two: 5.1 and 6.0 us for 300 tokens, 6.8 and 7.1 for 600 (into the cache), 7.5
// and 7.2 for 1000, 14.1 and 10.6 for 2000 (into the cache).  Four and eight tokens: 9.1 and 13.4 us for 1000, 14.8 (two: 15.7)
// and 17.9 for 4000, 31.3 (30.7) and 31.7 for 8191.
constexpr int kFewTokens = 768;
constexpr int kTokens = 2;
constexpr int kNone = -1;            // no cache

struct RopeKernelArgs {
  RopeArgs a;
  int heads;                         // of a workgroup
  int rows;                          // that many times TOK tokens to a workgroup, side by side
};

// Sum over the LG lanes that hold a vector, on each of them.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
}
template <int LG>
__device__ __forceinline__ float group_sum(float v) {
  v = dpp_add<0xB1>(v);                            // quad_perm [1,0,3,2]
  v = dpp_add<0x4E>(v);                            // quad_perm [2,3,0,1]
  if constexpr (LG >= 8) v = dpp_add<0x141>(v);    // row_half_mirror
  if constexpr (LG >= 16) v = dpp_add<0x140>(v);   // row_mirror
  if constexpr (LG >= 32) v += __shfl_xor(v, 16, kWave);
  return v;
}

// Two words of two 16-bit values each, sorted by even and odd place, and back.
__device__ __forceinline__ uint32_t evens(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ __forceinline__ uint32_t odds(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// What lanes choose by the kind of their head, from values: a choice between variables, or kernel arguments, would be one of
// addresses, and a trip to memory for each lane ahead of every load and store.
template <typename T>
__device__ __forceinline__ T pick(bool key, T q, T k) { return key ? k : q; }
template <typename T>
__device__ __forceinline__ T pick(bool key, bool value, T q, T k, T v) { return value ? v : key ? k : q; }
// Pointers are chosen as numbers, and are global memory's where they are used.
__device__ __forceinline__ uint64_t address(const void* p) { return reinterpret_cast<uint64_t>(p); }
__device__ __forceinline__ void* global(uint64_t at) { return (void*)reinterpret_cast<__attribute__((address_space(1))) char*>(at); }
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(1))) u32x2 global_u32x2;

// A lane's 8 elements: the first elements of its four pairs, then the second ones.
struct Eight {
  uint2 a, b;
  // at: the vector's address
  __device__ __forceinline__ void load(uint64_t at, int c0, int c1) {
    const u32x2 x = *reinterpret_cast<const global_u32x2*>(at + 2 * c0), y = *reinterpret_cast<const global_u32x2*>(at + 2 * c1);
    a = make_uint2(x[0], x[1]);
    b = make_uint2(y[0], y[1]);
  }
  template <bool STREAM>
  __device__ __forceinline__ void store(uint64_t at, int c0, int c1) const {
    global_u32x2 *x = reinterpret_cast<global_u32x2*>(at + 2 * c0), *y = reinterpret_cast<global_u32x2*>(at + 2 * c1);
    if constexpr (STREAM) {
      __builtin_nontemporal_store(u32x2{a.x, a.y}, x);
      __builtin_nontemporal_store(u32x2{b.x, b.y}, y);
    } else {
      *x = u32x2{a.x, a.y};
      *y = u32x2{b.x, b.y};
    }
  }
  __device__ __forceinline__ void pair_up(int neighbours) {
    if (!neighbours) return;
    const uint2 x = a, y = b;
    a = make_uint2(evens(x.x, x.y), evens(y.x, y.y));
    b = make_uint2(odds(x.x, x.y), odds(y.x, y.y));
  }
  __device__ __forceinline__ void take_apart(int neighbours) {
    if (!neighbours) return;
    const uint2 x = a, y = b;
    a = make_uint2(evens(x.x, y.x), odds(x.x, y.x));
    b = make_uint2(evens(x.y, y.y), odds(x.y, y.y));
  }
  template <int DT>
  __device__ __forceinline__ void to_f32(float (&v)[8]) const {
    const uint4 w = make_uint4(a.x, a.y, b.x, b.y);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = elem16<DT>(w, e);
  }
};

// SIDE: the heads fill no more than half of the groups, and several rows of TOK tokens stand side by side (33229 tokens of 8 + 1
// heads of 64 into the cache 29.7 -> 22.4 us).
// A lane group takes one head of TOK tokens at a time, then the next head that is the workgroup's groups further on: kind,
// weights and addresses are found once for the TOK rows, whose loads are all in flight, and the next head's replace them as they
// are worked on.
template <int DT, int FMT, int LG, int TOK, bool SIDE>
__global__ void __launch_bounds__(kThreads) k_qk_norm_rope(RopeKernelArgs ka) {
  constexpr int kGroups = kThreads / LG;
  // many rows are written past the caches: 8191 tokens took 32.7 us so and 38.2 with plain stores, four tokens to a workgroup
  constexpr bool kStream = TOK > 1;
  const RopeArgs& a = ka.a;
  // a token has two heads at the least, a head 4 LG pairs at the most
  constexpr int kMost = SIDE ? TOK * kGroups / 2 : TOK;
  __shared__ float2 s_turn[kMost][4 * LG];
  __shared__ int s_slot[kMost];
  constexpr bool kCodes = FMT != kNone && FMT != SPA_KV_NATIVE;
  __shared__ uint4 s_vec[kCodes ? kThreads : 1];
  const int lane = threadIdx.x % LG, group = threadIdx.x / LG;
  const int all = SIDE ? ka.rows * TOK : TOK;
  const int block_first = blockIdx.x * all, block_tokens = min(all, a.t - block_first);
  const int row = SIDE ? group / ka.heads * TOK : 0;    // this group's first token in the workgroup
  const int first = block_first + row, tokens = min(TOK, block_tokens - row);
  const int n_heads = a.hq + a.hkv * (FMT == kNone ? 1 : 2);   // queries, keys and, with a cache, values
  const int end = min((int)(blockIdx.y + 1) * ka.heads, n_heads);
  const bool in_head = lane * 8 < a.d, turns = lane * 8 < a.rot;
  const int c0 = a.neighbours || !turns ? 8 * lane : 4 * lane, c1 = a.neighbours || !turns ? c0 + 4 : a.rot / 2 + 4 * lane;
  // bytes between rows and between heads
  const uint64_t q_from = address(a.src[0]), k_from = address(a.src[1]), v_from = address(a.src[2]);
  const uint32_t q_row = 2 * (uint32_t)a.row[0], k_row = 2 * (uint32_t)a.row[1], v_row = 2 * (uint32_t)a.row[2];
  const uint32_t q_step = 2 * (uint32_t)a.head[0], k_step = 2 * (uint32_t)a.head[1], v_step = 2 * (uint32_t)a.head[2];
  const uint32_t k_first = (uint32_t)a.hq, v_first = (uint32_t)(a.hq + a.hkv);
  auto is_value = [&](int head) { return FMT != kNone && head >= (int)v_first; };
  auto is_key = [&](int head) { return head >= (int)k_first && !is_value(head); };
  auto load = [&](int head, Eight (&x)[TOK]) {
    const bool key = is_key(head), value = is_value(head);
    const uint32_t h = (uint32_t)head - pick(key, value, 0u, k_first, v_first);
    const uint32_t r = pick(key, value, q_row, k_row, v_row), st = pick(key, value, q_step, k_step, v_step);
    uint64_t at = pick(key, value, q_from, k_from, v_from);
    at += (uint64_t)(uint32_t)first * r + (uint64_t)h * st;
#pragma unroll
    for (int u = 0; u < TOK; ++u) {
      x[u].a = x[u].b = make_uint2(0, 0);
      if (head < end && u < tokens && in_head) x[u].load(at, c0, c1);
      at += r;
    }
  };

  // groups past the last row take no head
  int head = SIDE ? row < all ? group % ka.heads : end : (int)blockIdx.y * ka.heads + group;
  Eight x[TOK];
  load(head, x);
  const int pairs = a.rot / 2;
  for (int i = threadIdx.x; i < block_tokens * pairs; i += kThreads) {
    const int tok = i / pairs, f = i - tok * pairs;
    const double turn = (double)a.pos[block_first + tok] * ((double)a.freq[f] * 0.15915494309189535);
    float sn, cs;
    sincospif((float)(2.0 * (turn - rint(turn))), &sn, &cs);
    s_turn[tok][f] = make_float2(cs, sn);
  }
  if (FMT != kNone && (int)threadIdx.x < block_tokens) s_slot[threadIdx.x] = a.slots[block_first + threadIdx.x];
  __syncthreads();

  const int q_kind = a.norm[0].kind, k_kind = a.norm[1].kind;
  const uint64_t q_weight = address(a.norm[0].weight), k_weight = address(a.norm[1].weight);
  const uint64_t q_bias = address(a.norm[0].bias), k_bias = address(a.norm[1].bias);
  const uint64_t q_to = address(a.dst[0]), k_to = address(a.dst[1]);
  const uint32_t q_row_to = 2 * (uint32_t)a.drow[0], k_row_to = 2 * (uint32_t)a.drow[1];
  const uint32_t q_step_to = 2 * (uint32_t)a.dhead[0], k_step_to = 2 * (uint32_t)a.dhead[1];
  const uint64_t k_cells = address(a.pages[0]), v_cells = address(a.pages[1]);
  const uint64_t k_scale = address(a.scale[0]), v_scale = address(a.scale[1]);
  const float inv_d = 1.f / (float)a.d;
  for (; head < end; head += kGroups) {
    const bool key = is_key(head), value = is_value(head);
    const uint32_t h = (uint32_t)head - pick(key, value, 0u, k_first, v_first);
    const int norm = pick(key, value, q_kind, k_kind, (int)SPA_NORM_NONE);
    const uint64_t weight = pick(key, q_weight, k_weight), bias = pick(key, q_bias, k_bias);
    Eight w, b;                                        // the kind's weights and biases
    w.a = w.b = b.a = b.b = make_uint2(0, 0);
    if (in_head && norm != SPA_NORM_NONE) {
      if (weight) w.load(weight, c0, c1);
      if (bias) b.load(bias, c0, c1);
    }
    const uint32_t r_to = pick(key, q_row_to, k_row_to);
    uint64_t to = pick(key, q_to, k_to);
    const bool out = !value && to != 0 && in_head;
    to += (uint64_t)(uint32_t)first * r_to + (uint64_t)h * pick(key, q_step_to, k_step_to);
    Eight y[TOK];
#pragma unroll
    for (int u = 0; u < TOK; ++u) y[u] = x[u];
    load(head + kGroups, x);
    float wf[8], bf[8];
    w.pair_up(a.neighbours);
    b.pair_up(a.neighbours);
    w.to_f32<DT>(wf);
    b.to_f32<DT>(bf);
    if (!weight)
#pragma unroll
      for (int e = 0; e < 8; ++e) wf[e] = 1.f;
#pragma unroll
    for (int u = 0; u < TOK; ++u) {
      if (u >= tokens) break;
      if (!value) {
        y[u].pair_up(a.neighbours);
        float v[8];
        y[u].template to_f32<DT>(v);
        if (norm != SPA_NORM_NONE) {
          if (norm == SPA_NORM_LAYER) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += v[e];     // lanes past the head hold zeros
            const float mean = group_sum<LG>(s) * inv_d;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] -= in_head ? mean : 0.f;
          }
          float q = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) q += v[e] * v[e];
          const float r = rsqrtf(group_sum<LG>(q) * inv_d + a.eps);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = v[e] * r * wf[e];
          if (bias)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += bf[e];
        }
        if (turns) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 cs = s_turn[row + u][4 * lane + e];
            const float p = v[e], o = v[4 + e];
            v[e] = p * cs.x - o * cs.y;
            v[4 + e] = p * cs.y + o * cs.x;
          }
        }
        y[u].a = make_uint2(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]));
        y[u].b = make_uint2(pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7]));
        y[u].take_apart(a.neighbours);
        if (out) y[u].template store<kStream>(to, c0, c1);
        to += r_to;
      }
      if constexpr (FMT != kNone) {
        if (!key && !value) continue;
        const uint64_t cells = pick(value, k_cells, v_cells);
        const int slot = s_slot[row + u], page_size = (int)a.page.d;
        const int pg = slot >= 0 ? (int)a.page.div((uint32_t)slot) : a.n_pages;
        const bool there = slot >= 0 && pg < a.n_pages && in_head;
        const size_t block = (size_t)pg * (uint32_t)a.hkv + h;
        const int off = slot - pg * page_size;
        if constexpr (kCodes) {
          // 8 consecutive elements to a lane, for the scales
          uint2* mine = reinterpret_cast<uint2*>(s_vec + group * LG);
          if (in_head) mine[c0 / 4] = y[u].a, mine[c1 / 4] = y[u].b;
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
          __builtin_amdgcn_wave_barrier();
          __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
          const uint4 raw = in_head ? s_vec[group * LG + lane] : make_uint4(0, 0, 0, 0);
          __builtin_amdgcn_wave_barrier();
          store_vector<DT, FMT, LG>(global(cells), global(pick(value, k_scale, v_scale)), block, off, page_size, a.d, lane, there, raw);
        } else if (there) {
          y[u].template store<kStream>(cells + 2 * (block * page_size + off) * (uint32_t)a.d, c0, c1);
        }
      }
    }
  }
}

template <int DT, int FMT, int LG>
hipError_t go(const RopeArgs& a, hipStream_t st) {
  constexpr int kGroups = kThreads / LG;
  const int heads = a.hq + a.hkv * (FMT == kNone ? 1 : 2);
  RopeKernelArgs ka{a, heads, 1};
  if (a.t <= kFewTokens) {
    ka.heads = std::min(heads, kGroups);
    const dim3 grid(a.t, (heads + ka.heads - 1) / ka.heads);
    hipLaunchKernelGGL((k_qk_norm_rope<DT, FMT, LG, 1, false>), grid, dim3(kThreads), 0, st, ka);
  } else {
    ka.rows = std::max(kGroups / heads, 1);
    const int tokens = ka.rows * kTokens;
    const dim3 grid((a.t + tokens - 1) / tokens);
    if (ka.rows > 1) hipLaunchKernelGGL((k_qk_norm_rope<DT, FMT, LG, kTokens, true>), grid, dim3(kThreads), 0, st, ka);
    else hipLaunchKernelGGL((k_qk_norm_rope<DT, FMT, LG, kTokens, false>), grid, dim3(kThreads), 0, st, ka);
  }
  return hipGetLastError();
}
template <int DT, int FMT>
hipError_t by_width(const RopeArgs& a, hipStream_t st) {
  if (a.d <= 32) return go<DT, FMT, 4>(a, st);
  if (a.d <= 64) return go<DT, FMT, 8>(a, st);
  if (a.d <= 128) return go<DT, FMT, 16>(a, st);
  return go<DT, FMT, 32>(a, st);
}
template <int DT>
hipError_t by_format(int fmt, const RopeArgs& a, hipStream_t st) {
  if (fmt == kNone) return by_width<DT, kNone>(a, st);
  if (fmt == SPA_KV_NATIVE) return by_width<DT, SPA_KV_NATIVE>(a, st);
  if (fmt == SPA_KV_FP8) return by_width<DT, SPA_KV_FP8>(a, st);
  if (fmt == SPA_KV_MXFP4) return by_width<DT, SPA_KV_MXFP4>(a, st);
  return by_width<DT, SPA_KV_INT8>(a, st);
}

}  // namespace

hipError_t launch_qk_norm_rope(int dtype, const spa_kv_cache* cache, RopeArgs a, hipStream_t st) {
  int fmt = kNone;
  a.page = FastDiv(1u);
  if (cache) {
    fmt = cache->format;
    a.pages[0] = cache->k; a.pages[1] = cache->v;
    a.scale[0] = cache->k_scale; a.scale[1] = cache->v_scale;
    a.n_pages = cache->n_pages;
    a.page = FastDiv((uint32_t)cache->page_size);
  }
  return dtype == SPA_F16 ? by_format<SPA_F16>(fmt, a, st) : by_format<SPA_BF16>(fmt, a, st);
}

}  // namespace spa
