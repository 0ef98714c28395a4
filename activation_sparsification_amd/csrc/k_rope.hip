// Norm of each query and key head and its rotation by position in one pass, with the keys and values of a call put into the
// paged cache on the way:
//   u = N(x) over the head's d elements;  y_a = u_a cos - u_b sin,  y_b = u_a sin + u_b cos  for the pairs (a, b) of the first
//   r elements, at the angle position * inv_freq[i] of pair i;  the others are y = u.
//
// Bound by HBM for many rows, by latency for few.  A head is held by LG lanes, 8 elements each, taken so that both elements of
// a pair are in one lane: two runs of 4 elements, 4 i and r / 2 + 4 i (neighbours: 8 i and 8 i + 4).  Every byte moves once.
// Angles are turns: position * (inv_freq / 2 pi) in float64 keeps 2^-22 of a turn at any 32-bit position, where float32 would
// keep none at far ones; the whole turns go, and the sine and cosine of the rest are float32.  A workgroup forms them once for
// its tokens, in LDS, while its first rows are on their way.
#include <algorithm>

#include "spa_attn.h"
#include "spa_kv.h"
#include "spa_layer.h"

namespace spa {

namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 4;           // of a workgroup at the most
constexpr int kMaxPairs = 128;       // of a head of 256
constexpr int kNone = -1;            // no cache
constexpr int kAhead = 4;            // rows of a lane group in flight

struct RopeKernelArgs {
  RopeArgs a;
  FastDiv per;                       // heads of this workgroup's range
  int tokens;                        // of a workgroup
  int biased[2], to_keys;            // whether there are biases, and whether the keys go anywhere but the cache
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

// A lane's 8 elements: the first elements of its four pairs, then the second ones.
struct Eight {
  uint2 a, b;
  __device__ __forceinline__ void load(const uint16_t* p, int c0, int c1) {
    a = *reinterpret_cast<const uint2*>(p + c0);
    b = *reinterpret_cast<const uint2*>(p + c1);
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

// A kernel argument in a register of its own.  Where lanes choose between two arguments by the kind of head, the compiler
// otherwise reads the chosen one from memory for each lane, a trip to memory ahead of every load and store.
template <typename T>
__device__ __forceinline__ T held(T v) {
  asm volatile("" : "+s"(v));
  return v;
}

// One of three by the kind of head: queries, keys, values.
template <int FMT, typename T>
__device__ __forceinline__ T of_kind(bool key, bool value, T q, T k, T v) {
  const T x = key ? k : q;
  return FMT != kNone && value ? v : x;
}

template <int DT, int FMT, int LG>
__global__ void __launch_bounds__(kThreads) k_qk_norm_rope(RopeKernelArgs ka) {
  constexpr int kGroups = kThreads / LG;
  const RopeArgs& a = ka.a;
  __shared__ float2 s_turn[kTokens][kMaxPairs];
  __shared__ int s_slot[kTokens];
  constexpr bool kCodes = FMT != kNone && FMT != SPA_KV_NATIVE;
  __shared__ uint4 s_vec[kCodes ? kThreads : 1];
  const int lane = threadIdx.x % LG, group = threadIdx.x / LG;
  const int first = blockIdx.x * ka.tokens, tokens = min(ka.tokens, a.t - first);
  const int heads = (int)ka.per.d, h0 = blockIdx.y * heads;
  const int n_heads = a.hq + a.hkv * (FMT == kNone ? 1 : 2);   // queries, keys and, with a cache, values
  const int items = tokens * heads;
  const bool in_head = lane * 8 < a.d, turns = lane * 8 < a.rot;
  const int c0 = a.neighbours || !turns ? 8 * lane : 4 * lane, c1 = a.neighbours || !turns ? c0 + 4 : a.rot / 2 + 4 * lane;
  const uint16_t* src[3];
  uint16_t* dst[2];
  uint32_t row[3], step[3], drow[2], dstep[2];         // between rows and between heads
  int norm[2], biased[2];
  void *cells[2], *scales[2];
  const int to_keys = held(ka.to_keys);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    src[i] = held(a.src[i] + (size_t)first * a.row[i]);
    row[i] = held((uint32_t)a.row[i]);
    step[i] = held((uint32_t)a.head[i]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    dst[i] = held(a.dst[i] + (size_t)first * a.drow[i]);
    drow[i] = held((uint32_t)a.drow[i]);
    dstep[i] = held((uint32_t)a.dhead[i]);
    norm[i] = held(a.norm[i].kind);
    biased[i] = held(ka.biased[i]);
    cells[i] = held(a.pages[i]);
    scales[i] = held(a.scale[i]);
  }

  // item i: one head of one token
  struct Item { int tok, head; bool key, value, there; };
  auto find = [&](int i) {
    Item m;
    m.tok = (int)ka.per.div((uint32_t)i);
    m.head = h0 + i - m.tok * heads;
    m.there = i < items && m.head < n_heads;
    m.value = FMT != kNone && m.head >= a.hq + a.hkv;
    m.key = m.head >= a.hq && !m.value;
    m.head -= of_kind<FMT>(m.key, m.value, 0, a.hq, a.hq + a.hkv);
    return m;
  };
  auto load = [&](int i, Eight& x) {
    const Item m = find(i);
    x.a = x.b = make_uint2(0, 0);
    if (!m.there || !in_head) return;
    const uint16_t* p = of_kind<FMT>(m.key, m.value, src[0], src[1], src[2]);
    const uint32_t r = of_kind<FMT>(m.key, m.value, row[0], row[1], row[2]);
    const uint32_t h = of_kind<FMT>(m.key, m.value, step[0], step[1], step[2]);
    x.load(p + ((uint64_t)(uint32_t)m.tok * r + (uint64_t)(uint32_t)m.head * h), c0, c1);
  };

  Eight x[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) load(group + u * kGroups, x[u]);
  // each lane's weights of queries and keys, and their biases
  float w[2][8];
  Eight b[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[s][e] = 1.f;
    if (!in_head) continue;
    if (a.norm[s].weight) {
      Eight raw;
      raw.load(static_cast<const uint16_t*>(a.norm[s].weight), c0, c1);
      raw.pair_up(a.neighbours);
      raw.template to_f32<DT>(w[s]);
    }
    if (a.norm[s].bias) b[s].load(static_cast<const uint16_t*>(a.norm[s].bias), c0, c1);
    b[s].pair_up(a.neighbours);
  }
  const int pairs = a.rot / 2;
  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int tok = i / pairs, f = i - tok * pairs;
    const double turn = (double)a.pos[first + tok] * ((double)a.freq[f] * 0.15915494309189535);
    float sn, cs;
    sincospif((float)(2.0 * (turn - rint(turn))), &sn, &cs);
    s_turn[tok][f] = make_float2(cs, sn);
  }
  if (FMT != kNone && (int)threadIdx.x < tokens) s_slot[threadIdx.x] = a.slots[first + threadIdx.x];
  __syncthreads();

  const float inv_d = 1.f / (float)a.d;
  for (int base = group; base < items; base += kAhead * kGroups) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const Item m = find(base + u * kGroups);
      Eight y = x[u];
      load(base + (u + kAhead) * kGroups, x[u]);
      if (!m.there) continue;                                  // the whole group
      if (!m.value) {
        y.pair_up(a.neighbours);
        float v[8];
        y.to_f32<DT>(v);
        const int kind = m.key ? norm[1] : norm[0];
        if (kind != SPA_NORM_NONE) {
          if (kind == SPA_NORM_LAYER) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += v[e];             // lanes past the head hold zeros
            const float mean = group_sum<LG>(s) * inv_d;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] -= in_head ? mean : 0.f;
          }
          float q = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) q += v[e] * v[e];
          const float r = rsqrtf(group_sum<LG>(q) * inv_d + a.eps);
          if (m.key) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = v[e] * r * w[1][e];
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = v[e] * r * w[0][e];
          }
          if (m.key ? biased[1] : biased[0]) {
            float k[8];
            (m.key ? b[1] : b[0]).template to_f32<DT>(k);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += k[e];
          }
        }
        if (turns) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 cs = s_turn[m.tok][4 * lane + e];
            const float p = v[e], o = v[4 + e];
            v[e] = p * cs.x - o * cs.y;
            v[4 + e] = p * cs.y + o * cs.x;
          }
        }
        y.a = make_uint2(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]));
        y.b = make_uint2(pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7]));
        y.take_apart(a.neighbours);
        if ((FMT == kNone || !m.key || to_keys) && in_head) {
          const uint32_t r = m.key ? drow[1] : drow[0], h = m.key ? dstep[1] : dstep[0];
          uint16_t* to = (m.key ? dst[1] : dst[0]) + ((uint64_t)(uint32_t)m.tok * r + (uint64_t)(uint32_t)m.head * h);
          *reinterpret_cast<uint2*>(to + c0) = y.a;
          *reinterpret_cast<uint2*>(to + c1) = y.b;
        }
      }
      if constexpr (FMT != kNone) {
        if (!m.key && !m.value) continue;
        void* pages = m.value ? cells[1] : cells[0];
        const int slot = s_slot[m.tok], page_size = (int)a.page.d;
        const int pg = slot >= 0 ? (int)a.page.div((uint32_t)slot) : a.n_pages;
        const bool there = slot >= 0 && pg < a.n_pages && in_head;
        const size_t block = (size_t)pg * a.hkv + m.head;
        const int off = slot - pg * page_size;
        if constexpr (kCodes) {
          // 8 consecutive elements to a lane, for the scales
          uint2* mine = reinterpret_cast<uint2*>(s_vec + group * LG);
          if (in_head) mine[c0 / 4] = y.a, mine[c1 / 4] = y.b;
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
          __builtin_amdgcn_wave_barrier();
          __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
          const uint4 raw = in_head ? s_vec[group * LG + lane] : make_uint4(0, 0, 0, 0);
          __builtin_amdgcn_wave_barrier();
          store_vector<DT, FMT, LG>(pages, m.value ? scales[1] : scales[0], block, off, page_size, a.d, lane, there, raw);
        } else if (there) {
          uint16_t* to = static_cast<uint16_t*>(pages) + (block * page_size + off) * a.d;
          *reinterpret_cast<uint2*>(to + c0) = y.a;
          *reinterpret_cast<uint2*>(to + c1) = y.b;
        }
      }
    }
  }
}

template <int DT, int FMT, int LG>
hipError_t go(const RopeArgs& a, hipStream_t st) {
  constexpr int kGroups = kThreads / LG;
  const int heads = a.hq + a.hkv * (FMT == kNone ? 1 : 2);
  // few tokens: every group takes one head; many: a workgroup takes all heads of up to kTokens tokens
  const bool few = a.t <= 256;
  const int per = few ? std::min(heads, kGroups) : heads;
  const int tokens = few ? 1 : kTokens;
  const RopeKernelArgs ka{a, FastDiv((uint32_t)per), tokens, {a.norm[0].bias != nullptr, a.norm[1].bias != nullptr},
                          a.dst[1] != nullptr};
  const dim3 grid((a.t + tokens - 1) / tokens, (heads + per - 1) / per);
  hipLaunchKernelGGL((k_qk_norm_rope<DT, FMT, LG>), grid, dim3(kThreads), 0, st, ka);
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
