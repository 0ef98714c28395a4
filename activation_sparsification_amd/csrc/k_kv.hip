// The paged key-value cache: writing tokens' vectors (quantised on the way for the 8-bit formats) and reading
// the first positions of sequences back as dense rows.
//
// Both move every byte once: a vector of head_dim elements is held by a group of LG lanes, 8 elements each, so
// its largest magnitude is a butterfly over the group and nothing passes through memory twice.  A workgroup
// handles consecutive tokens of one head, keys and values together: consecutive tokens are consecutive positions of
// a page, so the codes and the 4-byte scales of a workgroup are runs.  8191 tokens by 8 heads of 128 into int8 pages:
// 11.5 us, 4.5 TB/s; twelve ragged sequences read back from them: 83 us, 4.7 TB/s (a large copy moves 4.9).
#include "spa_common.h"
#include "spa_attn.h"
#include "spa_layer.h"

namespace spa {

namespace {

constexpr int kThreads = 256;

struct KvArgs {
  const void* src[2];        // write: keys, values
  int64_t row_stride[2], head_stride[2];
  void* pages[2];
  float* scale[2];
  void* out[2];              // read: [total][heads][d]
  const int32_t* slots;      // write: [t]
  const int32_t* table;      // read
  const int32_t* cu;
  int t, heads, d, n_pages, n_seqs, max_pages;
  FastDiv page;
};

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

template <int DT, int FMT, int LG>
__global__ void __launch_bounds__(kThreads) k_kv_write(KvArgs a) {
  constexpr int ROWS = kThreads / LG;
  const int lane = threadIdx.x % LG;
  const int head = blockIdx.x % a.heads;
  const int tok = (blockIdx.x / a.heads) * ROWS + threadIdx.x / LG;
  // the vectors' loads do not wait for the slot: a skipped token's are read for nothing
  uint4 raw[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    raw[s] = make_uint4(0, 0, 0, 0);
    if (tok < a.t && lane * 8 < a.d)
      raw[s] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.src[s]) + (size_t)tok * a.row_stride[s] +
                                               (size_t)head * a.head_stride[s] + lane * 8);
  }
  const int slot = tok < a.t ? a.slots[tok] : -1;
  const int page_size = a.page.d;
  const int pg = slot >= 0 ? (int)a.page.div((uint32_t)slot) : a.n_pages;
  const bool ok = slot >= 0 && pg < a.n_pages;                  // the whole group agrees
  const bool live = ok && lane * 8 < a.d;
  const size_t cell = ((size_t)pg * a.heads + head) * page_size + (slot - pg * page_size);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if constexpr (FMT == SPA_KV_NATIVE) {
      if (live) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.pages[s]) + cell * a.d + lane * 8) = raw[s];
    } else {
      float x[8], scale;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = elem16<DT>(raw[s], e);
      const uint2 codes = quantise<FMT, LG>(x, scale);
      if (live) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.pages[s]) + cell * a.d + lane * 8) = codes;
      if (live && lane == 0) a.scale[s][cell] = scale;
    }
  }
}

// A wave takes kReadRows consecutive rows of one head.  Lane i finds row i's sequence, page and scales, all rows at
// once, and the groups get them by lane exchange; then every load of the wave's rows is in flight together.
constexpr int kReadRows = 16;
template <int DT, int FMT, int LG>
__global__ void __launch_bounds__(kThreads) k_kv_read(KvArgs a) {
  constexpr int PER = kWave / LG, STEPS = (kReadRows + PER - 1) / PER;      // rows side by side, and one after the other
  const int wl = threadIdx.x % kWave, lane = wl % LG;
  const int head = blockIdx.x % a.heads;
  const int first = (blockIdx.x / a.heads * (kThreads / kWave) + threadIdx.x / kWave) * kReadRows;
  if (first >= a.t) return;                                     // the whole wave
  const int row = first + wl % kReadRows;
  // a row's sequence: the number of offsets after the first that are at or below it
  int seq = 0;
  for (int base = 0; base < a.n_seqs; base += kWave) {
    const int end = base + wl < a.n_seqs ? a.cu[base + wl + 1] : INT32_MAX;
    const int low = __popcll(__ballot(end <= first)), high = __popcll(__ballot(end <= first + kReadRows - 1));
    seq += low;
    for (int i = low; i < high; ++i) seq += __shfl(end, i, kWave) <= row;      // sequences that end within the rows
  }
  const int page_size = a.page.d;
  bool ok = row < a.t && seq < a.n_seqs;
  const bool mine = ok;
  int cell = 0;
  if (ok) {
    const int pos = row - a.cu[seq];
    const int col = pos >= 0 ? (int)a.page.div((uint32_t)pos) : a.max_pages;
    const int pg = col < a.max_pages ? a.table[(size_t)seq * a.max_pages + col] : -1;
    ok = pg >= 0 && pg < a.n_pages;
    if (ok) cell = (pg * a.heads + head) * page_size + (pos - col * page_size);
  }
  float sc[2] = {0.f, 0.f};
  if constexpr (FMT != SPA_KV_NATIVE) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (ok) sc[s] = a.scale[s][cell];
  }
  const uint32_t there = (uint32_t)__ballot(ok), write = (uint32_t)__ballot(mine);
  constexpr int W = FMT == SPA_KV_NATIVE ? 4 : 2;
  uint32_t raw[STEPS][2][W];
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int r = i * PER + wl / LG;
    const size_t c = (uint32_t)__shfl(cell, r & (kReadRows - 1), kWave);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int w = 0; w < W; ++w) raw[i][s][w] = 0;
      if (r < kReadRows && (there >> r) & 1u && lane * 8 < a.d) {
        if constexpr (FMT == SPA_KV_NATIVE) {
          const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.pages[s]) + c * a.d + lane * 8);
          raw[i][s][0] = v.x; raw[i][s][1] = v.y; raw[i][s][2] = v.z; raw[i][s][3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.pages[s]) + c * a.d + lane * 8);
          raw[i][s][0] = v.x; raw[i][s][1] = v.y;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    const int r = i * PER + wl / LG;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint4 v;
      if constexpr (FMT == SPA_KV_NATIVE) {
        v = make_uint4(raw[i][s][0], raw[i][s][1], raw[i][s][2], raw[i][s][3]);
      } else {
        const float k = __shfl(sc[s], r & (kReadRows - 1), kWave);
        float x[8];
        codes_to_f32<FMT>(raw[i][s][0], x);
        codes_to_f32<FMT>(raw[i][s][1], x + 4);
        v = make_uint4(pack2<DT>(x[0] * k, x[1] * k), pack2<DT>(x[2] * k, x[3] * k), pack2<DT>(x[4] * k, x[5] * k),
                       pack2<DT>(x[6] * k, x[7] * k));
      }
      if (r < kReadRows && (write >> r) & 1u && lane * 8 < a.d)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out[s]) + ((size_t)(first + r) * a.heads + head) * a.d + lane * 8) = v;
    }
  }
}

template <int DT, int FMT, int LG>
hipError_t go(bool write, const KvArgs& a, hipStream_t st) {
  const int rows = write ? kThreads / LG : kThreads / kWave * kReadRows;      // of a workgroup
  const int64_t blocks = ((int64_t)a.t + rows - 1) / rows * a.heads;
  if (write) hipLaunchKernelGGL((k_kv_write<DT, FMT, LG>), dim3((uint32_t)blocks), dim3(kThreads), 0, st, a);
  else hipLaunchKernelGGL((k_kv_read<DT, FMT, LG>), dim3((uint32_t)blocks), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}
template <int DT, int FMT>
hipError_t by_width(bool write, const KvArgs& a, hipStream_t st) {
  if (a.d <= 32) return go<DT, FMT, 4>(write, a, st);
  if (a.d <= 64) return go<DT, FMT, 8>(write, a, st);
  if (a.d <= 128) return go<DT, FMT, 16>(write, a, st);
  return go<DT, FMT, 32>(write, a, st);
}
template <int DT>
hipError_t by_format(int fmt, bool write, const KvArgs& a, hipStream_t st) {
  if (fmt == SPA_KV_NATIVE) return by_width<DT, SPA_KV_NATIVE>(write, a, st);
  if (fmt == SPA_KV_FP8) return by_width<DT, SPA_KV_FP8>(write, a, st);
  return by_width<DT, SPA_KV_INT8>(write, a, st);
}
hipError_t dispatch(const spa_kv_cache& c, bool write, KvArgs& a, hipStream_t st) {
  a.pages[0] = c.k; a.pages[1] = c.v;
  a.scale[0] = c.k_scale; a.scale[1] = c.v_scale;
  a.heads = c.n_heads; a.d = c.head_dim; a.n_pages = c.n_pages;
  a.page = FastDiv((uint32_t)c.page_size);
  if (c.dtype == SPA_F16) return by_format<SPA_F16>(c.format, write, a, st);
  return by_format<SPA_BF16>(c.format, write, a, st);
}

}  // namespace

hipError_t launch_kv_write(const spa_heads& k, const spa_heads& v, int t, const int32_t* slots, const spa_kv_cache& c,
                           hipStream_t st) {
  KvArgs a{};
  const spa_heads* h[2] = {&k, &v};
  for (int s = 0; s < 2; ++s) {
    a.src[s] = h[s]->data;
    a.row_stride[s] = h[s]->row_stride;
    a.head_stride[s] = h[s]->head_stride;
  }
  a.slots = slots;
  a.t = t;
  return dispatch(c, true, a, st);
}

hipError_t launch_kv_read(const spa_kv_cache& c, const int32_t* table, int n_seqs, int max_pages, const int32_t* cu,
                          int total, void* k_out, void* v_out, hipStream_t st) {
  KvArgs a{};
  a.out[0] = k_out; a.out[1] = v_out;
  a.table = table; a.cu = cu;
  a.t = total; a.n_seqs = n_seqs; a.max_pages = max_pages;
  return dispatch(c, false, a, st);
}

}  // namespace spa
