// Attention of one new token per sequence over its paged cache: out = softmax(scale q K^T) V.
//
// Bound: the cache is read once for every 16 query heads that share it, and does little work: bound by HBM, at 0.71 to
// 0.79 of the rate of a stream that is only read (7.2 TB/s on this card; a copy moves 4.9).  A wave works on tiles of 32 positions of one (sequence, key-value head) and keeps
// everything in registers:
//   S^T = K Q^T on v_mfma_f32_16x16x32: a lane's K operand is 16 consecutive bytes of a cached row, so keys go
//         from memory to the matrix cores with no LDS; the 16 columns are the query heads (zeros past G);
//   O^T = V^T P^T: the scores' own registers are the P operand, each weight rounded to 16 bits, which is the output's own
//         unit roundoff (0.0023 of the 2-norm against 0.0017 for float32 weights, bfloat16 over e4m3; more bits would take
//         a second product).  The order of the 32 positions along the product is free, so it is taken as S^T leaves it:
//         lane group g holds 4g..4g+3 and 16+4g..16+4g+3.
//         A lane reads those 8 positions' rows, 16 lanes to a row, and turns its 8 x 8 block with byte
//         permutes into one V^T operand per dimension.
// The running maximum and sum are one column (query head) per lane.  The tiles of all sequences, end to end, are cut
// into equal shares, one for each workgroup of a head, whatever the lengths; every workgroup finds its share from
// the lengths on the device.  A sequence that is cut leaves unnormalised float32 sums with their maximum, and a
// second kernel joins them in a fixed order.
//
// 64 ragged sequences of up to 4099 positions (32 heads on 8 of 128, e4m3): 62 us, 5.1 TB/s; two of 100003 (int8,
// float16): 75 us, 5.6 TB/s; one of 61 (16 bits): 5.8 us.
#include <algorithm>

#include "spa_attn.h"
#include "spa_check_layer.h"
#include "spa_layer.h"

namespace spa {

namespace {

constexpr int kTile = 32;           // positions a wave takes at a time
constexpr int kWaves = 4;
constexpr int kMinTiles = 4;        // tiles of a piece at the least: one for each wave

struct DecodeAttnArgs {
  const uint16_t* q;
  int64_t q_row, q_head;
  const void* k;
  const void* v;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  const int32_t* lens;
  void* out;
  float* lse;
  float* part_o;             // [2 workgroups][n_q_heads][d]
  float2* part_ml;           // [2 workgroups][n_q_heads]
  int2* part_of;             // [n_seqs]: a sequence's first slot and its number of pieces
  int n_seqs, hq, hkv, group, d, n_pages, max_pages, head_tiles;
  int target;                // workgroups of a head at the most
  float c;                   // scale * log2 e
  FastDiv page;
};

// With an 8-bit cache a softmax weight carries its value vector's scale when it is rounded to 16 bits for the matrix
// product.  bfloat16 has the exponents for it.  For float16 the scales are taken relative to the largest that the wave
// has met, brought to 2^14: a weight then keeps its 11 bits down to 2^-28 of the largest, whatever the size of the values
// (with a constant factor instead, values of 1e-4 beside a heavy key were lost whole).  The reference is a power of two,
// so nothing is rounded twice, and the sums follow it as they follow the running maximum, when it rises.
template <int DT, int FMT> constexpr bool kFollowScale = FMT != SPA_KV_NATIVE && DT == SPA_F16;
struct ValueScale {
  static constexpr int kLow = 14;      // scales below 2^-112 are not brought up; a written vector's are above 2^-109
  int top = kLow;                      // the largest scale's exponent field, one value for the wave
  // Takes in a tile's largest scale; what sums so far are to be multiplied by, or 1.
  __device__ __forceinline__ float follow(float largest) {
    const int e = __builtin_amdgcn_readfirstlane((int)(__float_as_uint(largest) >> 23 & 0xFFu));
    const int before = top;
    top = max(top, e);
    return __uint_as_float((uint32_t)max(127 + before - top, 0) << 23);
  }
  __device__ __forceinline__ float up() const { return __uint_as_float((uint32_t)(267 - top) << 23); }       // 2^(140 - top)
  __device__ __forceinline__ float down() const { return __uint_as_float((uint32_t)(top - 13) << 23); }      // 2^(top - 140)
};

// Positions of sequence s that can count, and their tiles.
__device__ __forceinline__ int seq_len(const DecodeAttnArgs& a, int s) {
  return min(max(a.lens[s], 0), a.max_pages * (int)a.page.d);
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kTile - 1) / kTile; }

// What a workgroup works through: `per` consecutive tiles of all sequences' tiles laid end to end, so every
// workgroup of a head has the same share whatever the lengths.  An empty sequence stands as one tile of nothing.
struct Span {
  int per;
  int seq, local;              // where the next piece starts: sequence, tile within it
  int left;                    // tiles still to do
  bool fresh;                  // nothing done yet
  int lens;                    // lane i: the positions of sequence i < 64
};
// One piece of a sequence, for one key-value head and up to 16 of its query heads.
struct Piece {
  int seq, head, h0, heads;    // key-value head; first query head and their number
  int len;                     // positions of the sequence
  int begin, end;              // tiles
  bool whole;                  // the sequence is this piece alone
  int slot;                    // where the piece's sums go if not: two slots to a workgroup
};
__device__ __forceinline__ int seq_share(const DecodeAttnArgs& a, int s) { return max(tiles_of(seq_len(a, s)), 1); }

__device__ __forceinline__ bool find_span(const DecodeAttnArgs& a, Span& s) {
  const int lane = threadIdx.x & (kWave - 1);
  s.lens = lane < a.n_seqs ? seq_len(a, lane) : 0;
  const int c0 = lane < a.n_seqs ? max(tiles_of(s.lens), 1) : 0;
  const int incl0 = wave_scan(c0);
  long long total = __builtin_amdgcn_readlane(incl0, kWave - 1);
  for (int base = kWave; base < a.n_seqs; base += kWave) {
    long long c = base + lane < a.n_seqs ? seq_share(a, base + lane) : 0;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) c += __shfl_xor(c, off, kWave);
    total += c;
  }
  const int per = (int)max((total + a.target - 1) / a.target, (long long)kMinTiles);
  const long long start = (long long)blockIdx.x * per;
  if (start >= total) return false;
  long long before = 0;
  int c = c0, incl = incl0, base = 0;
  uint64_t past;
  while (!(past = __ballot(before + incl > start))) {
    before += __builtin_amdgcn_readlane(incl, kWave - 1);
    base += kWave;
    if (base >= a.n_seqs) return false;
    c = base + lane < a.n_seqs ? seq_share(a, base + lane) : 0;
    incl = wave_scan(c);
  }
  const int at = __ffsll((unsigned long long)past) - 1;
  s.per = per;
  s.seq = base + at;
  s.local = (int)(start - before) - __builtin_amdgcn_readlane(incl - c, at);
  s.left = (int)min((long long)per, total - start);
  s.fresh = true;
  return true;
}

__device__ __forceinline__ Piece next_piece(const DecodeAttnArgs& a, Span& s) {
  Piece p;
  p.seq = s.seq;
  const int ht = blockIdx.y / a.hkv;
  p.head = blockIdx.y % a.hkv;
  p.heads = min(a.group - 16 * ht, 16);
  p.h0 = p.head * a.group + 16 * ht;
  p.len = s.seq < kWave ? __builtin_amdgcn_readlane(s.lens, s.seq) : seq_len(a, s.seq);
  const int tiles = tiles_of(p.len), share = max(tiles, 1);
  const int take = min(share - s.local, s.left);
  p.begin = s.local;
  p.end = min(s.local + take, tiles);
  p.whole = take == share;
  // a piece that starts inside its sequence is its workgroup's first, one that ends inside its last
  p.slot = 2 * blockIdx.x + (s.local == 0 && !s.fresh);
  if (s.local == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    const int more = share - take;                              // tiles in the workgroups after this one
    a.part_of[p.seq] = make_int2(p.slot, 1 + (more + s.per - 1) / s.per);
  }
  s.left -= take;
  ++s.seq;
  s.local = 0;
  s.fresh = false;
  return p;
}

// Four 8-bit codes as two words of 16-bit values (exact in both types: e4m3 has 4 significant bits, int8 7).
template <int DT, int FMT>
__device__ __forceinline__ uint2 widen4(uint32_t c) {
  if constexpr (FMT == SPA_KV_FP8 && DT == SPA_BF16) {
    return make_uint2(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.f, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.f, true)));
  } else if constexpr (FMT == SPA_KV_FP8) {
    return make_uint2(__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.f, false)),
                      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.f, true)));
  } else {
    float x[4];
    codes_to_f32<FMT>(c, x);
    return make_uint2(pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]));
  }
}
// 8 consecutive elements of a cached row as a 16-bit matrix operand.
template <int DT, int FMT>
__device__ __forceinline__ uint4 widen8(uint2 c) {
  const uint2 lo = widen4<DT, FMT>(c.x), hi = widen4<DT, FMT>(c.y);
  return make_uint4(lo.x, lo.y, hi.x, hi.y);
}
// NV elements as stored, to pairs of 16-bit values.
template <int DT, int FMT, int NV, int VW>
__device__ __forceinline__ void widen_row(const uint32_t (&raw)[VW], uint32_t (&w)[NV / 2]) {
#pragma unroll
  for (int i = 0; i < VW; ++i) {
    if constexpr (FMT == SPA_KV_NATIVE) {
      w[i] = raw[i];
    } else {
      const uint2 x = widen4<DT, FMT>(raw[i]);
      w[2 * i] = x.x;
      w[2 * i + 1] = x.y;
    }
  }
}

// Largest of the four lanes that hold one column (lanes col, col + 16, + 32, + 48), on each of them.
__device__ __forceinline__ float across_groups_max(float v) {
  const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1]));
  const auto q = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

// Largest magnitude of a tile's scales, eight on each lane of a group, on every lane.
__device__ __forceinline__ float largest(const float (&vs)[8]) {
  float v = fabsf(vs[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) v = fmaxf(v, fabsf(vs[j]));
  return across_groups_max(v);
}

// The query operand of k step c: columns are query heads, elements q_at(c, g).. + 7.
template <int FMT>
__device__ __forceinline__ int q_at(int c, int g) {
  // 8-bit keys are read 16 bytes at a time, so two steps share 64 dimensions and a lane's 16 are consecutive
  if constexpr (FMT == SPA_KV_NATIVE) return 32 * c + 8 * g;
  else return 64 * (c / 2) + 16 * g + 8 * (c % 2);
}
template <int FMT, int KC>
__device__ __forceinline__ void load_q(const DecodeAttnArgs& a, const Piece& p, int col, int g, uint4 (&qf)[KC]) {
  const uint16_t* q = a.q + (size_t)p.seq * a.q_row + (size_t)(p.h0 + min(col, p.heads - 1)) * a.q_head;
#pragma unroll
  for (int c = 0; c < KC; ++c) {
    const int at = q_at<FMT>(c, g);
    qf[c] = make_uint4(0, 0, 0, 0);
    if (col < p.heads && at < a.d) qf[c] = *reinterpret_cast<const uint4*>(q + at);
  }
}

// 16 bytes, or a lane's share of a value row, that are read once.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint4 stream_load16(const void* p) {
  const u32x4 v = __builtin_nontemporal_load(static_cast<const u32x4*>(p));
  return make_uint4(v[0], v[1], v[2], v[3]);
}
// The same from an address of 8-byte alignment: rows of 8-bit codes where head_dim is an odd multiple of 8.
typedef uint32_t u32x4_by8 __attribute__((ext_vector_type(4), aligned(8)));
__device__ __forceinline__ uint4 stream_load16_by8(const void* p) {
  const u32x4_by8 v = __builtin_nontemporal_load(static_cast<const u32x4_by8*>(p));
  return make_uint4(v[0], v[1], v[2], v[3]);
}
// The first `live` of W words, the others 0 (live is W, W / 2 or 0: whole 8-element pieces).
template <int W>
__device__ __forceinline__ void stream_load(const char* p, int live, uint32_t (&w)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) w[i] = 0;
  if constexpr (W == 1) {
    if (live) w[0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p));
  } else {
    constexpr int kStep = W >= 8 ? 4 : 2;
#pragma unroll
    for (int i = 0; i < W; i += kStep) {
      if (i < live) {
        if constexpr (kStep == 4) {
          const uint4 v = stream_load16(p + 4 * i);
          w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
        } else {
          const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p + 4 * i));
          w[i] = v[0]; w[i + 1] = v[1];
        }
      }
    }
  }
}
template <int W>
__device__ __forceinline__ void stream_load(const char* p, uint32_t (&w)[W]) {
  if constexpr (W == 1) {
    w[0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p));
  } else if constexpr (W == 2) {
    const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p));
    w[0] = v[0]; w[1] = v[1];
  } else {
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const uint4 v = stream_load16(p + 4 * i);
      w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
    }
  }
}

// Joins the four waves and writes the piece's result: lane (col, g) holds dimensions NV * (4 g + r) + i of query
// head col, its maximum and its own positions' sum; `unit` is what one of o stands for.
template <int DT, int FMT, int DP>
__device__ __forceinline__ void finish(const DecodeAttnArgs& a, const Piece& p, const f32x4 (&o)[DP / 16], float unit, float m,
                                       float l) {
  constexpr int NV = DP / 16;
  __shared__ float s_o[kWaves][16][DP + 4];
  __shared__ float s_m[kWaves][16], s_l[kWaves][16];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int col = lane & 15, g = lane >> 4;
  l += __shfl_xor(l, 16, kWave);
  l += __shfl_xor(l, 32, kWave);
  if (g == 0) s_m[wave][col] = m, s_l[wave][col] = l;
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int i = 0; i < NV; ++i) s_o[wave][col][NV * (4 * g + r) + i] = kFollowScale<DT, FMT> ? o[i][r] * unit : o[i][r];
  __syncthreads();
  for (int e = threadIdx.x; e < p.heads * (DP / 2); e += kWaves * kWave) {
    const int h = e / (DP / 2), dim = e % (DP / 2) * 2;
    if (dim >= a.d) continue;
    float mx = s_m[0][h];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) mx = fmaxf(mx, s_m[w][h]);
    const float base = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f, x0 = 0.f, x1 = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = exp2_hw(s_m[w][h] - base);
      sum += f * s_l[w][h];
      x0 += f * s_o[w][h][dim];
      x1 += f * s_o[w][h][dim + 1];
    }
    if (p.whole) {
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const size_t to = (size_t)p.seq * a.hq + p.h0 + h;
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + to * a.d + dim) = pack2<DT>(x0 * inv, x1 * inv);
      if (dim == 0 && a.lse) a.lse[to] = sum == 0.f ? -INFINITY : kLn2 * (base + log2_hw(sum));
    } else {
      const size_t to = (size_t)p.slot * a.hq + p.h0 + h;
      *reinterpret_cast<float2*>(a.part_o + to * a.d + dim) = make_float2(x0, x1);
      if (dim == 0) a.part_ml[to] = make_float2(mx, sum);
    }
  }
  __syncthreads();      // the next piece writes here again
}

// Any page size: a lane finds one position's cell and the others get it by lane exchange.
template <int DT, int FMT, int DP>
__global__ void __launch_bounds__(kWaves * kWave) k_attention_decode(DecodeAttnArgs a) {
  constexpr int KC = DP / 32;      // k steps of S
  constexpr int NV = DP / 16;      // dimensions of V a lane holds
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int col = lane & 15, g = lane >> 4;
  Span span;
  if (!find_span(a, span)) return;
  do {
    const Piece p = next_piece(a, span);
    uint4 qf[KC];
    load_q<FMT, KC>(a, p, col, g, qf);

    f32x4 o[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    ValueScale vmax;

    for (int tile = p.begin + wave; tile < p.end; tile += kWaves) {
      // lane i < 32 finds position i's cell; a position that does not count is bit i of `gone`
      const int pos = tile * kTile + (lane & 31);
      const int p0 = min(pos, p.len - 1);
      const int pc = (int)a.page.div((uint32_t)p0);
      const int pg = a.table[(size_t)p.seq * a.max_pages + pc];
      const bool ok = pg >= 0 && pg < a.n_pages;
      const int cell = ok ? (pg * a.hkv + p.head) * (int)a.page.d + (p0 - pc * (int)a.page.d) : 0;
      const bool counts = pos < p.len && ok;
      const uint32_t gone = (uint32_t)__ballot(!counts);       // the scores are hidden and the values dropped
      float ksc = 1.f, vsc = 1.f;
      if constexpr (FMT != SPA_KV_NATIVE) {
        ksc = a.k_scale[cell];
        vsc = counts ? a.v_scale[cell] : 0.f;
      }
      float t[2][4];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const size_t kc = (size_t)(uint32_t)__shfl(cell, 16 * b + col, kWave);
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const int at = q_at<FMT>(c, g);
          uint4 kf = make_uint4(0, 0, 0, 0);
          if (at < a.d) {
            if constexpr (FMT == SPA_KV_NATIVE)
              kf = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.k) + kc * a.d + at);
            else
              kf = widen8<DT, FMT>(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(a.k) + kc * a.d + at));
          }
          s = mfma16<DT>(kf, qf[c], s);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = 16 * b + 4 * g + r;
          float x = s[r] * a.c;
          if constexpr (FMT != SPA_KV_NATIVE) x *= __shfl(ksc, i, kWave);
          t[b][r] = (gone >> i) & 1u ? -INFINITY : x;
        }
      }
      float mx = m;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r) mx = fmaxf(mx, t[b][r]);
      mx = fmaxf(mx, __shfl_xor(mx, 16, kWave));
      mx = fmaxf(mx, __shfl_xor(mx, 32, kWave));
      const float base = mx == -INFINITY ? 0.f : mx;           // nothing seen yet: every p is 0
      const float alpha = exp2_hw(m - base);
      m = mx;
      l *= alpha;
      float w[8], vs[8], grow = alpha;
      if constexpr (FMT != SPA_KV_NATIVE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) vs[j] = __shfl(vsc, 16 * (j / 4) + 4 * g + j % 4, kWave);
      }
      if constexpr (kFollowScale<DT, FMT>) grow *= vmax.follow(largest(vs));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        w[j] = exp2_hw(t[j / 4][j % 4] - base);
        l += w[j];
        if constexpr (kFollowScale<DT, FMT>) vs[j] *= vmax.up();
        if constexpr (FMT != SPA_KV_NATIVE) w[j] *= vs[j];
      }
      const uint4 pf = make_uint4(pack2<DT>(w[0], w[1]), pack2<DT>(w[2], w[3]), pack2<DT>(w[4], w[5]), pack2<DT>(w[6], w[7]));
      uint32_t vr[8][NV / 2];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = (j < 4 ? 4 * g + j : 16 + 4 * g + j - 4);
        const size_t vc = (size_t)(uint32_t)__shfl(cell, i, kWave);
        constexpr int ES = FMT == SPA_KV_NATIVE ? 2 : 1, VW = NV * ES / 4;
        uint32_t raw[VW];
        const bool live = NV * col < a.d && !((gone >> i) & 1u);
        const uint32_t* at = reinterpret_cast<const uint32_t*>(static_cast<const char*>(a.v) + (vc * a.d + NV * col) * ES);
#pragma unroll
        for (int e = 0; e < VW; ++e) raw[e] = live && NV * col + 4 / ES * e < a.d ? at[e] : 0u;
        widen_row<DT, FMT, NV>(raw, vr[j]);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t sel = i & 1 ? 0x07060302u : 0x05040100u;      // the high or low halves of two rows
        uint4 vf;
        vf.x = __builtin_amdgcn_perm(vr[1][i / 2], vr[0][i / 2], sel);
        vf.y = __builtin_amdgcn_perm(vr[3][i / 2], vr[2][i / 2], sel);
        vf.z = __builtin_amdgcn_perm(vr[5][i / 2], vr[4][i / 2], sel);
        vf.w = __builtin_amdgcn_perm(vr[7][i / 2], vr[6][i / 2], sel);
        o[i] *= grow;
        o[i] = mfma16<DT>(vf, pf, o[i]);
      }
    }

    finish<DT, FMT, DP>(a, p, o, vmax.down(), m, l);
  } while (span.left > 0);
}

// Pages of whole 16-position blocks: a block's rows are consecutive, so a tile has two bases that the whole wave
// shares.  EXACT: head_dim is DP; else pieces past it are not read and count as zeros.  The page numbers of a wave's next
// 32 tiles are held one to a lane; keys of the next tile are on their way while this tile's softmax and V product run, and
// values while its scores are formed.
template <int DT, int FMT, int DP, bool EXACT>
__global__ void __launch_bounds__(kWaves * kWave) k_attention_decode_blocks(DecodeAttnArgs a) {
  constexpr int KC = DP / 32, NV = DP / 16;
  constexpr int ES = FMT == SPA_KV_NATIVE ? 2 : 1;
  constexpr int KL = FMT == SPA_KV_NATIVE ? KC : KC / 2;     // 16-byte key loads of a lane per block
  constexpr int VW = NV * ES / 4;                            // 4-byte words of a lane's value load
  constexpr int kBatch = kWave / 2;                          // tiles whose page numbers are held
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int col = lane & 15, g = lane >> 4;
  Span span;
  if (!find_span(a, span)) return;
  do {
    const Piece p = next_piece(a, span);
    uint4 qf[KC];
    load_q<FMT, KC>(a, p, col, g, qf);

    f32x4 o[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    ValueScale vmax;

    const int first = p.begin + wave, n = (p.end - first + kWaves - 1) / kWaves;      // this wave's tiles
    int pages = -1;                      // lane i: the page of block i % 2 of tile i / 2 of the batch, -1 if there is none
    auto fetch_pages = [&](int it) {
      const int block = (first + kWaves * (it + lane / 2)) * 2 + (lane & 1);
      const int at = block * 16;
      pages = -1;
      if (at < p.len) {
        pages = a.table[(size_t)p.seq * a.max_pages + a.page.div((uint32_t)at)];
        if (pages >= a.n_pages) pages = -1;
      }
    };
    // the first cell of block b of tile number `it`, and whether its page is there (else cell 0 of the cache)
    auto base_of = [&](int it, int b, bool& there) {
      const int pg = __builtin_amdgcn_readlane(pages, 2 * (it % kBatch) + b);
      const uint32_t at = (uint32_t)((first + kWaves * it) * 2 + b) * 16;
      there = pg >= 0;
      const uint32_t cell = ((uint32_t)pg * a.hkv + p.head) * a.page.d + (at - a.page.div(at) * a.page.d);
      return there ? cell : 0u;
    };
    uint4 kr[2][KL];
    float4 ksc[2], vsc[2];
    const int d = EXACT ? DP : a.d;
    const uint32_t k_lane = (uint32_t)(col * d * ES + 16 * g), v_lane = (uint32_t)((4 * g * d + NV * col) * ES);
    const int v_live = EXACT ? VW : min(max((d - NV * col) / 4 * ES, 0), VW);      // words of a value row: ES for 4 elements
    auto load_k = [&](const uint32_t (&cell)[2]) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const char* base = static_cast<const char*>(a.k) + (size_t)cell[b] * (uint32_t)(d * ES);
#pragma unroll
        for (int c = 0; c < KL; ++c) {
          if constexpr (EXACT) {
            kr[b][c] = stream_load16(base + (k_lane + 64 * c));
          } else {
            uint32_t w[4] = {0, 0, 0, 0};
            const int bytes = d * ES - (16 * g + 64 * c);              // left in the row; whole 8-element pieces
            const char* from = base + (k_lane + 64 * c);
            if (bytes >= 16) {
              const uint4 v = FMT == SPA_KV_NATIVE ? stream_load16(from) : stream_load16_by8(from);
              w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
            } else if (bytes > 0) {
              w[0] = reinterpret_cast<const uint32_t*>(from)[0];
              w[1] = reinterpret_cast<const uint32_t*>(from)[1];
            }
            kr[b][c] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        if constexpr (FMT != SPA_KV_NATIVE) {
          ksc[b] = *reinterpret_cast<const float4*>(a.k_scale + (size_t)cell[b] + 4 * g);
          vsc[b] = *reinterpret_cast<const float4*>(a.v_scale + (size_t)cell[b] + 4 * g);
        }
      }
    };

    uint32_t cell[2];
    bool there[2] = {true, true};
    if (n > 0) {
      fetch_pages(0);
#pragma unroll
      for (int b = 0; b < 2; ++b) cell[b] = base_of(0, b, there[b]);
      load_k(cell);
    }
    for (int it = 0; it < n; ++it) {
      const int tile = first + kWaves * it;
      // values of this tile
      uint32_t vraw[8][VW];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const char* base = static_cast<const char*>(a.v) + (size_t)cell[j / 4] * (uint32_t)(d * ES);
        if constexpr (EXACT) stream_load<VW>(base + (v_lane + (j % 4) * DP * ES), vraw[j]);
        else stream_load<VW>(base + (v_lane + (j % 4) * d * ES), v_live, vraw[j]);
      }
      // scores
      f32x4 s[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        s[b] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          uint4 kf;
          if constexpr (FMT == SPA_KV_NATIVE) kf = kr[b][c];
          else kf = widen8<DT, FMT>(c % 2 ? make_uint2(kr[b][c / 2].z, kr[b][c / 2].w) : make_uint2(kr[b][c / 2].x, kr[b][c / 2].y));
          s[b] = mfma16<DT>(kf, qf[c], s[b]);
        }
      }
      float t[8], vs[8];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const float kq[4] = {ksc[b].x, ksc[b].y, ksc[b].z, ksc[b].w}, vq[4] = {vsc[b].x, vsc[b].y, vsc[b].z, vsc[b].w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          t[4 * b + r] = s[b][r] * a.c;
          if constexpr (FMT != SPA_KV_NATIVE) t[4 * b + r] *= kq[r];
          vs[4 * b + r] = FMT != SPA_KV_NATIVE ? vq[r] : 1.f;
        }
      }
      // the last tile's end and absent pages: what does not count is removed from the scores, the values and their scales
      const bool cut = (tile + 1) * kTile > p.len || !there[0] || !there[1];
      uint32_t gone = 0;
      if (cut) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int pos = tile * kTile + 16 * (j / 4) + 4 * g + j % 4;
          if (pos >= p.len || !there[j / 4]) {
            gone |= 1u << j;
            t[j] = -INFINITY;
            vs[j] = 0.f;
          }
        }
      }
      // keys of the next tile
      if (it + 1 < n) {
        if ((it + 1) % kBatch == 0) fetch_pages(it + 1);
#pragma unroll
        for (int b = 0; b < 2; ++b) cell[b] = base_of(it + 1, b, there[b]);
        load_k(cell);
      }
      // softmax
      float mx = t[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) mx = fmaxf(mx, t[j]);
      mx = across_groups_max(mx);
      if (__any(mx > m)) {
        const float now = fmaxf(m, mx), alpha = exp2_hw(m - (now == -INFINITY ? 0.f : now));
        m = now;
        l *= alpha;
#pragma unroll
        for (int i = 0; i < NV; ++i) o[i] *= alpha;
      }
      const float base = m == -INFINITY ? 0.f : m;           // nothing seen yet: every weight is 0
      if constexpr (kFollowScale<DT, FMT>) {
        const float grow = vmax.follow(largest(vs));
        if (grow != 1.f) {
#pragma unroll
          for (int i = 0; i < NV; ++i) o[i] *= grow;
        }
      }
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        w[j] = exp2_hw(t[j] - base);
        l += w[j];
        if constexpr (kFollowScale<DT, FMT>) vs[j] *= vmax.up();
        if constexpr (FMT != SPA_KV_NATIVE) w[j] *= vs[j];
      }
      const uint4 pf = make_uint4(pack2<DT>(w[0], w[1]), pack2<DT>(w[2], w[3]), pack2<DT>(w[4], w[5]), pack2<DT>(w[6], w[7]));
      if (cut) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if ((gone >> j) & 1u)
#pragma unroll
            for (int i = 0; i < VW; ++i) vraw[j][i] = 0;
      }
      // one stored word of the eight rows at a time: PW pairs of dimensions
      constexpr int PW = 2 / ES;
#pragma unroll
      for (int i = 0; i < VW; ++i) {
        uint32_t vr[8][PW];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t raw[1] = {vraw[j][i]};
          widen_row<DT, FMT, 2 * PW, 1>(raw, vr[j]);
        }
#pragma unroll
        for (int e = 0; e < 2 * PW; ++e) {
          const uint32_t sel = e & 1 ? 0x07060302u : 0x05040100u;      // the high or low halves of two rows
          uint4 vf;
          vf.x = __builtin_amdgcn_perm(vr[1][e / 2], vr[0][e / 2], sel);
          vf.y = __builtin_amdgcn_perm(vr[3][e / 2], vr[2][e / 2], sel);
          vf.z = __builtin_amdgcn_perm(vr[5][e / 2], vr[4][e / 2], sel);
          vf.w = __builtin_amdgcn_perm(vr[7][e / 2], vr[6][e / 2], sel);
          o[2 * PW * i + e] = mfma16<DT>(vf, pf, o[2 * PW * i + e]);
        }
      }
    }
    finish<DT, FMT, DP>(a, p, o, vmax.down(), m, l);
  } while (span.left > 0);
}

// Joins a sequence's pieces in a fixed order.  A thread takes four dimensions of one head, brings the pieces' sums to
// their common maximum and adds them; with RUNS > 1 that many threads take every RUNS-th piece of the same four
// dimensions, and the first of them adds the runs up.
constexpr int kJoinThreads = 256;
struct JoinSums {
  float m, sum;
  float4 x;
};
__device__ __forceinline__ void rescale(JoinSums& j, float m) {
  const float f = exp2_hw(j.m - (m == -INFINITY ? 0.f : m));
  j.m = m;
  j.sum *= f;
  j.x.x *= f; j.x.y *= f; j.x.z *= f; j.x.w *= f;
}
template <int DT, int FMT, int RUNS>
__global__ void __launch_bounds__(kJoinThreads) k_attention_decode_join(DecodeAttnArgs a) {
  constexpr int kCols = kJoinThreads / RUNS, U = RUNS > 1 ? 4 : 8;
  __shared__ JoinSums s_run[RUNS > 1 ? RUNS : 1][RUNS > 1 ? kCols : 1];
  const int2 of = a.part_of[blockIdx.x];
  if (of.y == 1) return;
  const int quads = a.d / 4;
  const int run = threadIdx.x / kCols, at = blockIdx.y * kCols + threadIdx.x % kCols;
  const int head = at / quads, dim = at % quads * 4;
  const bool live = head < a.hq;
  const int next = of.x & ~1;                  // piece k > 0 is in the first slot of the k-th workgroup after
  JoinSums j{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  if (live) {
    for (int i = run; i < of.y; i += U * RUNS) {
      float2 s[U];
      float4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = min(i + u * RUNS, of.y - 1);
        const size_t row = (size_t)(k ? next + 2 * k : of.x) * a.hq + head;
        s[u] = a.part_ml[row];
        v[u] = *reinterpret_cast<const float4*>(a.part_o + row * a.d + dim);
        if (i + u * RUNS >= of.y) {               // none: not a piece of weight 0, whose infinities would give NaN
          s[u].x = -INFINITY;
          v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
      float now = j.m;
#pragma unroll
      for (int u = 0; u < U; ++u) now = fmaxf(now, s[u].x);
      rescale(j, now);
      const float base = now == -INFINITY ? 0.f : now;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float f = exp2_hw(s[u].x - base);
        j.sum += f * s[u].y;
        j.x.x += f * v[u].x; j.x.y += f * v[u].y; j.x.z += f * v[u].z; j.x.w += f * v[u].w;
      }
    }
  }
  if constexpr (RUNS > 1) {
    s_run[run][threadIdx.x % kCols] = j;
    __syncthreads();
    if (run) return;
    float m = j.m;
#pragma unroll
    for (int r = 1; r < RUNS; ++r) m = fmaxf(m, s_run[r][threadIdx.x].m);
    rescale(j, m);
#pragma unroll
    for (int r = 1; r < RUNS; ++r) {
      JoinSums o = s_run[r][threadIdx.x];
      rescale(o, m);
      j.sum += o.sum;
      j.x.x += o.x.x; j.x.y += o.x.y; j.x.z += o.x.z; j.x.w += o.x.w;
    }
  }
  if (!live) return;
  const float inv = j.sum == 0.f ? 0.f : 1.f / j.sum;
  const size_t to = (size_t)blockIdx.x * a.hq + head;
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + to * a.d + dim) =
      make_uint2(pack2<DT>(j.x.x * inv, j.x.y * inv), pack2<DT>(j.x.z * inv, j.x.w * inv));
  if (dim == 0 && a.lse) a.lse[to] = j.sum == 0.f ? -INFINITY : kLn2 * (j.m + log2_hw(j.sum));
}

template <int DT, int FMT, int DP>
hipError_t go(const DecodeAttnArgs& a, hipStream_t st) {
  // no more workgroups than the table has room for
  const int64_t room = ((int64_t)a.max_pages * a.page.d + kTile - 1) / kTile;
  const int units = (int)std::min<int64_t>(a.target, (std::max<int64_t>(room, 1) * a.n_seqs + kMinTiles - 1) / kMinTiles);
  const dim3 grid(units, a.hkv * a.head_tiles), block(kWaves * kWave);
  if (a.page.d % 16 == 0 && a.d == DP)
    hipLaunchKernelGGL((k_attention_decode_blocks<DT, FMT, DP, true>), grid, block, 0, st, a);
  else if (a.page.d % 16 == 0)
    hipLaunchKernelGGL((k_attention_decode_blocks<DT, FMT, DP, false>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_attention_decode<DT, FMT, DP>), grid, block, 0, st, a);
  if (hipError_t e = hipGetLastError()) return e;
  // one workgroup to a head cuts nothing
  if (units == 1) return hipSuccess;
  // runs side by side where a sequence has 8 pieces or more on the average: four sequences of up to 30000 on 2 heads take
  // 18.5 us so and 29.0 us in one run; where most have few, more workgroups only cost their start
  const int quads = a.hq * (a.d / 4);
  if (units >= 8 * a.n_seqs) {
    const dim3 join(a.n_seqs, (quads + kJoinThreads / 8 - 1) / (kJoinThreads / 8));
    hipLaunchKernelGGL((k_attention_decode_join<DT, FMT, 8>), join, dim3(kJoinThreads), 0, st, a);
  } else {
    const dim3 join(a.n_seqs, (quads + kJoinThreads - 1) / kJoinThreads);
    hipLaunchKernelGGL((k_attention_decode_join<DT, FMT, 1>), join, dim3(kJoinThreads), 0, st, a);
  }
  return hipGetLastError();
}
template <int DT, int FMT>
hipError_t by_dim(const DecodeAttnArgs& a, hipStream_t st) {
  if (a.d <= 64) return go<DT, FMT, 64>(a, st);
  if (a.d <= 128) return go<DT, FMT, 128>(a, st);
  return go<DT, FMT, 256>(a, st);
}
template <int DT>
hipError_t by_format(int fmt, const DecodeAttnArgs& a, hipStream_t st) {
  if (fmt == SPA_KV_NATIVE) return by_dim<DT, SPA_KV_NATIVE>(a, st);
  if (fmt == SPA_KV_FP8) return by_dim<DT, SPA_KV_FP8>(a, st);
  return by_dim<DT, SPA_KV_INT8>(a, st);
}

}  // namespace

hipError_t launch_attention_decode(const spa_heads& q, int n_seqs, int n_q_heads, const spa_kv_cache& c,
                                   const int32_t* table, int max_pages, const int32_t* lens, float scale, void* out,
                                   float* lse, float* part_o, float* part_ml, int32_t* part_of, hipStream_t st) {
  DecodeAttnArgs a{};
  a.q = static_cast<const uint16_t*>(q.data);
  a.q_row = q.row_stride; a.q_head = q.head_stride;
  a.k = c.k; a.v = c.v; a.k_scale = c.k_scale; a.v_scale = c.v_scale;
  a.table = table; a.lens = lens; a.out = out; a.lse = lse;
  a.part_o = part_o; a.part_ml = reinterpret_cast<float2*>(part_ml);
  a.part_of = reinterpret_cast<int2*>(part_of);
  a.n_seqs = n_seqs; a.hq = n_q_heads; a.hkv = c.n_heads; a.group = n_q_heads / c.n_heads;
  a.d = c.head_dim; a.n_pages = c.n_pages; a.max_pages = max_pages;
  a.head_tiles = spa_check::head_tiles(n_q_heads, c.n_heads);
  a.target = spa_check::decode_groups(n_q_heads, c.n_heads, c.head_dim);
  a.c = scale * kLog2e;
  a.page = FastDiv((uint32_t)c.page_size);
  return c.dtype == SPA_F16 ? by_format<SPA_F16>(c.format, a, st) : by_format<SPA_BF16>(c.format, a, st);
}

}  // namespace spa
