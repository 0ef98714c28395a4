// What the decode attention kernels share (internal to them): how the sequences' tiles are divided among the workgroups, how
// a piece's sums are written, and how the pieces of a sequence are joined.
#pragma once

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
  const void* k_scale;       // float32, or the bytes of SPA_KV_MXFP4
  const void* v_scale;
  const int32_t* table;
  const int32_t* lens;
  void* out;
  float* lse;
  float* part_o;             // [2 workgroups][n_q_heads][d]
  float2* part_ml;           // [2 workgroups][n_q_heads]
  int2* part_of;             // [n_seqs]: a sequence's first slot and its number of pieces
  int n_seqs, hq, hkv, group, d, n_pages, max_pages, head_tiles;
  int target;                // workgroups of a head at the most
  int whole;                 // 1: one to each sequence, and nothing is cut (with START only)
  float c;                   // scale * log2 e
  FastDiv page;
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
  int lens;                    // lane i: the positions of sequence i < 64; of the only one where nothing is cut
};
// One piece of a sequence, for one key-value head and up to 16 of its query heads.
struct Piece {
  int seq, head, h0, heads;    // key-value head; first query head and their number
  int len;                     // positions of the sequence
  int begin, end;              // tiles
  int whole;                   // 1: the sequence is this piece alone
  int slot;                    // where the piece's sums go if not: two slots to a workgroup
};
// START: what beginning a sequence costs a workgroup, in tiles; every sequence's share has so many ahead of its own.
template <int START>
__device__ __forceinline__ int seq_share(const DecodeAttnArgs& a, int s) {
  return max(tiles_of(seq_len(a, s)), 1) + START;
}

// The least share of a workgroup.  With START: less where it gives a sequence few pieces to join.  One sequence of 4000 by 8 heads
// of 128: 10.3 us with 8, 12.0 with 16; of 16000 13.3 and 12.4, of 71180 on one head 18.0 and 15.3.
constexpr int kFewTiles = 256;       // of a sequence on the average
template <int START>
__device__ __forceinline__ int least_share(const DecodeAttnArgs& a, long long total) {
  if (START == 0) return kMinTiles;
  return total <= (long long)kFewTiles * a.n_seqs ? 8 : 16;
}

template <int START = 0>
__device__ __forceinline__ bool find_span(const DecodeAttnArgs& a, Span& s) {
  const int lane = threadIdx.x & (kWave - 1);
  if (START > 0 && a.whole) {
    s.lens = seq_len(a, blockIdx.x);
    s.seq = blockIdx.x;
    s.local = 0;
    s.left = s.per = max(tiles_of(s.lens), 1) + START;
    s.fresh = true;
    return true;
  }
  s.lens = lane < a.n_seqs ? seq_len(a, lane) : 0;
  const int c0 = lane < a.n_seqs ? max(tiles_of(s.lens), 1) + START : 0;
  const int incl0 = wave_scan(c0);
  long long total = __builtin_amdgcn_readlane(incl0, kWave - 1);
  for (int base = kWave; base < a.n_seqs; base += kWave) {
    long long c = base + lane < a.n_seqs ? seq_share<START>(a, base + lane) : 0;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) c += __shfl_xor(c, off, kWave);
    total += c;
  }
  const int per = (int)max((total + a.target - 1) / a.target, (long long)least_share<START>(a, total));
  const long long start = (long long)blockIdx.x * per;
  if (start >= total) return false;
  long long before = 0;
  int c = c0, incl = incl0, base = 0;
  uint64_t past;
  while (!(past = __ballot(before + incl > start))) {
    before += __builtin_amdgcn_readlane(incl, kWave - 1);
    base += kWave;
    if (base >= a.n_seqs) return false;
    c = base + lane < a.n_seqs ? seq_share<START>(a, base + lane) : 0;
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

// The next piece of a workgroup's share; false if the share ends in a sequence's START, whose tiles are the next workgroup's.
template <int START>
__device__ __forceinline__ bool next_piece(const DecodeAttnArgs& a, Span& s, Piece& p) {
  p.seq = s.seq;
  const int ht = blockIdx.y / a.hkv;
  p.head = blockIdx.y % a.hkv;
  p.heads = min(a.group - 16 * ht, 16);
  p.h0 = p.head * a.group + 16 * ht;
  p.len = START > 0 && a.whole ? s.lens : s.seq < kWave ? __builtin_amdgcn_readlane(s.lens, s.seq) : seq_len(a, s.seq);
  const int tiles = tiles_of(p.len), share = max(tiles, 1) + START;
  const int take = min(share - s.local, s.left), upto = s.local + take;
  const bool some = upto > START, begins = some && s.local <= START;
  p.begin = max(s.local - START, 0);
  p.end = min(upto - START, tiles);
  p.whole = begins && upto == share;
  // a piece that starts inside its sequence is its workgroup's first, one that ends inside its last
  p.slot = 2 * blockIdx.x + (s.local == 0 && !s.fresh);
  if (begins && blockIdx.y == 0 && threadIdx.x == 0) {
    const int more = share - upto;                              // tiles in the workgroups after this one
    a.part_of[p.seq] = make_int2(p.slot, 1 + (more + s.per - 1) / s.per);
  }
  s.left -= take;
  ++s.seq;
  s.local = 0;
  s.fresh = false;
  return some;
}
__device__ __forceinline__ Piece next_piece(const DecodeAttnArgs& a, Span& s) {
  Piece p;
  next_piece<0>(a, s, p);
  return p;
}

// Largest of the four lanes that hold one column (lanes col, col + 16, + 32, + 48), on each of them.
__device__ __forceinline__ float across_groups_max(float v) {
  const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1]));
  const auto q = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}

// 16 bytes that are read once.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint4 stream_load16(const void* p) {
  const u32x4 v = __builtin_nontemporal_load(static_cast<const u32x4*>(p));
  return make_uint4(v[0], v[1], v[2], v[3]);
}
// Joins the waves and writes the piece's result: lane (col, g) holds dimensions NV * (4 g + r) + i of query
// head col, its maximum and its own positions' sum; with SCALED, `unit` is what
// one of o stands for.
template <int DT, int DP, bool SCALED, int WAVES = kWaves>
__device__ __forceinline__ void finish(const DecodeAttnArgs& a, const Piece& p, const f32x4 (&o)[DP / 16], float unit, float m,
                                       float l) {
  constexpr int NV = DP / 16;
  __shared__ float s_o[WAVES][16][DP + 4];
  __shared__ float s_m[WAVES][16], s_l[WAVES][16];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int col = lane & 15, g = lane >> 4;
  l += __shfl_xor(l, 16, kWave);
  l += __shfl_xor(l, 32, kWave);
  if (g == 0) s_m[wave][col] = m, s_l[wave][col] = l;
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int i = 0; i < NV; ++i) s_o[wave][col][NV * (4 * g + r) + i] = SCALED ? o[i][r] * unit : o[i][r];
  __syncthreads();
  for (int e = threadIdx.x; e < p.heads * (DP / 2); e += WAVES * kWave) {
    const int h = e / (DP / 2), dim = e % (DP / 2) * 2;
    if (dim >= a.d) continue;
    float mx = s_m[0][h];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) mx = fmaxf(mx, s_m[w][h]);
    const float base = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f, x0 = 0.f, x1 = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
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
template <int DT, int RUNS>
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

// Workgroups of a head: no more than the table has room for.
inline int units_of(const DecodeAttnArgs& a, int start = 0) {
  const int64_t room = ((int64_t)a.max_pages * a.page.d + kTile - 1) / kTile;
  const int64_t total = (std::max<int64_t>(room, 1) + start) * a.n_seqs, few = (int64_t)kFewTiles * a.n_seqs;
  int64_t most = (total + kMinTiles - 1) / kMinTiles;
  if (start) most = std::max((std::min(total, few) + 7) / 8, (total + 15) / 16);   // by either of the least shares
  return (int)std::min<int64_t>(a.target, most);
}
template <int DT>
hipError_t join_pieces(const DecodeAttnArgs& a, int units, hipStream_t st) {
  // one workgroup to a head cuts nothing
  if (units == 1) return hipSuccess;
  // runs side by side where a sequence has 8 pieces or more on the average: four sequences of up to 30000 on 2 heads take
  // 18.5 us so and 29.0 us in one run; where most have few, more workgroups only cost their start
  const int quads = a.hq * (a.d / 4);
  if (units >= 8 * a.n_seqs) {
    const dim3 join(a.n_seqs, (quads + kJoinThreads / 8 - 1) / (kJoinThreads / 8));
    hipLaunchKernelGGL((k_attention_decode_join<DT, 8>), join, dim3(kJoinThreads), 0, st, a);
  } else {
    const dim3 join(a.n_seqs, (quads + kJoinThreads - 1) / kJoinThreads);
    hipLaunchKernelGGL((k_attention_decode_join<DT, 1>), join, dim3(kJoinThreads), 0, st, a);
  }
  return hipGetLastError();
}
inline DecodeAttnArgs decode_args(const spa_heads& q, int n_seqs, int n_q_heads, const spa_kv_cache& c, const int32_t* table,
                                  int max_pages, const int32_t* lens, float scale, void* out, float* lse, float* part_o,
                                  float* part_ml, int32_t* part_of) {
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
  return a;
}

}  // namespace

}  // namespace spa
