// Attention over packed prompts: out = softmax(scale Q K^T + mask) V with grouped heads.
//
// A workgroup of four waves takes 128 query rows of one head, 32 to a wave, and passes once over the keys it
// can see in tiles of BN, with the running maximum and sum of the softmax in registers.
//   S^T = K Q^T on v_mfma_f32_32x32x16: a lane's 32 x 32 result column is one query, so the row maximum and sum
//         are in-lane but for one exchange with lane ^ 32, and one query's statistics are one register;
//   O^T = V^T P^T: the result registers of S^T are, packed to 16 bits, the P^T operand as they stand (the order
//         of the keys along the product is free); V^T operands are read from LDS by the transposing 64-bit read.
// K and V tiles go from memory to LDS directly, two stages deep, the next tile on its way while this one is
// worked on.  A row's 16-byte pieces are stored at piece ^ swz(row): both the K reads (one piece of 16 rows)
// and the V reads (four pieces of four rows) then fall on distinct banks.  Where few query rows meet many keys, a
// tile's keys are divided over workgroups and a second kernel joins the pieces.
//
// Bound by the matrix cores and the vector unit together (32 exponentials of 16 cycles beside 32 matrix instructions
// of 32 per lane and 64 keys).  One causal prompt of 8192 by 32 heads of 128 on 8: 522 us, 1053 TFLOP/s (a large
// library product reaches 1112 on the same card), matrix cores busy 54 % at a sustained 1.98 GHz, no bank conflicts.
// Nine prompts of up to 1531: 94 us; three pieces over 4093 cached keys by 16 heads of 64: 30 us.
#include "spa_attn.h"
#include "spa_layer.h"

namespace spa {

namespace {

constexpr int kThreads = 256;
constexpr int kWaveRows = 32;
constexpr int kBM = kThreads / kWave * kWaveRows;

// The sums are kept relative to a reference that follows the running maximum only when that has risen by more than
// a factor of 2^kSlack for some row of the wave: weights then reach 2^8 at most, which both 16-bit types hold with
// their full precision, and the 64 multiplications per lane of a rescale are rare after the first tiles.
constexpr float kSlack = 8.f;

struct PrefillAttnArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_row, q_head, k_row, k_head, v_row, v_head;
  const int32_t* cu_q;
  const int32_t* cu_k;
  uint16_t* out;
  float* lse;
  float* part_o;             // splits > 1: [splits][tq][hq][d]
  float2* part_ml;           // splits > 1: [splits][tq][hq]
  int tq, tk, hq, hkv, group, d, n_seqs, causal;
  int splits;                // pieces of a tile's keys at the most
  float c;                   // scale * log2 e
};

__device__ __forceinline__ int clamp_to(int v, int lo, int hi) { return min(max(v, lo), hi); }
// Rows [first, first + count) of sequence s; offsets that are not ascending or run past the rows are cut.
__device__ __forceinline__ void seq_rows(const int32_t* cu, int s, int total, int& first, int& count) {
  first = clamp_to(cu[s], 0, total);
  count = clamp_to(cu[s + 1], first, total) - first;
}

// Where 16-byte piece p of a row is stored (CH pieces to a row).  Four rows 4i..4i+3 differ in the bits that
// select a quarter of the banks, 16 consecutive rows take 16 different places.
template <int CH>
__device__ __forceinline__ int swz(int row) {
  if constexpr (CH == 8) return (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
  else return ((row & 3) << 2) | ((row >> 2) & 3);
}

// One tile of queries: its sequence and rows, and the keys it can see.
struct Tile {
  int q_first, lq, k_first, lk;
  int m0;                      // first row within the sequence
  int k_end;                   // keys that any of its rows sees
};
__device__ __forceinline__ int visible_end(int row, int lq, int lk, int causal) {
  return causal ? clamp_to(row + lk - lq + 1, 0, lk) : lk;
}
// Fills in m0 and k_end of the tile that lies `from_end` tiles before its sequence's last.
__device__ __forceinline__ void place_tile(const PrefillAttnArgs& a, Tile& t, int from_end) {
  t.m0 = ((t.lq + kBM - 1) / kBM - 1 - from_end) * kBM;
  t.k_end = visible_end(min(t.m0 + kBM, t.lq) - 1, t.lq, t.lk, a.causal);
}
// Keys of one piece when a tile's are divided: whole BN steps, evenly, at least kMinSteps of them.
constexpr int kMinSteps = 4;
template <int BN>
__device__ __forceinline__ int piece_keys(int k_end, int splits) {
  const int steps = (k_end + BN - 1) / BN;
  return max((steps + splits - 1) / splits, kMinSteps) * BN;
}

// The tile with this number; the last tile of a sequence's queries, which sees the most keys, comes first.  Up to
// 64 sequences' offsets are read once, one to a lane.  Where the workgroups would fill the chip fewer than three
// times, the tiles of all causal sequences are ordered by their last one's keys less their distance from it (in steps
// of kBM), so that the longest work is not the last to start: 16 prompts of up to 1000 by 20 heads of 64 take 41 us so
// and 45.5 us in the sequences' order.  With more, equal work that starts together also waits together: nine prompts
// of up to 1531 by 32 heads of 128 take 97 us so and 92 us in order.
template <int DP>
__device__ __forceinline__ bool find_tile(const PrefillAttnArgs& a, int index, Tile& t) {
  constexpr uint32_t kPlaces = DP <= 64 ? 768 : DP <= 128 ? 512 : 256;      // workgroups on the chip at a time
  int seq, from_end = 0;
  if (a.n_seqs <= kWave) {
    const int lane = threadIdx.x & (kWave - 1);
    int qf = 0, lq = 0, kf = 0, lk = 0;
    if (lane < a.n_seqs) {
      seq_rows(a.cu_q, lane, a.tq, qf, lq);
      seq_rows(a.cu_k, lane, a.tk, kf, lk);
    }
    const int n = (lq + kBM - 1) / kBM;
    seq = kWave;
    if (a.causal && a.n_seqs > 1 && gridDim.x < 3 * kPlaces) {
      const int top = (lk + kBM - 1) / kBM;
      int level = n ? top : INT32_MIN, low = n ? top - n : INT32_MAX;        // levels (top - n, top] hold a lane's tiles
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) {
        level = max(level, __shfl_xor(level, off, kWave));
        low = min(low, __shfl_xor(low, off, kWave));
      }
      for (; level > low; --level) {
        uint64_t at = __ballot(level <= top && level > top - n);
        const int count = __popcll(at);
        if (index < count) {
          for (int i = 0; i < index; ++i) at &= at - 1;
          seq = __ffsll((unsigned long long)at) - 1;
          from_end = __shfl(top, seq, kWave) - level;
          break;
        }
        index -= count;
      }
    } else {
      const int incl = wave_scan(n);
      const uint64_t past = __ballot(incl > index);
      if (past) {
        seq = __ffsll((unsigned long long)past) - 1;
        from_end = index - __shfl(incl - n, seq, kWave);
      }
    }
    if (seq == kWave) return false;
    seq = __builtin_amdgcn_readfirstlane(seq);
    t.q_first = __builtin_amdgcn_readlane(qf, seq);
    t.lq = __builtin_amdgcn_readlane(lq, seq);
    t.k_first = __builtin_amdgcn_readlane(kf, seq);
    t.lk = __builtin_amdgcn_readlane(lk, seq);
  } else {
    locate(index, a.n_seqs, [&](int s) {
      int first, count;
      seq_rows(a.cu_q, s, a.tq, first, count);
      return (count + kBM - 1) / kBM;
    }, seq, from_end);
    if (seq >= a.n_seqs) return false;
    seq = __builtin_amdgcn_readfirstlane(seq);
    seq_rows(a.cu_q, seq, a.tq, t.q_first, t.lq);
    seq_rows(a.cu_k, seq, a.tk, t.k_first, t.lk);
  }
  place_tile(a, t, from_end);
  return true;
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
// 64 bits per lane, transposed in each group of 16 lanes: lane i gets element i % 4 of lanes i/4, 4 + i/4,
// 8 + i/4 and 12 + i/4.
__device__ __forceinline__ uint2 lds_read_tr(const char* p) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
}

// What a wave of workgroup `block` works on: 32 query rows of one head and the keys of its workgroup's piece.
struct Place {
  int head, kvh, split;
  int q_first, lq, k_first, lk;
  int k_begin, k_end;          // the piece's keys
  bool whole;                  // the piece is all of the tile's keys
  int w0;                      // the wave's first row within the sequence
  int full, wave_end;          // keys that all its rows see, and the end of the piece's that any does
};
// The number of block's tile, for find_tile.
__device__ __forceinline__ int tile_number(const PrefillAttnArgs& a, int block) {
  return block / a.hkv / a.group / a.splits;
}
// False if the tile has no keys for the workgroup's piece.
template <int BN>
__device__ __forceinline__ bool place_wave(const PrefillAttnArgs& a, int block, int wave, const Tile& t, Place& p) {
  // key-value heads fastest (one XCD keeps to as few of them as there are), then the query heads that share one
  p.kvh = block % a.hkv;
  const int rest = block / a.hkv;
  p.head = p.kvh * a.group + rest % a.group;
  p.split = rest / a.group % a.splits;
  // one value for the wave, whichever way it was found: tile bases stay in scalar registers
  p.q_first = __builtin_amdgcn_readfirstlane(t.q_first), p.lq = __builtin_amdgcn_readfirstlane(t.lq);
  p.k_first = __builtin_amdgcn_readfirstlane(t.k_first), p.lk = __builtin_amdgcn_readfirstlane(t.lk);
  const int m0 = __builtin_amdgcn_readfirstlane(t.m0), tile_end = __builtin_amdgcn_readfirstlane(t.k_end);
  const int per = piece_keys<BN>(tile_end, a.splits);
  p.k_begin = p.split * per;                                    // this piece's keys: [k_begin, k_end)
  p.k_end = min(p.k_begin + per, tile_end);
  p.whole = tile_end <= per;
  p.w0 = m0 + wave * kWaveRows;
  p.full = visible_end(p.w0, p.lq, p.lk, a.causal);
  p.wave_end = min(visible_end(p.w0 + kWaveRows - 1, p.lq, p.lk, a.causal), p.k_end);
  return !p.split || p.k_begin < tile_end;
}

// A 16-bit value into its half of a word: itself if it is finite; else 1 into `plus` for +inf, `minus` for -inf, both for NaN.
template <int DT> constexpr uint32_t kOne16 = DT == SPA_BF16 ? 0x3F80u : 0x3C00u;
template <int DT>
__device__ __forceinline__ void take_out(uint32_t h, int sh, uint32_t& v, uint32_t& plus, uint32_t& minus) {
  constexpr uint32_t kInf = DT == SPA_BF16 ? 0x7F80u : 0x7C00u;
  const uint32_t size = h & 0x7FFFu;
  if (size < kInf) v |= h << sh;
  if (size > kInf || h == kInf) plus |= kOne16<DT> << sh;
  if (size > kInf || h == (kInf | 0x8000u)) minus |= kOne16<DT> << sh;
}

// Hides what a lane's row does not see of the scores of tile j0: register r of block b is key 32 b + 8 (r / 4) + 4 g + r % 4.
template <int BN>
__device__ __forceinline__ void hide(f32x16 (&s)[BN / 32], int j0, int full, int sees, int g) {
  if (j0 + BN <= full) return;
  const int hidden = sees - j0 - 4 * g;
#pragma unroll
  for (int b = 0; b < BN / 32; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r)
      if (32 * b + 8 * (r / 4) + r % 4 >= hidden) s[b][r] = -INFINITY;
}
// The largest score of the row, both halves of the wave, in the exponent's unit.
template <int NB>
__device__ __forceinline__ float row_max(const f32x16 (&s)[NB], float c) {
  float v = s[0][0];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) v = fmaxf(v, s[b][r]);
  const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1])) * c;
}
// The reference m and what is relative to it follow the tile's maximum mx.
template <int N>
__device__ __forceinline__ void follow(float mx, float& m, float& l, f32x16 (&o)[N]) {
  if (__any(mx > m + kSlack)) {
    const float now = fmaxf(mx, m), alpha = exp2_hw(m - (now == -INFINITY ? 0.f : now));
    m = now;
    l *= alpha;
#pragma unroll
    for (int b = 0; b < N; ++b) o[b] *= alpha;
  }
}
// Scores to weights, rounded to the 16-bit type as operands of the product with V; their sum, unrounded, goes to l.  The
// rounding is the output's own unit roundoff on each weight: 0.0021 of the 2-norm against 0.0016 for float32 weights
// (8192 bfloat16 keys); two 16-bit parts of a weight would double the product with V, half of all matrix work.
template <int DT, int NB>
__device__ __forceinline__ void weights(f32x16 (&s)[NB], uint4 (&pf)[2 * NB], float c, float m, float& l) {
  const float base = m == -INFINITY ? 0.f : m;
  float sum = 0.f;
#pragma unroll
  for (int t = 0; t < 2 * NB; ++t) {
    f32x16& p = s[t / 2];
    const int r0 = t % 2 * 8;
#pragma unroll
    for (int r = r0; r < r0 + 8; ++r) {
      p[r] = exp2_hw(fmaf(p[r], c, -base));
      sum += p[r];
    }
    pf[t] = make_uint4(pack2<DT>(p[r0], p[r0 + 1]), pack2<DT>(p[r0 + 2], p[r0 + 3]), pack2<DT>(p[r0 + 4], p[r0 + 5]),
                       pack2<DT>(p[r0 + 6], p[r0 + 7]));
  }
  l += sum;
  asm volatile("" : "+v"(l));      // the sum is taken here, not after the product that follows
}

// Writes blocks of 32 dimensions, from `first` on, of the wave's outputs or of its piece of them; l is the row's sum.
template <int DT, int N>
__device__ __forceinline__ void store_blocks(const PrefillAttnArgs& a, const Place& p, int row, int g, const f32x16 (&o)[N],
                                             int first, float m, float l) {
  if (row >= p.lq) return;
  const size_t to = (size_t)(p.q_first + row) * a.hq + p.head;
  const bool stats = first == 0 && g == 0;
  if (!p.whole) {
    const size_t at = (size_t)p.split * a.tq * a.hq + to;
#pragma unroll
    for (int b = 0; b < N; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int dim = 32 * (first + b) + 8 * r + 4 * g;
        if (dim < a.d)
          *reinterpret_cast<float4*>(a.part_o + at * a.d + dim) =
              make_float4(o[b][4 * r], o[b][4 * r + 1], o[b][4 * r + 2], o[b][4 * r + 3]);
      }
    if (stats) a.part_ml[at] = make_float2(m, l);
    return;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int b = 0; b < N; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int at = 32 * (first + b) + 8 * r + 4 * g;
      if (at < a.d)
        *reinterpret_cast<uint2*>(a.out + to * a.d + at) =
            make_uint2(pack2<DT>(o[b][4 * r] * inv, o[b][4 * r + 1] * inv),
                       pack2<DT>(o[b][4 * r + 2] * inv, o[b][4 * r + 3] * inv));
    }
  if (a.lse && stats) a.lse[to] = l == 0.f ? -INFINITY : kLn2 * (m + log2_hw(l));
}

// The wave's work again, by itself, from memory and 32 dimensions at a time: infinities and NaN are taken out of the values,
// and two more products with 1 for each key that a row sees find the rows that they belong to.  The arguments and the place
// are found anew, so that nothing for this stays in registers beside the first walk.
template <int DT, int DP, int BN>
__device__ __forceinline__ void walk_again(int wave) {
  constexpr int KS = DP / 16, NB = BN / 32, DB = DP / 32;
  auto kernarg = __builtin_amdgcn_kernarg_segment_ptr();
  int block = blockIdx.x;
  asm volatile("" : "+s"(kernarg), "+s"(block));
  const PrefillAttnArgs a = *(const PrefillAttnArgs*)kernarg;
  Tile tile;
  Place p;
  if (!find_tile<DP>(a, tile_number(a, block), tile) || !place_wave<BN>(a, block, wave, tile, p)) return;
  const int lane = threadIdx.x & (kWave - 1), l32 = lane & 31, g = lane >> 5;
  const int row = p.w0 + l32, sees = visible_end(min(row, p.lq - 1), p.lq, p.lk, a.causal);
  const uint16_t* q = a.q + (size_t)(p.q_first + min(row, p.lq - 1)) * a.q_row + (size_t)p.head * a.q_head;
  const uint16_t* kbase = a.k + (size_t)p.k_first * a.k_row + (size_t)p.kvh * a.k_head;
  const uint16_t* vbase = a.v + (size_t)p.k_first * a.v_row + (size_t)p.kvh * a.v_head;
#pragma unroll 1
  for (int b = 0; b < DB; ++b) {
    const int dim = min(32 * b + l32, a.d - 1);
    f32x16 ob[1], zero;
#pragma unroll
    for (int r = 0; r < 16; ++r) ob[0][r] = zero[r] = 0.f;
    float m = -INFINITY, l = 0.f;
#pragma unroll 1
    for (int j0 = p.k_begin; j0 < p.wave_end; j0 += BN) {
      f32x16 s0[NB];
#pragma unroll
      for (int c = 0; c < NB; ++c) {
        s0[c] = zero;
        const uint16_t* k = kbase + (size_t)min(j0 + 32 * c + l32, p.lk - 1) * a.k_row;
#pragma unroll
        for (int t = 0; t < KS; ++t) {
          const int at = 16 * t + 8 * g;
          uint4 kf = make_uint4(0, 0, 0, 0), qf = kf;
          if (at < a.d) {
            kf = *reinterpret_cast<const uint4*>(k + at);
            qf = *reinterpret_cast<const uint4*>(q + at);
          }
          s0[c] = mfma32<DT>(kf, qf, s0[c]);
        }
      }
      hide<BN>(s0, j0, p.full, sees, g);
      follow(row_max(s0, a.c), m, l, ob);
      uint4 pf[BN / 16];
      weights<DT>(s0, pf, a.c, m, l);
#pragma unroll
      for (int t = 0; t < BN / 16; ++t) {
        uint32_t v[4] = {}, plus[4] = {}, minus[4] = {}, one[4] = {};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int key = j0 + 16 * t + 8 * (e / 4) + 4 * g + e % 4, sh = 16 * (e % 2);
          take_out<DT>(vbase[(size_t)min(key, p.lk - 1) * a.v_row + dim], sh, v[e / 2], plus[e / 2], minus[e / 2]);
          if (key < sees) one[e / 2] |= kOne16<DT> << sh;
        }
        const auto part = [](const uint32_t (&w)[4]) { return make_uint4(w[0], w[1], w[2], w[3]); };
        ob[0] = mfma32<DT>(part(v), pf[t], ob[0]);
        const f32x16 up = mfma32<DT>(part(plus), part(one), zero);
#pragma unroll
        for (int r = 0; r < 16; ++r) ob[0][r] = up[r] > 0.f ? ob[0][r] + INFINITY : ob[0][r];
        const f32x16 down = mfma32<DT>(part(minus), part(one), zero);
#pragma unroll
        for (int r = 0; r < 16; ++r) ob[0][r] = down[r] > 0.f ? ob[0][r] - INFINITY : ob[0][r];
      }
    }
    l += __shfl_xor(l, 32, kWave);
    store_blocks<DT>(a, p, row, g, ob, b, m, l);
  }
}

template <int DT, int DP, int BN>
__global__ void __launch_bounds__(kThreads, DP <= 128 ? 2 : 1) k_attention_prefill(PrefillAttnArgs a) {
  constexpr int CH = DP / 8;             // 16-byte pieces of a row
  constexpr int KS = DP / 16;            // k steps of S
  constexpr int NB = BN / 32;            // 32-key blocks of a tile
  constexpr int DB = DP / 32;            // 32-dimension blocks of O
  constexpr int kTileBytes = BN * DP * 2;
  constexpr bool kAhead = DP <= 128;     // the next tile's scores run beside this tile's softmax (registers allow it)
  constexpr int kLoads = BN * CH / kThreads;      // direct loads of a wave per tile and operand
  extern __shared__ __align__(16) char s_kv[];    // [K, V][2 stages][BN][CH] pieces

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int l32 = lane & 31, g = lane >> 5;

  Tile tile;
  if (!find_tile<DP>(a, tile_number(a, blockIdx.x), tile)) return;
  Place p;
  if (!place_wave<BN>(a, blockIdx.x, wave, tile, p)) return;
  const int head = p.head, kvh = p.kvh, q_first = p.q_first, lq = p.lq, k_first = p.k_first, lk = p.lk;
  const int k_begin = p.k_begin, k_end = p.k_end, full = p.full, wave_end = p.wave_end;
  const int row = p.w0 + l32;                                   // this lane's query
  const int sees = visible_end(min(row, lq - 1), lq, lk, a.causal);                       // its first hidden key

  // a tile's direct loads: lane -> (row, stored piece); rows past the end repeat the last one, pieces past
  // head_dim repeat the first (they meet zeros of Q, or give columns of O that are not stored; where they hold an infinity
  // the sums show it, and the second walk reads neither)
  const uint16_t* kbase = a.k + (size_t)k_first * a.k_row + (size_t)kvh * a.k_head;
  const uint16_t* vbase = a.v + (size_t)k_first * a.v_row + (size_t)kvh * a.v_head;
  auto stage = [&](const uint16_t* base, int64_t stride, int j0, uint32_t lds) {
    const int left = lk - 1 - j0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int slot = (wave * kLoads + i) * kWave + lane;
      const int r = slot / CH;
      int piece = (slot % CH) ^ swz<CH>(r);
      if (piece * 8 >= a.d) piece = 0;
      const uint32_t to = __builtin_amdgcn_readfirstlane(lds + (wave * kLoads + i) * kWave * 16);
      lds_dma16(base + (size_t)j0 * stride, (uint32_t)(min(r, left) * (int)stride + piece * 8) * 2, to);
    }
  };
  auto stage_k = [&](int j0, int buf) {
    if (j0 < k_end) stage(kbase, a.k_row, j0, lds_addr(s_kv) + buf * kTileBytes);
  };
  auto stage_v = [&](int j0, int buf) {
    if (j0 < k_end) stage(vbase, a.v_row, j0, lds_addr(s_kv) + (2 + buf) * kTileBytes);
  };

  // the first keys, the queries, the keys after and the first values: all on their way at once
  stage_k(k_begin, 0);
  uint4 qf[KS];
  {
    const uint16_t* q = a.q + (size_t)(q_first + min(row, lq - 1)) * a.q_row + (size_t)head * a.q_head;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int at = 16 * s + 8 * g;
      qf[s] = make_uint4(0, 0, 0, 0);
      if (at < a.d) qf[s] = *reinterpret_cast<const uint4*>(q + at);
    }
  }
  if constexpr (kAhead) stage_k(k_begin + BN, 1);
  stage_v(k_begin, 0);

  f32x16 o[DB];
#pragma unroll
  for (int b = 0; b < DB; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[b][r] = 0.f;
  float m = -INFINITY, l = 0.f, mx = -INFINITY;

  // the scores of the tile in K buffer `buf`: register r of block b is key 32 b + 8 (r / 4) + 4 g + r % 4
  auto scores = [&](f32x16 (&s)[NB], int buf) {
    const char* ks = s_kv + buf * kTileBytes;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int r = 0; r < 16; ++r) s[b][r] = 0.f;
      const int krow = 32 * b + l32;
#pragma unroll
      for (int t = 0; t < KS; ++t) {
        const uint4 kf = *reinterpret_cast<const uint4*>(ks + (krow * CH + ((2 * t + g) ^ swz<CH>(krow))) * 16);
        s[b] = mfma32<DT>(kf, qf[t], s[b]);
      }
    }
  };
  auto values = [&](const uint4 (&pf)[BN / 16], int buf) {
    const char* vs = s_kv + (2 + buf) * kTileBytes;
#pragma unroll
    for (int t = 0; t < BN / 16; ++t) {
      // lane (16-lane group q, i): row 16 t + 4 g + i / 4 (then + 8), dimensions 32 b + 16 (q % 2) + 4 (i % 4)
      const int vrow = 16 * t + 4 * g + ((lane & 15) >> 2);
      const int piece = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
#pragma unroll
      for (int b = 0; b < DB; ++b) {
        const uint2 lo = lds_read_tr(vs + (vrow * CH + ((4 * b + piece) ^ swz<CH>(vrow))) * 16 + 8 * (lane & 1));
        const uint2 hi = lds_read_tr(vs + ((vrow + 8) * CH + ((4 * b + piece) ^ swz<CH>(vrow + 8))) * 16 + 8 * (lane & 1));
        o[b] = mfma32<DT>(make_uint4(lo.x, lo.y, hi.x, hi.y), pf[t], o[b]);
      }
    }
  };
  // Tile j0, whose scores are in `cur` (their maximum in mx), and the scores of the one after it: the next tile's
  // K Q^T does not depend on this tile's exponentials, so matrix and vector instructions run side by side.
  auto arrive = [&](int j0, int buf) {
    wait_vm<0>(0);
    bare_barrier();
    if constexpr (kAhead) stage_k(j0 + 2 * BN, buf);
    else stage_k(j0 + BN, buf ^ 1);
    stage_v(j0 + BN, buf ^ 1);
  };
  // the order of a step's instructions: fragments a few reads ahead, vector work between the matrix instructions
  auto interleave = [&]() {
    constexpr int kRead = 0x100, kMfma = 0x8, kVector = 0x402;
    __builtin_amdgcn_sched_group_barrier(kRead, 4, 0);
#pragma unroll
    for (int i = 0; i < NB * KS; ++i) {
      __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kRead, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kVector, 40 / KS, 0);
    }
#pragma unroll
    for (int i = 0; i < BN / 16 * DB; ++i) {
      __builtin_amdgcn_sched_group_barrier(kRead, 2, 0);
      __builtin_amdgcn_sched_group_barrier(kVector, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kMfma, 1, 0);
    }
  };
  auto step = [&](f32x16 (&cur)[NB], f32x16 (&nxt)[NB], int j0, int buf) {
    arrive(j0, buf);
    follow(mx, m, l, o);
    uint4 pf[BN / 16];
    scores(nxt, buf ^ 1);
    weights<DT>(cur, pf, a.c, m, l);
    values(pf, buf);
    interleave();
    hide<BN>(nxt, j0 + BN, full, sees, g);
    mx = row_max(nxt, a.c);
  };
  auto last = [&](f32x16 (&cur)[NB], int j0, int buf) {
    arrive(j0, buf);
    follow(mx, m, l, o);
    uint4 pf[BN / 16];
    weights<DT>(cur, pf, a.c, m, l);
    values(pf, buf);
  };

  if (k_begin < k_end) {
    int j0 = k_begin, buf = 0;
    if constexpr (kAhead) {
      wait_vm<0>(0);
      bare_barrier();
    }
    if constexpr (!kAhead) {
      for (; j0 < wave_end; j0 += BN, buf ^= 1) {
        arrive(j0, buf);
        f32x16 s0[NB];
        scores(s0, buf);
        hide<BN>(s0, j0, full, sees, g);
        mx = row_max(s0, a.c);
        follow(mx, m, l, o);
        uint4 pf[BN / 16];
        weights<DT>(s0, pf, a.c, m, l);
        values(pf, buf);
      }
    } else if (j0 < wave_end) {
      f32x16 s0[NB], s1[NB];
      scores(s0, 0);
      hide<BN>(s0, j0, full, sees, g);
      mx = row_max(s0, a.c);
      for (; j0 + 2 * BN < wave_end; j0 += 2 * BN) {
        step(s0, s1, j0, 0);
        step(s1, s0, j0 + BN, 1);
      }
      if (j0 + BN < wave_end) {
        step(s0, s1, j0, 0);
        last(s1, j0 + BN, 1);
        j0 += 2 * BN;
      } else {
        last(s0, j0, 0);
        j0 += BN;
        buf = 1;
      }
    }
    for (; j0 < k_end; j0 += BN, buf ^= 1) arrive(j0, buf);      // the other waves' tiles: this wave brings its part
  }

  // A value that a row does not see has weight 0, and 0 times an infinity or NaN is NaN.  Such a value in a tile that some
  // row sees in part, or in the last key's copies past the end, shows in the wave's sums.
  float none[DB];
#pragma unroll
  for (int b = 0; b < DB; ++b) {
    none[b] = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) none[b] = fmaf(o[b][r], 0.f, none[b]);
    if (b) none[0] += none[b];
  }
  if (__any(none[0] != 0.f)) {                                  // one is NaN
    walk_again<DT, DP, BN>(wave);
    return;
  }
  l += __shfl_xor(l, 32, kWave);
  store_blocks<DT>(a, p, row, g, o, 0, m, l);
}

// One workgroup per row and 1024 of its outputs: the pieces of the row's tile brought to their common maximum and
// added in order.  A thread takes four dimensions of one head.
template <int DT, int BN>
__global__ void __launch_bounds__(kThreads) k_attention_prefill_join(PrefillAttnArgs a) {
  const int lane = threadIdx.x & (kWave - 1);
  const int row = blockIdx.x;
  int seq = 0;                 // the number of sequences that end at or before the row
  for (int base = 0; base < a.n_seqs; base += kWave) {
    const int end = base + lane < a.n_seqs ? a.cu_q[base + lane + 1] : INT32_MAX;
    seq += __popcll(__ballot(end <= row));
  }
  if (seq >= a.n_seqs) return;
  Tile t;
  seq_rows(a.cu_q, seq, a.tq, t.q_first, t.lq);
  seq_rows(a.cu_k, seq, a.tk, t.k_first, t.lk);
  if (row < t.q_first || row >= t.q_first + t.lq) return;
  place_tile(a, t, (t.lq + kBM - 1) / kBM - 1 - (row - t.q_first) / kBM);
  const int per = piece_keys<BN>(t.k_end, a.splits);
  const int pieces = (t.k_end + per - 1) / per;
  if (pieces <= 1) return;
  const int quads = a.d / 4;
  const int at = blockIdx.y * kThreads + threadIdx.x;
  const int head = at / quads, dim = at % quads * 4;
  if (head >= a.hq) return;
  const size_t to = (size_t)row * a.hq + head, step = (size_t)a.tq * a.hq;
  float m = -INFINITY, sum = 0.f;
  for (int i = 0; i < pieces; ++i) m = fmaxf(m, a.part_ml[to + i * step].x);
  const float base = m == -INFINITY ? 0.f : m;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < pieces; ++i) {
    const float2 ml = a.part_ml[to + i * step];
    const float4 v = *reinterpret_cast<const float4*>(a.part_o + (to + i * step) * a.d + dim);
    const float f = exp2_hw(ml.x - base);
    sum += f * ml.y;
    x.x += f * v.x; x.y += f * v.y; x.z += f * v.z; x.w += f * v.w;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *reinterpret_cast<uint2*>(a.out + to * a.d + dim) =
      make_uint2(pack2<DT>(x.x * inv, x.y * inv), pack2<DT>(x.z * inv, x.w * inv));
  if (dim == 0 && a.lse) a.lse[to] = sum == 0.f ? -INFINITY : kLn2 * (m + log2_hw(sum));
}

template <int DT, int DP, int BN>
hipError_t go(const PrefillAttnArgs& a, hipStream_t st) {
  const int tiles = a.tq / kBM + a.n_seqs;          // at least the sum over sequences of ceil(rows / kBM)
  hipLaunchKernelGGL((k_attention_prefill<DT, DP, BN>), dim3(tiles * a.hq * a.splits), dim3(kThreads), 4 * BN * DP * 2, st, a);
  if (hipError_t e = hipGetLastError()) return e;
  if (a.splits == 1) return hipSuccess;
  const int groups = (a.hq * (a.d / 4) + kThreads - 1) / kThreads;
  hipLaunchKernelGGL((k_attention_prefill_join<DT, BN>), dim3(a.tq, groups), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}
template <int DT>
hipError_t by_dim(const PrefillAttnArgs& a, hipStream_t st) {
  if (a.d <= 64) return go<DT, 64, 64>(a, st);
  if (a.d <= 128) return go<DT, 128, 64>(a, st);
  return go<DT, 256, 32>(a, st);
}

}  // namespace

hipError_t launch_attention_prefill(const spa_heads& q, const spa_heads& k, const spa_heads& v, int dtype, int tq,
                                    int tk, int n_q_heads, int n_kv_heads, int head_dim, const int32_t* cu_q,
                                    const int32_t* cu_k, int n_seqs, bool causal, float scale, void* out, float* lse,
                                    int splits, float* part_o, float* part_ml, hipStream_t st) {
  PrefillAttnArgs a{};
  a.q = static_cast<const uint16_t*>(q.data);
  a.k = static_cast<const uint16_t*>(k.data);
  a.v = static_cast<const uint16_t*>(v.data);
  a.q_row = q.row_stride; a.q_head = q.head_stride;
  a.k_row = k.row_stride; a.k_head = k.head_stride;
  a.v_row = v.row_stride; a.v_head = v.head_stride;
  a.cu_q = cu_q; a.cu_k = cu_k;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.tq = tq; a.tk = tk; a.hq = n_q_heads; a.hkv = n_kv_heads; a.group = n_q_heads / n_kv_heads; a.d = head_dim;
  a.n_seqs = n_seqs; a.causal = causal;
  a.splits = splits; a.part_o = part_o; a.part_ml = reinterpret_cast<float2*>(part_ml);
  a.c = scale * kLog2e;
  return dtype == SPA_F16 ? by_dim<SPA_F16>(a, st) : by_dim<SPA_BF16>(a, st);
}

}  // namespace spa
