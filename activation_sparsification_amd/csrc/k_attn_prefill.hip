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
// of 32 per lane and 64 keys).  One causal prompt of 8192 by 32 heads of 128 on 8: 523 us, 1051 TFLOP/s (a large
// library product reaches 1112 on the same card), matrix cores busy 54 % at a sustained 1.98 GHz, no bank conflicts.
// Nine prompts of up to 1531: 93 us; three pieces over 4093 cached keys by 16 heads of 64: 30 us.
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

  // key-value heads fastest (one XCD keeps to as few of them as there are), then the query heads that share one
  const int kvh = blockIdx.x % a.hkv;
  const int rest = blockIdx.x / a.hkv;
  const int head = kvh * a.group + rest % a.group;
  const int split = rest / a.group % a.splits;
  Tile t;
  if (!find_tile<DP>(a, rest / a.group / a.splits, t)) return;
  // one value for the wave, whichever way it was found: tile bases stay in scalar registers
  const int q_first = __builtin_amdgcn_readfirstlane(t.q_first), lq = __builtin_amdgcn_readfirstlane(t.lq);
  const int k_first = __builtin_amdgcn_readfirstlane(t.k_first), lk = __builtin_amdgcn_readfirstlane(t.lk);
  const int m0 = __builtin_amdgcn_readfirstlane(t.m0), tile_end = __builtin_amdgcn_readfirstlane(t.k_end);
  const int per = piece_keys<BN>(tile_end, a.splits);
  const int k_begin = split * per;                              // this piece's keys: [k_begin, k_end)
  if (split && k_begin >= tile_end) return;
  const int k_end = min(k_begin + per, tile_end);
  const bool whole = tile_end <= per;
  const int w0 = m0 + wave * kWaveRows;
  const int row = w0 + l32;                                     // this lane's query
  const int sees = visible_end(min(row, lq - 1), lq, lk, a.causal);                       // its first hidden key
  const int full = visible_end(w0, lq, lk, a.causal);                                     // keys that all its wave sees
  const int wave_end = min(visible_end(w0 + kWaveRows - 1, lq, lk, a.causal), k_end);     // and that any does

  // a tile's direct loads: lane -> (row, stored piece); rows past the end repeat the last one, pieces past
  // head_dim repeat the first (they meet zeros of Q, or give columns of O that are not stored)
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
  auto mask = [&](f32x16 (&s)[NB], int j0) {
    if (j0 + BN <= full) return;
    const int hidden = sees - j0 - 4 * g;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (32 * b + 8 * (r / 4) + r % 4 >= hidden) s[b][r] = -INFINITY;
  };
  auto row_max = [&](const f32x16 (&s)[NB]) {
    float v = s[0][0];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) v = fmaxf(v, s[b][r]);
    const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(h[0]), __uint_as_float(h[1])) * a.c;
  };
  auto follow = [&]() {
    if (__any(mx > m + kSlack)) {
      const float now = fmaxf(mx, m), alpha = exp2_hw(m - (now == -INFINITY ? 0.f : now));
      m = now;
      l *= alpha;
#pragma unroll
      for (int b = 0; b < DB; ++b) o[b] *= alpha;
    }
  };
  auto weights = [&](f32x16 (&s)[NB], uint4 (&pf)[BN / 16]) {
    const float base = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int t = 0; t < BN / 16; ++t) {
      f32x16& p = s[t / 2];
      const int r0 = t % 2 * 8;
#pragma unroll
      for (int r = r0; r < r0 + 8; ++r) {
        p[r] = exp2_hw(fmaf(p[r], a.c, -base));
        sum += p[r];
      }
      pf[t] = make_uint4(pack2<DT>(p[r0], p[r0 + 1]), pack2<DT>(p[r0 + 2], p[r0 + 3]), pack2<DT>(p[r0 + 4], p[r0 + 5]),
                         pack2<DT>(p[r0 + 6], p[r0 + 7]));
    }
    l += sum;
    asm volatile("" : "+v"(l));      // the sum is taken here, not after the product that follows
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
    follow();
    uint4 pf[BN / 16];
    scores(nxt, buf ^ 1);
    weights(cur, pf);
    values(pf, buf);
    interleave();
    mask(nxt, j0 + BN);
    mx = row_max(nxt);
  };
  auto last = [&](f32x16 (&cur)[NB], int j0, int buf) {
    arrive(j0, buf);
    follow();
    uint4 pf[BN / 16];
    weights(cur, pf);
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
        mask(s0, j0);
        mx = row_max(s0);
        follow();
        uint4 pf[BN / 16];
        weights(s0, pf);
        values(pf, buf);
      }
    } else if (j0 < wave_end) {
      f32x16 s0[NB], s1[NB];
      scores(s0, 0);
      mask(s0, j0);
      mx = row_max(s0);
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

  l += __shfl_xor(l, 32, kWave);
  if (row >= lq) return;
  const size_t to = (size_t)(q_first + row) * a.hq + head;
  if (!whole) {
    const size_t at = (size_t)split * a.tq * a.hq + to;
#pragma unroll
    for (int b = 0; b < DB; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int dim = 32 * b + 8 * r + 4 * g;
        if (dim < a.d)
          *reinterpret_cast<float4*>(a.part_o + at * a.d + dim) =
              make_float4(o[b][4 * r], o[b][4 * r + 1], o[b][4 * r + 2], o[b][4 * r + 3]);
      }
    if (g == 0) a.part_ml[at] = make_float2(m, l);
    return;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int b = 0; b < DB; ++b)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int at = 32 * b + 8 * r + 4 * g;
      if (at < a.d)
        *reinterpret_cast<uint2*>(a.out + to * a.d + at) =
            make_uint2(pack2<DT>(o[b][4 * r] * inv, o[b][4 * r + 1] * inv),
                       pack2<DT>(o[b][4 * r + 2] * inv, o[b][4 * r + 3] * inv));
    }
  if (a.lse && g == 0) a.lse[to] = l == 0.f ? -INFINITY : kLn2 * (m + log2_hw(l));
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
