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
// and the V reads (four pieces of four rows) then fall on distinct banks.
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
  int tq, tk, hq, hkv, group, d, n_seqs, causal;
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
  constexpr int kLoads = BN * CH / kThreads;      // direct loads of a wave per tile and operand
  extern __shared__ __align__(16) char s_kv[];    // [2 stages][K, V][BN][CH] pieces

  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int l32 = lane & 31, g = lane >> 5;

  const int kvh = blockIdx.x % a.hkv;
  const int rest = blockIdx.x / a.hkv;
  const int head = kvh * a.group + rest % a.group;
  int seq, local;
  locate(rest / a.group, a.n_seqs, [&](int s) {
    int first, count;
    seq_rows(a.cu_q, s, a.tq, first, count);
    return (count + kBM - 1) / kBM;
  }, seq, local);
  if (seq >= a.n_seqs) return;
  seq = __builtin_amdgcn_readfirstlane(seq);
  local = __builtin_amdgcn_readfirstlane(local);
  int q_first, lq, k_first, lk;
  seq_rows(a.cu_q, seq, a.tq, q_first, lq);
  seq_rows(a.cu_k, seq, a.tk, k_first, lk);
  // a sequence's last tile of queries sees the most keys: it comes first
  const int m0 = ((lq + kBM - 1) / kBM - 1 - local) * kBM;
  const int shift = lk - lq;                                    // query i sees keys 0..i + shift
  const int row = m0 + wave * kWaveRows + l32;                  // this lane's query
  const int sees = a.causal ? clamp_to(min(row, lq - 1) + shift + 1, 0, lk) : lk;        // its first hidden key
  const int m_last = min(m0 + kBM, lq) - 1;
  const int k_end = a.causal ? clamp_to(m_last + shift + 1, 0, lk) : lk;                 // the workgroup's
  const int full = a.causal ? clamp_to(m0 + wave * kWaveRows + shift + 1, 0, lk) : lk;   // keys that all rows see
  const int wave_end = a.causal ? clamp_to(m0 + wave * kWaveRows + kWaveRows + shift, 0, lk) : lk;   // keys that any sees

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

  // a tile's direct loads: lane -> (row, stored piece); rows past the end repeat the last one, pieces past
  // head_dim repeat the first (they meet zeros of Q, or give columns of O that are not stored)
  const uint16_t* kbase = a.k + (size_t)k_first * a.k_row + (size_t)kvh * a.k_head;
  const uint16_t* vbase = a.v + (size_t)k_first * a.v_row + (size_t)kvh * a.v_head;
  auto stage = [&](int j0, int buf) {
    const uint32_t lds = lds_addr(s_kv) + buf * 2 * kTileBytes;
    const int left = lk - 1 - j0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int slot = (wave * kLoads + i) * kWave + lane;
      const int r = slot / CH;
      int piece = (slot % CH) ^ swz<CH>(r);
      if (piece * 8 >= a.d) piece = 0;
      const int rr = min(r, left);
      const uint32_t to = __builtin_amdgcn_readfirstlane(lds + (wave * kLoads + i) * kWave * 16);
      lds_dma16(kbase + (size_t)j0 * a.k_row, (uint32_t)(rr * (int)a.k_row + piece * 8) * 2, to);
      lds_dma16(vbase + (size_t)j0 * a.v_row, (uint32_t)(rr * (int)a.v_row + piece * 8) * 2, to + kTileBytes);
    }
  };

  f32x16 o[DB];
#pragma unroll
  for (int b = 0; b < DB; ++b)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[b][r] = 0.f;
  float m = -INFINITY, l = 0.f;

  if (k_end > 0) stage(0, 0);
  int buf = 0;
  for (int j0 = 0; j0 < k_end; j0 += BN, buf ^= 1) {
    wait_vm<0>(0);
    bare_barrier();
    if (j0 + BN < k_end) stage(j0 + BN, buf ^ 1);
    if (j0 >= wave_end) continue;        // every row of this wave ends before this tile
    const char* ks = s_kv + buf * 2 * kTileBytes;
    const char* vs = ks + kTileBytes;

    f32x16 s[NB];
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
    // register r of block b is key j0 + 32 b + 8 (r / 4) + 4 g + r % 4
    if (j0 + BN > full) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (j0 + 32 * b + 8 * (r / 4) + 4 * g + r % 4 >= sees) s[b][r] = -INFINITY;
    }
    float mx = s[0][0];
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[b][r]);
    mx = fmaxf(mx, __shfl_xor(mx, 32, kWave)) * a.c;
    if (__any(mx > m + kSlack)) {
      const float now = fmaxf(mx, m), alpha = exp2_hw(m - (now == -INFINITY ? 0.f : now));
      m = now;
      l *= alpha;
#pragma unroll
      for (int b = 0; b < DB; ++b) o[b] *= alpha;
    }
    const float base = m == -INFINITY ? 0.f : m;
    float sum = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[b][r] = exp2_hw(fmaf(s[b][r], a.c, -base));
        sum += s[b][r];
      }
    l += sum;
#pragma unroll
    for (int t = 0; t < BN / 16; ++t) {
      const f32x16& p = s[t / 2];
      const int r0 = t % 2 * 8;
      const uint4 pf = make_uint4(pack2<DT>(p[r0], p[r0 + 1]), pack2<DT>(p[r0 + 2], p[r0 + 3]),
                                  pack2<DT>(p[r0 + 4], p[r0 + 5]), pack2<DT>(p[r0 + 6], p[r0 + 7]));
      // lane (16-lane group q, i): row 16 t + 4 g + i / 4 (then + 8), dimensions 32 b + 16 (q % 2) + 4 (i % 4)
      const int vrow = 16 * t + 4 * g + ((lane & 15) >> 2);
      const int piece = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
#pragma unroll
      for (int b = 0; b < DB; ++b) {
        const uint2 lo = lds_read_tr(vs + (vrow * CH + ((4 * b + piece) ^ swz<CH>(vrow))) * 16 + 8 * (lane & 1));
        const uint2 hi = lds_read_tr(vs + ((vrow + 8) * CH + ((4 * b + piece) ^ swz<CH>(vrow + 8))) * 16 + 8 * (lane & 1));
        o[b] = mfma32<DT>(make_uint4(lo.x, lo.y, hi.x, hi.y), pf, o[b]);
      }
    }
  }

  l += __shfl_xor(l, 32, kWave);
  if (row >= lq) return;
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const size_t to = (size_t)(q_first + row) * a.hq + head;
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
  if (a.lse && g == 0) a.lse[to] = l > 0.f ? kLn2 * (m + log2_hw(l)) : -INFINITY;
}

template <int DT, int DP, int BN>
hipError_t go(const PrefillAttnArgs& a, hipStream_t st) {
  const int tiles = a.tq / kBM + a.n_seqs;          // at least the sum over sequences of ceil(rows / kBM)
  hipLaunchKernelGGL((k_attention_prefill<DT, DP, BN>), dim3(tiles * a.hq), dim3(kThreads), 4 * BN * DP * 2, st, a);
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
                                    hipStream_t st) {
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
  a.c = scale * kLog2e;
  return dtype == SPA_F16 ? by_dim<SPA_F16>(a, st) : by_dim<SPA_BF16>(a, st);
}

}  // namespace spa
