// Attention of one new token per sequence over its paged cache: out = softmax(scale q K^T) V.
//
// Bound: the cache is read once and every cached vector meets only the G query heads that share it, so the
// call is bound by HBM.  A wave works on tiles of 32 positions of one (sequence, key-value head) and keeps
// everything in registers:
//   S^T = K Q^T on v_mfma_f32_16x16x32: a lane's K operand is 16 consecutive bytes of a cached row, so keys go
//         from memory to the matrix cores with no LDS; the 16 columns are the query heads (zeros past G);
//   O^T = V^T P^T: the scores' own registers are the P operand (the order of the 32 positions along the
//         product is free, so it is taken as S^T leaves it: lane group g holds 4g..4g+3 and 16+4g..16+4g+3).
//         A lane reads those 8 positions' rows, 16 lanes to a row, and turns its 8 x 8 block with byte
//         permutes into one V^T operand per dimension.
// The running maximum and sum are one column (query head) per lane.  A sequence is cut into pieces so that
// there are about 1024 workgroups whatever the lengths; the cut is computed by every workgroup from the lengths
// on the device.  Pieces leave unnormalised float32 sums with their maximum, and a second kernel joins them in
// a fixed order.
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
  float* part_o;             // [units][n_q_heads][d]
  float2* part_ml;           // [units][n_q_heads]
  int n_seqs, hq, hkv, group, d, n_pages, max_pages, head_tiles;
  int target;                // pieces wanted over all sequences
  float c;                   // scale * log2 e
  FastDiv page;
};

// P is multiplied by the value vector's scale before it is rounded to 16 bits; a constant power of two keeps
// that product of ordinary values near 1 (it leaves with the final division).  Scales are max / 448 and
// max / 127: with a largest value of 1, 2^8 / 448 and 2^6 / 127 are about a half.
template <int FMT> constexpr float kPScale = FMT == SPA_KV_FP8 ? 256.f : FMT == SPA_KV_INT8 ? 64.f : 1.f;

__device__ __forceinline__ int seq_tiles(const DecodeAttnArgs& a, int s) {
  const int cap = a.max_pages * (int)a.page.d;
  return (min(max(a.lens[s], 0), cap) + kTile - 1) / kTile;
}

// The tiles of a piece: total tiles over the pieces wanted, the same on every wave.
__device__ __forceinline__ int piece_tiles(const DecodeAttnArgs& a) {
  const int lane = threadIdx.x & (kWave - 1);
  long long total = 0;
  for (int base = 0; base < a.n_seqs; base += kWave) total += base + lane < a.n_seqs ? seq_tiles(a, base + lane) : 0;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) total += __shfl_xor(total, off, kWave);
  const long long per = (total + a.target - 1) / a.target;
  return (int)max(per, (long long)kMinTiles);
}
__device__ __forceinline__ int seq_pieces(const DecodeAttnArgs& a, int s, int per) {
  return max((seq_tiles(a, s) + per - 1) / per, 1);       // an empty sequence is one piece, of nothing
}

// 8 consecutive elements of a cached row as a 16-bit matrix operand.
template <int DT, int FMT>
__device__ __forceinline__ uint4 widen8(uint2 c) {
  float x[8];
  codes_to_f32<FMT>(c.x, x);
  codes_to_f32<FMT>(c.y, x + 4);
  return make_uint4(pack2<DT>(x[0], x[1]), pack2<DT>(x[2], x[3]), pack2<DT>(x[4], x[5]), pack2<DT>(x[6], x[7]));
}

// NV consecutive elements of a cached row, as pairs of 16-bit values.
template <int DT, int FMT, int NV>
__device__ __forceinline__ void load_row(const void* base, size_t cell, int d, int at, bool live, uint32_t (&w)[NV / 2]) {
  if (!live) {
#pragma unroll
    for (int i = 0; i < NV / 2; ++i) w[i] = 0;
    return;
  }
  if constexpr (FMT == SPA_KV_NATIVE) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(base) + cell * d + at);
#pragma unroll
    for (int i = 0; i < NV / 2; ++i) w[i] = p[i];
  } else {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(base) + cell * d + at);
#pragma unroll
    for (int i = 0; i < NV / 4; ++i) {
      float x[4];
      codes_to_f32<FMT>(p[i], x);
      w[2 * i] = pack2<DT>(x[0], x[1]);
      w[2 * i + 1] = pack2<DT>(x[2], x[3]);
    }
  }
}

template <int DT, int FMT, int DP>
__global__ void __launch_bounds__(kWaves * kWave) k_attention_decode(DecodeAttnArgs a) {
  constexpr int KC = DP / 32;      // k steps of S
  constexpr int NV = DP / 16;      // dimensions of V a lane holds
  __shared__ float s_o[kWaves][16][DP + 4];
  __shared__ float s_m[kWaves][16], s_l[kWaves][16];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int col = lane & 15, g = lane >> 4;
  const int per = piece_tiles(a);
  int seq, piece;
  locate(blockIdx.x, a.n_seqs, [&](int s) { return seq_pieces(a, s, per); }, seq, piece);
  if (seq >= a.n_seqs) return;
  const int head = blockIdx.y % a.hkv, ht = blockIdx.y / a.hkv;     // key-value head, tile of 16 query heads
  const int heads = min(a.group - 16 * ht, 16);                     // query heads of this tile
  const int h0 = head * a.group + 16 * ht;
  const int len = min(max(a.lens[seq], 0), a.max_pages * (int)a.page.d);
  const int tile_end = min((len + kTile - 1) / kTile, (piece + 1) * per);

  uint4 qf[KC];
  {
    const uint16_t* q = a.q + (size_t)seq * a.q_row + (size_t)(h0 + min(col, heads - 1)) * a.q_head;
#pragma unroll
    for (int c = 0; c < KC; ++c) {
      const int at = 32 * c + 8 * g;
      qf[c] = make_uint4(0, 0, 0, 0);
      if (col < heads && at < a.d) qf[c] = *reinterpret_cast<const uint4*>(q + at);
    }
  }

  f32x4 o[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;

  for (int tile = piece * per + wave; tile < tile_end; tile += kWaves) {
    // lane i < 32 finds position i's cell; a position that does not count is bit i of `gone`
    const int pos = tile * kTile + (lane & 31);
    const int p0 = min(pos, len - 1);
    const int pc = (int)a.page.div((uint32_t)p0);
    const int pg = a.table[(size_t)seq * a.max_pages + pc];
    const bool ok = pg >= 0 && pg < a.n_pages;
    const int cell = ok ? (pg * a.hkv + head) * (int)a.page.d + (p0 - pc * (int)a.page.d) : 0;
    const uint32_t gone = (uint32_t)__ballot(pos >= len || !ok);
    const uint32_t bad = (uint32_t)__ballot(!ok);            // its cell is not the sequence's: the values are dropped
    float ksc = 1.f, vsc = 1.f;
    if constexpr (FMT != SPA_KV_NATIVE) {
      ksc = a.k_scale[cell];
      vsc = ok ? a.v_scale[cell] : 0.f;
    }
    float t[2][4];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const size_t kc = (size_t)(uint32_t)__shfl(cell, 16 * b + col, kWave);
      f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const int at = 32 * c + 8 * g;
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
    float p[8];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float e = exp2_hw(t[b][r] - base);
        l += e;
        if constexpr (FMT != SPA_KV_NATIVE) e *= __shfl(vsc, 16 * b + 4 * g + r, kWave) * kPScale<FMT>;
        p[4 * b + r] = e;
      }
    const uint4 pf = make_uint4(pack2<DT>(p[0], p[1]), pack2<DT>(p[2], p[3]), pack2<DT>(p[4], p[5]), pack2<DT>(p[6], p[7]));
    uint32_t vr[8][NV / 2];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = (j < 4 ? 4 * g + j : 16 + 4 * g + j - 4);
      const size_t vc = (size_t)(uint32_t)__shfl(cell, i, kWave);
      load_row<DT, FMT, NV>(a.v, vc, a.d, NV * col, NV * col < a.d && !((bad >> i) & 1u), vr[j]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t sel = i & 1 ? 0x07060302u : 0x05040100u;      // the high or low halves of two rows
      uint4 vf;
      vf.x = __builtin_amdgcn_perm(vr[1][i / 2], vr[0][i / 2], sel);
      vf.y = __builtin_amdgcn_perm(vr[3][i / 2], vr[2][i / 2], sel);
      vf.z = __builtin_amdgcn_perm(vr[5][i / 2], vr[4][i / 2], sel);
      vf.w = __builtin_amdgcn_perm(vr[7][i / 2], vr[6][i / 2], sel);
      o[i] *= alpha;
      o[i] = mfma16<DT>(vf, pf, o[i]);
    }
  }

  // join the four waves; lane (col, g) holds dimensions NV * (4 g + r) + i of query head col
  l += __shfl_xor(l, 16, kWave);
  l += __shfl_xor(l, 32, kWave);
  if (g == 0) s_m[wave][col] = m, s_l[wave][col] = l;
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int i = 0; i < NV; ++i) s_o[wave][col][NV * (4 * g + r) + i] = o[i][r];
  __syncthreads();
  const bool whole = seq_pieces(a, seq, per) == 1;
  for (int e = threadIdx.x; e < heads * (DP / 2); e += kWaves * kWave) {
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
    if (whole) {
      const float inv = sum > 0.f ? 1.f / (sum * kPScale<FMT>) : 0.f;
      const size_t to = (size_t)seq * a.hq + h0 + h;
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + to * a.d + dim) = pack2<DT>(x0 * inv, x1 * inv);
      if (dim == 0 && a.lse) a.lse[to] = sum > 0.f ? kLn2 * (base + log2_hw(sum)) : -INFINITY;
    } else {
      const size_t to = (size_t)blockIdx.x * a.hq + h0 + h;
      *reinterpret_cast<float2*>(a.part_o + to * a.d + dim) = make_float2(x0, x1);
      if (dim == 0) a.part_ml[to] = make_float2(mx, sum);
    }
  }
}

// One wave per (sequence, query head): the pieces' sums brought to their common maximum and added in order.
template <int DT, int FMT>
__global__ void __launch_bounds__(kWave) k_attention_decode_join(DecodeAttnArgs a) {
  const int lane = threadIdx.x;
  const int seq = blockIdx.x / a.hq, head = blockIdx.x % a.hq;
  const int per = piece_tiles(a);
  const int pieces = seq_pieces(a, seq, per);
  if (pieces == 1) return;
  int first = 0;
  for (int base = 0; base < seq; base += kWave) first += base + lane < seq ? seq_pieces(a, base + lane, per) : 0;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) first += __shfl_xor(first, off, kWave);
  float mx = -INFINITY;
  for (int i = lane; i < pieces; i += kWave) mx = fmaxf(mx, a.part_ml[(size_t)(first + i) * a.hq + head].x);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off, kWave));
  const float base = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f, x[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < pieces; ++i) {
    const size_t row = (size_t)(first + i) * a.hq + head;
    const float2 ml = a.part_ml[row];
    const float f = exp2_hw(ml.x - base);
    sum += f * ml.y;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (lane + kWave * e < a.d) x[e] += f * a.part_o[row * a.d + lane + kWave * e];
  }
  const float inv = sum > 0.f ? 1.f / (sum * kPScale<FMT>) : 0.f;
  const size_t to = (size_t)seq * a.hq + head;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (lane + kWave * e < a.d)
      static_cast<uint16_t*>(a.out)[to * a.d + lane + kWave * e] = (uint16_t)pack2<DT>(x[e] * inv, 0.f);
  if (lane == 0 && a.lse) a.lse[to] = sum > 0.f ? kLn2 * (base + log2_hw(sum)) : -INFINITY;
}

template <int DT, int FMT, int DP>
hipError_t go(const DecodeAttnArgs& a, hipStream_t st) {
  const int units = spa_check::decode_units(a.n_seqs, a.hq, a.hkv);
  hipLaunchKernelGGL((k_attention_decode<DT, FMT, DP>), dim3(units, a.hkv * a.head_tiles), dim3(kWaves * kWave), 0, st, a);
  if (hipError_t e = hipGetLastError()) return e;
  hipLaunchKernelGGL((k_attention_decode_join<DT, FMT>), dim3(a.n_seqs * a.hq), dim3(kWave), 0, st, a);
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
                                   float* lse, float* part_o, float* part_ml, hipStream_t st) {
  DecodeAttnArgs a{};
  a.q = static_cast<const uint16_t*>(q.data);
  a.q_row = q.row_stride; a.q_head = q.head_stride;
  a.k = c.k; a.v = c.v; a.k_scale = c.k_scale; a.v_scale = c.v_scale;
  a.table = table; a.lens = lens; a.out = out; a.lse = lse;
  a.part_o = part_o; a.part_ml = reinterpret_cast<float2*>(part_ml);
  a.n_seqs = n_seqs; a.hq = n_q_heads; a.hkv = c.n_heads; a.group = n_q_heads / c.n_heads;
  a.d = c.head_dim; a.n_pages = c.n_pages; a.max_pages = max_pages;
  a.head_tiles = spa_check::head_tiles(n_q_heads, c.n_heads);
  a.target = spa_check::decode_units(n_seqs, n_q_heads, c.n_heads) - n_seqs;
  a.c = scale * kLog2e;
  a.page = FastDiv((uint32_t)c.page_size);
  return c.dtype == SPA_F16 ? by_format<SPA_F16>(c.format, a, st) : by_format<SPA_BF16>(c.format, a, st);
}

}  // namespace spa
