// Attention of one new token per sequence over a cache held in 4 bits (SPA_KV_MXFP4): out = softmax(scale q K^T) V.
//
// Bound by HBM like the other formats (k_attn_decode.hip; the division into pieces is the same), with half the bytes of an
// 8-bit cache, so there is half the time to unpack them.  Keys are not unpacked at all:
//   S^T = K Q^T on v_mfma_scale_f32_16x16x128_f8f6f4, whose A operand is e2m1 with one power-of-two scale to 32 elements:
//         a lane's 16 bytes of a cached row and the scale byte beside them, as they are.  The B operand, the queries, is
//         e4m3, cut into pieces that together hold them: of each 32 elements (the operand's own blocks) the largest is
//         brought below 16, and a piece is the nearest integer, the next one 32 times what is left.  Integers up to 16
//         times codes up to 6 are whole multiples of one half below 2^7, so the sum over 32 elements, which share the query's
//         scale and the key's, is exact: the unit aligns the products of 16 elements to the largest and drops what is 2^-14 of
//         it, which a plain split of the queries into e4m3 numbers loses bits to.  Blocks of 32 and pieces are added in
//         float32.  Four pieces hold an element to 2^-19 of the largest.
//   O^T = V^T P^T on v_mfma_f32_16x16x32_bf16: values are unpacked, with their scales, by v_cvt_scalef32_pk_bf16_fp4 (exact: a
//         code has two significant bits), pairs of positions brought together by byte permutes.  A softmax weight is taken as
//         two bfloat16 numbers in two products (16 bits, and bfloat16 has the scales' range).  One, its 8 bits, would be off by
//         more than the rounding of a bfloat16 output where values cancel, and save 1 to 8 % (64 ragged sequences of up to
//         8191 52.4 -> 50.6 us, 32 of up to 8000 by 16 + 4 heads of 96 23.7 -> 21.9).
//
// 64 ragged sequences of up to 8191 positions by 8 heads of 128: 52 us with the join, 4.7 TB/s; two of 200003 79 us, 5.5 TB/s (a
// stream that is only read reaches 7.2); one of 61 5.6 us.  The choices below were timed with
// a bfloat16 call's weights in one product.
#include "spa_attn_decode.h"

namespace spa {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kGroup = 32;           // elements of one scale
// What beginning a sequence costs a workgroup, in tiles: its query, the first loads' way, the join of the waves.  64 ragged
// sequences of up to 8191 positions: 57.7 us without it, 54.8 with 6, 52.5 with 10 to 16; 40 of up to 1500: 23.5, 19.1, 18.6.
constexpr int kStart = 12;
// Tables of up to so many tiles to a sequence: a workgroup takes a sequence whole, and there is no join.  The table's width
// decides, not the lengths in it, which the host does not know: in tables four times as wide one sequence of 500 takes 10.6 us
// instead of 7.9, 128 of up to 500 by 20 heads 44.8 instead of 36.2.  With 8 heads of 128, one
// sequence of 500 takes 7.5 us so and 10.5 divided, of 1000 11.2 and 11.2, of 2000 17.4 and 11.2; 16 ragged ones of up to 1000 11.7 and
// 13.9, 128 of up to 500 by 20 heads 41.6 and 59.1.
constexpr int kWholeTiles = 32;
constexpr int kUnits = 256;          // compute units
constexpr int kPieces = 4;           // of a query element, 5 bits each, at the least

template <int CTRL>
__device__ __forceinline__ float row_turned(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, 0xF, 0xF, false));
}

// The query operands.  The matrix product has 16 columns and 128 places along k, and takes
//   PACK pieces of 16 / PACK heads side by side (4 of up to 4 heads, 2 of up to 8), whose results are added up over the columns;
//   with 64 dimensions or fewer, two pieces one behind the other, the keys standing twice in the k step.
// So a k step of 128 dimensions takes ceil(kPieces / slots) products, and the columns hold every head's scores PACK times.
template <int DP, int PACK>
struct Query {
  static constexpr int KS = DP == 64 ? 1 : DP / 128;                       // k steps
  static constexpr int kSlots = PACK * (DP == 64 ? 2 : 1);
  static constexpr int kProducts = (kPieces + kSlots - 1) / kSlots;
  i32x8 w[KS][kProducts];
  int scale[KS][kProducts];
};

__device__ __forceinline__ uint32_t fp8_quad(const float* x) { return fp8_pair(x[0], x[1]) | fp8_pair(x[2], x[3]) << 16; }

// What a lane reads of its column's head: for each k step, the 16 elements of each half.
template <int DP>
struct RawQuery {
  static constexpr int kHalves = DP == 64 ? 1 : DP / 64;
  uint4 r[kHalves][2];
};
template <int DP, int PACK>
__device__ __forceinline__ void read_query(const DecodeAttnArgs& a, const Piece& p, int col, int g, RawQuery<DP>& raw) {
  const int head = col % (16 / PACK);
  const uint16_t* q = a.q + (size_t)p.seq * a.q_row + (size_t)(p.h0 + min(head, p.heads - 1)) * a.q_head;
#pragma unroll
  for (int h = 0; h < RawQuery<DP>::kHalves; ++h)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = 64 * h + 16 * g + 8 * i;
      raw.r[h][i] = make_uint4(0, 0, 0, 0);
      if (head < p.heads && at < a.d) raw.r[h][i] = *reinterpret_cast<const uint4*>(q + at);
    }
}
// 16 elements, brought so that the largest of the 32 that they are one half of (the other is 16 lanes away) is in [8, 16);
// returns the exponent byte of their unit.
template <int DT>
__device__ __forceinline__ int bring(const uint4 (&raw)[2], float (&x)[16]) {
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = elem16<DT>(raw[e / 8], e % 8);
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 16; ++e) top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
  top = max(top, (uint32_t)__shfl_xor((int)top, 16, kWave));
  const int up = max((int)(top >> 23), 24);                    // a block below 2^-103 is taken to 2^-122
  const float k = __uint_as_float((uint32_t)(257 - up) << 23);      // 2^(130 - up)
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] *= k;
  return up - 3;
}
// Piece p of 16 elements: the digit of 32^-p, in -16 .. 16, with 32^p in `at`.  Every operation is exact; an infinity or a NaN
// gives NaN.
__device__ __forceinline__ void digits(const float (&x)[16], float at, int* out) {
  const float before = at * 0.03125f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float n[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) n[e] = rintf(x[4 * i + e] * at) - 32.f * rintf(x[4 * i + e] * before);
    out[i] = (int)fp8_quad(n);
  }
}

template <int DT, int DP, int PACK>
__device__ __forceinline__ void cut_query(const RawQuery<DP>& raw, int col, int g, Query<DP, PACK>& qp) {
  using Q = Query<DP, PACK>;
  const int side = col / (16 / PACK);                          // this column's piece of PACK
  const float step = __uint_as_float((uint32_t)(127 + 5 * side) << 23);    // 32^side
  const int other = col + 32 * (g & 1);                        // a lane with the block of dimensions 32 (g % 2), 64 + 32 (g % 2)
  // lane (col, g) holds dimensions 16 g .. + 15 in the first half of a k step and 64 + 16 g .. in the second, and gives the
  // scale of dimensions 32 g .. + 31
  if constexpr (DP == 64) {
    float x[16];
    const int unit = bring<DT>(raw.r[0], x);
    const int mine = __shfl(unit, other, kWave);
#pragma unroll
    for (int i = 0; i < Q::kProducts; ++i) {
      int lo[4], hi[4];
      const float at = step * (float)(1ll << (5 * PACK * 2 * i));
      digits(x, at, lo);
      digits(x, at * (float)(1ll << (5 * PACK)), hi);
#pragma unroll
      for (int j = 0; j < 4; ++j) qp.w[0][i][j] = lo[j], qp.w[0][i][4 + j] = hi[j];
      qp.scale[0][i] = max(mine - 5 * (PACK * (2 * i + (g >> 1)) + side), 0);
    }
  } else {
#pragma unroll
    for (int s = 0; s < Q::KS; ++s) {
      float x[16], y[16];
      const int u0 = bring<DT>(raw.r[2 * s], x), u1 = bring<DT>(raw.r[2 * s + 1], y);
      const int a0 = __shfl(u0, other, kWave), a1 = __shfl(u1, other, kWave);
      const int mine = g < 2 ? a0 : a1;                        // of dimensions 128 s + 32 g .. + 31
#pragma unroll
      for (int i = 0; i < Q::kProducts; ++i) {
        int lo[4], hi[4];
        const float at = step * (float)(1ll << (5 * PACK * i));
        digits(x, at, lo);
        digits(y, at, hi);
#pragma unroll
        for (int j = 0; j < 4; ++j) qp.w[s][i][j] = lo[j], qp.w[s][i][4 + j] = hi[j];
        qp.scale[s][i] = max(mine - 5 * (PACK * i + side), 0);
      }
    }
  }
}

// S^T of 16 positions: lane (row, g) gives 16 bytes of position row and their scale for each k step.
template <int DP, int PACK>
__device__ __forceinline__ f32x4 scores(const uint4 (&k)[Query<DP, PACK>::KS], const int (&ks)[Query<DP, PACK>::KS],
                                        const Query<DP, PACK>& q) {
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < Query<DP, PACK>::KS; ++c) {
    const i32x8 kf = {(int)k[c].x, (int)k[c].y, (int)k[c].z, (int)k[c].w, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < Query<DP, PACK>::kProducts; ++i)
      s = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(kf, q.w[c][i], s, 4, 0, 0, ks[c], 0, q.scale[c][i]);
  }
  // the pieces in other columns: 4 and 8 lanes away within the row of 16
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    if constexpr (PACK == 4) s[r] += row_turned<0x124>(s[r]);
    if constexpr (PACK >= 2) s[r] += row_turned<0x128>(s[r]);
  }
  return s;
}

// The exponent byte b of a word as the scale that the conversions take.
__device__ __forceinline__ float scale_of(uint32_t w, int b) { return __uint_as_float(((w >> (8 * b)) & 0xFFu) << 23); }

template <int SEL>
__device__ __forceinline__ uint32_t widen2(uint32_t w, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL));
}

// Adds this lane's 8 positions to o.  raw: their value rows' codes, NV dimensions each; w: their softmax weights, each cut into
// a bfloat16 number and what that leaves.
template <int NV>
__device__ __forceinline__ void add_values(const uint32_t (&raw)[8][NV > 8 ? NV / 8 : 1], const float (&vs)[8], const float (&w)[8],
                                           f32x4 (&o)[NV]) {
  uint4 pf[2];
  {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      hi[j] = pack2<SPA_BF16>(w[2 * j], w[2 * j + 1]);
      lo[j] = pack2<SPA_BF16>(w[2 * j] - bf16_to_f32(hi[j] & 0xFFFFu), w[2 * j + 1] - bf16_to_f32(hi[j] >> 16));
    }
    pf[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    pf[1] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
#pragma unroll
  for (int i = 0; i < NV / 2; ++i) {
    uint32_t vr[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t r = raw[j][i / 4];
      vr[j] = i % 4 == 0 ? widen2<0>(r, vs[j]) : i % 4 == 1 ? widen2<1>(r, vs[j]) : i % 4 == 2 ? widen2<2>(r, vs[j]) : widen2<3>(r, vs[j]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint32_t sel = e ? 0x07060302u : 0x05040100u;      // the high or low halves of two rows
      uint4 vf;
      vf.x = __builtin_amdgcn_perm(vr[1], vr[0], sel);
      vf.y = __builtin_amdgcn_perm(vr[3], vr[2], sel);
      vf.z = __builtin_amdgcn_perm(vr[5], vr[4], sel);
      vf.w = __builtin_amdgcn_perm(vr[7], vr[6], sel);
#pragma unroll
      for (const uint4& part : pf) o[2 * i + e] = mfma16<SPA_BF16>(vf, part, o[2 * i + e]);
    }
  }
}

// The running maximum, sum and outputs take in a tile's scores t, of which c times is the exponent; w receives its weights.
template <int NV>
__device__ __forceinline__ void softmax_step(const float (&t)[8], float c, float& m, float& l, f32x4 (&o)[NV], float (&w)[8]) {
  float mx = t[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) mx = fmaxf(mx, t[j]);
  mx = across_groups_max(mx);
  if (__any(mx > m)) {
    const float now = fmaxf(m, mx), alpha = exp2_hw((m - (now == -INFINITY ? 0.f : now)) * c);
    m = now;
    l *= alpha;
#pragma unroll
    for (int i = 0; i < NV; ++i) o[i] *= alpha;
  }
  const float base = m == -INFINITY ? 0.f : -m * c;            // nothing seen yet: every weight is 0
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    w[j] = exp2_hw(t[j] * c + base);
    l += w[j];
  }
}

// `bytes` of a row's codes from p (whole 4-byte pieces of 8 elements; 16 at the most), the others 0.
__device__ __forceinline__ uint4 load_codes(const char* p, int bytes) {
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (4 * i < bytes) w[i] = reinterpret_cast<const uint32_t*>(p)[i];
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// NV elements of a value row, at NV * col: NV / 2 bytes, none past the row's end.
template <int NV>
__device__ __forceinline__ void load_value(const char* row, int col, int bytes, bool live, uint32_t (&w)[NV > 8 ? NV / 8 : 1]) {
  const int at = NV / 2 * col;
#pragma unroll
  for (int i = 0; i < (NV > 8 ? NV / 8 : 1); ++i) {
    w[i] = 0;
    if (!live || at + 4 * i >= bytes) continue;
    if constexpr (NV == 4) w[0] = *reinterpret_cast<const uint16_t*>(row + at);
    else w[i] = *reinterpret_cast<const uint32_t*>(row + at + 4 * i);
  }
}

// Any page size: a lane finds one position's place and the others get it by lane exchange.
template <int DT, int DP>
__global__ void __launch_bounds__(kWaves * kWave, DP <= 128 ? 2 : 1) k_attention_decode_mx(DecodeAttnArgs a) {
  constexpr int NV = DP / 16, VW = NV > 8 ? NV / 8 : 1, KS = Query<DP, 1>::KS;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int col = lane & 15, g = lane >> 4;
  const int kg = DP == 64 ? g & 1 : g;                         // this lane's 32 dimensions of a k step
  const int bytes = a.d / 2, groups = (a.d + kGroup - 1) / kGroup, page = (int)a.page.d;
  const uint8_t *k_scale = static_cast<const uint8_t*>(a.k_scale), *v_scale = static_cast<const uint8_t*>(a.v_scale);
  Span span;
  if (!find_span<kStart>(a, span)) return;
  Piece p;
  while (next_piece<kStart>(a, span, p)) {
    RawQuery<DP> raw_q;
    Query<DP, 1> qp;
    read_query<DP, 1>(a, p, col, g, raw_q);
    cut_query<DT, DP, 1>(raw_q, col, g, qp);
    f32x4 o[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    for (int tile = p.begin + wave; tile < p.end; tile += kWaves) {
      // lane i < 32 finds position i's place; a position that does not count is bit i of `gone`
      const int pos = tile * kTile + (lane & 31);
      const int p0 = min(pos, p.len - 1);
      const int pc = (int)a.page.div((uint32_t)p0);
      const int pg = a.table[(size_t)p.seq * a.max_pages + pc];
      const bool ok = pg >= 0 && pg < a.n_pages;
      const int block = ok ? pg * a.hkv + p.head : 0, off = ok ? p0 - pc * page : 0;       // page and head; place in it
      const uint32_t gone = (uint32_t)__ballot(pos >= p.len || !ok);
      float t[8];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const size_t kb = (uint32_t)__shfl(block, 16 * b + col, kWave);
        const int ko = __shfl(off, 16 * b + col, kWave);
        uint4 kf[KS];
        int ks[KS];
#pragma unroll
        for (int c = 0; c < KS; ++c) {
          const int at = 64 * c + 16 * kg;
          kf[c] = load_codes(static_cast<const char*>(a.k) + (kb * page + ko) * bytes + at, bytes - at);
          ks[c] = at < bytes ? k_scale[(kb * groups + at / 16) * page + ko] : 127;
        }
        const f32x4 s = scores<DP, 1>(kf, ks, qp);
#pragma unroll
        for (int r = 0; r < 4; ++r) t[4 * b + r] = (gone >> (16 * b + 4 * g + r)) & 1u ? -INFINITY : s[r];
      }
      float w[8], vs[8];
      softmax_step<NV>(t, a.c, m, l, o, w);
      uint32_t raw[8][VW];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = 16 * (j / 4) + 4 * g + j % 4;
        const size_t vb = (uint32_t)__shfl(block, i, kWave);
        const int vo = __shfl(off, i, kWave);
        const bool live = !((gone >> i) & 1u) && NV * col < a.d;
        load_value<NV>(static_cast<const char*>(a.v) + (vb * page + vo) * bytes, col, bytes, live, raw[j]);
        vs[j] = live ? scale_of(v_scale[(vb * groups + NV * col / kGroup) * page + vo], 0) : 1.f;
      }
      add_values<NV>(raw, vs, w, o);
    }
    finish<DT, DP, false>(a, p, o, 1.f, m * a.c, l);
    if (span.left <= 0) break;
  }
}

// A cached row: of the kernel's DP dimensions; of whole 16-byte lanes (a multiple of 32 dimensions); of 4-byte words.
constexpr int kFull = 0, kLines = 1, kWordsOnly = 2;

// A table entry that a whole wave reads, by the scalar unit: nothing writes the table during the call.
typedef const __attribute__((address_space(4))) int32_t* table_ptr;

// A wave's way through a piece, the same on every lane.
struct Walk {
  int first, n;                // its first tile and how many it takes, every WAVES-th
  int len;
  uint32_t head;
  table_ptr table;             // the sequence's row
};
template <int WAVES>
__device__ __forceinline__ Walk walk_of(const DecodeAttnArgs& a, const Piece& p, int wave) {
  Walk w;
  w.first = __builtin_amdgcn_readfirstlane(p.begin) + wave;
  w.n = (__builtin_amdgcn_readfirstlane(p.end) - w.first + WAVES - 1) / WAVES;
  w.len = __builtin_amdgcn_readfirstlane(p.len);
  w.head = (uint32_t)__builtin_amdgcn_readfirstlane(p.head);
  w.table = (table_ptr)(a.table + (size_t)__builtin_amdgcn_readfirstlane(p.seq) * a.max_pages);
  return w;
}

// Waves of a workgroup, and of a SIMD as the registers allow: the workgroups of a compute unit (three, two or one, by the head's
// dimensions) fill it.  The division counts two for 128 dimensions also where the registers leave room for three: they serve
// calls of more workgroups (128 sequences of up to 500 by 20 heads 41.5 -> 34.1 us).
template <int DP, int PACK> constexpr int kBlockWaves = DP == 256 && PACK > 1 ? 8 : 4;
template <int DP, int ROW, int PACK>
constexpr int kSimdWaves = (DP == 64 || (DP == 128 && ROW == kFull && PACK == 4) ? 3 : DP == 128 ? 2 : 1) * kBlockWaves<DP, PACK> / 4;

// Pages of whole 16-position blocks: a block's rows are consecutive, so a tile has two bases that the whole wave shares.
// ROW: other than kFull, what lies past head_dim meets zeros of the query or is not written.  Two tiles are on their way while one is worked
// on, and the page numbers of the next one; at the end of a piece they are the next piece's.  Every load of the loop is issued
// whatever the tile (past the last one it is read again): a load that only some rounds issue would make the waits drain all
// of them.
template <int DT, int DP, int ROW, int PACK>
__global__ void __launch_bounds__((kBlockWaves<DP, PACK> * kWave), (kSimdWaves<DP, ROW, PACK>)) k_attention_decode_mx_blocks(DecodeAttnArgs a) {
  constexpr int kWaves = kBlockWaves<DP, PACK>;
  constexpr int NV = DP / 16, VW = NV > 8 ? NV / 8 : 1, KS = Query<DP, PACK>::KS;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int col = lane & 15, g = lane >> 4;
  const int kg = DP == 64 ? g & 1 : g;                       // this lane's 32 dimensions of a k step
  const int d = ROW == kFull ? DP : a.d, bytes = d / 2, groups = (d + kGroup - 1) / kGroup, page = (int)a.page.d;
  const bool in_row = ROW == kFull || NV * col < d;
  const uint32_t k_at = (uint32_t)(col * bytes + 16 * kg), ks_at = (uint32_t)(kg * page + col);
  const uint32_t vs_at = (uint32_t)((in_row ? NV * col / kGroup : 0) * page + 4 * g);
  uint32_t v_at[VW];                   // this lane's dimensions; past the row's end they are not written, whatever was read
#pragma unroll
  for (int i = 0; i < VW; ++i) {
    const int at = NV / 2 * col + 4 * i;
    v_at[i] = (uint32_t)(4 * g * bytes + (ROW == kFull ? at : min(at, bytes - (NV == 4 ? 2 : 4))));
  }
  // Of the workgroups on a unit the one that came first is served first, and the later ones end after it, alone: 66 and 79 us of a
  // call of 82.  The n-th to come (from 0) therefore goes first for n / (n + 1) of a piece, and they end together (two sequences of
  // 200003 81.3 -> 78.2 us, 64 ragged ones of up to 8191 53.3 -> 51.9, two of 100000 by 20 heads 118.4 -> 113.0; one workgroup
  // to a unit: the same).
  const int nth = a.whole ? 0 : (int)(blockIdx.x + gridDim.x * blockIdx.y) / kUnits;
  Span span;
  if (!find_span<kStart>(a, span)) return;

  struct Tile {
    uint4 k[2][KS];
    int ks[2][KS];
    uint32_t v[8][VW], vs[2];
    int there;                   // bit b: block b's page is there
  };
  // the first position of block b of a walk's tile number `it` (or of its last tile), as far as the sequence has it
  auto block_at = [&](const Walk& w, int it, int b) {
    return (uint32_t)min((w.first + kWaves * min(it, w.n - 1)) * kTile + 16 * b, (w.len - 1) & ~15);
  };
  int pages[2];                        // of the tile that is read next
  auto find_pages = [&](const Walk& w, int it) {
#pragma unroll
    for (int b = 0; b < 2; ++b) pages[b] = w.table[a.page.div(block_at(w, it, b))];
  };
  auto load = [&](Tile& x, const Walk& w, int it) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      // an absent page: the cache's first one stands in
      const bool there = pages[b] >= 0 && pages[b] < a.n_pages;
      x.there = (b ? x.there : 0) | (int)there << b;
      const uint32_t at = block_at(w, it, b), off = there ? at - a.page.div(at) * (uint32_t)page : 0u;
      const uint32_t block = there ? (uint32_t)pages[b] * (uint32_t)a.hkv + w.head : 0u;
      const size_t codes = ((size_t)block * (uint32_t)page + off) * (uint32_t)bytes;
      const size_t scales = (size_t)block * (uint32_t)(groups * page) + off;
      const char *k = static_cast<const char*>(a.k) + codes, *v = static_cast<const char*>(a.v) + codes;
      const uint8_t *ks = static_cast<const uint8_t*>(a.k_scale) + scales, *vs = static_cast<const uint8_t*>(a.v_scale) + scales;
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        if constexpr (ROW == kFull) {
          x.k[b][c] = stream_load16(k + (k_at + 64 * c));
          x.ks[b][c] = ks[ks_at + (uint32_t)(4 * c * page)];
        } else {
          // past the row's end the query is 0, and any codes will do: 32 ragged sequences of up to 8000 by 16 + 4 heads of 96 take
          // 21.7 us so, 26.7 with lanes that read nothing
          const int from = 64 * c + 16 * kg;
          const uint32_t row = (uint32_t)(col * bytes);
          if constexpr (ROW == kLines) {
            x.k[b][c] = stream_load16(k + (row + (uint32_t)min(from, bytes - 16)));
          } else {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint32_t*>(k + (row + (uint32_t)min(from + 4 * i, bytes - 4)));
            x.k[b][c] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          x.ks[b][c] = ks[(uint32_t)(min(4 * c + kg, groups - 1) * page + col)];
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (ROW == kFull) {
          load_value<NV>(v + ((uint32_t)(4 * g * bytes) + (uint32_t)(r * bytes)), col, bytes, true, x.v[4 * b + r]);
        } else {
#pragma unroll
          for (int i = 0; i < VW; ++i) {
            const char* from = v + (v_at[i] + (uint32_t)(r * bytes));
            if constexpr (NV == 4) x.v[4 * b + r][i] = *reinterpret_cast<const uint16_t*>(from);
            else x.v[4 * b + r][i] = *reinterpret_cast<const uint32_t*>(from);
          }
        }
      }
      x.vs[b] = *reinterpret_cast<const uint32_t*>(vs + vs_at);
    }
  };
  Tile x[2];
  auto start = [&](const Walk& w) {
    if (w.n <= 0) return;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      find_pages(w, u);
      load(x[u], w, u);
    }
  };

  Piece p;
  if (!next_piece<kStart>(a, span, p)) return;
  Walk now = walk_of<kWaves>(a, p, wave);
  RawQuery<DP> raw_q;
  // 256 dimensions leave no registers to read a piece's tiles and query while the one before ends
  constexpr bool kAhead = DP < 256;
  if constexpr (kAhead) {
    read_query<DP, PACK>(a, p, col, g, raw_q);
    start(now);
  }
  for (;;) {
    bool more = __builtin_amdgcn_readfirstlane(span.left) > 0;
    Piece next = p;
    if (more) more = __builtin_amdgcn_readfirstlane((int)next_piece<kStart>(a, span, next));
    const Walk then = walk_of<kWaves>(a, next, wave);
    Query<DP, PACK> qp;
    if constexpr (!kAhead) read_query<DP, PACK>(a, p, col, g, raw_q);
    cut_query<DT, DP, PACK>(raw_q, col, g, qp);
    if constexpr (!kAhead) start(now);
    f32x4 o[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    const int steps = now.n > 0 ? (now.n + 1) & ~1 : 0;
    const bool ahead = kAhead && more && then.n > 0;                     // past this piece's tiles the next one's are read
    // the tile to read at place `it`, of this piece or the next one
    auto source = [&](int it, Walk& w) {
      const bool far = it >= steps && ahead;
      w.first = far ? then.first : now.first; w.n = far ? then.n : now.n; w.len = far ? then.len : now.len;
      w.head = far ? then.head : now.head; w.table = far ? then.table : now.table;
      return far ? it - steps : it;
    };
    if (steps) {
      Walk from;
      const int place = source(2, from);
      find_pages(from, place);
    }
    for (int base = 0; base < steps; base += 2) {
      if (DP < 256 && nth) {
        if (base * (nth + 1) < steps * nth) __builtin_amdgcn_s_setprio(1);
        else __builtin_amdgcn_s_setprio(0);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int it = base + u, tile = now.first + kWaves * it;
        if (it < now.n) {
          float t[8], vs[8], w[8];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            int unit[KS];
#pragma unroll
            for (int c = 0; c < KS; ++c) unit[c] = ROW != kFull && 64 * c + 16 * kg >= bytes ? 127 : x[u].ks[b][c];
            const f32x4 s = scores<DP, PACK>(x[u].k[b], ROW == kFull ? x[u].ks[b] : unit, qp);
#pragma unroll
            for (int r = 0; r < 4; ++r) t[4 * b + r] = s[r];
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) vs[j] = scale_of(x[u].vs[j / 4], j % 4);
          // the last tile's end and absent pages: what does not count is removed from the scores and the values
          if ((tile + 1) * kTile > now.len || x[u].there != 3) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (tile * kTile + 16 * (j / 4) + 4 * g + j % 4 >= now.len || !(x[u].there >> (j / 4) & 1)) {
                t[j] = -INFINITY;
                vs[j] = 1.f;
#pragma unroll
                for (int i = 0; i < VW; ++i) x[u].v[j][i] = 0;
              }
          }
          softmax_step<NV>(t, a.c, m, l, o, w);
          add_values<NV>(x[u].v, vs, w, o);
        }
        Walk from;
        int place = source(it + 2, from);
        load(x[u], from, place);
        place = source(it + 3, from);
        find_pages(from, place);
      }
    }
    if (kAhead && more) read_query<DP, PACK>(a, next, col, g, raw_q);
    finish<DT, DP, false, kWaves>(a, p, o, 1.f, m * a.c, l);
    if (!more) break;
    if (kAhead && steps == 0) start(then);                     // nothing was read ahead
    p = next;
    now = then;
  }
}

template <int DT, int DP, int PACK>
void launch_blocks(const DecodeAttnArgs& a, dim3 grid, hipStream_t st) {
  const dim3 block(kBlockWaves<DP, PACK> * kWave);
  if (a.d == DP) hipLaunchKernelGGL((k_attention_decode_mx_blocks<DT, DP, kFull, PACK>), grid, block, 0, st, a);
  else if (a.d % 32 == 0) hipLaunchKernelGGL((k_attention_decode_mx_blocks<DT, DP, kLines, PACK>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_attention_decode_mx_blocks<DT, DP, kWordsOnly, PACK>), grid, block, 0, st, a);
}
template <int DT, int DP>
hipError_t go(DecodeAttnArgs a, hipStream_t st) {
  a.whole = a.page.d % 16 == 0 && (int64_t)a.max_pages * a.page.d <= kWholeTiles * kTile;
  const int units = a.whole ? a.n_seqs : units_of(a, kStart);
  const dim3 grid(units, a.hkv * a.head_tiles);
  if (a.page.d % 16) hipLaunchKernelGGL((k_attention_decode_mx<DT, DP>), grid, dim3(kWaves * kWave), 0, st, a);
  else if (a.group <= 4) launch_blocks<DT, DP, 4>(a, grid, st);
  else if (a.group <= 8) launch_blocks<DT, DP, 2>(a, grid, st);
  else launch_blocks<DT, DP, 1>(a, grid, st);
  if (hipError_t e = hipGetLastError()) return e;
  return a.whole ? hipSuccess : join_pieces<DT>(a, units, st);
}
template <int DT>
hipError_t by_dim(const DecodeAttnArgs& a, hipStream_t st) {
  if (a.d <= 64) return go<DT, 64>(a, st);
  if (a.d <= 128) return go<DT, 128>(a, st);
  return go<DT, 256>(a, st);
}

}  // namespace

hipError_t launch_attention_decode_mx(const spa_heads& q, int n_seqs, int n_q_heads, const spa_kv_cache& c,
                                      const int32_t* table, int max_pages, const int32_t* lens, float scale, void* out,
                                      float* lse, float* part_o, float* part_ml, int32_t* part_of, hipStream_t st) {
  const DecodeAttnArgs a = decode_args(q, n_seqs, n_q_heads, c, table, max_pages, lens, scale, out, lse, part_o, part_ml, part_of);
  return c.dtype == SPA_F16 ? by_dim<SPA_F16>(a, st) : by_dim<SPA_BF16>(a, st);
}

}  // namespace spa
