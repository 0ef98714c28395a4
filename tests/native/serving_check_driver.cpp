// Host-only sweep of the argument checks of the page planning, the norm and rotation of queries and keys, and the 4-bit cache,
// meant to be built with AddressSanitizer and UndefinedBehaviorSanitizer: every check runs on a fixed pseudo-random set of
// valid and hostile arguments, and what is accepted must be what the kernels assume.  Prints "ok <calls> accepted <counts>" or
// the failures, and exits non-zero on any.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>

#include "spa.h"
#include "spa_check_layer.h"

namespace {

uint64_t g_state = 0x243F6A8885A308D3ull;
uint64_t next_u64() {  // splitmix64
  uint64_t z = (g_state += 0x9E3779B97F4A7C15ull);
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}
int g_fails = 0;
long g_calls = 0, g_ok[3] = {0, 0, 0};
#define EXPECT(cond, ...)                                   \
  do {                                                      \
    if (!(cond) && g_fails++ < 20) {                        \
      std::printf("fail %s:%d: ", __FILE__, __LINE__);      \
      std::printf(__VA_ARGS__);                             \
      std::printf("\n");                                    \
    }                                                       \
  } while (0)

int32_t pick(int32_t lo, int32_t hi) { return lo + (int32_t)(next_u64() % (uint64_t)((int64_t)hi - lo + 1)); }
bool hostile() { return next_u64() % 40 == 0; }
int32_t pick_n(int32_t lo, int32_t hi) {
  static const int32_t edge[] = {0, -1, INT32_MAX, INT32_MIN, 1 << 30, (1 << 30) + 1, 1 << 20, (1 << 20) + 1, 4097, 1 << 24};
  return hostile() ? edge[next_u64() % 10] : pick(lo, hi);
}
// Addresses that are never read.
template <typename T>
T* at(uint64_t bytes) { return reinterpret_cast<T*>((uintptr_t)bytes); }
const int32_t* pick_ints() {
  if (hostile()) return nullptr;
  return at<const int32_t>(0x100000 + next_u64() % 64 * 0x100000 + 4 * (next_u64() % 8));
}
bool apart(const void* a, int64_t n, const void* b, int64_t m) {   // in bytes
  const __int128 x = (__int128)(uintptr_t)a, y = (__int128)(uintptr_t)b;
  return n == 0 || m == 0 || x + n <= y || y + m <= x;
}

void sweep_plan() {
  for (int it = 0; it < 300000; ++it) {
    const int32_t n = pick_n(0, 300), width = pick_n(0, 64), page = pick_n(1, 300), t = pick_n(0, 9000);
    spa_page_pool pool{const_cast<int32_t*>(pick_ints()), pick_ints(), const_cast<int32_t*>(pick_ints()), pick_n(0, 4000)};
    if (next_u64() % 2) pool.count = pool.count_out;
    const int32_t *lens = pick_ints(), *fresh = pick_ints(), *done = next_u64() % 2 ? pick_ints() : nullptr, *table = pick_ints();
    const int32_t* lens_out = next_u64() % 2 ? lens : pick_ints();
    const int32_t *slots = pick_ints(), *pos = pick_ints(), *cq = pick_ints(), *ck = pick_ints();
    const spa_page_pool* pp = next_u64() % 100 ? &pool : nullptr;
    const spa_status s = spa_check::check_kv_plan(lens, fresh, done, n, table, width, page, pp, t, slots, pos, cq, ck, lens_out);
    ++g_calls;
    EXPECT(s == SPA_OK || s == SPA_ERR_INVALID || s == SPA_ERR_UNSUPPORTED, "status %d", (int)s);
    if (s != SPA_OK) continue;
    ++g_ok[0];
    EXPECT(n >= 0 && n <= 1 << 20 && width >= 0 && page >= 1 && t >= 0 && t <= 1 << 30 && pool.n_pages >= 0, "sizes");
    EXPECT((int64_t)width * page + t <= INT32_MAX, "positions pass 31 bits");
    EXPECT((int64_t)pool.n_pages * page <= INT32_MAX, "slots pass 31 bits");
    EXPECT(pool.count && pool.count_out && cq && ck && (!pool.n_pages || pool.pages), "pointers");
    EXPECT(!n || (lens && fresh && lens_out && (!width || table)), "sequences");
    EXPECT(!t || (slots && pos), "rows");
    struct { const void* p; int64_t bytes; } out[] = {{lens_out, 4ll * n}, {pool.count_out, 8}, {slots, 4ll * t}, {pos, 4ll * t},
        {cq, 4ll * n + 4}, {ck, 4ll * n + 4}, {table, 4ll * n * width}, {pool.pages, 4ll * pool.n_pages}};
    for (auto& a : out) {
      for (auto& b : out) EXPECT(&a == &b || apart(a.p, a.bytes, b.p, b.bytes), "outputs overlap");
      EXPECT(apart(a.p, a.bytes, fresh, 4ll * n) && (!done || apart(a.p, a.bytes, done, 4ll * n)), "an output on an input");
      EXPECT(a.p == lens || apart(a.p, a.bytes, lens, 4ll * n), "an output on the lengths");
      EXPECT(a.p == pool.count || apart(a.p, a.bytes, pool.count, 4), "an output on the count");
    }
  }
}

int64_t pick_stride(int64_t least) {
  static const int64_t edge[] = {-8, INT64_MIN, INT64_MAX, (int64_t(1) << 23) + 8, int64_t(1) << 23, 0, 4, 12};
  return hostile() ? edge[next_u64() % 8] : least + 8 * (int64_t)pick(0, 3) * (next_u64() % 2);
}
const void* pick_data() {
  if (hostile()) return nullptr;
  return at<const void>(0x10000000ull * (1 + next_u64() % 8) + (hostile() ? 4 : 0));
}
spa_heads pick_heads(int32_t heads, int32_t d) {
  const int64_t head = pick_stride(d);
  return spa_heads{pick_data(), pick_stride(head > 0 && head < 1 << 20 ? head * heads : 64), head};
}
spa_kv_cache pick_cache(int32_t dtype, int32_t h, int32_t d) {
  spa_kv_cache c{};
  c.dtype = hostile() ? pick(-1, 4) : dtype;
  c.format = hostile() ? pick(-1, 5) : pick(0, 3);
  c.n_pages = pick_n(1, 4000);
  c.page_size = pick_n(1, 300);
  c.n_heads = hostile() ? pick(0, 16) : h;
  c.head_dim = hostile() ? pick(0, 300) : d;
  c.k = const_cast<void*>(pick_data());
  c.v = const_cast<void*>(pick_data());
  c.k_scale = const_cast<void*>(pick_data());
  c.v_scale = const_cast<void*>(pick_data());
  return c;
}
void expect_heads(const spa_heads* h, const char* name) {
  EXPECT(h && h->data && (uintptr_t)h->data % 16 == 0, "%s: data", name);
  if (!h) return;
  EXPECT(h->row_stride >= 0 && h->row_stride % 8 == 0 && h->row_stride <= 1 << 23, "%s: rows", name);
  EXPECT(h->head_stride >= 0 && h->head_stride % 8 == 0 && h->head_stride <= 1 << 23, "%s: heads", name);
}
// Whether two vectors of a written tensor share an element, by going through the pairs of a few rows and heads.
void expect_apart(const spa_heads* h, int32_t t, int32_t heads, int32_t d, const char* name) {
  const int64_t rows = t < 4 ? t : 4, cols = heads < 6 ? heads : 6;
  for (int64_t a = 0; a < rows * cols; ++a)
    for (int64_t b = 0; b < a; ++b) {
      const int64_t x = a / cols * h->row_stride + a % cols * h->head_stride, y = b / cols * h->row_stride + b % cols * h->head_stride;
      EXPECT(x + d <= y || y + d <= x, "%s: vectors overlap (strides %lld %lld, %d of %d)", name, (long long)h->row_stride,
             (long long)h->head_stride, heads, d);
    }
}

void sweep_rope() {
  for (int it = 0; it < 300000; ++it) {
    const int32_t dtype = hostile() ? pick(-1, 4) : pick(1, 2), t = pick_n(0, 9000), hq = pick_n(1, 16), hkv = pick_n(1, 16);
    const int32_t d = hostile() ? pick(-1, 300) : 8 * pick(1, 32);
    const spa_heads q = pick_heads(hq, d), k = pick_heads(hkv, d), v = pick_heads(hkv, d);
    spa_heads qo = pick_heads(hq, d), ko = pick_heads(hkv, d);
    if (next_u64() % 4 == 0) qo = q;
    if (next_u64() % 4 == 0) ko = k;
    const spa_kv_cache c = pick_cache(dtype, hkv, d);
    const bool cached = next_u64() % 2;
    const spa_kv_cache* cp = cached ? &c : nullptr;
    const spa_heads* vp = cached != hostile() ? &v : nullptr;
    const int32_t* slots = cached != hostile() ? pick_ints() : nullptr;
    const spa_heads* kop = cached && next_u64() % 2 ? nullptr : &ko;
    const spa_rope rope{hostile() ? nullptr : at<const float>(0x5000), hostile() ? pick(-8, 300) : d > 8 ? 8 * pick(0, d / 8) : 8, pick(0, 1)};
    const spa_rope* rp = next_u64() % 8 ? &rope : nullptr;
    const spa_norm n1{hostile() ? pick(-2, 5) : pick(0, 2), pick_data(), nullptr}, n2{pick(0, 2), nullptr, pick_data()};
    const spa_norm *np = next_u64() % 2 ? &n1 : nullptr, *mp = next_u64() % 2 ? &n2 : nullptr;
    const float eps = hostile() ? NAN : hostile() ? -1.f : hostile() ? INFINITY : 1e-5f;
    const int32_t* pos = pick_ints();
    const spa_status s = spa_check::check_qk_norm_rope(&q, &k, vp, dtype, t, hq, hkv, d, pos, rp, np, mp, eps, &qo, kop, slots, cp);
    ++g_calls;
    EXPECT(s == SPA_OK || s == SPA_ERR_INVALID || s == SPA_ERR_UNSUPPORTED, "status %d", (int)s);
    if (s != SPA_OK) continue;
    ++g_ok[1];
    EXPECT((dtype == SPA_F16 || dtype == SPA_BF16) && d >= 8 && d <= 256 && d % 8 == 0, "types");
    EXPECT(t >= 0 && hq >= 1 && hkv >= 1 && eps >= 0.f && eps < 2e30f, "sizes");
    if (rp) EXPECT(rope.rotary_dim >= 0 && rope.rotary_dim <= d && rope.rotary_dim % 8 == 0 && (!rope.rotary_dim || rope.inv_freq), "rotation");
    if (!t) continue;
    EXPECT((int64_t)t * (hq + 2 * hkv) * 32 <= INT32_MAX, "threads of the launch");
    EXPECT(!rp || !rope.rotary_dim || pos, "positions");
    expect_heads(&q, "q"), expect_heads(&k, "k"), expect_heads(&qo, "q_out");
    if (kop) expect_heads(kop, "k_out");
    expect_apart(&qo, t, hq, d, "q_out");
    if (kop) expect_apart(kop, t, hkv, d, "k_out");
    EXPECT(cp || kop, "the keys go nowhere");
    EXPECT(qo.data != k.data && (!kop || (kop->data != q.data && kop->data != qo.data)), "an output on another's vectors");
    if (qo.data == q.data && t > 1 && hq > 1) EXPECT(qo.row_stride == q.row_stride && qo.head_stride == q.head_stride, "in place");
    if (kop && kop->data == k.data && t > 1 && hkv > 1) EXPECT(kop->row_stride == k.row_stride && kop->head_stride == k.head_stride, "in place");
    if (cp) {
      expect_heads(vp, "v");
      EXPECT(slots && qo.data != v.data && (!kop || kop->data != v.data), "values");
      EXPECT(c.dtype == dtype && c.n_heads == hkv && c.head_dim == d, "another cache");
      EXPECT(c.format >= SPA_KV_NATIVE && c.format <= SPA_KV_MXFP4, "format %d", c.format);
    }
  }
}

void sweep_cache() {
  for (int it = 0; it < 300000; ++it) {
    const int32_t d = hostile() ? pick(-1, 300) : 8 * pick(1, 32), h = pick_n(1, 16);
    spa_kv_cache c = pick_cache(pick(1, 2), h, d);
    c.format = SPA_KV_MXFP4;
    const spa_status s = spa_check::check_cache(&c);
    ++g_calls;
    if (s != SPA_OK) continue;
    ++g_ok[2];
    EXPECT(c.head_dim % 8 == 0 && c.head_dim <= 256 && (c.dtype == SPA_F16 || c.dtype == SPA_BF16), "vectors");
    EXPECT((__int128)c.n_pages * c.page_size * c.n_heads <= INT32_MAX, "cells pass 31 bits");
    for (const void* p : {(const void*)c.k, (const void*)c.v, (const void*)c.k_scale, (const void*)c.v_scale})
      EXPECT(p && (uintptr_t)p % 16 == 0, "pages and scales");
  }
}

}  // namespace

int main() {
  sweep_plan();
  sweep_rope();
  sweep_cache();
  if (g_fails) {
    std::printf("failures %d of %ld calls\n", g_fails, g_calls);
    return 1;
  }
  std::printf("ok %ld calls accepted %ld %ld %ld\n", g_calls, g_ok[0], g_ok[1], g_ok[2]);
  return 0;
}
