// Host-only sweep of the argument checks and workspace layouts of the cache, attention and norm entry points, and of
// the division their kernels use, meant to be built with AddressSanitizer and UndefinedBehaviorSanitizer: every check
// runs on a fixed pseudo-random set of valid and hostile arguments, and what is accepted must be what the kernels
// assume.  Prints "ok <calls> accepted <counts>" or the failures, and exits non-zero on any.
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "spa.h"
#include "spa_check_layer.h"
#include "spa_div.h"

namespace {

uint64_t g_state = 0x9E3779B97F4A7C15ull;
uint64_t next_u64() {  // splitmix64
  uint64_t z = (g_state += 0x9E3779B97F4A7C15ull);
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}
int g_fails = 0;
long g_calls = 0, g_ok[5] = {0, 0, 0, 0, 0};
#define EXPECT(cond, ...)                                   \
  do {                                                      \
    if (!(cond) && g_fails++ < 20) {                        \
      std::printf("fail %s:%d: ", __FILE__, __LINE__);      \
      std::printf(__VA_ARGS__);                             \
      std::printf("\n");                                    \
    }                                                       \
  } while (0)

int32_t pick(int32_t lo, int32_t hi) { return lo + (int32_t)(next_u64() % (uint64_t)((int64_t)hi - lo + 1)); }
bool hostile() { return next_u64() % 12 == 0; }
int32_t odd_int() {
  static const int32_t edge[] = {0, -1, INT32_MAX, INT32_MIN, 1 << 30, (1 << 30) + 1, 1 << 20, (1 << 20) + 1, 4097, 1 << 24};
  return edge[next_u64() % 10];
}
int32_t pick_n(int32_t lo, int32_t hi) { return hostile() ? odd_int() : pick(lo, hi); }
int64_t pick_stride() {
  static const int64_t edge[] = {-8, INT64_MIN, INT64_MAX, (int64_t(1) << 23) + 8, int64_t(1) << 23, 0, 4, 12};
  return hostile() ? edge[next_u64() % 8] : 8 * (int64_t)pick(0, 4096);
}
alignas(64) unsigned char g_buf[256];
const void* pick_ptr() {
  const uint64_t r = next_u64() % 24;
  return r == 0 ? nullptr : r == 1 ? (const void*)(g_buf + 4) : (const void*)(g_buf + 16 * (r % 4));
}
spa_heads pick_heads() { return spa_heads{pick_ptr(), pick_stride(), pick_stride()}; }
float pick_scale() {
  static const float edge[] = {0.f, -1.f, NAN, INFINITY, -INFINITY, 1e31f, 1e-38f};
  return hostile() ? edge[next_u64() % 7] : 0.125f;
}
spa_kv_cache pick_cache() {
  spa_kv_cache c{};
  c.dtype = hostile() ? pick(-1, 4) : pick(1, 2);
  c.format = hostile() ? pick(-1, 4) : pick(0, 2);
  c.n_pages = pick_n(1, 4000);
  c.page_size = pick_n(1, 300);
  c.n_heads = pick_n(1, 16);
  c.head_dim = hostile() ? odd_int() : hostile() ? pick(1, 300) : 8 * pick(1, 32);
  c.k = const_cast<void*>(pick_ptr());
  c.v = const_cast<void*>(pick_ptr());
  c.k_scale = (float*)const_cast<void*>(pick_ptr());
  c.v_scale = (float*)const_cast<void*>(pick_ptr());
  return c;
}
bool known(spa_status s) { return s == SPA_OK || s == SPA_ERR_INVALID || s == SPA_ERR_UNSUPPORTED; }

void expect_cache(const spa_kv_cache& c) {
  EXPECT(c.dtype == SPA_F16 || c.dtype == SPA_BF16, "dtype %d", c.dtype);
  EXPECT(c.n_pages >= 1 && c.page_size >= 1 && c.n_heads >= 1, "sizes");
  EXPECT((__int128)c.n_pages * c.page_size * c.n_heads <= INT32_MAX, "cells pass 31 bits");
  EXPECT(c.head_dim >= 8 && c.head_dim <= 256 && c.head_dim % 8 == 0, "head_dim %d", c.head_dim);
  EXPECT(c.k && c.v && (uintptr_t)c.k % 16 == 0 && (uintptr_t)c.v % 16 == 0, "pages");
  if (c.format != SPA_KV_NATIVE) EXPECT(c.k_scale && c.v_scale, "scales");
}
void expect_heads(const spa_heads& h) {
  EXPECT(h.data && (uintptr_t)h.data % 16 == 0, "data");
  EXPECT(h.row_stride >= 0 && h.row_stride % 8 == 0 && h.head_stride >= 0 && h.head_stride % 8 == 0, "strides");
  // a tile of 64 rows and a row of pieces are addressed in 32 bits
  EXPECT(63 * h.row_stride * 2 + 512 < (int64_t(1) << 32) && h.head_stride <= (1 << 23), "stride range");
}

void sweep() {
  const int32_t* ints = reinterpret_cast<const int32_t*>(g_buf);
  for (int it = 0; it < 300000; ++it) {
    const spa_kv_cache c = pick_cache();
    const spa_kv_cache* cp = next_u64() % 50 ? &c : nullptr;
    const spa_heads q = pick_heads(), k = pick_heads(), v = pick_heads();
    const spa_heads* qp = next_u64() % 50 ? &q : nullptr;
    const int32_t* opt = next_u64() % 30 ? ints : nullptr;
    const void* out = pick_ptr();

    const int32_t t = pick_n(0, 9000);
    spa_status s = spa_check::check_kv_write(qp, &v, t, opt, cp);
    ++g_calls;
    EXPECT(known(s), "status %d", (int)s);
    if (s == SPA_OK) {
      ++g_ok[0];
      expect_cache(c);
      EXPECT(t >= 0, "t %d", t);
      if (t) {
        EXPECT(opt, "no slots");
        EXPECT((int64_t)t * c.n_heads * 32 < (int64_t(1) << 32), "threads of the launch");
        expect_heads(q);
        expect_heads(v);
      }
    }

    const int32_t n = pick_n(0, 300), pages = pick_n(0, 400), total = pick_n(0, 20000);
    const void* out2 = pick_ptr();
    s = spa_check::check_kv_read(cp, opt, n, pages, ints, total, out, out2);
    ++g_calls;
    EXPECT(known(s), "status %d", (int)s);
    if (s == SPA_OK) {
      ++g_ok[1];
      expect_cache(c);
      EXPECT(n >= 0 && total >= 0 && pages >= 0, "sizes");
      if (n && total) EXPECT(opt && out && out2 && pages >= 1, "pointers");
    }

    const int32_t hq = hostile() ? odd_int() : (c.n_heads > 0 && c.n_heads < 100 ? c.n_heads * pick(1, 20) : pick(1, 64));
    const float scale = pick_scale();
    s = spa_check::check_attention_decode(qp, n, hq, cp, opt, pages, ints, scale, out);
    ++g_calls;
    EXPECT(known(s), "status %d", (int)s);
    if (s == SPA_OK) {
      ++g_ok[2];
      expect_cache(c);
      EXPECT(scale > 0 && std::isfinite(scale), "scale");
      EXPECT(hq >= 1 && hq % c.n_heads == 0, "heads %d / %d", hq, c.n_heads);
      if (n) {
        expect_heads(q);
        EXPECT(pages == 0 || opt, "no table");
        EXPECT((int64_t)pages * c.page_size <= (1 << 29), "positions of a sequence");
        const spa_check::DecodeAttnPlan p = spa_check::decode_attn_plan(n, hq, c.n_heads, c.head_dim);
        const int64_t groups = spa_check::decode_groups(hq, c.n_heads, c.head_dim);
        const int64_t tiles = spa_check::head_tiles(hq, c.n_heads);
        EXPECT(groups >= 1 && groups * c.n_heads * tiles < (1 << 16) + 768, "groups %lld", (long long)groups);
        EXPECT(c.n_heads * tiles <= 65535, "second grid axis");
        EXPECT(tiles * 16 * c.n_heads >= hq, "heads uncovered");
        const size_t rows = (size_t)2 * groups * hq;
        EXPECT(p.o == 0 && p.ml >= rows * c.head_dim * 4 && p.of - p.ml >= rows * 8 && p.bytes - p.of >= (size_t)n * 8 &&
                   p.ml % 256 == 0 && p.of % 256 == 0, "plan");
      }
    }

    const int32_t tq = pick_n(0, 9000), tk = pick_n(0, 9000), hkv = pick_n(1, 16), d = c.head_dim;
    const int32_t hq2 = hostile() ? odd_int() : (hkv > 0 && hkv < 100 ? hkv * pick(1, 20) : 8);
    s = spa_check::check_attention_prefill(qp, &k, &v, c.dtype, tq, tk, hq2, hkv, d, opt, ints, n, scale, out);
    ++g_calls;
    EXPECT(known(s), "status %d", (int)s);
    if (s == SPA_OK) {
      ++g_ok[3];
      EXPECT(d >= 8 && d <= 256 && d % 8 == 0 && (c.dtype == SPA_F16 || c.dtype == SPA_BF16), "dtype, head_dim");
      EXPECT(hq2 >= 1 && hkv >= 1 && hq2 % hkv == 0 && scale > 0 && std::isfinite(scale), "heads");
      if (tq && n) {
        expect_heads(q);
        if (tk) {
          expect_heads(k);
          expect_heads(v);
        }
        EXPECT(opt && out, "pointers");
        const spa_check::PrefillAttnPlan p = spa_check::prefill_attn_plan(tq, tk, n, hq2, d);
        EXPECT(p.splits >= 1 && p.splits <= 8, "splits %d", p.splits);
        EXPECT(((int64_t)tq / 128 + n) * hq2 * p.splits <= (int64_t(1) << 24), "workgroups of the grid");
        if (p.splits > 1) {
          const size_t rows = (size_t)p.splits * tq * hq2;
          EXPECT(p.o == 0 && p.ml >= rows * d * 4 && p.bytes - p.ml >= rows * 8, "plan");
        } else {
          EXPECT(p.bytes == 0, "bytes without splits");
        }
      }
    }

    spa_norm post{hostile() ? pick(-1, 4) : pick(0, 2), pick_ptr(), pick_ptr()}, pre = post;
    const int32_t ch = pick_n(1, 70000), dt = hostile() ? pick(-1, 4) : pick(0, 2), st = hostile() ? pick(-1, 4) : dt;
    const int32_t rows = hostile() ? odd_int() : next_u64() % 2 ? t : pick(0, 1);
    const void* gate = rows ? g_buf : nullptr;
    const float eps = hostile() ? pick_scale() : 1e-5f;
    s = spa_check::check_norm(pick_ptr(), dt, t, ch, pick_ptr(), st, next_u64() % 9 ? &post : nullptr, gate, rows, 1.f, &pre, eps,
                              out, out2);
    ++g_calls;
    EXPECT(known(s), "status %d", (int)s);
    if (s == SPA_OK) {
      ++g_ok[4];
      EXPECT(dt >= 0 && dt <= 2 && st >= 0 && st <= 2 && t >= 0, "types");
      EXPECT(eps >= 0 && std::isfinite(eps), "eps");
      if (t) EXPECT((st == dt || st == SPA_F32) && ch >= 1 && ch <= 65536 && (out || out2) &&
                    (rows == 0 || rows == 1 || rows == t), "sizes");
    }
  }
}

void sweep_div() {
  const uint32_t top = 0x7FFFFFFFu;
  for (int it = 0; it < 200000; ++it) {
    uint32_t d = it < 2000 ? (uint32_t)it + 1 : (uint32_t)(next_u64() >> (33 + next_u64() % 31));
    if (d == 0 || d > top) d = top;
    const spa::FastDiv f(d);
    const uint32_t near = (uint32_t)(next_u64() % top) / d * d;
    const uint32_t xs[] = {0, 1, d - 1, d, d + 1 <= top ? d + 1 : top, near, near ? near - 1 : 0, top, top - 1,
                           (uint32_t)(next_u64() % top)};
    for (uint32_t x : xs) {
      ++g_calls;
      if (x > top) continue;
      EXPECT(f.div(x) == x / d, "%u / %u = %u", x, d, f.div(x));
    }
  }
}

}  // namespace

int main() {
  sweep();
  sweep_div();
  if (g_fails) {
    std::printf("failures %d of %ld calls\n", g_fails, g_calls);
    return 1;
  }
  std::printf("ok %ld calls accepted %ld %ld %ld %ld %ld\n", g_calls, g_ok[0], g_ok[1], g_ok[2], g_ok[3], g_ok[4]);
  return 0;
}
