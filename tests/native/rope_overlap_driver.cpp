// Host-only check of where the norm and rotation of queries and keys may write, meant to be built with AddressSanitizer and
// UndefinedBehaviorSanitizer: the overlap of two sets of vectors against marking every byte, and calls that are accepted or
// refused by what lies where.  Nothing is read or written at the addresses.  Prints "ok <sets> <overlapping> <calls>" or the
// failures, and exits non-zero on any.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "spa.h"
#include "spa_check_layer.h"

namespace {

uint64_t g_state = 0x13198A2E03707344ull;
uint64_t next_u64() {  // splitmix64
  uint64_t z = (g_state += 0x9E3779B97F4A7C15ull);
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}
int64_t pick(int64_t lo, int64_t hi) { return lo + (int64_t)(next_u64() % (uint64_t)(hi - lo + 1)); }
int g_fails = 0;
long g_sets = 0, g_overlapping = 0, g_calls = 0;

using spa_check::Vectors;

// Every byte of every vector, marked: the definition.
bool marked(const Vectors& a, const Vectors& b, bool& ranges) {
  constexpr int64_t kBase = 1 << 16;
  std::vector<char> seen(1 << 15);
  int64_t a_end = 0, b_end = 0;
  bool hit = false;
  for (int64_t r = 0; r < a.rows; ++r)
    for (int64_t h = 0; h < a.heads; ++h)
      for (int64_t i = 0; i < a.bytes; ++i) {
        const int64_t at = (int64_t)a.at - kBase + r * a.row + h * a.head + i;
        seen.at(at) = 1;
        if (at + 1 > a_end) a_end = at + 1;
      }
  for (int64_t r = 0; r < b.rows; ++r)
    for (int64_t h = 0; h < b.heads; ++h)
      for (int64_t i = 0; i < b.bytes; ++i) {
        const int64_t at = (int64_t)b.at - kBase + r * b.row + h * b.head + i;
        hit |= seen.at(at) != 0;
        if (at + 1 > b_end) b_end = at + 1;
      }
  ranges = a.bytes && b.bytes && (int64_t)a.at - kBase < b_end && (int64_t)b.at - kBase < a_end;
  return hit;
}
Vectors random_vectors(int64_t row, int64_t head, int64_t bytes) {
  Vectors v{(uintptr_t)(65536 + pick(0, 700)), 0, pick(1, 6), pick(1, 5), row, head, next_u64() % 20 ? bytes : 0};
  if (v.rows == 1 || row == 0) v.rows = 1, v.row = 0;
  if (v.heads == 1 || head == 0) v.heads = 1, v.head = 0;
  v.end = v.at + (uintptr_t)((v.rows - 1) * v.row + (v.heads - 1) * v.head + v.bytes);
  return v;
}
void sweep() {
  for (int it = 0; it < 60000; ++it) {
    const int64_t d = 2 * pick(1, 12), head = next_u64() % 8 ? d * pick(1, 4) : pick(0, 90);
    const int64_t row = next_u64() % 3 ? head * pick(1, 6) + pick(0, 3) * d : next_u64() % 2 ? d * pick(1, 3) : pick(0, 400);
    const Vectors a = random_vectors(row, next_u64() % 3 ? head : row * 6, d);
    const Vectors b = random_vectors(next_u64() % 4 ? row : pick(0, 400), next_u64() % 3 ? a.head : next_u64() % 2 ? head : pick(0, 300),
                                     next_u64() % 4 ? d : pick(1, 900));
    bool ranges;
    const bool want = marked(a, b, ranges), other_rows = a.rows > 1 && b.rows > 1 && a.row != b.row;
    for (int way = 0; way < 2; ++way) {
      const bool got = way ? spa_check::overlap(b, a) : spa_check::overlap(a, b);
      if (got != (other_rows ? ranges : want) && g_fails++ < 20)
        std::printf("fail: %d for {%ld x %ld of %ld at %ld, strides %ld %ld} and {%ld x %ld of %ld at %ld, strides %ld %ld}\n", got, (long)a.rows,
                    (long)a.heads, (long)a.bytes, (long)a.at, (long)a.row, (long)a.head, (long)b.rows, (long)b.heads, (long)b.bytes, (long)b.at,
                    (long)b.row, (long)b.head);
    }
    ++g_sets;
    g_overlapping += want;
  }
}

// A call on a packed projection x [t, 12, 64] of bfloat16 at 1 MiB (8 query, 2 key and 2 value heads); everything else in memory
// of its own.
constexpr int kT = 4, kD = 64;
constexpr uint64_t kX = 0x100000, kY = 0x200000, kInts = 0x300000, kCache = 0x400000;
spa_heads view(uint64_t base, int64_t head, int64_t row = 0, int64_t row_stride = 12 * kD, int64_t head_stride = kD) {
  return spa_heads{reinterpret_cast<const void*>((uintptr_t)(base + 2 * (row * row_stride + head * head_stride))), row_stride, head_stride};
}
template <typename T = void>
T* mem(uint64_t at) { return reinterpret_cast<T*>((uintptr_t)at); }
struct Call {
  spa_heads q = view(kX, 0), k = view(kX, 8), v = view(kX, 10), q_out = view(kY, 0), k_out = view(kY, 8);
  const int32_t *pos = mem<const int32_t>(kInts), *slots = mem<const int32_t>(kInts + 4096);
  spa_rope rope{mem<const float>(kInts + 8192), kD, 0};
  spa_norm qn{SPA_NORM_LAYER, mem<const void>(kInts + 12288), mem<const void>(kInts + 12544)};
  spa_norm kn{SPA_NORM_LAYER, mem<const void>(kInts + 12800), mem<const void>(kInts + 13056)};
  spa_kv_cache c{SPA_BF16, SPA_KV_MXFP4, 4, 16, 2, kD, mem(kCache), mem(kCache + 65536), mem(kCache + 131072), mem(kCache + 196608)};
  bool cached = true, keys = true;
  int t = kT;
  spa_status operator()() const {
    ++g_calls;
    return spa_check::check_qk_norm_rope(&q, &k, cached ? &v : nullptr, SPA_BF16, t, 8, 2, kD, pos, &rope, &qn, &kn, 1e-5f, &q_out,
                                         keys ? &k_out : nullptr, cached ? slots : nullptr, cached ? &c : nullptr);
  }
};
template <typename F>
void is(spa_status want, const char* name, F change) {
  for (int cached = 0; cached < 2; ++cached) {
    Call call;
    call.cached = cached;
    change(call);
    const spa_status got = call();
    if (got != want && g_fails++ < 20) std::printf("fail: %s (cache %d): status %d, not %d\n", name, (int)call.cached, (int)got, (int)want);
  }
}
template <typename F>
void refused(const char* name, F change) { is(SPA_ERR_INVALID, name, change); }
template <typename F>
void accepted(const char* name, F change) { is(SPA_OK, name, change); }

void calls() {
  accepted("apart", [](Call&) {});
  accepted("in place", [](Call& c) { c.q_out = c.q, c.k_out = c.k; });
  accepted("keys in place", [](Call& c) { c.k_out = c.k; });
  accepted("interleaved heads in place", [](Call& c) {      // [t, heads, 3, d] with as many heads of queries as of keys, and more
    c.q = c.q_out = view(kX, 0, 0, 24 * kD, 3 * kD);
    c.k = c.k_out = view(kX + 2 * kD, 0, 0, 24 * kD, 3 * kD);
    c.v = view(kX + 4 * kD, 0, 0, 24 * kD, 3 * kD);
  });
  accepted("heads outermost, in place", [](Call& c) {
    c.q = c.q_out = view(kX, 0, 0, kD, kT * kD);
    c.k = c.k_out = view(kX, 8, 0, kD, kT * kD);
    c.v = view(kX, 10, 0, kD, kT * kD);
  });
  accepted("one row, in place, strides that do not count", [](Call& c) {
    c.t = 1;
    c.q_out = c.q, c.k_out = c.k;
    c.q.row_stride = 0, c.k_out.row_stride = 8;
  });
  accepted("queries' place taken by keys of another buffer's rows", [](Call& c) { c.q_out = view(kY, 4), c.k_out = view(kY, 2); });
  accepted("the same vector for every row, elsewhere", [](Call& c) { c.q.row_stride = c.k.row_stride = c.v.row_stride = 0; });
  accepted("values read beside the keys that are written", [](Call& c) { c.k_out = c.k; });

  refused("queries a head further on", [](Call& c) { c.q_out = view(kX, 1), c.k_out = c.k; });
  refused("queries a head further on, keys elsewhere", [](Call& c) { c.q_out = view(kX, 1); });
  refused("queries a head before", [](Call& c) { c.q = view(kX, 1), c.q_out = view(kX, 0), c.k = view(kY, 8), c.k_out = view(kY, 8); });
  refused("queries a row further on", [](Call& c) { c.q_out = view(kX, 0, 1); });
  refused("queries half a vector further on", [](Call& c) { c.q_out.data = mem<const void>(kX + kD); });
  refused("queries and keys share a head", [](Call& c) { c.k_out = view(kY, 7); });
  refused("queries and keys share a head, keys first", [](Call& c) { c.q_out = view(kY, 2), c.k_out = view(kY, 1); });
  refused("keys a head further on", [](Call& c) { c.k_out = view(kX, 9); });
  refused("keys within the queries", [](Call& c) { c.k_out = view(kX, 3); });
  refused("keys a row further on", [](Call& c) { c.k_out = view(kX, 8, 1); });
  refused("queries over the keys' last head", [](Call& c) { c.q_out = view(kX, 9); c.k_out = view(kY, 20); });
  refused("queries in place, keys the same tensor", [](Call& c) { c.k = c.q, c.q_out = c.q; });
  refused("other strides on the same memory", [](Call& c) { c.q_out = view(kX, 0, 0, 24 * kD, kD); });
  refused("heads outermost over heads innermost", [](Call& c) { c.q_out = view(kX, 0, 0, kD, kT * kD); });
  refused("in place, the same vector for every row", [](Call& c) { c.q.row_stride = 0, c.q_out = view(kX, 0); });
  const uint64_t last = kY + 2 * (3 * 12 * kD + 8 * kD) - 16;                 // the queries' last 16 bytes
  refused("positions", [=](Call& c) { c.pos = mem<const int32_t>(last); });
  refused("positions that end in the first vector", [](Call& c) { c.pos = mem<const int32_t>(kY - 4 * (kT - 1)); });
  accepted("positions that end before it", [](Call& c) { c.pos = mem<const int32_t>(kY - 4 * kT); });
  accepted("positions behind the last", [=](Call& c) { c.pos = mem<const int32_t>(last + 16), c.k_out = view(kX + 0x40000, 0); });
  refused("frequencies", [=](Call& c) { c.rope.inv_freq = mem<const float>(last); });
  accepted("frequencies that are not read", [=](Call& c) { c.rope.inv_freq = mem<const float>(last), c.rope.rotary_dim = 0; });
  refused("queries' weights", [=](Call& c) { c.qn.weight = mem<const void>(last); });
  refused("queries' biases", [=](Call& c) { c.qn.bias = mem<const void>(last); });
  refused("keys' weights", [=](Call& c) { c.kn.weight = mem<const void>(last); });
  refused("keys' biases", [=](Call& c) { c.kn.bias = mem<const void>(last); });
  accepted("weights that are not read", [=](Call& c) { c.kn = spa_norm{SPA_NORM_NONE, mem<const void>(last), mem<const void>(last)}; });

  auto with_cache = [](auto change) {
    return [=](Call& c) {
      c.cached = true;
      change(c);
    };
  };
  accepted("keys into the cache alone", with_cache([](Call& c) { c.keys = false; }));
  refused("slots", with_cache([=](Call& c) { c.slots = mem<const int32_t>(last); }));
  refused("queries over the values", with_cache([](Call& c) { c.q_out = view(kX, 10); }));
  refused("keys over the values", with_cache([](Call& c) { c.k_out = view(kX, 10); }));
  refused("keys over the values' second head", with_cache([](Call& c) { c.k_out = view(kX, 11); }));
  const uint64_t codes = 4 * 16 * 2 * kD / 2, bytes = 4 * 16 * 2 * kD / 32;   // of the pages, of their scales
  for (int part = 0; part < 4; ++part) {
    const uint64_t at = kCache + 65536 * part, end = at + (part < 2 ? codes : bytes);
    refused("queries on a cache", with_cache([=](Call& c) { c.q_out.data = mem<const void>(end - 16); }));
    refused("keys on a cache", with_cache([=](Call& c) { c.k_out.data = mem<const void>(at); }));
    accepted("queries behind a cache", with_cache([=](Call& c) { c.q_out.data = mem<const void>(end); }));
    refused("values in a cache", with_cache([=](Call& c) { c.v.data = mem<const void>(end - 16); }));
    refused("positions in a cache", with_cache([=](Call& c) { c.pos = mem<const int32_t>(end - 4); }));
    refused("slots in a cache", with_cache([=](Call& c) { c.slots = mem<const int32_t>(end - 4); }));
  }
  // the formats' sizes
  const int64_t cells = 4 * 16 * 2, sizes[4][2] = {{cells * kD * 2, 0}, {cells * kD, cells * 4}, {cells * kD, cells * 4}, {cells * kD / 2, cells * 2}};
  for (int f = 0; f < 4; ++f)
    for (int part = 0; part < 4; ++part) {
      const int64_t n = sizes[f][part >= 2];
      const uint64_t at = kCache + 65536 * part;
      if (n) refused("a format's last bytes", with_cache([=](Call& c) { c.c.format = f, c.q_out.data = mem<const void>(at + n - 16); }));
      accepted("behind a format's last bytes", with_cache([=](Call& c) { c.c.format = f, c.q_out.data = mem<const void>(at + n); }));
    }
}

}  // namespace

int main() {
  sweep();
  calls();
  if (g_fails) {
    std::printf("failures %d\n", g_fails);
    return 1;
  }
  std::printf("ok %ld %ld %ld\n", g_sets, g_overlapping, g_calls);
  return 0;
}
