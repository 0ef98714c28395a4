// Division by a number fixed for a launch (host and device).
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define SPA_DIV_HD __host__ __device__ __forceinline__
#else
#define SPA_DIV_HD inline
#endif

namespace spa {

// floor(x / d) for x below 2^31 and d of 1..2^31 - 1: with s = ceil(log2 d) and m = ceil(2^(31 + s) / d), it is
// floor(x * m / 2^(31 + s)).  The excess of m over 2^(31+s) / d is below 1, so the product is high by less than
// x / 2^(31+s) <= 1 / d, which never reaches the next whole number.
struct FastDiv {
  uint32_t d, m, s;
  FastDiv() = default;
  explicit SPA_DIV_HD FastDiv(uint32_t div) : d(div) {
    s = 0;
    while ((1ull << s) < div) ++s;
    m = (uint32_t)(((1ull << (31 + s)) + div - 1) / div);       // below 2^32: 2^s < 2 d
  }
  SPA_DIV_HD uint32_t div(uint32_t x) const { return (uint32_t)(((uint64_t)x * m) >> (31 + s)); }
};

}  // namespace spa
