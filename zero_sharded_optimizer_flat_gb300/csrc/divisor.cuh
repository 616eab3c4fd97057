// Division by a number the host knows.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace zopt {

// n / d for n < 2^31 by a multiplication (division by invariant integers, Granlund and Montgomery).
struct Divisor {
  uint32_t d, m, s;
  Divisor() = default;
  explicit Divisor(uint32_t d_) : d(d_), m(0), s(0) {
    while (s < 32 && (1ull << s) < d) ++s;
    m = static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - d)) / d + 1);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (__umulhi(m, n) + n) >> s; }
};

}  // namespace zopt
