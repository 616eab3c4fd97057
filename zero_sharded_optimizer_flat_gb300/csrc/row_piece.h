// Pieces of rows that start anywhere.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace zopt {
namespace lm {

// Eight bf16 elements from s, those from n on zero.
__host__ __device__ __forceinline__ uint4 row_piece8(const uint16_t* s, long long n) {
  const unsigned mis = static_cast<unsigned>(reinterpret_cast<uintptr_t>(s)) & 15u;
  if (n >= 8 && mis == 0) return *reinterpret_cast<const uint4*>(s);
  if (n >= 8 && (mis & 7u) == 0) {
    const uint2 a = reinterpret_cast<const uint2*>(s)[0], b = reinterpret_cast<const uint2*>(s)[1];
    return make_uint4(a.x, a.y, b.x, b.y);
  }
  if (n >= 8) {
    // words, each a whole one of memory: of a row that starts in the middle of one, four and a half, shifted together
    // (what lies behind the eighth element may be nobody's)
    const uint32_t* const w = reinterpret_cast<const uint32_t*>(reinterpret_cast<uintptr_t>(s) & ~uintptr_t{3});
    uint32_t x[5];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = w[k];
    x[4] = (mis & 2u) != 0 ? s[7] : 0u;
    if ((mis & 2u) == 0) return make_uint4(x[0], x[1], x[2], x[3]);
    return make_uint4((x[0] >> 16) | (x[1] << 16), (x[1] >> 16) | (x[2] << 16), (x[2] >> 16) | (x[3] << 16),
                      (x[3] >> 16) | (x[4] << 16));
  }
  uint32_t x[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = k < n ? s[k] : 0u;
  return make_uint4(x[0] | (x[1] << 16), x[2] | (x[3] << 16), x[4] | (x[5] << 16), x[6] | (x[7] << 16));
}

}  // namespace lm
}  // namespace zopt
