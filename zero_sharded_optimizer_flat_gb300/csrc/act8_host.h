// Host side of the 8-bit checkpoints, shared with the feed-forward block (not part of the ABI).
#pragma once

#include <cuda_runtime.h>

#include "internal.h"

namespace zopt {
namespace act8 {

constexpr long long kMaxDim = 1LL << 30;

size_t scale_bytes(long long rows, long long cols, int parts);
// The checkpoint's own consistency (shape, pointers, alignment).
zopt_status check(const char* fn, const zopt_act8& c);
// A checked checkpoint's values as bf16 rows of ld elements.
zopt_status unpack(const char* fn, const zopt_act8& c, uint16_t* out, long long ld, cudaStream_t s);

}  // namespace act8
}  // namespace zopt
