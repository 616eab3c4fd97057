// The feed-forward block's forward for a few tokens (not part of the ABI).
#pragma once

#include <cuda_runtime.h>

#include "internal.h"

namespace zopt {
namespace few {

constexpr long long kFewTokens = 4;

// Whether this path takes the job: few tokens, a grid that covers the shape and, for three tokens and
// more, weights that it reads sooner than the tensor cores' path.
bool takes(const zopt_ffn_job& job);
// fp32 elements of the partial sums of a job it takes: gate and up's, y's.
void partial_elems(const zopt_ffn_job& job, long long* gate_up, long long* y);
// y (and what is kept) of a checked job it takes.
zopt_status ffn_forward(const zopt_ffn_job& job, float* gate_up, float* y, cudaStream_t s);

}  // namespace few
}  // namespace zopt
