// Linear cross entropy's forward for a few tokens (not part of the ABI).
#pragma once

#include <cuda_runtime.h>

#include "internal.h"

namespace zopt {
namespace few {

// Whether this path takes the job's forward.
bool takes(const zopt_linear_ce_job& job);
// The (maximum, sum) pairs that it leaves for each token: one a CTA.
int ce_parts(const zopt_linear_ce_job& job);
// part[p][token], p < ce_parts, and the targets' logits of a checked job it takes.
zopt_status ce_logits(const zopt_linear_ce_job& job, float2* part, float* tlogit, cudaStream_t s);

}  // namespace few
}  // namespace zopt
