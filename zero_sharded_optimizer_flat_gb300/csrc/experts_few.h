// The experts' forward for a few slots (not part of the ABI).
#pragma once

#include <cuda_runtime.h>

#include "internal.h"

namespace zopt {
namespace few {

// Whether this path takes the job.
bool takes(const zopt_experts_job& job);
// fp32 elements of the partial sums of a job it takes: gate and up's, y's.
void partial_elems(const zopt_experts_job& job, long long* gate_up, long long* y);
// y (and what is kept) of a checked job it takes.
zopt_status experts_forward(const zopt_experts_job& job, float* gate_up, float* y, cudaStream_t s);

}  // namespace few
}  // namespace zopt
