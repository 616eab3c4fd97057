// The experts' products: batches whose rows belong to one expert after another (not part of the ABI).
#pragma once

#include "lm_gemm.cuh"

namespace zopt {
namespace lm {

constexpr int kGroupRows = 64;  // an expert's rows are filled up to a multiple of these

// The maps of a grouped job's operands: activations (rows of all experts, `rows` of them; 64 to a box) or, deeper,
// the experts' weights, `stride` elements apart. mn: the inner length is the rows, not the columns.
zopt_status map_rows(const char* fn, CUtensorMap* m, const void* base, long long rows, long long cols, long long pitch);
zopt_status map_weights(const char* fn, CUtensorMap* m, const void* base, long long rows, long long cols,
                        long long pitch, long long experts, long long stride, int mn, int box);

// Fills a grouped job's tiling from kind, M (by_inner), N, K (else), a_mn, b_mn and kept_mode.
void set_group_tiles(Job& j);
// Launches the batch with the kernel for `kinds` (kStore, kGluFwd or kGluBwd). most_tiles: row tiles that there
// can be.
zopt_status launch_grouped(const char* fn, Batch& b, int kinds, long long most_tiles, cudaStream_t s);

}  // namespace lm
}  // namespace zopt
