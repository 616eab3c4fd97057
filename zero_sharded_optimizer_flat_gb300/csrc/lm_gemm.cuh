// The matrix products of the training operators (linear_ce.cu, ffn.cu) on CTA pairs, each with the
// epilogue its operator needs: what a launch is made of, on both sides of the launch.
//
// A launch is a batch of jobs. A job is one product D = P Q, D of M x N with inner length K,
// fp32 accumulation over bf16 operands, cut into tiles of 256 x 256 or 256 x 128 (kGluFwd: 128 or 64
// gate and the matching up columns) and, where a launch would leave most CTA pairs idle, into runs
// of k-blocks as well. Operands come through 2-D tensor maps: P's rows and Q's columns either with the
// inner length contiguous ("K-major") or with the other one ("MN-major", a_mn / b_mn).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "divisor.cuh"
#include "internal.h"

namespace zopt {
namespace lm {

constexpr int kTileM = 256, kTileN = 256, kTileK = 64;
constexpr int kPairs = 76;  // GB300's CTA pairs, what work is shared out for
constexpr int kStages = 6;
constexpr int kHalfBytes = 128 * kTileK * 2;  // one CTA's half of a stage's P or Q: 16 KiB
constexpr int kMnBoxBytes = 64 * kTileK * 2;  // one 64 (MN) x 64 (K) box of an MN-major operand
constexpr int kEpiWarps = 8;
constexpr int kFirstEpi = 3;  // warp 0 loads P, warp 1 issues the MMAs, warp 2 loads Q, warps 3 .. 10 epilogue
constexpr int kThreads = 32 * (kFirstEpi + kEpiWarps);
constexpr int kBoxBytes = 32 * 128;  // an epilogue warp's results on their way to memory: 32 rows of 128 bytes
constexpr int kSwapBytes = 4 * 64 * 2;  // kGluFwd: two warps' block exponents for each quarter of the rows
constexpr int kSmemBytes = kStages * 2 * kHalfBytes + kEpiWarps * kBoxBytes + kSwapBytes + 1024 + 256;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");
constexpr int kMaxJobs = 3;
constexpr float kLog2e = 1.4426950408889634f;
// The longest inner length: an epilogue waits for a whole tile's products (those that are not cut) with a
// limit (tc::kWaitLimitNs, 4 s), so they have to end well before it. These are 2^20 k-blocks: 0.43 s where
// all pairs share one operand and read the other from HBM (cross entropy forward, 256 x 2^19 x 19456:
// 0.41 us a k-block), twice that if they shared none.
constexpr long long kMaxInner = 1LL << 26;

// What an epilogue makes of its accumulators.
enum Kind : int {
  kStore = 1,   // D (+ add), rounded to bf16 or kept in fp32
  kCeFwd = 2,   // softmax statistics of the logits
  kCeBwd = 4,   // the logits' gradient
  kGluFwd = 8,  // h = a(gate) * up, gate and up kept
  kGluBwd = 16  // dgate, dup and h from dh
};

enum OutMode : int { kOutBf16 = 0, kOutF32 = 1 };                   // kStore
enum KeptMode : int { kKeepNone = 0, kKeepBf16 = 1, kKeep8 = 2 };  // kGluFwd, kGluBwd

struct Job {
  CUtensorMap P, Q, Up;  // Up: kGluFwd's up columns (Q: its gate's)
  int kind;
  int M, N, K;
  int a_mn, b_mn;
  int tile_n;  // columns of a tile: 256 or 128
  int a_rows;  // rows of P (K-major) a CTA loads at a time: 128, or M rounded up to 8 where M <= 128
  int tx;      // bytes of a stage, both CTAs'
  int tiles_m, tiles_n, tiles;
  Divisor per_split, per_line;  // by tiles; by the tiles that follow one another (set at the launch)
  int nk, kb_per_split, splits;
  int whole;      // its inner length is not cut
  int rows_fast;  // consecutive tiles walk down a tile column (else along a tile row)
  // D, or what the epilogue makes of it: kCeBwd's dl; kGluFwd's h; kGluBwd's dgate, its dup N columns
  // later, and h (out_h, rows of ld_h)
  void* out;
  long long ld_out;
  void* out_h;
  long long ld_h;
  // kStore
  int out_mode;
  long long split_stride;  // split_stride: elements between the partial sums of one tile's runs of k
  const float* add;                // fp32 M x N added to D; null: none
  long long ld_add;
  const float* alpha;  // (D + add) is multiplied by *alpha; null: 1
  // kCeFwd, kCeBwd
  const int64_t* target;
  int64_t ignore, vocab, col0;  // the job's columns are vocabulary entries col0 ...
  const float* lse;
  const float* dloss;
  const float* unit;  // kCeBwd: dl is stored in this unit (it is its products' alpha)
  float2* part;   // kCeFwd: (max, sum) of half a tile's logits times kLog2e, at [2 tile column + half][row]
  float* tlogit;  // kCeFwd: the target's logit
  // kGluFwd, kGluBwd
  int act, kept_mode;
  void* kept;  // gate and up as the caller keeps them: row r's gate at r * ld_kept, its up hidden later
  long long ld_kept;
  uint8_t* kept_scale;  // kKeep8: row r's block exponents at r * 2 blocks, the gate's first
  int hidden;           // the gate's width, N
};

// Units of work are numbered job by job, a job's runs of k one after another. Pair p takes units p,
// p + pairs, ...; or, in a launch of unequal units few enough for it, those that the host gave it:
// order[first[p]] .. order[first[p + 1] - 1].
constexpr int kMaxListed = 512;

struct Batch {
  int n;
  int start[kMaxJobs + 1];
  int listed;
  int* err;
  Job job[kMaxJobs];
  uint16_t first[kPairs + 1];
  uint16_t order[kMaxListed];
};

// ------------------------------------------------------------------ host side

// The maps of a tiled job's operands: P's M rows and Q's columns (`columns` of them as stored), stored
// with the inner length contiguous, or as its transpose where MN-major; `pitch` elements (a multiple
// of 8) between the rows as stored.
zopt_status map_p(const char* fn, Job& j, const void* base, long long pitch);
zopt_status map_q(const char* fn, Job& j, const void* base, long long columns, long long pitch);
zopt_status map_up(const char* fn, Job& j, const void* base, long long columns, long long pitch);

// Fills a job's tiling from kind, M, N, K, a_mn, b_mn and kept_mode.
void set_tiles(Job& j);
// Cuts the inner length of the batch's kStore jobs so that no pair's run of k-blocks is much longer
// than the launch's average (none where there are tiles enough). Depends on the shapes alone.
void plan_splits(Job* jobs, int n);
// fp32 elements of a job's partial sums (0 without splits): splits matrices of M x split_pitch(N).
inline long long split_pitch(long long n) { return (n + 3) / 4 * 4; }
inline long long split_elems(const Job& j) {
  return j.splits > 1 ? static_cast<long long>(j.splits) * j.M * split_pitch(j.N) : 0;
}
// Launches the batch with the kernel for `kinds` (a union of Kind values it was built for).
zopt_status launch(const char* fn, Batch& b, int kinds, cudaStream_t s);

// After a launch with splits: out = the sum of each job's partial sums in split order, as bf16.
struct SumJob {
  const float* part;
  long long split_stride, pitch;
  int splits;
  long long M, N;
  uint16_t* out;
  long long ld_out;
  const float* alpha;
};
struct SumBatch {
  int n;
  long long start[kMaxJobs + 1];  // in groups of four columns
  SumJob job[kMaxJobs];
};
zopt_status launch_sums(const char* fn, const SumBatch& b, cudaStream_t s);

// dst[r][c] = src[r][c] for c < cols, 0 for cols <= c < dst_cols: an operand that the TMA cannot read
// where it is.
zopt_status launch_stage(const char* fn, uint16_t* dst, long long dst_pitch, long long dst_cols, const uint16_t* src,
                         long long src_pitch, long long rows, long long cols, cudaStream_t s);

// Blocks of 256 threads for `items` threads' work, at most eight per SM.
unsigned blocks_for(long long items, int sms);

// Eight bf16 elements from s, those from n on zero.
__device__ __forceinline__ uint4 row_piece8(const uint16_t* s, long long n) {
  if (n >= 8 && (reinterpret_cast<uintptr_t>(s) & 15u) == 0) return *reinterpret_cast<const uint4*>(s);
  uint32_t x[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) x[k] = k < n ? s[k] : 0u;
  return make_uint4(x[0] | (x[1] << 16), x[2] | (x[3] << 16), x[4] | (x[5] << 16), x[6] | (x[7] << 16));
}

inline long long round_up(long long x, long long a) { return (x + a - 1) / a * a; }

}  // namespace lm
}  // namespace zopt
