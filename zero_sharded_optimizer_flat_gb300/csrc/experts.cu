// The experts' feed-forward block, forward and backward.
//
// The plan: one cluster counts the experts' slots, gives every expert a run of rows (a multiple of 64) and
// every slot a row of its expert's run, in the slots' order, so that a call's results do not depend on
// which thread came first. Then
//   forward:   x's rows copied into that order; gate and up with the activation, the weight and the
//              product in the epilogue; down; every token's parts added up.
//   backward:  x's and dy's rows copied; dh, whose epilogue reads the kept gate and up and writes dgate,
//              dup, h and the parts of dweight; dx's parts, dgate_up and ddown in one launch; every
//              token's parts added up.
// (A forward of a few slots takes experts_few.cu.)
//
// Measured (GB300, 8192 tokens' 6 slots among 64 experts, 2048 x 1408): forward with bf16 kept 725 us = 1.17
// PFLOP/s: the products 350 and 180 by themselves (tensor pipe 87 and 79 % of elapsed at the clock that the power
// cap leaves; what is lost beside it are the experts' last row tiles), the rows in and out 36 and 42, the plan
// 14. Backward, 8 bits kept, 1385 to 1466 us: by themselves dh and its epilogue take 240, the three products behind
// it 950, rows in 78, out 44.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "act8.cuh"
#include "act8_host.h"
#include "divisor.cuh"
#include "experts_few.h"
#include "experts_gemm.h"
#include "guarded.h"
#include "launch.cuh"
#include "ns_internal.h"
#include "per_device.h"
#include "tc.cuh"

namespace zopt {
namespace lm {
namespace {

constexpr int kMaxExperts = 1024, kMaxTopK = 32;
constexpr long long kMaxSlots = 1LL << 26;
constexpr long long kMaxLd = 1LL << 32, kMaxStride = 1LL << 38;
constexpr long long kMaxElems = 1LL << 44;  // of any matrix: tile numbers stay well below 2^31

// ---------------------------------------------------------------------- the plan

constexpr int kPlanCtas = 8, kPlanWarps = 32;
constexpr int kPlanKept = 8;  // times 32 slots that a warp keeps in registers

struct PlanArgs {
  const int32_t* index;
  const float* weight;
  long long slots;
  int experts, tile_rows;
  int* head;
  int4* tiles;
  int2* info;
  int* used;     // the experts that have a slot
  int2* row;     // [rows] slot and weight
  int* row_of;   // [slots] its row; -1: none; -2: an index that is none
};

__device__ __forceinline__ int read_remote(const int* p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(tc::map_to_rank(tc::smem_u32(p), rank)) : "memory");
  return v;
}

// Every warp has a run of the slots, and counts its experts' 32 at a time; sums over the warps, the
// cluster's blocks and the experts before give each warp the first row of each expert's slots in its
// run, and the run is gone through again.
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(32 * kPlanWarps) plan_kernel(const PlanArgs a) {
  extern __shared__ int smem[];
  int* count = smem;                               // [warps][experts]
  int* mine = count + kPlanWarps * a.experts;      // [experts] this block's
  __shared__ uint32_t sums[2][kPlanWarps];
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.experts;
  const uint32_t rank = tc::cluster_rank();
  const long long per = (a.slots + 32 * kPlanCtas * kPlanWarps - 1) / (32 * kPlanCtas * kPlanWarps) * 32;
  const long long s0 = (static_cast<long long>(rank) * kPlanWarps + warp) * per, s1 = min(a.slots, s0 + per);
  int* const my = count + warp * E;
  for (int e = lane; e < E; e += 32) my[e] = 0;
  __syncwarp();
  int kept[kPlanKept];  // the first of the run's, and which of the 32 are the same
  unsigned same[kPlanKept];
#pragma unroll
  for (int k = 0; k < kPlanKept; ++k) {
    const long long s = s0 + 32 * k + lane;
    kept[k] = s < s1 ? a.index[s] : -1;
  }
#pragma unroll
  for (int k = 0; k < kPlanKept; ++k) {
    if (s0 + 32 * k >= s1) break;
    same[k] = __match_any_sync(0xFFFFFFFFu, kept[k]);
    if (kept[k] >= 0 && kept[k] < E && lane == __ffs(same[k]) - 1) my[kept[k]] += __popc(same[k]);
    __syncwarp();
  }
  for (long long s = s0 + 32 * kPlanKept; s < s1; s += 32) {
    const int e = s + lane < s1 ? a.index[s + lane] : -1;
    const unsigned m = __match_any_sync(0xFFFFFFFFu, e);
    if (e >= 0 && e < E && lane == __ffs(m) - 1) my[e] += __popc(m);
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 32 * kPlanWarps) {  // (once: E <= 1024)
    int run = 0;
#pragma unroll 8
    for (int w = 0; w < kPlanWarps; ++w) {
      const int c = count[w * E + e];
      count[w * E + e] = run;
      run += c;
    }
    mine[e] = run;
  }
  tc::cluster_sync();
  const int e = threadIdx.x;
  int before = 0, all = 0;
  if (e < E) {
    for (uint32_t r = 0; r < kPlanCtas; ++r) {
      const int c = read_remote(mine + e, r);
      before += r < rank ? c : 0;
      all += c;
    }
  }
  // the experts before: their rows, and in one word their row tiles (fewer than 2^20) and how many have a slot
  constexpr int kTileBits = 21;
  static_assert(kMaxSlots / 128 + kMaxExperts < 1LL << kTileBits && static_cast<long long>(kMaxExperts) << kTileBits < 1LL << 32, "the word");
  const int rows = (all + kGroupRows - 1) / kGroupRows * kGroupRows, tiles = (all + a.tile_rows - 1) / a.tile_rows;
  const uint32_t word = static_cast<uint32_t>(tiles) | (all > 0 ? 1u << kTileBits : 0u);
  int r = rows;
  uint32_t t = word;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, r, d);
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, t, d);
    if (lane >= d) r += x, t += y;
  }
  if (lane == 31) sums[0][warp] = static_cast<uint32_t>(r), sums[1][warp] = t;
  __syncthreads();
  if (warp == 0) {
    uint32_t x = sums[0][lane], y = sums[1][lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, x, d), v = __shfl_up_sync(0xFFFFFFFFu, y, d);
      if (lane >= d) x += u, y += v;
    }
    sums[0][lane] = x, sums[1][lane] = y;
  }
  __syncthreads();
  const int first = r - rows + (warp > 0 ? static_cast<int>(sums[0][warp - 1]) : 0);
  const uint32_t before_it = t - word + (warp > 0 ? sums[1][warp - 1] : 0u), sum = sums[1][kPlanWarps - 1];
  const int first_tile = static_cast<int>(before_it & ((1u << kTileBits) - 1u));
  if (rank == 0 && threadIdx.x == 0)
    a.head[0] = static_cast<int>(sum & ((1u << kTileBits) - 1u)), a.head[1] = static_cast<int>(sum >> kTileBits);
  tc::cluster_sync();  // every block has read `mine`
  if (e < E) {
    mine[e] = first + before;
    if (rank == 0) a.info[e] = make_int2(first, all);
    if (rank == 0 && all > 0) a.used[before_it >> kTileBits] = e;
    for (int i = static_cast<int>(rank); i < tiles; i += kPlanCtas)
      a.tiles[first_tile + i] = make_int4(e, first + i * a.tile_rows, min(first + rows, first + (i + 1) * a.tile_rows),
                                          min(all - i * a.tile_rows, a.tile_rows) <= kTileM / 2 ? 1 : 0);
    for (int i = all + static_cast<int>(rank); i < rows; i += kPlanCtas) a.row[first + i] = make_int2(-1, 0);
  }
  __syncthreads();
  auto place = [&](long long s, int x, unsigned same, float weight) {  // 32 slots from s on
    const bool on = x >= 0 && x < E;
    int at = x == -1 ? -1 : -2;
    if (on) {
      at = mine[x] + my[x] + __popc(same & ((1u << lane) - 1u));
      a.row[at] = make_int2(static_cast<int>(s) + lane, __float_as_int(weight));
    }
    if (s + lane < s1) a.row_of[s + lane] = at;
    __syncwarp();
    if (on && lane == __ffs(same) - 1) my[x] += __popc(same);
    __syncwarp();
  };
  float weight[kPlanKept];
#pragma unroll
  for (int k = 0; k < kPlanKept; ++k) weight[k] = kept[k] >= 0 && kept[k] < E ? a.weight[s0 + 32 * k + lane] : 0.0f;
#pragma unroll
  for (int k = 0; k < kPlanKept; ++k) {
    if (s0 + 32 * k >= s1) break;
    place(s0 + 32 * k, kept[k], same[k], weight[k]);
  }
  for (long long s = s0 + 32 * kPlanKept; s < s1; s += 32) {
    const int x = s + lane < s1 ? a.index[s + lane] : -1;
    place(s, x, __match_any_sync(0xFFFFFFFFu, x), x >= 0 && x < E ? a.weight[s + lane] : 0.0f);
  }
}

// ---------------------------------------------------------------------- rows in and out

struct Source {
  const uint16_t* x;  // rows of ld elements; null: none
  long long ld;
  const uint8_t *q, *scale;  // or a checkpoint (x null)
  uint16_t* to;              // rows of `pitch` elements
};
// An operand that the TMA cannot read where it is: dst[e][r][c] = src[e][r][c] for c < cols, 0 up to dst_cols. Of
// experts that have a slot alone: no unit reads another's.
struct Copy {
  uint16_t* dst;
  const uint16_t* src;
  long long dst_cols, ld, stride, rows, cols;
  long long chunk;  // at most 2^30 rows, of fewer than 2^31 pieces less a grid's threads
  Divisor per_row, per_expert;
};
// The kept rows of the slots that have an expert, gate and up each from a 16-byte boundary on, zeros behind them
// (the epilogue that reads them takes 16 bytes of a row at a time; rows that start anywhere, a lane each, would
// take it 32 times as long).
struct KeptCopy {
  uint8_t* dst;  // rows of two parts of `part` bytes; null: none
  const void* src;
  long long ld, hidden, part;
  int size;  // of an entry
};
struct GatherArgs {
  Source from[2];
  int n;
  long long tokens, cols, pitch;
  const int* row_of;
  const int2* info;
  const int *head, *used;
  int top_k, experts;
  int fill;  // the backward multiplies by the rows that only fill up
  Copy copy[3];
  int copies;
  KeptCopy kept;
};

// 16 bytes of a token's row, zeros behind the last column.
__device__ __forceinline__ uint4 piece_of(const Source& f, long long cols, long long token, int p) {
  if (f.x != nullptr) return row_piece8(f.x + token * f.ld + 8 * p, cols - 8 * p);
  const uint8_t* const q = f.q + token * cols;  // (a piece of eight columns lies in one block of 128)
  uint32_t w[4];
  const float power = act8::scale(f.scale[token * act8::blocks_of(cols) + (p >> 4)]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long c = 8 * p + 2 * i;
    const uint32_t two = (c < cols ? q[c] : 0u) | ((c + 1 < cols ? q[c + 1] : 0u) << 8);
    const float2 v = act8::decode2(two);
    const __nv_bfloat162 h = __floats2bfloat162_rn(v.x * power, v.y * power);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// (Where a piece lies is found without divisions: with 64-bit ones a forward of 64 x 6 slots of 64 experts, 2047 x 1407,
// takes 850 us for 806. `chunk` rows at a time, their pieces' numbers below 2^31.)
__device__ __forceinline__ void copy_rows(const Copy& c, const int* used, int n, uint32_t thread, uint32_t threads) {
  const long long rows = n * c.rows;
  for (long long row0 = 0; row0 < rows; row0 += c.chunk) {
    const long long k0 = row0 / c.rows;
    const uint32_t r0 = static_cast<uint32_t>(row0 - k0 * c.rows);
    const uint32_t all = static_cast<uint32_t>(min(c.chunk, rows - row0)) * c.per_row.d;
#pragma unroll 2
    for (uint32_t g = thread; g < all; g += threads) {
      const uint32_t row = c.per_row(g), k = c.per_expert(r0 + row);
      const long long col = (g - row * c.per_row.d) * 8, r = r0 + row - k * c.per_expert.d, e = used[k0 + k];
      *reinterpret_cast<uint4*>(c.dst + (e * c.rows + r) * c.dst_cols + col) = row_piece8(c.src + e * c.stride + r * c.ld + col, c.cols - col);
    }
  }
}
__device__ __forceinline__ void copy_kept(const KeptCopy& c, const int* row_of, long long slots, int lane, int warp, int warps) {
  const long long pieces = 2 * c.part / 16;
  const int per = 16 / c.size;
  for (long long s = warp; s < slots; s += warps) {
    if (__ldcg(row_of + s) < 0) continue;
#pragma unroll 4
    for (long long p = lane; p < pieces; p += 32) {
      const long long col = (p * 16 < c.part ? p : p - c.part / 16) * per, at = s * c.ld + (p * 16 < c.part ? 0 : c.hidden) + col;
      uint4 v;
      if (c.size == 2) {
        v = row_piece8(static_cast<const uint16_t*>(c.src) + at, c.hidden - col);
      } else {
        uint32_t w[4] = {};
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (col + i < c.hidden) w[i / 4] |= static_cast<uint32_t>(static_cast<const uint8_t*>(c.src)[at + i]) << (8 * (i % 4));
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
      *reinterpret_cast<uint4*>(c.dst + s * 2 * c.part + 16 * p) = v;
    }
  }
}

// Rows of x (and dy) in the plan's order, zeros behind the last column and (fill) where a row only fills up. A warp
// reads a token's row, 1024 columns of it at a time, and writes it wherever the token's slots have theirs;
// bound by what it writes. What else has to be copied first is, in the same launch.
__global__ void __launch_bounds__(256) gather_kernel(const GatherArgs a) {
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  constexpr int kAtOnce = 4;
  const int lane = threadIdx.x & 31, warps = gridDim.x * 8, me = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int pieces = static_cast<int>(a.pitch / 8), chunks = (pieces + 32 * kAtOnce - 1) / (32 * kAtOnce);
  const long long items = a.tokens * a.n * chunks;
  for (long long i = me; i < items; i += warps) {
    const long long token = i / (a.n * chunks);
    const int k = static_cast<int>(i - token * (a.n * chunks)), from = k / chunks, p0 = (k - from * chunks) * 32 * kAtOnce + lane;
    const int mine = lane < a.top_k ? __ldcg(a.row_of + token * a.top_k + lane) : -1;
    if (!__any_sync(0xFFFFFFFFu, mine >= 0)) continue;  // (a row that nobody takes is not read)
    const Source& f = a.from[from];
    uint4 v[kAtOnce];
#pragma unroll
    for (int q = 0; q < kAtOnce; ++q)
      if (p0 + 32 * q < pieces) v[q] = piece_of(f, a.cols, token, p0 + 32 * q);
    for (int j = 0; j < a.top_k; ++j) {
      const int r = __shfl_sync(0xFFFFFFFFu, mine, j);
      if (r < 0) continue;
      uint16_t* const to = f.to + r * a.pitch;
#pragma unroll
      for (int q = 0; q < kAtOnce; ++q)
        if (p0 + 32 * q < pieces) *reinterpret_cast<uint4*>(to + 8 * (p0 + 32 * q)) = v[q];
    }
  }
  if (a.copies > 0) {
    const int n = a.head[1];
    for (int k = 0; k < a.copies; ++k) copy_rows(a.copy[k], a.used, n, blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
  }
  if (a.kept.dst != nullptr) copy_kept(a.kept, a.row_of, a.tokens * a.top_k, lane, me, warps);
  if (!a.fill) return;
  for (int i = me; i < a.experts * (kGroupRows - 1); i += warps) {  // the rows that only fill up
    const int e = i / (kGroupRows - 1), k = i - e * (kGroupRows - 1);
    const int2 at = __ldcg(a.info + e);
    if (k >= (kGroupRows - at.y % kGroupRows) % kGroupRows) continue;
    for (int q = 0; q < a.n; ++q)
      for (int p = lane; p < pieces; p += 32)
        *reinterpret_cast<uint4*>(a.from[q].to + (at.x + at.y + k) * a.pitch + 8 * p) = make_uint4(0, 0, 0, 0);
  }
}

struct CombineArgs {
  const uint16_t* parts;  // rows of `pitch` elements, fp16 in units of `scale`, at [64 columns][row]
  long long pitch;
  const float* scale;
  long long rows_ld;
  const int* row_of;
  uint16_t* out;
  long long ld;
  long long tokens, cols;
  int top_k, chunks;  // chunks: of 256 columns, and in the backward one more
  // the weights' gradient (backward): n_dots parts of each row's
  const float* dots;
  int n_dots;
  float* dweight;
};

// A token's parts added up in the order of its slots. A warp takes 256 columns of a token, or (behind the
// last ones, in the backward) its weights' gradients.
__global__ void __launch_bounds__(256) combine_kernel(const CombineArgs a) {
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long n = a.tokens * a.chunks;
  for (long long i = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < n; i += static_cast<long long>(gridDim.x) * 8) {
    const long long t = i / a.chunks;
    const int chunk = static_cast<int>(i - t * a.chunks), col = 256 * chunk + 8 * lane;
    const int mine = lane < a.top_k ? a.row_of[t * a.top_k + lane] : -1;
    if (256LL * chunk >= a.cols) {
#pragma unroll 4
      for (int j = 0; j < a.top_k; ++j) {  // (a row's parts lie side by side)
        const int r = __shfl_sync(0xFFFFFFFFu, mine, j);
        float x = 0.0f;
        if (r >= 0) {
          for (int p = lane; p < a.n_dots; p += 32) x += __ldcg(a.dots + static_cast<long long>(r) * a.n_dots + p);
        }
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, d);
        if (lane == j) a.dweight[t * a.top_k + j] = r == -2 ? __uint_as_float(0x7FC00000u) : x;
      }
      continue;
    }
    float acc[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) acc[k] = 0.0f;
#pragma unroll 4
    for (int j = 0; j < a.top_k; ++j) {
      const int r = __shfl_sync(0xFFFFFFFFu, mine, j);
      if (r >= 0 && col < a.cols) {
        const uint4 v = __ldcg(reinterpret_cast<const uint4*>(a.parts + r * a.pitch + col));
        const float unit = __ldcg(a.scale + (col >> 6) * a.rows_ld + r);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
          acc[2 * k] = fmaf(x.x, unit, acc[2 * k]);
          acc[2 * k + 1] = fmaf(x.y, unit, acc[2 * k + 1]);
        }
      }
    }
    if (__any_sync(0xFFFFFFFFu, mine == -2)) {
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = __uint_as_float(0x7FC00000u);
    }
    if (col < a.cols) {
      uint16_t* const o = a.out + t * a.ld + col;
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(acc[2 * k], acc[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      }
      if (col + 8 <= a.cols && (reinterpret_cast<uintptr_t>(o) & 15u) == 0) {
        *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (col + k < a.cols) o[k] = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
      }
    }
  }
}

// dst[e][r][c] = 0 for c < cols
__global__ void __launch_bounds__(256) zero_kernel(uint16_t* dst, long long ld, long long stride, long long experts, long long rows,
                                                   long long cols) {
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const long long n = experts * rows * cols, step = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long g = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; g < n; g += step) {
    const long long row = g / cols, e = row / rows;
    dst[e * stride + (row - e * rows) * ld + (g - row * cols)] = 0;
  }
}

// ---------------------------------------------------------------------- host

struct Layout {
  long long dp, fp, gp;  // dim, hidden and 2 hidden rounded up to 8
  long long slots, rows, tiles;
  int tile_rows;
  bool stage_gate, stage_up, stage_down, stage_kept;
  long long kept_row;  // bytes of a part of a staged row
  size_t head, tile, info, used, row, row_of, gate, up, down, xs, dys, h, dgu, parts, scales, dots, kept, few_gate_up, few_y, total;
  int dot_parts;
  bool few;
};

size_t take(size_t& at, long long bytes) {
  const size_t here = at;
  at += static_cast<size_t>(round_up(bytes, 1024));
  return here;
}

bool sizes_ok(const zopt_experts_job& c) {
  if (c.tokens < 0 || c.dim < 1 || c.hidden < 1 || c.experts < 1 || c.top_k < 1) return false;
  if (c.experts > kMaxExperts || c.top_k > kMaxTopK || c.tokens > kMaxSlots / c.top_k) return false;
  if (c.dim > kMaxInner || c.hidden > kMaxInner / 2) return false;
  const long long rows = c.tokens * c.top_k + kGroupRows * c.experts;
  return rows * c.dim <= kMaxElems && rows * 2 * c.hidden <= kMaxElems && c.experts * c.dim * 2 * c.hidden <= kMaxElems;
}

bool ld_ok(int64_t ld, int64_t least) { return ld >= least && ld <= kMaxLd; }
// (the last row of a matrix need not be followed by the rest of its distance)
bool stride_ok(int64_t stride, int64_t experts, int64_t rows, int64_t ld, int64_t cols) {
  return experts == 1 || (stride >= (rows - 1) * ld + cols && stride <= kMaxStride);
}
bool weights_ok(const zopt_experts_job& c) {
  return ld_ok(c.ld_gate_up, 2 * c.hidden) && ld_ok(c.ld_down, c.dim) &&
         stride_ok(c.stride_gate_up, c.experts, c.dim, c.ld_gate_up, 2 * c.hidden) &&
         stride_ok(c.stride_down, c.experts, c.hidden, c.ld_down, c.dim);
}

void group_job(Job& j, int kind, bool by_inner, long long m, long long n, long long k) {
  j = Job{};
  j.kind = kind;
  j.by_inner = by_inner;
  j.M = static_cast<int>(m), j.N = static_cast<int>(n), j.K = static_cast<int>(k);
  set_group_tiles(j);
}

Layout layout(const zopt_experts_job& c, bool backward) {
  Layout p{};
  const long long D = c.dim, F = c.hidden, E = c.experts;
  p.slots = c.tokens * c.top_k;
  p.dp = round_up(D, 8), p.fp = round_up(F, 8), p.gp = round_up(2 * F, 8);
  const long long used = std::min<long long>(E, p.slots);
  p.rows = round_up(p.slots + (kGroupRows - 1) * used, kGroupRows);
  // Tiles of 128 rows throughout where those of 256 (with half of one left over for every expert) would leave
  // pairs idle: the gate's product has the fewest columns (backward, 1023 x 2 slots
  // of 256 x 768 in eight experts: 37 us for 45, with the rounds of units in turn and back).
  p.tile_rows = (p.slots / kTileM + (used + 1) / 2) * ((F + kTileN - 1) / kTileN) <= kPairs ? kTileM / 2 : kTileM;
  p.tiles = p.slots / p.tile_rows + used;
  // (a tensor map's strides are multiples of 16 bytes, and the outer one of the inner)
  p.stage_gate = c.ld_gate_up % 8 != 0 || (E > 1 && c.stride_gate_up % c.ld_gate_up != 0);
  p.stage_up = p.stage_gate || F % 8 != 0;  // (the forward reads up's columns from column hidden on)
  p.stage_down = c.ld_down % 8 != 0 || (E > 1 && c.stride_down % c.ld_down != 0);
  size_t at = 0;
  p.head = take(at, 8);
  p.tile = take(at, 16 * p.tiles);
  p.info = take(at, 8 * E);
  p.used = take(at, 4 * E);
  p.row = take(at, 8 * p.rows);
  p.row_of = take(at, 4 * p.slots);
  if (p.stage_gate) p.gate = take(at, E * D * p.gp * 2);
  if (p.stage_down) p.down = take(at, E * F * p.dp * 2);
  p.xs = take(at, p.rows * p.dp * 2);
  p.h = take(at, p.rows * p.fp * 2);
  p.scales = take(at, p.rows * ((D + 63) / 64) * 4);
  p.total = at;
  if (p.stage_up) p.up = take(p.total, E * D * p.fp * 2);
  p.parts = p.xs;  // the forward's y parts, when x has been read
  p.few = few::takes(c);
  if (p.few) {
    long long gate_up, y;
    few::partial_elems(c, &gate_up, &y);
    size_t end = 0;
    p.few_gate_up = take(end, gate_up * 4);
    p.few_y = take(end, y * 4);
    p.total = end;
  }
  if (!backward) return p;
  p.dys = take(at, p.rows * p.dp * 2);
  p.dgu = take(at, p.rows * p.gp * 2);
  // dx's parts; before them, where they have to be copied, the kept rows (of whichever format: a query may not
  // know which, nor the distance of their rows, which it then has as 0)
  const long long size = c.kept8 != nullptr ? 1 : 2;
  p.stage_kept = F * size % 16 != 0 || (c.kept8 == nullptr && c.ld_kept % 8 != 0);
  p.kept_row = round_up(F * size, 16);
  const bool may = F % 16 != 0 || c.ld_kept == 0 || c.ld_kept % 8 != 0;
  p.kept = p.parts = take(at, std::max(p.rows * p.dp * 2, may ? p.slots * 2 * round_up(2 * F, 16) : 0));
  p.dot_parts = static_cast<int>((F + 63) / 64);
  p.dots = take(at, 4 * p.rows * p.dot_parts);
  p.total = std::max(p.total, at);
  return p;
}

zopt_status check(const char* fn, const zopt_experts_job* c, bool backward, void* d_ws, size_t ws_bytes) {
  const std::string f(fn);
  auto bad = [&](const char* what) { return fail(ZOPT_EINVAL, f + ": " + what); };
  if (c == nullptr) return bad("NULL job");
  if (c->dtype != ZOPT_BF16) return fail(ZOPT_EUNSUPPORTED, f + ": dtype must be ZOPT_BF16");
  if (c->act != ZOPT_ACT_SILU && c->act != ZOPT_ACT_GELU) return bad("act must be ZOPT_ACT_SILU or ZOPT_ACT_GELU");
  if (c->tokens < 0 || c->dim < 1 || c->hidden < 1) return bad("tokens < 0, dim < 1 or hidden < 1");
  if (c->experts < 1 || c->experts > kMaxExperts) return bad("experts outside 1 .. 1024");
  if (c->top_k < 1 || c->top_k > kMaxTopK) return bad("top_k outside 1 .. 32");
  if (!sizes_ok(*c)) return bad("tokens top_k above 2^26, dim above 2^26, hidden above 2^25 or a matrix above 2^44 elements");
  const int64_t T = c->tokens, D = c->dim, F = c->hidden, S = T * c->top_k;
  if (!weights_ok(*c)) return bad("a weight's row distance below its row or above 2^32, or a stride below its matrix or above 2^38");
  if (c->w_gate_up == nullptr || c->w_down == nullptr) return bad("NULL weight");
  if (!aligned16(c->w_gate_up) || !aligned16(c->w_down)) return bad("matrices must be 16-byte aligned");
  if (c->kept != nullptr && c->kept8 != nullptr) return bad("both kept and kept8");
  if (c->kept != nullptr && (!ld_ok(c->ld_kept, 2 * F) || !aligned16(c->kept))) return bad("kept: row distance or alignment");
  if (c->kept8 != nullptr) {
    const zopt_status st = act8::check(fn, *c->kept8);
    if (st != ZOPT_OK) return st;
    if (c->kept8->rows != S || c->kept8->cols != 2 * F || c->kept8->parts != 2)
      return bad("kept8 must be tokens top_k x 2 hidden in two parts");
  }
  if (backward) {
    if (c->dw_gate_up == nullptr || c->dw_down == nullptr) return bad("NULL dw_gate_up or dw_down");
    if (!ld_ok(c->ld_dx, D) || !ld_ok(c->ld_dw_gate_up, 2 * F) || !ld_ok(c->ld_dw_down, D) ||
        !stride_ok(c->stride_dw_gate_up, c->experts, D, c->ld_dw_gate_up, 2 * F) ||
        !stride_ok(c->stride_dw_down, c->experts, F, c->ld_dw_down, D))
      return bad("a gradient's row distance below its row or above 2^32, or a stride below its matrix or above 2^38");
    if (!aligned16(c->dx) || !aligned16(c->dw_gate_up) || !aligned16(c->dw_down)) return bad("matrices must be 16-byte aligned");
  }
  if (!backward && c->x8 != nullptr) return bad("the forward takes x in bf16");
  if (T == 0) return ok();
  if (c->index == nullptr || c->weight == nullptr) return bad("NULL index or weight");
  if (reinterpret_cast<uintptr_t>(c->index) % 4 != 0 || reinterpret_cast<uintptr_t>(c->weight) % 4 != 0)
    return bad("index and weight must be aligned to their elements");
  if ((c->x != nullptr) == (c->x8 != nullptr)) return bad("exactly one of x and x8 is wanted");
  if (c->x8 != nullptr) {
    const zopt_status st = act8::check(fn, *c->x8);
    if (st != ZOPT_OK) return st;
    if (c->x8->rows != T || c->x8->cols != D || c->x8->parts != 1) return bad("x8 must be tokens x dim in one part");
  } else if (!ld_ok(c->ld_x, D) || !aligned16(c->x)) {
    return bad("x: row distance or alignment");
  }
  if (backward) {
    if (c->kept == nullptr && c->kept8 == nullptr) return bad("the backward needs kept or kept8");
    if (c->dy == nullptr || !ld_ok(c->ld_dy, D) || !aligned16(c->dy)) return bad("dy: NULL, row distance or alignment");
    if (c->dx == nullptr || c->dweight == nullptr || reinterpret_cast<uintptr_t>(c->dweight) % 4 != 0)
      return bad("NULL dx or dweight, or dweight not aligned to its element");
  } else {
    if (c->y == nullptr || !ld_ok(c->ld_y, D) || !aligned16(c->y)) return bad("y: NULL, row distance or alignment");
  }
  if (d_ws == nullptr || !aligned16(d_ws)) return bad("the workspace must be 16-byte aligned");
  if (ws_bytes < layout(*c, backward).total) return bad("workspace too small");
  return ok();
}

#define TRY(expr)                   \
  do {                              \
    const zopt_status st_ = (expr); \
    if (st_ != ZOPT_OK) return st_; \
  } while (0)

// The experts' matrices as the TMA reads them: in place, or copied into the workspace.
struct Weights {
  const uint16_t *gate, *up, *down;
  long long pg, sg, pu, su, pd, sd;  // row distance and stride of each
};

struct Call {
  const char* fn;
  const zopt_experts_job& c;
  const Layout& p;
  uint8_t* ws;
  int* err;
  int sms;
  cudaStream_t s;

  template <typename T>
  T* at(size_t off) const {
    return reinterpret_cast<T*>(ws + off);
  }

  void copy(GatherArgs& a, size_t off, long long pitch, const uint16_t* src, long long ld, long long stride, long long rows,
            long long cols, const uint16_t** to, long long* pitch_to, long long* stride_to) const {
    uint16_t* d = at<uint16_t>(off);
    *to = d, *pitch_to = pitch, *stride_to = rows * pitch;
    const long long per_row = pitch / 8, chunk = std::max<long long>(1, std::min<long long>(1LL << 30, ((1LL << 31) - (1LL << 22)) / per_row));
    a.copy[a.copies++] = Copy{d, src, pitch, ld, stride, rows, cols, chunk, Divisor(static_cast<uint32_t>(per_row)), Divisor(static_cast<uint32_t>(rows))};
  }
  // The forward reads gate's and up's columns, the backward gate_up's rows whole.
  Weights weights(bool backward, GatherArgs& a) const {
    const long long D = c.dim, F = c.hidden;
    Weights w{c.w_gate_up, c.w_gate_up + F, c.w_down, c.ld_gate_up, c.stride_gate_up, c.ld_gate_up, c.stride_gate_up,
              c.ld_down, c.stride_down};
    if (p.stage_gate)
      copy(a, p.gate, p.gp, c.w_gate_up, c.ld_gate_up, c.stride_gate_up, D, backward ? 2 * F : F, &w.gate, &w.pg, &w.sg);
    if (p.stage_up && !backward) copy(a, p.up, p.fp, c.w_gate_up + F, c.ld_gate_up, c.stride_gate_up, D, F, &w.up, &w.pu, &w.su);
    if (p.stage_down) copy(a, p.down, p.dp, c.w_down, c.ld_down, c.stride_down, F, D, &w.down, &w.pd, &w.sd);
    return w;
  }
  zopt_status plan() const {
    const size_t smem = static_cast<size_t>(kPlanWarps + 1) * c.experts * 4;
    ZOPT_CUDA_TRY(once_per_device([] {
      return cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (kPlanWarps + 1) * kMaxExperts * 4);
    }));
    const PlanArgs a{c.index, c.weight, p.slots, c.experts, p.tile_rows, at<int>(p.head), at<int4>(p.tile), at<int2>(p.info), at<int>(p.used), at<int2>(p.row),
                     at<int>(p.row_of)};
    return launch_pdl(plan_kernel, dim3(kPlanCtas), dim3(32 * kPlanWarps), smem, s, a);
  }
  zopt_status gather(bool backward, GatherArgs& a) const {
    a.n = backward ? 2 : 1;
    a.from[0] = Source{c.x, c.ld_x, nullptr, nullptr, at<uint16_t>(p.xs)};
    if (c.x8 != nullptr) a.from[0] = Source{nullptr, 0, c.x8->q, c.x8->scale, at<uint16_t>(p.xs)};
    if (backward) a.from[1] = Source{c.dy, c.ld_dy, nullptr, nullptr, at<uint16_t>(p.dys)};
    a.tokens = c.tokens, a.cols = c.dim, a.pitch = p.dp;
    a.row_of = at<int>(p.row_of), a.info = at<int2>(p.info);
    a.head = at<int>(p.head), a.used = at<int>(p.used);
    a.top_k = c.top_k, a.experts = c.experts, a.fill = backward;
    long long threads = 32 * a.n * c.tokens * ((p.dp + 1023) / 1024);
    const long long used = std::min<long long>(c.experts, p.slots);
    for (int k = 0; k < a.copies; ++k) threads = std::max(threads, used * a.copy[k].rows * (a.copy[k].dst_cols / 8));
    if (a.kept.dst != nullptr) threads = std::max(threads, 32 * p.slots);
    if (backward) threads = std::max(threads, 32 * (kGroupRows - 1) * used);  // a warp a row to fill up
    return launch_pdl(gather_kernel, dim3(blocks_for(threads, sms)), dim3(256), 0, s, a);
  }
  zopt_status combine(bool backward) const {
    CombineArgs a{};
    a.parts = at<uint16_t>(p.parts), a.pitch = p.dp;
    a.scale = at<float>(p.scales), a.rows_ld = p.rows;
    a.row_of = at<int>(p.row_of);
    a.out = backward ? c.dx : c.y, a.ld = backward ? c.ld_dx : c.ld_y;
    a.tokens = c.tokens, a.cols = c.dim;
    a.top_k = c.top_k, a.chunks = static_cast<int>((c.dim + 255) / 256) + (backward ? 1 : 0);
    if (backward) a.dots = at<float>(p.dots), a.n_dots = p.dot_parts, a.dweight = c.dweight;
    return launch_pdl(combine_kernel, dim3(blocks_for(32 * a.tokens * a.chunks, sms)), dim3(256), 0, s, a);
  }
  void begin(Batch& b, int n) const {
    b.err = err;
    b.n = n;
    b.groups = Groups{at<int>(p.head), at<int4>(p.tile), at<int2>(p.info), at<int2>(p.row), c.experts, static_cast<int>(p.tiles)};
  }
  void parts(Job& j) const {
    j.out = at<uint16_t>(p.parts);
    j.ld_out = p.dp;
    j.part_scale = at<float>(p.scales);
    j.rows_ld = p.rows;
  }
  void glu(Job& j) const {
    j.act = c.act;
    j.hidden = static_cast<int>(c.hidden);
    j.kept_up = c.hidden;
    if (c.kept8 != nullptr) {
      j.kept_mode = kKeep8;
      j.kept = c.kept8->q;
      j.ld_kept = 2 * c.hidden;
      j.kept_scale = c.kept8->scale;
    } else if (c.kept != nullptr) {
      j.kept_mode = kKeepBf16;
      j.kept = c.kept;
      j.ld_kept = c.ld_kept;
    }
  }
  // The kept rows where the epilogue can read them.
  void stage_kept(Job& j, GatherArgs& a) const {
    const int size = c.kept8 != nullptr ? 1 : 2;
    a.kept = KeptCopy{at<uint8_t>(p.kept), j.kept, j.ld_kept, c.hidden, p.kept_row, size};
    j.kept = a.kept.dst;
    j.ld_kept = 2 * p.kept_row / size, j.kept_up = p.kept_row / size;
  }

  zopt_status forward() const {
    if (p.few) return few::experts_forward(c, at<float>(p.few_gate_up), at<float>(p.few_y), s);
    GatherArgs rows{};
    const Weights w = weights(false, rows);
    TRY(plan());
    TRY(gather(false, rows));
    const long long D = c.dim, F = c.hidden;
    {
      Batch b{};
      begin(b, 1);
      Job& j = b.job[0];
      group_job(j, kGluFwd, false, 0, F, D);
      j.b_mn = 1;
      glu(j);
      TRY(map_rows(fn, &j.P, at<uint16_t>(p.xs), p.rows, D, p.dp));
      TRY(map_weights(fn, &j.Q, w.gate, D, F, w.pg, c.experts, w.sg, 1, 0));
      TRY(map_weights(fn, &j.Up, w.up, D, F, w.pu, c.experts, w.su, 1, 0));
      j.out = at<uint16_t>(p.h);
      j.ld_out = p.fp;
      TRY(launch_grouped(fn, b, kGluFwd, p.tiles, s));
    }
    Batch b{};
    begin(b, 1);
    Job& j = b.job[0];
    group_job(j, kStore, false, 0, D, F);
    j.b_mn = 1;
    TRY(map_rows(fn, &j.P, at<uint16_t>(p.h), p.rows, F, p.fp));
    TRY(map_weights(fn, &j.Q, w.down, F, D, w.pd, c.experts, w.sd, 1, 0));
    parts(j);
    TRY(launch_grouped(fn, b, kStore, p.tiles, s));
    return combine(false);
  }

  zopt_status backward() const {
    GatherArgs rows{};
    const Weights w = weights(true, rows);
    TRY(plan());
    const long long D = c.dim, F = c.hidden;
    uint16_t *const xs = at<uint16_t>(p.xs), *const dys = at<uint16_t>(p.dys), *const h = at<uint16_t>(p.h),
             *const dgu = at<uint16_t>(p.dgu);
    {
      Batch b{};
      begin(b, 1);
      Job& j = b.job[0];
      group_job(j, kGluBwd, false, 0, F, D);
      glu(j);
      if (p.stage_kept) stage_kept(j, rows);
      TRY(gather(true, rows));
      TRY(map_rows(fn, &j.P, dys, p.rows, D, p.dp));
      TRY(map_weights(fn, &j.Q, w.down, F, D, w.pd, c.experts, w.sd, 0, j.tile_n / 2));
      j.out = dgu, j.ld_out = p.gp;
      j.out_h = h, j.ld_h = p.fp;
      j.dots = at<float>(p.dots), j.n_dots = p.dot_parts;
      TRY(map_results(fn, b, p.rows));
      TRY(launch_grouped(fn, b, kGluBwd, p.tiles, s));
    }
    Batch b{};
    begin(b, 3);
    {
      Job& j = b.job[0];  // dx's parts
      group_job(j, kStore, false, 0, D, 2 * F);
      TRY(map_rows(fn, &j.P, dgu, p.rows, 2 * F, p.gp));
      TRY(map_weights(fn, &j.Q, w.gate, D, 2 * F, w.pg, c.experts, w.sg, 0, j.tile_n / 2));
      parts(j);
    }
    {
      Job& j = b.job[1];  // dgate_up
      group_job(j, kStore, true, D, 2 * F, 0);
      j.a_mn = j.b_mn = 1;
      TRY(map_rows(fn, &j.P, xs, p.rows, D, p.dp));
      TRY(map_rows(fn, &j.Q, dgu, p.rows, 2 * F, p.gp));
      j.out = c.dw_gate_up, j.ld_out = c.ld_dw_gate_up, j.out_stride = c.stride_dw_gate_up;
    }
    {
      Job& j = b.job[2];  // ddown
      group_job(j, kStore, true, F, D, 0);
      j.a_mn = j.b_mn = 1;
      TRY(map_rows(fn, &j.P, h, p.rows, F, p.fp));
      TRY(map_rows(fn, &j.Q, dys, p.rows, D, p.dp));
      j.out = c.dw_down, j.ld_out = c.ld_dw_down, j.out_stride = c.stride_dw_down;
    }
    TRY(launch_grouped(fn, b, kStore, p.tiles, s));
    return combine(true);
  }

  zopt_status zero_gradients() const {
    const long long D = c.dim, F = c.hidden, E = c.experts;
    TRY(launch_pdl(zero_kernel, dim3(blocks_for(E * D * 2 * F, sms)), dim3(256), 0, s, c.dw_gate_up,
                   static_cast<long long>(c.ld_dw_gate_up), static_cast<long long>(c.stride_dw_gate_up), E, D, 2 * F));
    return launch_pdl(zero_kernel, dim3(blocks_for(E * F * D, sms)), dim3(256), 0, s, c.dw_down,
                      static_cast<long long>(c.ld_dw_down), static_cast<long long>(c.stride_dw_down), E, F, D);
  }
};

zopt_status run(const char* fn, const zopt_experts_job* cp, bool backward, void* d_ws, size_t ws_bytes, cudaStream_t s) {
  TRY(check(fn, cp, backward, d_ws, ws_bytes));
  const zopt_experts_job& c = *cp;
  if (c.tokens == 0 && !backward) return ok();
  const int sms = sm_count();
  if (sms < 1) return fail(ZOPT_ECUDA, std::string(fn) + ": no CUDA device");
  const Layout p = layout(c, backward);
  Call call{fn, c, p, static_cast<uint8_t*>(d_ws), nullptr, sms, s};
  if (c.tokens == 0) return call.zero_gradients();
  TRY(ns::take_error_word(fn, &call.err));
  return backward ? call.backward() : call.forward();
}

}  // namespace
}  // namespace lm
}  // namespace zopt

extern "C" size_t zopt_experts_workspace(const zopt_experts_job* job, int32_t backward) {
  using namespace zopt::lm;
  if (job == nullptr || !sizes_ok(*job) || !weights_ok(*job)) return 0;
  const size_t n = layout(*job, backward != 0).total;
  return n < 16 ? 16 : n;
}

extern "C" zopt_status zopt_experts_forward(const zopt_experts_job* job, void* d_ws, size_t ws_bytes, zopt_stream stream) {
  return zopt::guarded([&] { return zopt::lm::run("zopt_experts_forward", job, false, d_ws, ws_bytes, stream); });
}

extern "C" zopt_status zopt_experts_backward(const zopt_experts_job* job, void* d_ws, size_t ws_bytes, zopt_stream stream) {
  return zopt::guarded([&] { return zopt::lm::run("zopt_experts_backward", job, true, d_ws, ws_bytes, stream); });
}
