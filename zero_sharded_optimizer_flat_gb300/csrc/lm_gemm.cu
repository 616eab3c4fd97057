// The batches of products over whole matrices: the kernel of lm_kernel.cuh built for them, its host
// launcher, the sum of split products and the copy that stages operands.
#include <algorithm>
#include <cmath>
#include <cudaTypedefs.h>

#include <string>

#include "launch.cuh"
#include "lm_gemm.cuh"
#include "lm_kernel.cuh"
#include "ns_internal.h"
#include "tc.cuh"

namespace zopt {
namespace ns {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();
}
namespace lm {
namespace {

// Partial sums added in split order, so a call's result does not depend on which pair ran when. Bound
// by its launch and L2: 3.5 us for 3 MB of parts, 6.5 us for 18 MB.
__global__ void __launch_bounds__(256) sum_kernel(const __grid_constant__ SumBatch B) {
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long g = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; g < B.start[B.n]; g += stride) {
    int ji = 0;
    while (ji + 1 < B.n && g >= B.start[ji + 1]) ++ji;
    const SumJob& j = B.job[ji];
    const long long per_row = j.pitch / 4, l = g - B.start[ji];
    const long long row = l / per_row, col = (l - row * per_row) * 4;
    const float* p = j.part + row * j.pitch + col;
    float4 a = *reinterpret_cast<const float4*>(p);
    for (int s = 1; s < j.splits; ++s) {
      const float4 v = *reinterpret_cast<const float4*>(p + s * j.split_stride);
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    }
    const float alpha = j.alpha != nullptr ? __ldcg(j.alpha) : 1.0f;
    a.x *= alpha, a.y *= alpha, a.z *= alpha, a.w *= alpha;
    uint16_t* o = j.out + row * j.ld_out + col;
    if (col + 4 <= j.N && (reinterpret_cast<uintptr_t>(o) & 7u) == 0) {
      *reinterpret_cast<uint2*>(o) = make_uint2(pack2(a.x, a.y), pack2(a.z, a.w));
    } else {
      const float v[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (col + k < j.N) o[k] = __bfloat16_as_ushort(__float2bfloat16_rn(v[k]));
    }
  }
}

// One pass over an operand: 4 bytes an entry, 5 us for 1000 x 2732 (most of it the launch).
__global__ void __launch_bounds__(256) stage_kernel(uint16_t* dst, long long dst_pitch, long long dst_cols,
                                                    const uint16_t* src, long long src_pitch, long long rows,
                                                    long long cols) {
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const long long per_row = dst_cols / 8, n = rows * per_row;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long g = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; g < n; g += stride) {
    const long long row = g / per_row, col = (g - row * per_row) * 8;
    *reinterpret_cast<uint4*>(dst + row * dst_pitch + col) = row_piece8(src + row * src_pitch + col, cols - col);
  }
}

}  // namespace

unsigned blocks_for(long long items, int sms) {
  const long long want = (items + 255) / 256, most = 8LL * sms;
  return static_cast<unsigned>(want < 1 ? 1 : (want < most ? want : most));
}

// ---------------------------------------------------------------------- host side

namespace {
// A bf16 row-major matrix [outer][inner] with `pitch` elements between rows, boxes of 64 x box_outer.
zopt_status make_map(const char* fn, CUtensorMap* m, const void* base, long long inner, long long outer,
                     long long pitch, int box_outer) {
  auto enc = ns::encode_fn();
  if (enc == nullptr) return fail(ZOPT_ECUDA, std::string(fn) + ": cuTensorMapEncodeTiled is unavailable");
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch) * 2};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_outer)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(ZOPT_ECUDA, std::string(fn) + ": cuTensorMapEncodeTiled failed (" + std::to_string(r) + ")");
  return ok();
}
}  // namespace

zopt_status map_p(const char* fn, Job& j, const void* base, long long pitch) {
  return j.a_mn ? make_map(fn, &j.P, base, j.M, j.K, pitch, 64) : make_map(fn, &j.P, base, j.K, j.M, pitch, j.a_rows);
}
zopt_status map_q(const char* fn, Job& j, const void* base, long long columns, long long pitch) {
  return j.b_mn ? make_map(fn, &j.Q, base, columns, j.K, pitch, 64)
                : make_map(fn, &j.Q, base, j.K, columns, pitch, j.tile_n / 2);
}

zopt_status map_up(const char* fn, Job& j, const void* base, long long columns, long long pitch) {
  return make_map(fn, &j.Up, base, columns, j.K, pitch, 64);
}

zopt_status map_results(const char* fn, Batch& b, long long rows) {
  Job& j = b.job[0];
  j.bulk = j.N % 8 == 0 && j.ld_out % 8 == 0 && j.ld_h % 8 == 0 && aligned16(j.out) && aligned16(j.out_h);
  if (!j.bulk) return ok();
  auto enc = ns::encode_fn();
  if (enc == nullptr) return fail(ZOPT_ECUDA, std::string(fn) + ": cuTensorMapEncodeTiled is unavailable");
  void* const base[3] = {j.out, static_cast<uint16_t*>(j.out) + j.N, j.out_h};
  for (int k = 0; k < 3; ++k) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(j.N), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(k == 2 ? j.ld_h : j.ld_out) * 2};
    const cuuint32_t box[2] = {32, 32}, estr[2] = {1, 1};
    const CUresult r = enc(&b.outs[k], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base[k], dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(ZOPT_ECUDA, std::string(fn) + ": cuTensorMapEncodeTiled failed (" + std::to_string(r) + ")");
  }
  return ok();
}

void set_tiles(Job& j) {
  j.tiles_m = (j.M + kTileM - 1) / kTileM;
  j.nk = (j.K + kTileK - 1) / kTileK;
  j.kb_per_split = j.nk;
  j.splits = 1;
  auto columns = [&](int tile_n) {
    const int width = j.kind == kGluFwd ? tile_n / 2 : tile_n;
    return (j.N + width - 1) / width;
  };
  // Tiles half as wide cost more than half as much (P is read again for each: 0.7 of a k-block's
  // time, and half of an epilogue's, which counts as 16 k-blocks), but where there are few of the
  // wide ones they keep twice as many pairs busy. kStore cuts its inner length instead (with narrow
  // tiles cross entropy backward, 512 x 256 x 4096, took 32 us for 23), and a tile that makes 8-bit
  // blocks has to be one block wide.
  j.tile_n = kTileN;
  if (j.kind != kStore && !(j.kind == kGluFwd && j.kept_mode == kKeep8)) {
    auto waves = [&](int tile_n) { return (static_cast<long long>(j.tiles_m) * columns(tile_n) + kPairs - 1) / kPairs; };
    if (waves(128) * (0.7 * j.nk + 8) < waves(256) * (1.0 * j.nk + 16)) j.tile_n = 128;
  }
  j.tiles_n = columns(j.tile_n);
  // P's rows beyond M are not loaded where a single box holds them all: loads of rows that are not
  // there take the TMA longer than loads of rows that are.
  j.a_rows = !j.a_mn && j.M <= 128 ? (j.M + 7) / 8 * 8 : 128;
  j.tx = (j.a_rows < 128 ? j.a_rows : 256) * kTileK * 2 + j.tile_n * kTileK * 2;
  // The larger operand is streamed once: tiles that run together share its rows (or columns) and
  // walk the smaller one, which stays in L2.
  j.rows_fast = j.N >= j.M ? 1 : 0;
}

void plan_splits(Job* jobs, int n) {
  // In k-blocks' time (0.27 us): an epilogue takes about 12; adding up partial sums a launch, about
  // eight (with four, y of 1023 x 256 x 768 is cut in three: 15.8 us a forward for 13.8; with twelve,
  // cross entropy backward of 2000 x 2048 x 5000 is not cut: 90 us for 85), and their bytes, one for
  // every 4 MiB. A run is at least four k-blocks.
  constexpr long long kLeast = 4, kEpilogue = 12, kSum = 8;
  long long longest = 0;
  for (int i = 0; i < n; ++i)
    if (!jobs[i].whole) longest = std::max<long long>(longest, jobs[i].nk);
  // what a launch with runs of at most `run` takes: a single job's in turn, several jobs' dealt out
  auto cost = [&](long long run) {
    long long all = 0, count = 0, most = 0, bytes = 0;
    for (int i = 0; i < n; ++i) {
      const Job& j = jobs[i];
      const long long s = j.kind == kStore && !j.whole ? std::max<long long>(1, (j.nk + run - 1) / run) : 1, kb = (j.nk + s - 1) / s;
      const long long tiles = static_cast<long long>(j.tiles_m) * j.tiles_n;
      all += tiles * s * (kb + kEpilogue), count += tiles * s, most = std::max(most, kb + kEpilogue);
      if (s > 1) bytes += s * j.M * split_pitch(j.N) * 4;
    }
    const long long waves = (count + kPairs - 1) / kPairs;
    return (n == 1 ? waves * most : std::max(most, all / kPairs + most / 2)) + (bytes > 0 ? kSum + (bytes >> 22) : 0);
  };
  long long best = longest, least = cost(std::max(longest, kLeast));
  for (int s = 2; s <= 64 && longest > kLeast; ++s) {
    const long long run = std::max(kLeast, (longest + s - 1) / s), c = cost(run);
    if (c < least) least = c, best = run;
    if (run == kLeast) break;
  }
  for (int i = 0; i < n; ++i) {
    Job& j = jobs[i];
    if (j.kind != kStore || j.whole || j.nk <= best) continue;
    j.splits = static_cast<int>((j.nk + best - 1) / best);
    j.kb_per_split = (j.nk + j.splits - 1) / j.splits;
    j.splits = (j.nk + j.kb_per_split - 1) / j.kb_per_split;
  }
}

namespace {
// Gives each unit, the longest first, to the pair with the least to do so far (a unit's k-blocks, and
// 12 for its epilogue).
void list_units(Batch& b, int total, int pairs) {
  struct Entry {
    int cost;
    uint16_t unit;
  };
  Entry e[kMaxListed];
  for (int i = 0, u = 0; i < b.n; ++i) {
    const Job& j = b.job[i];
    for (; u < b.start[i + 1]; ++u) {
      const int split = (u - b.start[i]) / j.tiles, kb0 = split * j.kb_per_split;
      e[u] = Entry{std::min(j.kb_per_split, j.nk - kb0) + 12, static_cast<uint16_t>(u)};
    }
  }
  std::stable_sort(e, e + total, [](const Entry& x, const Entry& y) { return x.cost > y.cost; });
  int load[kPairs] = {}, count[kPairs] = {};
  uint8_t owner[kMaxListed];
  for (int u = 0; u < total; ++u) {
    const int p = static_cast<int>(std::min_element(load, load + pairs) - load);
    load[p] += e[u].cost;
    ++count[p];
    owner[u] = static_cast<uint8_t>(p);
  }
  int at[kPairs];
  b.first[0] = 0;
  for (int p = 0; p < kPairs; ++p) b.first[p + 1] = static_cast<uint16_t>(b.first[p] + (p < pairs ? count[p] : 0));
  for (int p = 0; p < pairs; ++p) at[p] = b.first[p];
  for (int u = 0; u < total; ++u) b.order[at[owner[u]]++] = e[u].unit;
}
}  // namespace

zopt_status launch(const char* fn, Batch& b, int kinds, cudaStream_t s) {
  long long total = 0;
  for (int i = 0; i < b.n; ++i) {
    Job& j = b.job[i];
    const long long tiles = static_cast<long long>(j.tiles_m) * j.tiles_n;
    const long long units = tiles * j.splits;
    if (tiles < 1 || total + units > 0x7FFFFFFFLL) return fail(ZOPT_EINVAL, std::string(fn) + ": too many tiles");
    j.tiles = static_cast<int>(tiles);
    j.per_split = Divisor(static_cast<uint32_t>(tiles));
    j.per_line = Divisor(static_cast<uint32_t>(j.rows_fast ? j.tiles_m : j.tiles_n));
    b.start[i] = static_cast<int>(total);
    total += units;
  }
  b.start[b.n] = static_cast<int>(total);
  const int sms = sm_count();
  if (sms < 2) return fail(ZOPT_ECUDA, std::string(fn) + ": no CUDA device");
  const long long pairs = std::min<long long>(total, std::min(sms / 2, kPairs));
  // In turn, unequal units would leave pairs idle: 1537 tokens of a 1000 x 2732 block, 188 units of 43
  // and 25 k-blocks, 125 for the last pair where 86 do.
  b.listed = b.n > 1 && total > pairs && total <= kMaxListed;
  if (b.listed) list_units(b, static_cast<int>(total), static_cast<int>(pairs));
  const dim3 grid(static_cast<unsigned>(2 * pairs));
  switch (kinds) {
    case kStore: return launch_kinds<false, kStore>(b, grid, s);
    case kCeFwd: return launch_kinds<false, kCeFwd>(b, grid, s);
    case kStore | kCeBwd: return launch_kinds<false, kStore | kCeBwd>(b, grid, s);
    case kGluFwd:
    case kGluBwd:
      return b.job[0].act == ZOPT_ACT_GELU ? launch_glu<false, ZOPT_ACT_GELU>(b, grid, s) : launch_glu<false, ZOPT_ACT_SILU>(b, grid, s);
  }
  return fail(ZOPT_EINVAL, std::string(fn) + ": internal: no kernel for these epilogues");
}

zopt_status launch_sums(const char* fn, const SumBatch& b, cudaStream_t s) {
  const int sms = sm_count();
  if (sms < 1) return fail(ZOPT_ECUDA, std::string(fn) + ": no CUDA device");
  return launch_pdl(sum_kernel, dim3(blocks_for(b.start[b.n], sms)), dim3(256), 0, s, b);
}

zopt_status launch_stage(const char* fn, uint16_t* dst, long long dst_pitch, long long dst_cols, const uint16_t* src,
                         long long src_pitch, long long rows, long long cols, cudaStream_t s) {
  const int sms = sm_count();
  if (sms < 1) return fail(ZOPT_ECUDA, std::string(fn) + ": no CUDA device");
  return launch_pdl(stage_kernel, dim3(blocks_for(rows * (dst_cols / 8), sms)), dim3(256), 0, s, dst, dst_pitch,
                    dst_cols, src, src_pitch, rows, cols);
}

}  // namespace lm
}  // namespace zopt
