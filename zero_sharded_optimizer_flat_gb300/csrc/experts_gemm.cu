// The batches of products over experts' rows: the kernel of lm_kernel.cuh built for them, and its host
// launcher.
//
// A unit is a tile of at most 256 rows of one expert, or a tile of one expert's weight gradient with
// the expert's rows as its inner length. How many rows an expert has is known on the device alone:
// units are found through the row tiles' table that the plan leaves (experts.cu), so nothing waits
// for the host and a captured call follows whatever the tokens choose.
//
// An expert's last tile is full by half on average. With tiles of 256 rows alone the experts of 8192 x 6 slots
// (768 rows each) multiply 16 % of rows that nobody has; tiles of at most 128 rows on the M = 128 MMA, in half
// the time, leave 8 % (forward 758 us for 740; 4096 x 2 slots of 2048 x 5632 in eight experts 431 for 411).
#include <algorithm>
#include <cudaTypedefs.h>

#include <string>

#include "experts_gemm.h"
#include "lm_kernel.cuh"

namespace zopt {
namespace ns {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();
}
namespace lm {
namespace {

zopt_status make_map3(const char* fn, CUtensorMap* m, const void* base, long long inner, long long outer, long long depth,
                      long long pitch, long long stride, int box_outer) {
  auto enc = ns::encode_fn();
  if (enc == nullptr) return fail(ZOPT_ECUDA, std::string(fn) + ": cuTensorMapEncodeTiled is unavailable");
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer), static_cast<cuuint64_t>(depth)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch) * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_outer), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(ZOPT_ECUDA, std::string(fn) + ": cuTensorMapEncodeTiled failed (" + std::to_string(r) + ")");
  return ok();
}

}  // namespace

zopt_status map_rows(const char* fn, CUtensorMap* m, const void* base, long long rows, long long cols, long long pitch) {
  return make_map3(fn, m, base, cols, rows, 1, pitch, pitch, 64);
}
zopt_status map_weights(const char* fn, CUtensorMap* m, const void* base, long long rows, long long cols,
                        long long pitch, long long experts, long long stride, int mn, int box) {
  return make_map3(fn, m, base, cols, rows, experts, pitch, experts > 1 ? stride : pitch, mn ? 64 : box);
}

void set_group_tiles(Job& j) {
  auto columns = [&](int tile_n) {
    const int width = j.kind == kGluFwd ? tile_n / 2 : tile_n;
    return (j.N + width - 1) / width;
  };
  j.tile_n = kTileN;
  j.tiles_n = columns(j.tile_n);
  j.a_rows = 128;
  j.tx = 256 * kTileK * 2 + j.tile_n * kTileK * 2;
  j.splits = 1;
  if (j.by_inner) {
    j.tiles_m = (j.M + kTileM - 1) / kTileM;
    j.tiles = j.tiles_m * j.tiles_n;
    j.rows_fast = j.N >= j.M ? 1 : 0;
    j.per_split = Divisor(static_cast<uint32_t>(j.tiles));
    j.per_line = Divisor(static_cast<uint32_t>(j.rows_fast ? j.tiles_m : j.tiles_n));
  } else {
    j.nk = (j.K + kTileK - 1) / kTileK;
    j.per_line = Divisor(static_cast<uint32_t>(j.tiles_n));
  }
}

zopt_status launch_grouped(const char* fn, Batch& b, int kinds, long long most_tiles, cudaStream_t s) {
  long long total = 0;
  for (int i = 0; i < b.n; ++i) {
    const Job& j = b.job[i];
    total += j.by_inner ? static_cast<long long>(j.tiles_m) * j.tiles_n * b.groups.experts : most_tiles * j.tiles_n;
  }
  if (total > 0x7FFFFFFFLL) return fail(ZOPT_EINVAL, std::string(fn) + ": too many tiles");
  const int sms = sm_count();
  if (sms < 2) return fail(ZOPT_ECUDA, std::string(fn) + ": no CUDA device");
  b.listed = 0;
  const dim3 grid(static_cast<unsigned>(2 * std::min<long long>(total, std::min(sms / 2, kPairs))));
  if (kinds == kStore) return launch_kinds<true, kStore>(b, grid, s);
  return b.job[0].act == ZOPT_ACT_GELU ? launch_glu<true, ZOPT_ACT_GELU>(b, grid, s) : launch_glu<true, ZOPT_ACT_SILU>(b, grid, s);
}

}  // namespace lm
}  // namespace zopt
