// The products of the training operators on tcgen05 tensor cores: one persistent CTA-pair kernel
// over a batch of jobs (lm_gemm.cuh), as lm_gemm.cu and experts_gemm.cu build it.
//
// A cluster of two CTAs computes a 256 x 256 tile with tcgen05.mma.cta_group::2: each CTA holds its
// 128 rows of P and its 128 columns of Q, so a 64-deep k-block brings 32 KiB per SM and the ring
// holds six stages (with five, units of eight k-blocks take 8 % longer, with four 25 %), the gated block's backward
// five, whose epilogue needs the room more than its loads do. A thread of
// each CTA for each operand streams it by TMA (all complete on the leader's stage barrier), one
// thread of the leader issues the M=256, N=256, K=16 MMAs into one of two TMEM accumulators, and
// eight epilogue warps (two per quarter of the TMEM lanes, each 128 of the 256 columns) turn the
// other accumulator into the operator's outputs meanwhile. A lane holds whole row pieces, so softmax
// statistics and the 8-bit blocks need no exchange between lanes.
//
// A grouped batch (kGrouped) has the rows of many experts one after another: its units are found through
// tables in device memory (Groups in lm_gemm.cuh), weights come through maps with the expert as a third
// coordinate, and a tile of at most 128 rows takes the pair's M = 128 MMA.
//
// Bound by the tensor cores where the inner length is long enough to hide a tile's epilogue (12 to 30
// k-blocks' time): 521 cycles a k-block of 512, tensor pipe 92 % of elapsed in the cross entropy's
// forward (4096 x 768 x 50304), 89 % in the block's first product and 90 % in its backward's second
// launch (8192 x 2048 x 5632), all three at the clock that the power cap leaves; 61 % (137 us) in the
// backward's first launch, whose epilogue (three results and two kept inputs an entry) outlasts its
// 32 k-blocks; 76 % in y, 256 tiles over 76 pairs.
#pragma once

#include <cuda_fp16.h>

#include "act8.cuh"
#include "f2.cuh"
#include "launch.cuh"
#include "lm_gemm.cuh"
#include "per_device.h"
#include "row_bytes.h"
#include "tc.cuh"

namespace zopt {
namespace lm {
namespace {

// ---------------------------------------------------------------------- device helpers

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(F2 a) {
  const float2 x = f2(a);
  return pack2(x.x, x.y);
}

// True in one lane of a converged warp. The copies and MMAs take their operands from uniform
// registers: behind this predicate the compiler knows that one thread issues them, behind a
// comparison of lanes it has to issue them lane by lane (680 against 521 cycles a k-block of 8192^3,
// whose MMAs take 512).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// ---------------------------------------------------------------------- results to memory
//
// A warp's results are 32 rows, one lane each; memory wants consecutive lanes along a row. So a lane
// writes its row (128 bytes) into the warp's 4 KiB box and the warp stores the box row by row. The
// box's 16-byte piece q of row r lies at piece q ^ r', r' the low three bits of r in reverse: eight
// lanes at a time meet every bank once, whether they are eight rows' one piece, one row's eight, two
// rows' four or four rows' two. (Through 2 KiB boxes handed to the TMA a tile of bf16 results took its
// warps 6000 cycles, this way 3700.)
// Boxes of 64-byte rows (kRow), which the TMA takes to memory, hold piece q at q ^ r', r' the row's bits 1 and 2: its
// 64-byte swizzle. Eight lanes meet every bank once where they are eight rows' one piece.
template <int kRow = 128>
__device__ __forceinline__ uint32_t box_piece(uint32_t box, int row, int q) {
  if constexpr (kRow == 64) return box + static_cast<uint32_t>(row * 64) + ((static_cast<uint32_t>(q) ^ (static_cast<uint32_t>(row >> 1) & 3u)) << 4);
  return box + static_cast<uint32_t>(row * 128) + ((static_cast<uint32_t>(q) ^ (__brev(static_cast<uint32_t>(row & 7)) >> 29)) << 4);
}
// Pieces q0 .. of the lane's row. (box is a multiple of 128.)
template <int kWords>
__device__ __forceinline__ void box_put(uint32_t box, int lane, int q0, const uint32_t (&o)[kWords]) {
  const uint32_t at = box_piece(box, lane, 0);
#pragma unroll
  for (int q = 0; q < kWords / 4; ++q)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at ^ static_cast<uint32_t>((q0 + q) << 4)), "r"(o[4 * q]),
                 "r"(o[4 * q + 1]), "r"(o[4 * q + 2]), "r"(o[4 * q + 3])
                 : "memory");
}

template <int kRow = 128>
__device__ __forceinline__ void box_put4(uint32_t box, int lane, int q, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box_piece<kRow>(box, lane, 0) ^ static_cast<uint32_t>(q << 4)), "r"(a),
               "r"(b), "r"(c), "r"(d)
               : "memory");
}

// Pieces of kPiece bytes, for rows whose start or length is not a multiple of 16 bytes.
template <typename Piece, int kBytes>
__device__ __noinline__ void rows_out_odd(uint32_t box, uint8_t* base, long long pitch, int bytes, int rows, int skip, int lane) {
  constexpr int kPiece = sizeof(Piece), kAll = kBytes / kPiece, kPerRow = kAll < 32 ? kAll : 32, kAtOnce = 32 / kPerRow;
#pragma unroll
  for (int o = 0; o < kAll / kPerRow; ++o) {
    const int off = (lane % kPerRow + o * kPerRow) * kPiece, in = off + skip;
    uint8_t* p = base + lane / kPerRow * pitch + off;
#pragma unroll 8
    for (int row = lane / kPerRow; row < 32; row += kAtOnce) {
      const Piece v = *reinterpret_cast<const Piece*>(__cvta_shared_to_generic(box_piece(box, row, in >> 4) + (in & 15)));
      if (row < rows && off + kPiece <= bytes) *reinterpret_cast<Piece*>(p) = v;
      p += kAtOnce * pitch;
    }
  }
}
template <int kBytes>
__device__ __noinline__ void rows_out_any(uint32_t box, uint8_t* base, long long pitch, int bytes, int rows, int skip, int lane) {
  const unsigned mis = static_cast<unsigned>(reinterpret_cast<uintptr_t>(base)) | static_cast<unsigned>(pitch) |
                       static_cast<unsigned>(bytes);
  if ((mis & 15u) == 0) {
    rows_out_odd<uint4, kBytes>(box, base, pitch, bytes, rows, skip, lane);
  } else if ((mis & 7u) == 0) {
    rows_out_odd<uint2, kBytes>(box, base, pitch, bytes, rows, skip, lane);
  } else if ((mis & 3u) == 0) {
    rows_out_odd<uint32_t, kBytes>(box, base, pitch, bytes, rows, skip, lane);
  } else if ((mis & 1u) == 0) {
    rows_out_odd<uint16_t, kBytes>(box, base, pitch, bytes, rows, skip, lane);
  } else {
    rows_out_odd<uint8_t, kBytes>(box, base, pitch, bytes, rows, skip, lane);
  }
}

// Row by row, a byte (or two) a lane: rows that lie anywhere and start anywhere, or end within the part.
template <int kBytes>
__device__ __noinline__ void scatter_any(uint32_t box, uint8_t* base, long long pitch, int bytes, int slot, int skip, int lane) {
  const unsigned mis = static_cast<unsigned>(reinterpret_cast<uintptr_t>(base)) | static_cast<unsigned>(pitch) | static_cast<unsigned>(bytes);
#pragma unroll 1
  for (int row = 0; row < 32; ++row) {
    const int to = __shfl_sync(0xFFFFFFFFu, slot, row);
    if (to < 0) continue;
    uint8_t* p = base + to * pitch;
    if ((mis & 1u) == 0) {
      const int off = 2 * lane, in = off + skip;
      if (off + 2 <= bytes)
        *reinterpret_cast<uint16_t*>(p + off) =
            *reinterpret_cast<const uint16_t*>(__cvta_shared_to_generic(box_piece(box, row, in >> 4) + (in & 15)));
    } else {
      for (int off = lane; off < bytes; off += 32) {
        const int in = off + skip;
        p[off] = *reinterpret_cast<const uint8_t*>(__cvta_shared_to_generic(box_piece(box, row, in >> 4) + (in & 15)));
      }
    }
  }
}

// Where a warp's part of a result goes: its 32 rows from a first column on, kBytes of each row at a
// time. What does not change within a tile is worked out once (the addresses of a lane's pieces; that
// every row is there and every piece whole), since a store costs little more than its instructions.
template <int kBytes>
struct Out {
  static constexpr int kPerRow = kBytes / 16, kAtOnce = 32 / kPerRow;
  uint8_t* base;
  uint8_t* mine;    // the lane's first piece
  long long pitch;  // bytes
  int bytes, rows;  // from base to the row's end (or the warp's part's), and rows there are
  bool whole;
  // columns col .. of rows row0 .. of M rows and n columns of `size` bytes
  __device__ __forceinline__ Out(void* matrix, long long ld, int size, int row0, int M, int col, int n, int lane) {
    pitch = ld * size;
    base = static_cast<uint8_t*>(matrix) + row0 * pitch + static_cast<long long>(col) * size;
    bytes = row_bytes(n, col, size);
    rows = min(32, M - row0);
    mine = base + lane / kPerRow * pitch + 16 * (lane % kPerRow);
    whole = rows == 32 && ((static_cast<unsigned>(reinterpret_cast<uintptr_t>(base)) | static_cast<unsigned>(pitch)) & 15u) == 0;
  }
  // kBytes of each of the box's rows, from byte kSkip on, to byte `at` of the result's rows
  template <int kSkip>
  __device__ __forceinline__ void put(uint32_t box, int lane, int at) const {
    if (whole && at + kBytes <= bytes) {
      const int q = lane % kPerRow, r0 = lane / kPerRow;
      uint8_t* p = mine + at;
      uint4 v[kPerRow];
#pragma unroll
      for (int i = 0; i < kPerRow; ++i)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[i].x), "=r"(v[i].y), "=r"(v[i].z), "=r"(v[i].w)
                     : "r"(box_piece(box, r0 + i * kAtOnce, kSkip / 16 + q)));
#pragma unroll
      for (int i = 0; i < kPerRow; ++i) {
        *reinterpret_cast<uint4*>(p) = v[i];
        p += kAtOnce * pitch;
      }
    } else if (at < bytes) {
      rows_out_any<kBytes>(box, base + at, pitch, min(kBytes, bytes - at), rows, kSkip, lane);
    }
  }
};

// The same for rows that lie anywhere: the lane's row is row `slot` of the matrix, -1: it goes nowhere.
template <int kBytes>
struct Scatter {
  static constexpr int kPerRow = kBytes / 16, kAtOnce = 32 / kPerRow;
  uint8_t* base;  // row 0's first byte of the warp's part
  long long pitch;
  int bytes, slot;
  bool aligned;
  __device__ __forceinline__ Scatter(void* matrix, long long ld, int size, int slot_, int col, int n) {
    pitch = ld * size;
    base = static_cast<uint8_t*>(matrix) + static_cast<long long>(col) * size;
    bytes = row_bytes(n, col, size);
    slot = slot_;
    aligned = ((static_cast<unsigned>(reinterpret_cast<uintptr_t>(base)) | static_cast<unsigned>(pitch)) & 15u) == 0;
  }
  template <int kSkip>
  __device__ __forceinline__ void put(uint32_t box, int lane, int at) const {
    if (at >= bytes) return;
    if (aligned && at + kBytes <= bytes) {
      const int q = lane % kPerRow, r0 = lane / kPerRow;
      uint8_t* p = base + at + 16 * q;
#pragma unroll
      for (int i = 0; i < kPerRow; ++i) {
        const int to = __shfl_sync(0xFFFFFFFFu, slot, r0 + i * kAtOnce);
        uint4 v;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "r"(box_piece(box, r0 + i * kAtOnce, kSkip / 16 + q)));
        if (to >= 0) *reinterpret_cast<uint4*>(p + to * pitch) = v;
      }
    } else {
      scatter_any<kBytes>(box, base + at, pitch, min(kBytes, bytes - at), slot, kSkip, lane);
    }
  }
};
// A warp's part of a result, in rows that follow one another or anywhere.
template <int kBytes, bool kAnywhere>
__device__ __forceinline__ auto part_of(void* matrix, long long ld, int size, int row0, int M, int slot, int col, int n, int lane) {
  if constexpr (kAnywhere) {
    return Scatter<kBytes>(matrix, ld, size, slot, col, n);
  } else {
    return Out<kBytes>(matrix, ld, size, row0, M, col, n, lane);
  }
}

// A unit of work: one tile of one job over one run of k-blocks.
struct Unit {
  int tj, split, kb0, kb1;
  int row0, rows;    // the tile's first row, and where the rows of D end
  int expert, krow;  // grouped: whose matrices; by_inner: the row of both operands that k = 0 is
  bool half;         // grouped: a tile of at most 128 rows
};
// A warp's part of a tile: its first row, and its columns (kGluFwd: hidden ones) in the accumulator and in D.
//
// A tile of 256 rows gives each CTA 128, a TMEM lane each, and all columns (the pair's MMA with M = 256); one
// of 128 rows gives each CTA 64, whose first half of the columns lies in lanes 0 .. 63 and whose second in
// lanes 64 .. 127 (M = 128), in half the accumulator's columns and half the time.
struct Part {
  int row0, tcol, col, width;
};
template <bool kGrouped>
__device__ __forceinline__ Part part_of_tile(const Unit& w, int width, uint32_t rank, int quad, int h) {
  if (kGrouped && w.half)
    return Part{w.row0 + static_cast<int>(rank) * 64 + 32 * (quad & 1), (width >> 2) * h,
                w.tj * width + (width >> 1) * (quad >> 1) + (width >> 2) * h, width >> 2};
  return Part{w.row0 + static_cast<int>(rank) * 128 + 32 * quad, (width >> 1) * h, w.tj * width + (width >> 1) * h, width >> 1};
}
// (tile: grouped, by rows: the unit's row tile, where it has been read already)
template <bool kGrouped>
__device__ __forceinline__ Unit unit_of(const Batch& B, const Job& j, int u, const int4* tile = nullptr) {
  Unit w;
  if (kGrouped && !j.by_inner) {  // columns of a row tile one after another
    const int line = static_cast<int>(j.per_line(static_cast<uint32_t>(u)));
    const int4 t = tile != nullptr ? *tile : __ldcg(B.groups.tiles + line);
    w.tj = u - line * j.tiles_n;
    w.split = 0, w.kb0 = 0, w.kb1 = j.nk;
    w.expert = t.x, w.row0 = t.y, w.rows = t.z, w.krow = 0;
    w.half = t.w != 0;
    return w;
  }
  w.split = static_cast<int>(j.per_split(static_cast<uint32_t>(u)));
  u -= w.split * j.tiles;
  const int line = static_cast<int>(j.per_line(static_cast<uint32_t>(u))), at = u - line * static_cast<int>(j.per_line.d);
  const int ti = j.rows_fast ? at : line;
  w.tj = j.rows_fast ? line : at;
  w.row0 = ti * kTileM, w.rows = j.M;
  w.expert = 0, w.krow = 0;
  w.half = false;
  if (kGrouped) {
    const int2 e = __ldcg(B.groups.info + w.split);
    w.expert = w.split, w.split = 0;
    w.krow = e.x;
    w.kb0 = 0, w.kb1 = (e.y + kTileK - 1) / kTileK;
  } else {
    w.kb0 = w.split * j.kb_per_split;
    w.kb1 = min(w.kb0 + j.kb_per_split, j.nk);
  }
  return w;
}
// Pair p's i-th unit, or a number beyond the last.
// (Grouped: units are the longer the earlier they come, and those that begin every other round go to the
// pairs whose last ones were the shortest.)
template <bool kGrouped>
__device__ __forceinline__ int unit_at(const Batch& b, int pair, int npairs, int i) {
  if constexpr (kGrouped) return i * npairs + ((i & 1) != 0 ? npairs - 1 - pair : pair);
  if (!b.listed) return pair + i * npairs;
  const int at = b.first[pair] + i;
  return at < b.first[pair + 1] ? b.order[at] : 0x7FFFFFFF;
}
// Where each job's units begin, and where the last one's end.
template <bool kGrouped>
struct Starts {
  int at[kMaxJobs + 1];
  int4 tile0;  // the pair's first unit's row tile, on its way beside their number (job 0 is by rows)
  __device__ __forceinline__ Starts(const Batch& b, int pair) {
    if constexpr (kGrouped) {  // (as many row tiles as the tokens' choices made)
      tile0 = __ldcg(b.groups.tiles + min(static_cast<int>(b.job[0].per_line(static_cast<uint32_t>(pair))), b.groups.most_tiles - 1));
      const int tiles = __ldcg(b.groups.head);
      at[0] = 0;
#pragma unroll
      for (int j = 0; j < kMaxJobs; ++j)
        at[j + 1] = at[j] + (j >= b.n ? 0 : b.job[j].by_inner ? b.groups.experts * b.job[j].tiles : tiles * b.job[j].tiles_n);
    }
  }
  __device__ __forceinline__ int total(const Batch& b) const { return kGrouped ? at[kMaxJobs] : b.start[b.n]; }
  __device__ __forceinline__ int job(const Batch& b, int t) const {
    if constexpr (kGrouped) return t >= at[2] && b.n > 2 ? 2 : t >= at[1] && b.n > 1 ? 1 : 0;
    int j = 0;
    while (j + 1 < b.n && t >= b.start[j + 1]) ++j;
    return j;
  }
  __device__ __forceinline__ const int4* tile(int job, int i) const { return kGrouped && job == 0 && i == 0 ? &tile0 : nullptr; }
  __device__ __forceinline__ int start(const Batch& b, int j) const {
    if constexpr (kGrouped) return j == 0 ? 0 : j == 1 ? at[1] : at[2];
    return b.start[j];
  }
};

// Grouped: the slot and the weight of the lane's row (row0 + lane) of a tile; slot -1: a row that is only
// there to fill up, of zeros.
struct Row {
  int slot;
  float weight;
  template <bool kGrouped>
  static __device__ __forceinline__ Row at(const Batch& b, int row, int rows) {
    Row r{-1, 0.0f};
    if (kGrouped && row < rows) {
      const int2 v = __ldcg(b.groups.row + row);
      r = Row{v.x, __int_as_float(v.y)};
    }
    return r;
  }
};

// A bounded wait for an mbarrier (given by its shared-memory address) that costs the two threads
// feeding the tensor cores as little as a wait can: the clock and the error word (in host memory)
// are only looked at every 256th failed try. Each try may sleep in the hardware until the phase
// completes.
template <bool kCluster>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (kCluster) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  }
  return ok != 0;
}
template <bool kCluster>
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, int* err) {
  unsigned long long t0 = 0;
  for (uint32_t spin = 1;; ++spin) {
    if (try_wait<kCluster>(bar, parity)) return true;
    if ((spin & 255u) == 0) {
      const unsigned long long t = tc::globaltimer();
      if (t0 == 0) t0 = t;
      if (err != nullptr && t - t0 > 1000000ull && *reinterpret_cast<volatile int*>(err) != 0) return false;
      if (t - t0 > tc::kWaitLimitNs) {
        if (err != nullptr) atomicExch(err, 1);
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, int* err) {
  return try_wait<false>(bar, parity) || wait_slow<false>(bar, parity, err);
}
// For a barrier on which threads of the other CTA arrive.
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity, int* err) {
  return try_wait<true>(bar, parity) || wait_slow<true>(bar, parity, err);
}
// The same without an error to report or heed: for copies and products that must have ended before
// their memory is given up.
__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity) { wait(bar, parity, nullptr); }

// A thread that gives up leaves the others to their own waits, so one of the four threads that load may
// have sent copies that no barrier was armed for and nobody waits for. Whoever gives up says so in both
// CTAs, and when no thread of the pair loads any more (behind the last cluster barrier) both stay for a
// millisecond, hundreds of times what a copy takes, before their shared memory is given up.
constexpr unsigned long long kSettleNs = 1000000ull;
__device__ __forceinline__ void tell_pair(uint32_t* word) {
  for (uint32_t r = 0; r < 2; ++r)
    asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(tc::map_to_rank(tc::smem_u32(word), r)), "r"(1u) : "memory");
}
__device__ __forceinline__ void settle() {
  const unsigned long long t0 = tc::globaltimer();
  while (tc::globaltimer() - t0 < kSettleNs) __nanosleep(1000);
}

template <bool kGrouped>
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* m, uint32_t bar_cluster, int c0, int c1, int c2) {
  if constexpr (kGrouped) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
        "%4, %5}], [%2];" ::"r"(dst),
        "l"(m), "r"(bar_cluster), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
    return;
  }
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4}], [%2];" ::"r"(dst),
      "l"(m), "r"(bar_cluster), "r"(c0), "r"(c1)
      : "memory");
}

// a(z) = z s(phi(z)) with the logistic s and phi(z) = z (c1 + c3 z^2): c1 = 1, c3 = 0 for SiLU; for the
// tanh form of GELU c1 = 2 sqrt(2/pi), c3 = 0.044715 c1, since (1 + tanh y) / 2 = s(2 y). Beyond
// |z| = 100 s is 0 or 1 in fp32: GELU's z is held there inside phi, so that no infinity meets a zero.
template <int kAct>
__device__ __forceinline__ void gate(F2 z, F2& a, F2& da) {
  const F2 one = f2(1.0f, 1.0f);
  F2 t, dphi = one;
  if constexpr (kAct == ZOPT_ACT_GELU) {
    const float c1 = 1.5957691216057308f, c3 = 0.071354816f;
    const float2 x = f2(z);
    const F2 zc = f2(fminf(fmaxf(x.x, -100.0f), 100.0f), fminf(fmaxf(x.y, -100.0f), 100.0f)), z2 = zc * zc;
    dphi = fma2(z2, f2(3.0f * c3, 3.0f * c3), f2(c1, c1));
    t = zc * fma2(z2, f2(-kLog2e * c3, -kLog2e * c3), f2(-kLog2e * c1, -kLog2e * c1));
  } else {
    t = z * f2(-kLog2e, -kLog2e);
  }
  const float2 e = f2(t);
  const float2 d = f2(f2(ex2(e.x), ex2(e.y)) + one);
  const F2 s = f2(rcp(d.x), rcp(d.y));
  a = z * s;
  da = a * fma2(s, f2(-1.0f, -1.0f), one);
  if constexpr (kAct == ZOPT_ACT_GELU) {
    da = fma2(da, dphi, s);
  } else {
    da = da + s;
  }
}

// ---------------------------------------------------------------------- epilogues
//
// Each turns one warp's part of a tile into outputs: 32 rows from row0 on and half h of the columns,
// a lane one row. `acc` reads the accumulators and gives them back to the MMAs as soon as the warp
// has read its last ones, while the arithmetic and the stores on them still run; every epilogue
// reads all it needs and calls done() once.
struct Acc {
  uint32_t base;         // the TMEM address of the warp's lanes, the tile's column 0
  uint32_t release_bar;  // the leader's barrier of this accumulator
  int lane;
  __device__ __forceinline__ void read32(int c, uint32_t (&v)[32]) const {
    tc::tmem_ld32(base + static_cast<uint32_t>(c), v);
    tc::tmem_wait_ld();
  }
  __device__ __forceinline__ void read64(int c, uint32_t (&v)[2][32]) const {
    tc::tmem_ld32(base + static_cast<uint32_t>(c), v[0]);
    tc::tmem_ld32(base + static_cast<uint32_t>(c + 32), v[1]);
    tc::tmem_wait_ld();
  }
  __device__ __forceinline__ void done() const {
    tc::fence_before_sync();
    __syncwarp();
    // What passes to the MMAs is the TMEM columns alone. PTX orders the tcgen05 operations of two threads
    // by the first's completed reads (wait::ld) and fence::before_thread_sync, an arrival and a wait at
    // a scope that holds both threads, relaxed ones too, and the second's fence::after_thread_sync. So
    // the arrival is relaxed, at cluster scope (wait_cluster is the other side): a release would wait for
    // the warp's stores in flight as well (777 x 768 x 50177 cross entropy backward 158 us for 166,
    // 1537 x 1000 x 2732 block both ways 126.7 for 131.5, the large shapes 0 to 1 %).
    if (lane == 0)
      asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(release_bar) : "memory");
  }
};
__device__ __forceinline__ float f(uint32_t x) { return __uint_as_float(x); }

// The parts of a token's sum are not rounded to bf16, which would add as much error as the sum's own
// rounding: 64 columns of a row share a power of two that brings the largest finite magnitude to
// 2^14 .. 2^15, and an entry is fp16 in that unit, three bits more in the same two bytes (2^-12 of an entry
// down to 2^-29 of the largest, a fixed step below). Returns the unit.
__device__ __forceinline__ float half_words(const uint32_t (&v)[2][32], uint32_t (&words)[32]) {
  float top[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < 64; ++k) top[k & 3] = act8::amax_step(top[k & 3], f(v[k >> 5][k & 31]));
  const uint32_t e = __float_as_uint(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]))) >> 23;
  const uint32_t up = min(127u + 127u + 14u - max(e, 1u), 253u);  // 2^(14 - exponent), at most 2^126
  const F2 scale = f2(__uint_as_float(up << 23), __uint_as_float(up << 23));
#pragma unroll
  for (int k = 0; k < 32; ++k) {
    const float2 x = f2(f2(f(v[k >> 4][2 * (k & 15)]), f(v[k >> 4][2 * (k & 15) + 1])) * scale);
    const __half2 h = __floats2half2_rn(x.x, x.y);
    words[k] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return __uint_as_float((254u - up) << 23);
}

template <bool kGrouped>
__device__ __forceinline__ void epi_store(const Job& j, const Unit& w, const Part& part, const Acc& acc, int lane, uint32_t box) {
  const int row0 = part.row0, row = row0 + lane;
  const float alpha = !kGrouped && j.alpha != nullptr && j.splits == 1 ? __ldcg(j.alpha) : 1.0f;
  const bool wide = !kGrouped && j.out_mode == kOutF32;
  const int width = part.width;
  void* const first = kGrouped ? static_cast<void*>(static_cast<uint16_t*>(j.out) + w.expert * j.out_stride)
                      : wide   ? static_cast<void*>(static_cast<float*>(j.out) + w.split * j.split_stride)
                               : j.out;
  const Out<128> out(first, j.ld_out, wide ? 4 : 2, row0, w.rows, part.col, j.N, lane);
  if (kGrouped && w.kb1 == 0 && width == 128 && out.whole && out.bytes >= 256) {  // a sum of nothing, without a look at the accumulator
    acc.done();
    uint8_t* p = out.base + lane / 16 * out.pitch + 16 * (lane % 16);
#pragma unroll
    for (int r = 0; r < 32; r += 2) {
      *reinterpret_cast<uint4*>(p) = make_uint4(0, 0, 0, 0);
      p += 2 * out.pitch;
    }
    return;
  }
#pragma unroll 1
  for (int half = 0; 64 * half < width; ++half) {
    uint32_t v[2][32];
    acc.read64(part.tcol + 64 * half, v);
    if (64 * half + 64 == width) acc.done();
    const int col0 = part.col + 64 * half;
    if (col0 >= j.N || row0 >= w.rows) continue;  // (warp-uniform)
    if (kGrouped && w.kb1 == 0) {  // a sum of nothing
#pragma unroll
      for (int k = 0; k < 64; ++k) v[k >> 5][k & 31] = 0u;
    }
    if (!kGrouped && j.add != nullptr && row < w.rows) {
      const float* a = j.add + static_cast<long long>(row) * j.ld_add + col0;
      if (col0 + 64 <= j.N) {
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const float4 x = reinterpret_cast<const float4*>(a)[q];
          uint32_t* o = &v[q >> 3][4 * (q & 7)];
          o[0] = __float_as_uint(f(o[0]) + x.x), o[1] = __float_as_uint(f(o[1]) + x.y);
          o[2] = __float_as_uint(f(o[2]) + x.z), o[3] = __float_as_uint(f(o[3]) + x.w);
        }
      } else {
#pragma unroll
        for (int k = 0; k < 64; ++k)
          if (col0 + k < j.N) v[k >> 5][k & 31] = __float_as_uint(f(v[k >> 5][k & 31]) + a[k]);
      }
    }
    if (alpha != 1.0f) {
#pragma unroll
      for (int k = 0; k < 64; ++k) v[k >> 5][k & 31] = __float_as_uint(f(v[k >> 5][k & 31]) * alpha);
    }
    if (kGrouped && j.part_scale != nullptr) {
      uint32_t words[32];
      j.part_scale[static_cast<long long>(col0 >> 6) * j.rows_ld + row] = half_words(v, words);
      box_put(box, lane, 0, words);
      __syncwarp();
      out.template put<0>(box, lane, 128 * half);
      __syncwarp();
    } else if (wide) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        box_put(box, lane, 0, v[c]);
        __syncwarp();
        out.put<0>(box, lane, 256 * half + 128 * c);
        __syncwarp();
      }
    } else {
      uint32_t words[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) words[k] = pack2(f(v[k >> 4][2 * (k & 15)]), f(v[k >> 4][2 * (k & 15) + 1]));
      box_put(box, lane, 0, words);
      __syncwarp();
      out.put<0>(box, lane, 128 * half);
      __syncwarp();
    }
  }
}

// The maximum m and the sum s = sum 2^(x - m) of the row's 128 logits times log2(e), 64 at a time.
// Columns beyond the vocabulary take no part; where all logits are -inf, m = -inf and s = 0.
__device__ __forceinline__ void epi_ce_fwd(const Job& j, const Unit& w, const Acc& acc, int row0, int lane, int h) {
  const int row = row0 + lane;
  const long long tgt = row < j.M ? j.target[row] : -1;
  float m = -INFINITY, s = 0.0f;
  const int width = j.tile_n >> 1;
#pragma unroll 1
  for (int half = 0; 64 * half < width; ++half) {
    uint32_t v[2][32];
    acc.read64(width * h + 64 * half, v);
    if (64 * half + 64 == width) acc.done();
    const int col = w.tj * j.tile_n + width * h + 64 * half;
    if (tgt >= col && tgt < col + 64 && tgt < j.N) {
      float t = 0.0f;
#pragma unroll
      for (int k = 0; k < 64; ++k)
        if (col + k == tgt) t = f(v[k >> 5][k & 31]);
      j.tlogit[row] = t;
    }
    if (col + 64 > j.N) {
#pragma unroll
      for (int k = 0; k < 64; ++k)
        if (col + k >= j.N) v[k >> 5][k & 31] = 0xFF800000u;
    }
    float top[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) top[i] = f(v[0][i]);
#pragma unroll
    for (int k = 8; k < 64; ++k) top[k & 7] = fmaxf(top[k & 7], f(v[k >> 5][k & 31]));
#pragma unroll
    for (int d = 4; d >= 1; d >>= 1)
#pragma unroll
      for (int i = 0; i < d; ++i) top[i] = fmaxf(top[i], top[i + d]);
    const float mn = fmaxf(m, top[0] * kLog2e);
    const float base = mn == -INFINITY ? 0.0f : mn;
    F2 part[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) part[i] = f2(0.0f, 0.0f);
    const F2 scale = f2(kLog2e, kLog2e), minus = f2(-base, -base);
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      const float2 x = f2(fma2(f2(f(v[k >> 4][2 * (k & 15)]), f(v[k >> 4][2 * (k & 15) + 1])), scale, minus));
      part[k & 3] = part[k & 3] + f2(ex2(x.x), ex2(x.y));
    }
    const float2 sum = f2((part[0] + part[1]) + (part[2] + part[3]));
    s = fmaf(s, ex2(m - base), sum.x + sum.y);
    m = mn;
  }
  if (row < j.M) j.part[static_cast<long long>(2 * w.tj + h) * j.M + row] = make_float2(m, s);
}

// (p - [column = target]) dloss / unit as bf16, p = 2^(logit log2(e) - lse log2(e)). A row without a
// loss is exactly zero whatever its logits; a row with a target outside the vocabulary is NaN.
// Rounding this gradient to bf16 is what lets both products that read it run on the tensor cores.
// The unit is the largest dloss: where all rows weigh the same (a mean), the target's entry, most of
// a row's norm, is p - 1, close to a bf16 value for a small p; times 1 / n it would carry one and the
// same rounding error, up to 2^-8, into every row (8192 x 2048 x 32000: gradients 2.8e-3 off in
// 64 bits' norm without the unit).
__device__ __forceinline__ void epi_ce_bwd(const Job& j, const Unit& w, const Acc& acc, int row0, int lane, int h,
                                           uint32_t box) {
  const int row = row0 + lane;
  const int width = j.tile_n >> 1;
  const Out<128> out(j.out, j.ld_out, 2, row0, j.M, w.tj * j.tile_n + width * h, j.N, lane);
  long long tgt = j.ignore;
  float lse2 = 0.0f, dl = 0.0f;
  if (row < j.M) {
    tgt = j.target[row];
    if (tgt != j.ignore) {
      lse2 = j.lse[row] * kLog2e;
      dl = (tgt < 0 || tgt >= j.vocab) ? __uint_as_float(0x7FC00000u) : j.dloss[row] / __ldcg(j.unit);
    }
  }
  const bool live = tgt != j.ignore;
  const long long at = tgt - j.col0;  // the target's column in this job
#pragma unroll 1
  for (int half = 0; 64 * half < width; ++half) {
    uint32_t v[2][32];
    acc.read64(width * h + 64 * half, v);
    if (64 * half + 64 == width) acc.done();
    const int col = w.tj * j.tile_n + width * h + 64 * half;
    if (col >= j.N || row0 >= j.M) continue;
    const F2 scale = f2(kLog2e, kLog2e), minus = f2(-lse2, -lse2), weight = f2(dl, dl);
    uint32_t words[32];
    if (at < col || at >= col + 64) {
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float2 x = f2(fma2(f2(f(v[k >> 4][2 * (k & 15)]), f(v[k >> 4][2 * (k & 15) + 1])), scale, minus));
        words[k] = pack2(f2(ex2(x.x), ex2(x.y)) * weight);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float2 x = f2(fma2(f2(f(v[k >> 4][2 * (k & 15)]), f(v[k >> 4][2 * (k & 15) + 1])), scale, minus));
        words[k] = pack2((ex2(x.x) - (col + 2 * k == at ? 1.0f : 0.0f)) * dl, (ex2(x.y) - (col + 2 * k + 1 == at ? 1.0f : 0.0f)) * dl);
      }
    }
    if (!live) {
#pragma unroll
      for (int k = 0; k < 32; ++k) words[k] = 0u;
    }
    box_put(box, lane, 0, words);
    __syncwarp();
    out.put<0>(box, lane, 128 * half);
    __syncwarp();
  }
}

// Whether all of the warps (`threads` in all) that share barrier `bar` bring ok. Every lane of them has to come.
__device__ __forceinline__ bool both_warps(int ok, int bar, int threads) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok), "r"(bar), "r"(threads)
      : "memory");
  return r != 0;
}

// The first half of a tile's TMEM columns hold the gate, the second the up product of the same 128 (or
// 64) hidden columns; the warp's are half h of each. Where 8 bits are kept a tile is one block wide
// (128): a block's largest magnitude is found within a lane and its partner in the warp that has the
// other half, through `swap` (two bytes a lane; the two warps share barrier `bar`).
template <int kAct, int kKept, bool kGrouped>
__device__ __forceinline__ void epi_glu_fwd(const Job& j, const Unit& w, const Part& part, const Acc& acc, const Row& mine, int lane,
                                            int h, uint32_t box, uint16_t* swap, int quad) {
  // the gate's columns in the accumulator, and the up's behind them
  const int row0 = part.row0, count = part.width, up = kGrouped && w.half ? 2 * part.width : (kKept == kKeep8 ? 128 : j.tile_n >> 1);
  const int row = kGrouped ? mine.slot : row0 + lane;
  if (row0 >= w.rows) {  // (the partner warps have the same rows)
    acc.done();
    return;
  }
  float inv[2] = {1.0f, 1.0f};
  if constexpr (kKept == kKeep8) {
    uint32_t e[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      uint32_t v[2][32];
      float top[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      const int n = j.hidden - part.col;
      if (kGrouped && w.half) {
        tc::tmem_ld32(acc.base + static_cast<uint32_t>(up * p + part.tcol), v[0]);
        tc::tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (k < n) top[k & 3] = act8::amax_step(top[k & 3], f(v[0][k]));
      } else {
        acc.read64(128 * p + 64 * h, v);
        if (n >= 64) {
#pragma unroll
          for (int k = 0; k < 64; ++k) top[k & 3] = act8::amax_step(top[k & 3], f(v[k >> 5][k & 31]));
        } else {
#pragma unroll
          for (int k = 0; k < 64; ++k)
            if (k < n) top[k & 3] = act8::amax_step(top[k & 3], f(v[k >> 5][k & 31]));
        }
      }
      e[p] = act8::exponent_byte(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
    }
    // (both_warps comes between this and the same warps' next; the byte grows with the magnitude)
    if (kGrouped && w.half) {  // four warps have the block's columns: two quarters' two halves
      uint16_t* const all = swap - 64 * quad + 256 + 128 * (quad & 1);  // (not where pairs have theirs)
      all[32 * (2 * (quad >> 1) + h) + lane] = static_cast<uint16_t>(e[0] | (e[1] << 8));
      asm volatile("bar.sync %0, 128;" ::"r"(5 + (quad & 1)) : "memory");
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t other = all[32 * q + lane];
        e[0] = max(e[0], other & 255u), e[1] = max(e[1], other >> 8);
      }
    } else {
      swap[32 * h + lane] = static_cast<uint16_t>(e[0] | (e[1] << 8));
      asm volatile("bar.sync %0, 64;" ::"r"(1 + quad) : "memory");
      const uint32_t other = swap[32 * (1 - h) + lane];
      e[0] = max(e[0], other & 255u), e[1] = max(e[1], other >> 8);
    }
    const long long nb = act8::blocks_of(j.hidden);
    if ((kGrouped ? row >= 0 : row < w.rows) && !(kGrouped && w.half && quad >= 2))
      j.kept_scale[static_cast<long long>(row) * 2 * nb + h * nb + w.tj] = static_cast<uint8_t>(h == 0 ? e[0] : e[1]);
    inv[0] = act8::inv_scale(e[0]), inv[1] = act8::inv_scale(e[1]);
  }
  constexpr int kSize = kKept == kKeep8 ? 1 : 2;
  const int first = part.col;
  const Out<64> out(j.out, j.ld_out, 2, row0, w.rows, first, j.hidden, lane);
  const auto gate_out = part_of<32 * kSize, kGrouped>(j.kept, j.ld_kept, kSize, row0, w.rows, row, first, j.hidden, lane);
  const auto up_out = part_of<32 * kSize, kGrouped>(static_cast<uint8_t*>(j.kept) + static_cast<long long>(j.hidden) * kSize,
                                                    j.ld_kept, kSize, row0, w.rows, row, first, j.hidden, lane);
#pragma unroll 1
  for (int c = 0; 32 * c < count; ++c) {
    uint32_t g[32], u[32];
    tc::tmem_ld32(acc.base + static_cast<uint32_t>(part.tcol + 32 * c), g);
    tc::tmem_ld32(acc.base + static_cast<uint32_t>(up + part.tcol + 32 * c), u);
    tc::tmem_wait_ld();
    if (32 * c + 32 >= count) acc.done();
    if (first + 32 * c >= j.hidden) continue;
    if constexpr (kKept == kKeepBf16) {  // a box: a row's 32 gates, then its 32 ups
      uint32_t words[32];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        words[k] = pack2(f(g[2 * k]), f(g[2 * k + 1]));
        words[16 + k] = pack2(f(u[2 * k]), f(u[2 * k + 1]));
      }
      box_put(box, lane, 0, words);
      __syncwarp();
      gate_out.template put<0>(box, lane, 64 * c);
      up_out.template put<64>(box, lane, 64 * c);
      __syncwarp();
    } else if constexpr (kKept == kKeep8) {  // a box: a row's 32 gate bytes, its 32 up bytes, its 32 h
      uint32_t words[16];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        words[q] = act8::encode4(f(g[4 * q]), f(g[4 * q + 1]), f(g[4 * q + 2]), f(g[4 * q + 3]), inv[0]);
        words[8 + q] = act8::encode4(f(u[4 * q]), f(u[4 * q + 1]), f(u[4 * q + 2]), f(u[4 * q + 3]), inv[1]);
      }
      box_put(box, lane, 0, words);
    }
    uint32_t hh[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      F2 a, da;
      gate<kAct>(f2(f(g[2 * k]), f(g[2 * k + 1])), a, da);
      F2 hk = a * f2(f(u[2 * k]), f(u[2 * k + 1]));
      if (kGrouped) hk = hk * f2(mine.weight, mine.weight);
      hh[k] = pack2(hk);
    }
    box_put(box, lane, 4, hh);
    __syncwarp();
    if constexpr (kKept == kKeep8) {
      gate_out.template put<0>(box, lane, 32 * c);
      up_out.template put<32>(box, lane, 32 * c);
    }
    out.put<64>(box, lane, 64 * c);
    __syncwarp();
  }
}

// The words of 32 kept columns of one row and part as they lie in memory (bf16: 16 words, 8 bits: 8),
// zero beyond `bytes`.
template <int kWords, typename Piece>
__device__ __forceinline__ void words_in(const uint8_t* p, int bytes, uint32_t* x) {
  constexpr int kPiece = sizeof(Piece);
#pragma unroll
  for (int i = 0; i < 4 * kWords / kPiece; ++i) {
    Piece v{};
    if ((i + 1) * kPiece <= bytes) v = __ldg(reinterpret_cast<const Piece*>(p) + i);
    if constexpr (kPiece == 8) {
      x[2 * i] = v.x, x[2 * i + 1] = v.y;
    } else if constexpr (kPiece == 4) {
      x[i] = v;
    } else {
      const int shift = 8 * (i * kPiece & 3);
      x[i * kPiece / 4] = (shift == 0 ? 0u : x[i * kPiece / 4]) | (static_cast<uint32_t>(v) << shift);
    }
  }
}

// Gate and up of 32 rows' 32 columns. Where every row, and up's offset in it, is a multiple of 16 bytes
// (kWide) consecutive lanes load along a row, and the warp's box turns the pieces into rows, a lane
// each, when they are used: a load that takes 16 bytes of 32 rows keeps the L1 data path, which the
// epilogue shares with the MMAs' operands, busy four times as long (the backward's first launch of
// 8192 x 2048 x 5632, 8 bits kept: 144 us for 139). Else each lane loads its row.
template <int kKept, bool kWide, bool kGrouped>
struct Kept {
  static constexpr int kWords = kKept == kKeep8 ? 8 : 16, kSize = kKept == kKeep8 ? 1 : 2;
  static constexpr int kPerRow = kWords / 4, kAtOnce = 32 / kPerRow;  // pieces of a row's part, rows of a load
  uint32_t x[2][kWords];
  // from row row0 (of `rows`; grouped: the lane's row is row `slot`) and column col on
  __device__ __forceinline__ void load(const Job& j, int row0, int rows, int slot, int col, int lane) {
    if constexpr (kWide && kGrouped) {
      const int at = col * kSize + 16 * (lane % kPerRow);
      const long long pitch = j.ld_kept * kSize, up = static_cast<long long>(j.hidden) * kSize;
      const uint8_t* const p = static_cast<const uint8_t*>(j.kept) + at;
      const long long to_up = j.kept_up * kSize;
#pragma unroll
      for (int i = 0; i < kPerRow; ++i) {
        uint4 g = make_uint4(0, 0, 0, 0), u = g;
        const int from = __shfl_sync(0xFFFFFFFFu, slot, lane / kPerRow + i * kAtOnce);
        if (at < up && from >= 0) {
          g = __ldg(reinterpret_cast<const uint4*>(p + from * pitch));
          u = __ldg(reinterpret_cast<const uint4*>(p + from * pitch + to_up));
        }
        x[0][4 * i] = g.x, x[0][4 * i + 1] = g.y, x[0][4 * i + 2] = g.z, x[0][4 * i + 3] = g.w;
        x[1][4 * i] = u.x, x[1][4 * i + 1] = u.y, x[1][4 * i + 2] = u.z, x[1][4 * i + 3] = u.w;
      }
    } else if constexpr (kWide) {
      const int at = col * kSize + 16 * (lane % kPerRow);
      const long long pitch = j.ld_kept * kSize, up = static_cast<long long>(j.hidden) * kSize;
      int row = row0 + lane / kPerRow;
      const uint8_t* p = static_cast<const uint8_t*>(j.kept) + row * pitch + at;
#pragma unroll
      for (int i = 0; i < kPerRow; ++i) {
        uint4 g = make_uint4(0, 0, 0, 0), u = g;
        if (at < up && row < rows) g = __ldg(reinterpret_cast<const uint4*>(p)), u = __ldg(reinterpret_cast<const uint4*>(p + up));
        x[0][4 * i] = g.x, x[0][4 * i + 1] = g.y, x[0][4 * i + 2] = g.z, x[0][4 * i + 3] = g.w;
        x[1][4 * i] = u.x, x[1][4 * i + 1] = u.y, x[1][4 * i + 2] = u.z, x[1][4 * i + 3] = u.w;
        row += kAtOnce, p += kAtOnce * pitch;
      }
    } else {
      load_row(j, row0 + lane, row0 + lane < rows, col);
    }
  }
  // Piece q of a row of 64 bytes, where neither eight rows' one nor two pieces of four rows meet a bank twice.
  static __device__ __forceinline__ uint32_t piece(uint32_t box, int row, int q) {
    return box + static_cast<uint32_t>(row * 64) + ((static_cast<uint32_t>(q) ^ (__brev(static_cast<uint32_t>(row & 6)) >> 29)) << 4);
  }
  // What was loaded becomes the lane's row (through a box of 64-byte rows: both parts, or of bf16 one after the
  // other).
  __device__ __forceinline__ void turn(uint32_t box, int lane) {
    if constexpr (kWide) {
      constexpr int kParts = kKept == kKeep8 ? 2 : 1;  // at a time
#pragma unroll
      for (int p0 = 0; p0 < 2; p0 += kParts) {
#pragma unroll
        for (int part = 0; part < kParts; ++part)
#pragma unroll
          for (int i = 0; i < kPerRow; ++i) {
            const uint32_t* const v = x[p0 + part] + 4 * i;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             piece(box, lane / kPerRow + i * kAtOnce, part * kPerRow + lane % kPerRow)),
                         "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                         : "memory");
          }
        __syncwarp();
#pragma unroll
        for (int part = 0; part < kParts; ++part)
#pragma unroll
          for (int i = 0; i < kPerRow; ++i) {
            uint32_t* const v = x[p0 + part] + 4 * i;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                         : "r"(piece(box, lane, part * kPerRow + i))
                         : "memory");
          }
        __syncwarp();
      }
    }
  }
  __device__ __forceinline__ void load_row(const Job& j, int row, bool there, int col) {
    const bool in = there && col < j.hidden;
    const int bytes = in ? min(32, j.hidden - col) * kSize : 0;
    const uint8_t* p = static_cast<const uint8_t*>(j.kept) + (in ? (static_cast<long long>(row) * j.ld_kept + col) * kSize : 0);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const uint8_t* at = p + (in ? static_cast<long long>(part) * j.hidden * kSize : 0);
      const unsigned mis = static_cast<unsigned>(reinterpret_cast<uintptr_t>(at)) | static_cast<unsigned>(bytes);
      if ((mis & 7u) == 0) {
        words_in<kWords, uint2>(at, bytes, x[part]);
      } else if ((mis & 3u) == 0) {
        words_in<kWords, uint32_t>(at, bytes, x[part]);
      } else if (kSize == 2) {
        words_in<kWords, uint16_t>(at, bytes, x[part]);
      } else {
        words_in<kWords, uint8_t>(at, bytes, x[part]);
      }
    }
  }
  // Values 2 q and 2 q + 1 of a part.
  __device__ __forceinline__ F2 two(int part, int q, float sc) const {
    if constexpr (kKept == kKeep8) {
      const float2 v = act8::decode2(x[part][q >> 1] >> (16 * (q & 1)));
      return f2(v.x, v.y) * f2(sc, sc);
    }
    return f2(__uint_as_float(x[part][q & (kWords - 1)] << 16), __uint_as_float(x[part][q & (kWords - 1)] & 0xFFFF0000u));
  }
};
// The two powers of the lane's row in the 128 columns from col on (one block of each part).
struct Scales {
  float s[2] = {1.0f, 1.0f};
  __device__ __forceinline__ void load(const Job& j, int row, bool there, int col) {
    if (!there || col >= j.hidden) return;
    const long long nb = act8::blocks_of(j.hidden);
    const uint8_t* p = j.kept_scale + static_cast<long long>(row) * 2 * nb + (col >> 7);
    s[0] = act8::scale(p[0]);
    s[1] = act8::scale(p[nb]);
  }
};

// dgate = dh up a'(gate), dup = dh a(gate), h = a(gate) up, each rounded to bf16 once: they are
// operands of the three products that follow, and leave by the TMA, a box of 32 rows and columns each. (This is
// the longest epilogue, and what bounds it is the L1 data path, which the MMAs' operands and their copies keep
// busy: with boxes read back and stored row by row the experts' whole backward of 8192 x 6 slots, 2048 x 1408, 8
// bits kept, took 1480 us for 1452; sixteen warps in eight's place changed nothing.) `k` holds the kept values of the warp's first 32
// columns; while 32 columns are worked on the next ones are on their way, at a tile's end the next
// tile's first (from row next_row0 and column next_col on): gate and up come from HBM, and a tile that
// began by waiting for them would take longer than its products.
constexpr int kTurnBytes = 32 * 64;  // a box of 32 rows of 64 bytes
__device__ __forceinline__ void store_box(const CUtensorMap* m, uint32_t box, int col, int row) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(m), "r"(box), "r"(col), "r"(row)
               : "memory");
}

// Grouped, dg, du and h carry the row's weight, and the weight's own gradient, the sum over the columns
// of dh h without it, leaves in parts.
struct Next {  // the tile after this one
  int row0, rows, col;
  Row mine;
};
template <int kAct, int kKept, bool kWide, bool kGrouped>
__device__ __forceinline__ void epi_glu_bwd(const Job& j, const Unit& w, const Part& part, const Acc& acc, const Row& mine, int lane,
                                            uint32_t box, const CUtensorMap* maps, Kept<kKept, kWide, kGrouped>& k, Scales& sc,
                                            const Next& n) {
  const int row0 = part.row0, width = part.width, col0 = part.col;
  const Out<64> dgate(j.out, j.ld_out, 2, row0, w.rows, col0, j.N, lane);
  const Out<64> dup(static_cast<uint16_t*>(j.out) + j.N, j.ld_out, 2, row0, w.rows, col0, j.N, lane);
  const Out<64> hout(j.out_h, j.ld_h, 2, row0, w.rows, col0, j.N, lane);
  const uint32_t out = box + kTurnBytes;  // the results' boxes, one after another
  Scales next_sc;
  if constexpr (kKept == kKeep8)
    next_sc.load(j, kGrouped ? n.mine.slot : n.row0 + lane, kGrouped ? n.mine.slot >= 0 : n.row0 + lane < n.rows, n.col);
  const F2 weight = f2(mine.weight, mine.weight);
  F2 dot = f2(0.0f, 0.0f);
#pragma unroll 1
  for (int c = 0; 32 * c < width; ++c) {
    const int col = col0 + 32 * c;
    const bool last = 32 * c + 32 == width;
    uint32_t v[32];
    acc.read32(part.tcol + 32 * c, v);
    if (last) acc.done();
    Kept<kKept, kWide, kGrouped> next;
    next.load(j, last ? n.row0 : row0, last ? n.rows : w.rows, last ? n.mine.slot : mine.slot, last ? n.col : col + 32, lane);
    if (col < j.N && row0 < w.rows) {
      k.turn(box, lane);
      if (j.bulk) {  // (the boxes' last contents have been read)
        if (lane == 0) tc::bulk_wait_read<0>();
        __syncwarp();
      }
      if (kGrouped && mine.slot < 0) {  // a row of zeros, whatever the weights hold
#pragma unroll
        for (int p = 0; p < 32; ++p) v[p] = 0u;
      }
      uint32_t hh[16];
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // eight columns: a piece of each result
        uint32_t dg[4], du[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int p = 4 * q + i;
          const F2 g = k.two(0, p, sc.s[0]), u = k.two(1, p, sc.s[1]);
          F2 d = f2(f(v[2 * p]), f(v[2 * p + 1]));
          F2 a, da;
          gate<kAct>(g, a, da);
          F2 au = a * u;
          if (kGrouped) {
            dot = fma2(d, au, dot);
            d = d * weight;
            au = au * weight;
          }
          dg[i] = pack2(d * u * da);
          du[i] = pack2(d * a);
          hh[p] = pack2(au);
        }
        if (j.bulk) {
          box_put4<64>(out, lane, q, dg[0], dg[1], dg[2], dg[3]);
          box_put4<64>(out + kTurnBytes, lane, q, du[0], du[1], du[2], du[3]);
          box_put4<64>(out + 2 * kTurnBytes, lane, q, hh[4 * q], hh[4 * q + 1], hh[4 * q + 2], hh[4 * q + 3]);
        } else {
          box_put4(out, lane, q, dg[0], dg[1], dg[2], dg[3]);  // a row's 32 dgates, then its 32 dups
          box_put4(out, lane, 4 + q, du[0], du[1], du[2], du[3]);
        }
      }
      if (j.bulk) {
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
#pragma unroll
          for (int r = 0; r < 3; ++r) store_box(&maps[r], out + r * kTurnBytes, col, row0);
          tc::bulk_commit();
        }
      } else {
        __syncwarp();
        dgate.template put<0>(out, lane, 64 * c);
        dup.template put<64>(out, lane, 64 * c);
        __syncwarp();
        box_put(out, lane, 0, hh);
        __syncwarp();
        hout.template put<0>(out, lane, 64 * c);
        __syncwarp();
      }
    }
    if (kGrouped && (c & 1) != 0) {  // a part for every 64 columns
      const float2 two = f2(dot);
      if (mine.slot >= 0 && col - 32 < j.N) j.dots[static_cast<long long>(row0 + lane) * j.n_dots + (col >> 6)] = two.x + two.y;
      dot = f2(0.0f, 0.0f);
    }
    k = next;
  }
  sc = next_sc;
}

// ---------------------------------------------------------------------- the kernel

template <int kKinds, int kAct, int kKept, bool kWide, bool kGrouped>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    lm_gemm_kernel(const __grid_constant__ Batch B) {
  constexpr int kStages = stages_of(kKinds), kBox = box_bytes_of(kKinds);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kStages * kHalfBytes;
  uint8_t* sEpi = sB + kStages * kHalfBytes;
  uint16_t* sSwap = reinterpret_cast<uint16_t*>(sEpi + kEpiWarps * kBox);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(sSwap) + kSwapBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drain + 1);
  uint32_t* gave_up = tslot + 1;  // some thread of the pair has stopped waiting

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = tc::cluster_rank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int q = 0; q < kStages; ++q) {
      tc::mbar_init(full + q, 1);
      tc::mbar_init(empty + q, 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(tfull + b, 1);
      tc::mbar_init(tempty + b, 2 * kEpiWarps);  // both CTAs' epilogue warps, one arrival each (used in the leader)
    }
    tc::mbar_init(drain, 1);
    *gave_up = 0;
    tc::fence_mbar_init();
    for (int j = 0; j < B.n; ++j) {
      tc::prefetch_tmap(&B.job[j].P);
      tc::prefetch_tmap(&B.job[j].Q);
      if ((kKinds & kGluFwd) != 0) tc::prefetch_tmap(&B.job[j].Up);
    }
  }
  if (warp == 1) {
    tc::tmem_alloc_pair(tslot, 2 * kTileN);
    tc::tmem_relinquish_pair();
  }
  tc::fence_before_sync();
  tc::cluster_sync();  // the peer's barriers exist before anyone arrives on them
  tc::fence_after_sync();
  const uint32_t tmem = *tslot;
  tc::pdl_launch_dependents();
  tc::pdl_wait();  // the previous launch's outputs are complete and visible

  const Starts<kGrouped> starts(B, pair);
  const int total = starts.total(B);
  int* const err = B.err;
  const uint32_t full0 = tc::smem_u32(full), empty0 = tc::smem_u32(empty);
  if (warp == 0 || warp == 2) {
    if (elect_one()) {
      // ---------------------------------------------------------------- TMA producers (both CTAs)
      // One thread loads P, one Q. Every cycle of this loop counts: a k-block takes the MMAs 512
      // cycles, and a copy takes its thread about 100 (one thread for both operands, two boxes each
      // where they are MN-major, needed 600 a k-block). So everything that a job fixes is in
      // registers before its k-loop.
      const bool is_p = warp == 0;
      const uint32_t s0 = tc::smem_u32(is_p ? sA : sB);
      const uint32_t lead0 = tc::map_to_rank(full0, 0);  // all loads complete on the leader's barriers
      uint32_t s = 0, ph = 1;
      long long done = 0;  // stages armed so far
      bool ok = true;
      for (int i = 0, t; ok && (t = unit_at<kGrouped>(B, pair, npairs, i)) < total; ++i) {
        const int ji = starts.job(B, t);
        const Job& j = B.job[ji];
        const Unit w = unit_of<kGrouped>(B, j, t - starts.start(B, ji), starts.tile(ji, i));
        const bool up = (kKinds & kGluFwd) != 0 && !leader;  // one CTA has the gate's columns, the other up's
        const CUtensorMap* const map = is_p ? &j.P : up ? &j.Up : &j.Q;
        const bool mn = (is_p ? j.a_mn : j.b_mn) != 0;
        const int width = j.tile_n >> 1;  // this CTA's columns of Q
        // this CTA's first row of P, or column of Q
        const bool halved = kGrouped && w.half;
        const int first = is_p                        ? w.row0 + static_cast<int>(rank) * (halved ? 64 : 128)
                          : (kKinds & kGluFwd) != 0 ? w.tj * width + (halved ? static_cast<int>(rank) * 64 : 0)
                                                    : w.tj * j.tile_n + static_cast<int>(rank) * width;
        // (a single tile of at most 128 rows: the other rows' accumulators are of no use to anyone)
        const bool any = !is_p || leader || j.a_rows == 128, two = is_p || width == 128;
        const uint32_t tx = static_cast<uint32_t>(halved ? j.tx - 128 * kTileK * 2 : j.tx);
        // (grouped: activations are one matrix of all experts' rows, weights an expert's)
        const int depth = kGrouped && !is_p && !j.by_inner ? w.expert : 0, krow = kGrouped ? w.krow : 0;
        const int k_end = w.kb1 * kTileK;
        for (int k = w.kb0 * kTileK; k < k_end; k += kTileK) {
          if (!wait(empty0 + 8 * s, ph, err)) {
            ok = false;
            break;
          }
          if (is_p && leader) tc::mbar_arrive_expect_tx(full + s, tx);  // both operands' bytes, both CTAs'
          const uint32_t bar = lead0 + 8 * s, to = s0 + s * kHalfBytes;
          if (!mn) {
            if (any) load_box<kGrouped>(to, map, bar, k, first, depth);
            if (kGrouped && is_p && !halved) load_box<kGrouped>(to + kMnBoxBytes, map, bar, k, first + 64, depth);
          } else if ((kKinds & kGluFwd) != 0 && halved) {  // 64 gate and the matching up columns in either CTA
            load_box<kGrouped>(to, &j.Q, bar, first, krow + k, depth);
            load_box<kGrouped>(to + kMnBoxBytes, &j.Up, bar, first, krow + k, depth);
          } else {
            load_box<kGrouped>(to, map, bar, first, krow + k, depth);
            if (two) load_box<kGrouped>(to + kMnBoxBytes, map, bar, first + 64, krow + k, depth);
          }
          ++done;
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok) tell_pair(gave_up);
      if (!ok && is_p && leader) {  // the leader's stage barriers count all copies: leave none in flight
        for (long long q = done > kStages ? done - kStages : 0; q < done; ++q)
          wait_drain(full0 + 8 * static_cast<uint32_t>(q % kStages), static_cast<uint32_t>(q / kStages) & 1u);
      }
    }
  } else if (warp == 1) {
    if (leader && elect_one()) {
      // ---------------------------------------------------------------- MMA issuer (leader)
      uint32_t s = 0, ph = 0;
      int it = 0;
      bool ok = true;
      const uint32_t tempty0 = tc::smem_u32(tempty);
      for (int t; ok && (t = unit_at<kGrouped>(B, pair, npairs, it)) < total; ++it) {
        const int ji = starts.job(B, t);
        const Job& j = B.job[ji];
        const Unit w = unit_of<kGrouped>(B, j, t - starts.start(B, ji), starts.tile(ji, it));
        const bool amn = j.a_mn != 0, bmn = j.b_mn != 0;
        const uint32_t idesc = tc::idesc_bf16_f32(kGrouped && w.half ? 128 : kTileM, j.tile_n, amn, bmn);
        // a stage's descriptors differ in the address alone (16-byte units), and so do a stage's steps
        const uint64_t ad0 = tc::smem_desc_sw128(tc::smem_u32(sA), amn ? kMnBoxBytes : 16u, 1024u);
        const uint64_t bd0 = tc::smem_desc_sw128(tc::smem_u32(sB), bmn ? kMnBoxBytes : 16u, 1024u);
        const uint32_t astep = amn ? 128u : 2u, bstep = bmn ? 128u : 2u;
        const int b = it & 1;
        const uint32_t tph = static_cast<uint32_t>(it >> 1) & 1u;
        if (!wait_cluster(tempty0 + 8 * b, tph ^ 1u, err)) {
          ok = false;
          break;
        }
        tc::fence_after_sync();
        const uint32_t d = tmem + static_cast<uint32_t>(b * kTileN);
        uint32_t accumulate = 0;
        for (int kb = w.kb0; kb < w.kb1; ++kb) {
          if (!wait(full0 + 8 * s, ph, err)) {
            ok = false;
            break;
          }
          tc::fence_after_sync();
          const uint64_t ad = ad0 + s * (kHalfBytes / 16), bd = bd0 + s * (kHalfBytes / 16);
#pragma unroll
          for (uint32_t kk = 0; kk < kTileK / 16; ++kk) {
            tc::umma_bf16_pair(d, ad + kk * astep, bd + kk * bstep, idesc, accumulate);
            accumulate = 1;
          }
          tc::umma_commit_pair(empty + s, 3);  // both CTAs' stage s is free
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        tc::umma_commit_pair(tfull + b, 3);  // both CTAs' accumulator b is complete
      }
      if (!ok) tell_pair(gave_up);
      tc::umma_commit_pair(drain, 1);
      wait_drain(tc::smem_u32(drain), 0);
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int quad = warp & 3;          // this warp may read TMEM lanes [32 quad, 32 quad + 32)
    const int half = (warp - kFirstEpi) >> 2;   // and takes this half of the columns
    const uint32_t tempty_leader[2] = {tc::map_to_rank(tc::smem_u32(tempty), 0),
                                       tc::map_to_rank(tc::smem_u32(tempty + 1), 0)};
    const uint32_t box = tc::smem_u32(sEpi) + (warp - kFirstEpi) * kBox;
    uint16_t* swap = sSwap + 64 * quad;
    // a tile's columns of D (kGluFwd: hidden ones)
    auto columns = [](const Job& j) { return (kKinds & kGluFwd) == 0 ? j.tile_n : kKept == kKeep8 ? 128 : j.tile_n >> 1; };
    Kept<kKept, kWide, kGrouped> kept;
    Scales scales;
    Row mine{-1, 0.0f};
    auto first_of = [&](int t) {  // the warp's first row and column of unit t (kGluBwd), and its rows
      Next n{0, 0, 0, Row{-1, 0.0f}};
      if (t >= total) return n;
      const Unit w = unit_of<kGrouped>(B, B.job[0], t);
      const Part part = part_of_tile<kGrouped>(w, columns(B.job[0]), rank, quad, half);
      n.row0 = part.row0, n.rows = w.rows, n.col = part.col;
      n.mine = Row::at<kGrouped>(B, n.row0 + lane, n.rows);
      return n;
    };
    if constexpr ((kKinds & kGluBwd) != 0) {
      const Next n = first_of(unit_at<kGrouped>(B, pair, npairs, 0));
      mine = n.mine;
      kept.load(B.job[0], n.row0, n.rows, mine.slot, n.col, lane);
      if constexpr (kKept == kKeep8)
        scales.load(B.job[0], kGrouped ? mine.slot : n.row0 + lane, kGrouped ? mine.slot >= 0 : n.row0 + lane < n.rows, n.col);
    }
    int it = 0;
    for (int t; (t = unit_at<kGrouped>(B, pair, npairs, it)) < total;) {
      const int b = it & 1;
      const uint32_t tph = static_cast<uint32_t>(it >> 1) & 1u;
      ++it;
      const int ji = starts.job(B, t);
      const Job& j = B.job[ji];
      const Unit w = unit_of<kGrouped>(B, j, t - starts.start(B, ji), starts.tile(ji, it - 1));
      const Part part = part_of_tile<kGrouped>(w, columns(j), rank, quad, half);
      const int row0 = part.row0;
      Next next{};
      if constexpr ((kKinds & kGluBwd) != 0) next = first_of(unit_at<kGrouped>(B, pair, npairs, it));
      if constexpr (kGrouped && (kKinds & kGluFwd) != 0) mine = Row::at<kGrouped>(B, row0 + lane, w.rows);
      int ok = 1;
      if (lane == 0) ok = wait(tc::smem_u32(tfull + b), tph, err) ? 1 : 0;
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      // Two warps wait for one another within such a tile: if one's wait has run out, neither begins it.
      if constexpr ((kKinds & kGluFwd) != 0 && kKept == kKeep8) ok = kGrouped && w.half ? both_warps(ok, 5 + (quad & 1), 128) : both_warps(ok, 1 + quad, 64);
      if (!ok) {
        if (lane == 0) tell_pair(gave_up);
        break;
      }
      tc::fence_after_sync();
      const Acc acc{tmem + (static_cast<uint32_t>(32 * quad) << 16) + static_cast<uint32_t>(b * kTileN), tempty_leader[b], lane};
      if ((kKinds & kStore) && j.kind == kStore) epi_store<kGrouped>(j, w, part, acc, lane, box);
      if ((kKinds & kCeFwd) && j.kind == kCeFwd) epi_ce_fwd(j, w, acc, row0, lane, half);
      if ((kKinds & kCeBwd) && j.kind == kCeBwd) epi_ce_bwd(j, w, acc, row0, lane, half, box);
      if constexpr ((kKinds & kGluFwd) != 0)
        epi_glu_fwd<kAct, kKept, kGrouped>(j, w, part, acc, mine, lane, half, box, swap, quad);
      if constexpr ((kKinds & kGluBwd) != 0) {
        epi_glu_bwd<kAct, kKept, kWide, kGrouped>(j, w, part, acc, mine, lane, box, B.outs, kept, scales, next);
        mine = next.mine;
      }
    }
  }
  if ((kKinds & kGluBwd) != 0 && warp >= kFirstEpi && lane == 0) tc::bulk_wait_all();  // results on their way out of the boxes
  tc::fence_before_sync();
  tc::cluster_sync();  // every MMA, copy and remote arrival of the pair is done
  if (*reinterpret_cast<volatile uint32_t*>(gave_up) != 0) settle();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc_pair(tmem, 2 * kTileN);
  }
}

template <bool kGrouped, int kKinds, int kAct = 0, int kKept = kKeepNone, bool kWide = true>
zopt_status launch_kinds(Batch& b, dim3 grid, cudaStream_t s) {
  const auto kernel = lm_gemm_kernel<kKinds, kAct, kKept, kWide, kGrouped>;
  ZOPT_CUDA_TRY(once_per_device([=] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_of(kKinds)); }));
  return launch_pdl(kernel, grid, dim3(kThreads), static_cast<size_t>(smem_of(kKinds)), s, b);
}
template <bool kGrouped, int kAct>
zopt_status launch_glu(Batch& b, dim3 grid, cudaStream_t s) {
  const Job& j = b.job[0];
  if (j.kind == kGluFwd) {
    if (j.kept_mode == kKeepNone) return launch_kinds<kGrouped, kGluFwd, kAct>(b, grid, s);
    return j.kept_mode == kKeep8 ? launch_kinds<kGrouped, kGluFwd, kAct, kKeep8>(b, grid, s)
                                 : launch_kinds<kGrouped, kGluFwd, kAct, kKeepBf16>(b, grid, s);
  }
  const int size = j.kept_mode == kKeep8 ? 1 : 2;
  const bool wide = kGrouped || (aligned16(j.kept) && j.ld_kept * size % 16 == 0 && j.kept_up * size % 16 == 0);  // (grouped: always)
  if constexpr (!kGrouped) {
    if (!wide)
      return j.kept_mode == kKeep8 ? launch_kinds<kGrouped, kGluBwd, kAct, kKeep8, false>(b, grid, s)
                                   : launch_kinds<kGrouped, kGluBwd, kAct, kKeepBf16, false>(b, grid, s);
  }
  return j.kept_mode == kKeep8 ? launch_kinds<kGrouped, kGluBwd, kAct, kKeep8>(b, grid, s)
                               : launch_kinds<kGrouped, kGluBwd, kAct, kKeepBf16>(b, grid, s);
}

}  // namespace
}  // namespace lm
}  // namespace zopt
