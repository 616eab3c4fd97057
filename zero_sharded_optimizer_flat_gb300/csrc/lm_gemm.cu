// The products of the training operators on tcgen05 tensor cores: one persistent CTA-pair kernel
// over a batch of jobs (lm_gemm.cuh), its host launcher, the sum of split products and the copy
// that stages operands.
//
// A cluster of two CTAs computes a 256 x 256 tile with tcgen05.mma.cta_group::2: each CTA holds its
// 128 rows of P and its 128 columns of Q, so a 64-deep k-block brings 32 KiB per SM and the ring
// holds six stages (with five, units of eight k-blocks take 8 % longer, with four 25 %). A thread of
// each CTA for each operand streams it by TMA (all complete on the leader's stage barrier), one
// thread of the leader issues the M=256, N=256, K=16 MMAs into one of two TMEM accumulators, and
// eight epilogue warps (two per quarter of the TMEM lanes, each 128 of the 256 columns) turn the
// other accumulator into the operator's outputs meanwhile. A lane holds whole row pieces, so softmax
// statistics and the 8-bit blocks need no exchange between lanes.
//
// Bound by the tensor cores where the inner length is long enough to hide a tile's epilogue (12 to 30
// k-blocks' time): 521 cycles a k-block of 512, tensor pipe 92 % of elapsed in the cross entropy's
// forward (4096 x 768 x 50304), 89 % in the block's first product and 90 % in its backward's second
// launch (8192 x 2048 x 5632), all three at the clock that the power cap leaves; 61 % in the
// backward's first launch, whose epilogue (three results and two kept inputs an entry) outlasts its
// 32 k-blocks; 76 % in y, 256 tiles over 76 pairs.
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cudaTypedefs.h>

#include <string>

#include "act8.cuh"
#include "f2.cuh"
#include "launch.cuh"
#include "lm_gemm.cuh"
#include "ns_internal.h"
#include "per_device.h"
#include "row_bytes.h"
#include "tc.cuh"

namespace zopt {
namespace ns {
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();
}
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
__device__ __forceinline__ uint32_t box_piece(uint32_t box, int row, int q) {
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

__device__ __forceinline__ void box_put4(uint32_t box, int lane, int q, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box_piece(box, lane, 0) ^ static_cast<uint32_t>(q << 4)), "r"(a),
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

// A unit of work: one tile of one job over one run of k-blocks.
struct Unit {
  int ti, tj, split, kb0, kb1;
};
__device__ __forceinline__ Unit unit_of(const Job& j, int u) {
  Unit w;
  w.split = static_cast<int>(j.per_split(static_cast<uint32_t>(u)));
  u -= w.split * j.tiles;
  const int line = static_cast<int>(j.per_line(static_cast<uint32_t>(u))), at = u - line * static_cast<int>(j.per_line.d);
  w.ti = j.rows_fast ? at : line;
  w.tj = j.rows_fast ? line : at;
  w.kb0 = w.split * j.kb_per_split;
  w.kb1 = min(w.kb0 + j.kb_per_split, j.nk);
  return w;
}
// Pair p's i-th unit, or a number beyond the last.
__device__ __forceinline__ int unit_at(const Batch& b, int pair, int npairs, int i) {
  if (!b.listed) return pair + i * npairs;
  const int at = b.first[pair] + i;
  return at < b.first[pair + 1] ? b.order[at] : 0x7FFFFFFF;
}
__device__ __forceinline__ int job_of(const Batch& b, int t) {
  int j = 0;
  while (j + 1 < b.n && t >= b.start[j + 1]) ++j;
  return j;
}

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

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* m, uint32_t bar_cluster, int c0, int c1) {
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

__device__ __forceinline__ void epi_store(const Job& j, const Unit& w, const Acc& acc, int row0, int lane, int h,
                                          uint32_t box) {
  const int row = row0 + lane;
  const float alpha = j.alpha != nullptr && j.splits == 1 ? __ldcg(j.alpha) : 1.0f;
  const bool wide = j.out_mode == kOutF32;
  const int width = j.tile_n >> 1;
  const Out<128> out(wide ? static_cast<void*>(static_cast<float*>(j.out) + w.split * j.split_stride) : j.out, j.ld_out,
                     wide ? 4 : 2, row0, j.M, w.tj * j.tile_n + width * h, j.N, lane);
#pragma unroll 1
  for (int half = 0; 64 * half < width; ++half) {
    uint32_t v[2][32];
    acc.read64(width * h + 64 * half, v);
    if (64 * half + 64 == width) acc.done();
    const int col0 = w.tj * j.tile_n + width * h + 64 * half;
    if (col0 >= j.N || row0 >= j.M) continue;  // (warp-uniform)
    if (j.add != nullptr && row < j.M) {
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
    if (wide) {
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

// Whether both of the two warps that share barrier `bar` bring ok. Every lane of both has to come.
__device__ __forceinline__ bool both_warps(int ok, int bar) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "bar.red.and.pred q, %2, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(ok), "r"(bar)
      : "memory");
  return r != 0;
}

// The first half of a tile's TMEM columns hold the gate, the second the up product of the same 128 (or
// 64) hidden columns; the warp's are half h of each. Where 8 bits are kept a tile is one block wide
// (128): a block's largest magnitude is found within a lane and its partner in the warp that has the
// other half, through `swap` (two bytes a lane; the two warps share barrier `bar`).
template <int kAct, int kKept>
__device__ __forceinline__ void epi_glu_fwd(const Job& j, const Unit& w, const Acc& acc, int row0, int lane, int h,
                                            uint32_t box, uint16_t* swap, int bar) {
  const int width = kKept == kKeep8 ? 128 : j.tile_n >> 1;  // hidden columns of a tile
  const int row = row0 + lane, n0 = w.tj * width;
  if (row0 >= j.M) {  // (the partner warp has the same rows)
    acc.done();
    return;
  }
  float inv[2] = {1.0f, 1.0f};
  if constexpr (kKept == kKeep8) {
    uint32_t e[2];
    uint32_t v[2][32];
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      acc.read64(128 * part + 64 * h, v);
      float top[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      const int n = j.hidden - n0 - 64 * h;
      if (n >= 64) {
#pragma unroll
        for (int k = 0; k < 64; ++k) top[k & 3] = act8::amax_step(top[k & 3], f(v[k >> 5][k & 31]));
      } else {
#pragma unroll
        for (int k = 0; k < 64; ++k)
          if (k < n) top[k & 3] = act8::amax_step(top[k & 3], f(v[k >> 5][k & 31]));
      }
      e[part] = act8::exponent_byte(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
    }
    swap[32 * h + lane] = static_cast<uint16_t>(e[0] | (e[1] << 8));
    asm volatile("bar.sync %0, 64;" ::"r"(bar) : "memory");
    const uint32_t other = swap[32 * (1 - h) + lane];  // (both_warps comes between this and the next tile's)
    e[0] = max(e[0], other & 255u), e[1] = max(e[1], other >> 8);  // the byte grows with the magnitude
    const long long nb = act8::blocks_of(j.hidden);
    if (row < j.M)
      j.kept_scale[static_cast<long long>(row) * 2 * nb + h * nb + w.tj] = static_cast<uint8_t>(h == 0 ? e[0] : e[1]);
    inv[0] = act8::inv_scale(e[0]), inv[1] = act8::inv_scale(e[1]);
  }
  constexpr int kSize = kKept == kKeep8 ? 1 : 2;
  const int first = n0 + (width >> 1) * h;
  const Out<64> out(j.out, j.ld_out, 2, row0, j.M, first, j.hidden, lane);
  Out<32 * kSize> gate_out(j.kept, j.ld_kept, kSize, row0, j.M, first, j.hidden, lane);
  Out<32 * kSize> up_out(static_cast<uint8_t*>(j.kept) + static_cast<long long>(j.hidden) * kSize, j.ld_kept, kSize, row0, j.M,
                         first, j.hidden, lane);
#pragma unroll 1
  for (int c = 0; 64 * c < width; ++c) {
    uint32_t g[32], u[32];
    tc::tmem_ld32(acc.base + static_cast<uint32_t>((width >> 1) * h + 32 * c), g);
    tc::tmem_ld32(acc.base + static_cast<uint32_t>(width + (width >> 1) * h + 32 * c), u);
    tc::tmem_wait_ld();
    if (64 * c + 64 >= width) acc.done();
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
      hh[k] = pack2(a * f2(f(u[2 * k]), f(u[2 * k + 1])));
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
template <int kKept, bool kWide>
struct Kept {
  static constexpr int kWords = kKept == kKeep8 ? 8 : 16, kSize = kKept == kKeep8 ? 1 : 2;
  static constexpr int kPerRow = kWords / 4, kAtOnce = 32 / kPerRow;  // pieces of a row's part, rows of a load
  uint32_t x[2][kWords];
  // from row row0 and column col on
  __device__ __forceinline__ void load(const Job& j, int row0, int col, int lane) {
    if constexpr (kWide) {
      const int at = col * kSize + 16 * (lane % kPerRow);
      const long long pitch = j.ld_kept * kSize, up = static_cast<long long>(j.hidden) * kSize;
      int row = row0 + lane / kPerRow;
      const uint8_t* p = static_cast<const uint8_t*>(j.kept) + row * pitch + at;
#pragma unroll
      for (int i = 0; i < kPerRow; ++i) {
        uint4 g = make_uint4(0, 0, 0, 0), u = g;
        if (at < up && row < j.M) g = __ldg(reinterpret_cast<const uint4*>(p)), u = __ldg(reinterpret_cast<const uint4*>(p + up));
        x[0][4 * i] = g.x, x[0][4 * i + 1] = g.y, x[0][4 * i + 2] = g.z, x[0][4 * i + 3] = g.w;
        x[1][4 * i] = u.x, x[1][4 * i + 1] = u.y, x[1][4 * i + 2] = u.z, x[1][4 * i + 3] = u.w;
        row += kAtOnce, p += kAtOnce * pitch;
      }
    } else {
      load_row(j, row0 + lane, col);
    }
  }
  // What was loaded becomes the lane's row (through the warp's box).
  __device__ __forceinline__ void turn(uint32_t box, int lane) {
    if constexpr (kWide) {
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int i = 0; i < kPerRow; ++i)
          box_put4(box, lane / kPerRow + i * kAtOnce, part * kPerRow + lane % kPerRow, x[part][4 * i], x[part][4 * i + 1],
                   x[part][4 * i + 2], x[part][4 * i + 3]);
      __syncwarp();
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int i = 0; i < kPerRow; ++i)
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x[part][4 * i]), "=r"(x[part][4 * i + 1]), "=r"(x[part][4 * i + 2]), "=r"(x[part][4 * i + 3])
                       : "r"(box_piece(box, lane, part * kPerRow + i))
                       : "memory");
      __syncwarp();
    }
  }
  __device__ __forceinline__ void load_row(const Job& j, int row, int col) {
    const bool in = row < j.M && col < j.hidden;
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
  __device__ __forceinline__ void load(const Job& j, int row, int col) {
    if (row >= j.M || col >= j.hidden) return;
    const long long nb = act8::blocks_of(j.hidden);
    const uint8_t* p = j.kept_scale + static_cast<long long>(row) * 2 * nb + (col >> 7);
    s[0] = act8::scale(p[0]);
    s[1] = act8::scale(p[nb]);
  }
};

// dgate = dh up a'(gate), dup = dh a(gate), h = a(gate) up, each rounded to bf16 once: they are
// operands of the three products that follow. `k` holds the kept values of the warp's first 32
// columns; while 32 columns are worked on the next ones are on their way, at a tile's end the next
// tile's first (from row next_row0 and column next_col on): gate and up come from HBM, and a tile that
// began by waiting for them would take longer than its products.
template <int kAct, int kKept, bool kWide>
__device__ __forceinline__ void epi_glu_bwd(const Job& j, const Unit& w, const Acc& acc, int row0, int lane, int h,
                                            uint32_t box, Kept<kKept, kWide>& k, Scales& sc, int next_row0, int next_col) {
  const int width = j.tile_n >> 1;
  const int col0 = w.tj * j.tile_n + width * h;
  const Out<64> dgate(j.out, j.ld_out, 2, row0, j.M, col0, j.N, lane);
  const Out<64> dup(static_cast<uint16_t*>(j.out) + j.N, j.ld_out, 2, row0, j.M, col0, j.N, lane);
  const Out<64> hout(j.out_h, j.ld_h, 2, row0, j.M, col0, j.N, lane);
  Scales next_sc;
  if constexpr (kKept == kKeep8) next_sc.load(j, next_row0 + lane, next_col);
#pragma unroll 1
  for (int c = 0; 32 * c < width; ++c) {
    const int col = col0 + 32 * c;
    const bool last = 32 * c + 32 == width;
    uint32_t v[32];
    acc.read32(width * h + 32 * c, v);
    if (last) acc.done();
    Kept<kKept, kWide> next;
    next.load(j, last ? next_row0 : row0, last ? next_col : col + 32, lane);
    if (col < j.N && row0 < j.M) {
      k.turn(box, lane);
      uint32_t hh[16];
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // eight columns: a piece of each result
        uint32_t dg[4], du[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int p = 4 * q + i;
          const F2 g = k.two(0, p, sc.s[0]), u = k.two(1, p, sc.s[1]), d = f2(f(v[2 * p]), f(v[2 * p + 1]));
          F2 a, da;
          gate<kAct>(g, a, da);
          dg[i] = pack2(d * u * da);
          du[i] = pack2(d * a);
          hh[p] = pack2(a * u);
        }
        box_put4(box, lane, q, dg[0], dg[1], dg[2], dg[3]);  // a row's 32 dgates, then its 32 dups
        box_put4(box, lane, 4 + q, du[0], du[1], du[2], du[3]);
      }
      __syncwarp();
      dgate.put<0>(box, lane, 64 * c);
      dup.put<64>(box, lane, 64 * c);
      __syncwarp();
      box_put(box, lane, 0, hh);
      __syncwarp();
      hout.put<0>(box, lane, 64 * c);
      __syncwarp();
    }
    k = next;
  }
  sc = next_sc;
}

// ---------------------------------------------------------------------- the kernel

template <int kKinds, int kAct, int kKept, bool kWide>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    lm_gemm_kernel(const __grid_constant__ Batch B) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kStages * kHalfBytes;
  uint8_t* sEpi = sB + kStages * kHalfBytes;
  uint16_t* sSwap = reinterpret_cast<uint16_t*>(sEpi + kEpiWarps * kBoxBytes);
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
  const int total = B.start[B.n];
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
      for (int i = 0, t; ok && (t = unit_at(B, pair, npairs, i)) < total; ++i) {
        const int ji = job_of(B, t);
        const Job& j = B.job[ji];
        const Unit w = unit_of(j, t - B.start[ji]);
        const bool up = (kKinds & kGluFwd) != 0 && !leader;  // one CTA has the gate's columns, the other up's
        const CUtensorMap* const map = is_p ? &j.P : up ? &j.Up : &j.Q;
        const bool mn = (is_p ? j.a_mn : j.b_mn) != 0;
        const int width = j.tile_n >> 1;  // this CTA's columns of Q
        // this CTA's first row of P, or column of Q
        const int first = is_p                        ? w.ti * kTileM + static_cast<int>(rank) * 128
                          : (kKinds & kGluFwd) != 0 ? w.tj * width
                                                    : w.tj * j.tile_n + static_cast<int>(rank) * width;
        // (a single tile of at most 128 rows: the other rows' accumulators are of no use to anyone)
        const bool any = !is_p || leader || j.a_rows == 128, two = is_p || width == 128;
        const uint32_t tx = static_cast<uint32_t>(j.tx);
        const int k_end = w.kb1 * kTileK;
        for (int k = w.kb0 * kTileK; k < k_end; k += kTileK) {
          if (!wait(empty0 + 8 * s, ph, err)) {
            ok = false;
            break;
          }
          if (is_p && leader) tc::mbar_arrive_expect_tx(full + s, tx);  // both operands' bytes, both CTAs'
          const uint32_t bar = lead0 + 8 * s, to = s0 + s * kHalfBytes;
          if (!mn) {
            if (any) load_box(to, map, bar, k, first);
          } else {
            load_box(to, map, bar, first, k);
            if (two) load_box(to + kMnBoxBytes, map, bar, first + 64, k);
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
      for (int t; ok && (t = unit_at(B, pair, npairs, it)) < total; ++it) {
        const int ji = job_of(B, t);
        const Job& j = B.job[ji];
        const Unit w = unit_of(j, t - B.start[ji]);
        const bool amn = j.a_mn != 0, bmn = j.b_mn != 0;
        const uint32_t idesc = tc::idesc_bf16_f32(kTileM, j.tile_n, amn, bmn);
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
    const uint32_t box = tc::smem_u32(sEpi) + (warp - kFirstEpi) * kBoxBytes;
    uint16_t* swap = sSwap + 64 * quad;
    const int rows0 = static_cast<int>(rank) * 128 + 32 * quad;  // this warp's rows within a tile
    Kept<kKept, kWide> kept;
    Scales scales;
    auto first_of = [&](int t, int& row, int& col) {  // the warp's first row and column of unit t (kGluBwd)
      row = B.job[0].M, col = 0;
      if (t >= total) return;
      const Unit w = unit_of(B.job[0], t);
      row = w.ti * kTileM + rows0;
      col = w.tj * B.job[0].tile_n + (B.job[0].tile_n >> 1) * half;
    };
    if constexpr ((kKinds & kGluBwd) != 0) {
      int row, col;
      first_of(unit_at(B, pair, npairs, 0), row, col);
      kept.load(B.job[0], row, col, lane);
      if constexpr (kKept == kKeep8) scales.load(B.job[0], row + lane, col);
    }
    int it = 0;
    for (int t; (t = unit_at(B, pair, npairs, it)) < total;) {
      const int b = it & 1;
      const uint32_t tph = static_cast<uint32_t>(it >> 1) & 1u;
      ++it;
      const int ji = job_of(B, t);
      const Job& j = B.job[ji];
      const Unit w = unit_of(j, t - B.start[ji]);
      const int row0 = w.ti * kTileM + rows0;
      int ok = 1;
      if (lane == 0) ok = wait(tc::smem_u32(tfull + b), tph, err) ? 1 : 0;
      ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
      // Two warps wait for one another within such a tile: if one's wait has run out, neither begins it.
      if constexpr ((kKinds & kGluFwd) != 0 && kKept == kKeep8) ok = both_warps(ok, 1 + quad);
      if (!ok) {
        if (lane == 0) tell_pair(gave_up);
        break;
      }
      tc::fence_after_sync();
      const Acc acc{tmem + (static_cast<uint32_t>(32 * quad) << 16) + static_cast<uint32_t>(b * kTileN), tempty_leader[b], lane};
      if ((kKinds & kStore) && j.kind == kStore) epi_store(j, w, acc, row0, lane, half, box);
      if ((kKinds & kCeFwd) && j.kind == kCeFwd) epi_ce_fwd(j, w, acc, row0, lane, half);
      if ((kKinds & kCeBwd) && j.kind == kCeBwd) epi_ce_bwd(j, w, acc, row0, lane, half, box);
      if constexpr ((kKinds & kGluFwd) != 0) epi_glu_fwd<kAct, kKept>(j, w, acc, row0, lane, half, box, swap, 1 + quad);
      if constexpr ((kKinds & kGluBwd) != 0) {
        int row, col;
        first_of(unit_at(B, pair, npairs, it), row, col);
        epi_glu_bwd<kAct, kKept, kWide>(j, w, acc, row0, lane, half, box, kept, scales, row, col);
      }
    }
  }
  tc::fence_before_sync();
  tc::cluster_sync();  // every MMA, copy and remote arrival of the pair is done
  if (*reinterpret_cast<volatile uint32_t*>(gave_up) != 0) settle();
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc_pair(tmem, 2 * kTileN);
  }
}

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

template <int kKinds, int kAct = 0, int kKept = kKeepNone, bool kWide = true>
zopt_status launch_kinds(Batch& b, dim3 grid, cudaStream_t s) {
  const auto kernel = lm_gemm_kernel<kKinds, kAct, kKept, kWide>;
  ZOPT_CUDA_TRY(once_per_device([=] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes); }));
  return launch_pdl(kernel, grid, dim3(kThreads), static_cast<size_t>(kSmemBytes), s, b);
}
template <int kAct>
zopt_status launch_glu(Batch& b, dim3 grid, cudaStream_t s) {
  const Job& j = b.job[0];
  if (j.kind == kGluFwd) {
    if (j.kept_mode == kKeepNone) return launch_kinds<kGluFwd, kAct>(b, grid, s);
    return j.kept_mode == kKeep8 ? launch_kinds<kGluFwd, kAct, kKeep8>(b, grid, s)
                                 : launch_kinds<kGluFwd, kAct, kKeepBf16>(b, grid, s);
  }
  const int size = j.kept_mode == kKeep8 ? 1 : 2;
  const bool wide = aligned16(j.kept) && j.ld_kept * size % 16 == 0 && static_cast<long long>(j.hidden) * size % 16 == 0;
  if (j.kept_mode == kKeep8)
    return wide ? launch_kinds<kGluBwd, kAct, kKeep8>(b, grid, s) : launch_kinds<kGluBwd, kAct, kKeep8, false>(b, grid, s);
  return wide ? launch_kinds<kGluBwd, kAct, kKeepBf16>(b, grid, s) : launch_kinds<kGluBwd, kAct, kKeepBf16, false>(b, grid, s);
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
    case kStore: return launch_kinds<kStore>(b, grid, s);
    case kCeFwd: return launch_kinds<kCeFwd>(b, grid, s);
    case kStore | kCeBwd: return launch_kinds<kStore | kCeBwd>(b, grid, s);
    case kGluFwd:
    case kGluBwd:
      return b.job[0].act == ZOPT_ACT_GELU ? launch_glu<ZOPT_ACT_GELU>(b, grid, s) : launch_glu<ZOPT_ACT_SILU>(b, grid, s);
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
