// The products of the training operators on tcgen05 tensor cores: one persistent CTA-pair kernel
// over a batch of jobs (lm_gemm.cuh), its host launcher, the sum of split products and the copy
// that stages operands.
//
// A cluster of two CTAs computes a 256 x 256 tile with tcgen05.mma.cta_group::2: each CTA holds its
// 128 rows of P and its 128 columns of Q, so a 64-deep k-block brings 32 KiB per SM and the ring
// holds six stages. Warp 0 of each CTA streams the operands by TMA (all complete on the leader's
// stage barrier), one thread of the leader issues the M=256, N=256, K=16 MMAs into one of two TMEM
// accumulators, and eight epilogue warps (two per quarter of the TMEM lanes, each 128 of the 256
// columns) turn the other accumulator into the operator's outputs meanwhile. A lane holds whole
// row pieces, so softmax statistics and the 8-bit blocks need no exchange between lanes.
#include <cuda_fp16.h>

#include <cmath>
#include <cudaTypedefs.h>

#include <string>

#include "act8.cuh"
#include "launch.cuh"
#include "lm_gemm.cuh"
#include "ns_internal.h"
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

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Row `lane` of a 32 x 32 bf16 box under the 64-byte swizzle: row r at 64 r, its 16-byte piece q at
// piece q ^ ((r >> 1) & 3).
__device__ __forceinline__ void box_row(uint8_t* box, int lane, const float (&o)[32]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint4 u;
    u.x = pack2(o[8 * q + 0], o[8 * q + 1]);
    u.y = pack2(o[8 * q + 2], o[8 * q + 3]);
    u.z = pack2(o[8 * q + 4], o[8 * q + 5]);
    u.w = pack2(o[8 * q + 6], o[8 * q + 7]);
    *reinterpret_cast<uint4*>(box + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) = u;
  }
}

// Hands a warp's output boxes to the TMA in turn: a box is written again only when the store that
// read it kBoxes stores earlier has finished reading.
struct Boxes {
  uint8_t* mine;
  int next;
  __device__ __forceinline__ void store(const CUtensorMap* m, int lane, const float (&o)[32], int col, int row) {
    uint8_t* box = mine + next * kBoxBytes;
    if (lane == 0) tc::bulk_wait_read<kBoxes - 1>();
    __syncwarp();
    box_row(box, lane, o);
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tc::tma_store_2d(m, box, col, row);
      tc::bulk_commit();
    }
    next = next + 1 == kBoxes ? 0 : next + 1;
  }
};

// 32 values to a row of bf16 in global memory, columns beyond n left out.
__device__ __forceinline__ void put_bf16(__nv_bfloat16* p, const float (&o)[32], int n) {
  if (n >= 32 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      reinterpret_cast<uint4*>(p)[q] = make_uint4(pack2(o[8 * q], o[8 * q + 1]), pack2(o[8 * q + 2], o[8 * q + 3]),
                                                  pack2(o[8 * q + 4], o[8 * q + 5]), pack2(o[8 * q + 6], o[8 * q + 7]));
  } else {
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (k < n) p[k] = __float2bfloat16_rn(o[k]);
  }
}

__device__ __forceinline__ void ld32(uint32_t taddr, float (&o)[32]) {
  uint32_t v[32];
  tc::tmem_ld32(taddr, v);
  tc::tmem_wait_ld();
#pragma unroll
  for (int k = 0; k < 32; ++k) o[k] = __uint_as_float(v[k]);
}

// A unit of work: one tile of one job over one run of k-blocks.
struct Unit {
  int ti, tj, split, kb0, kb1;
};
__device__ __forceinline__ Unit unit_of(const Job& j, int u) {
  Unit w;
  w.split = u / j.tiles;
  u -= w.split * j.tiles;
  if (j.rows_fast) {
    w.tj = u / j.tiles_m;
    w.ti = u - w.tj * j.tiles_m;
  } else {
    w.ti = u / j.tiles_n;
    w.tj = u - w.ti * j.tiles_n;
  }
  w.kb0 = w.split * j.kb_per_split;
  w.kb1 = min(w.kb0 + j.kb_per_split, j.nk);
  return w;
}
__device__ __forceinline__ int job_of(const Batch& b, int t) {
  int j = 0;
  while (j + 1 < b.n && t >= b.start[j + 1]) ++j;
  return j;
}

// True in one lane of a converged warp. The copies and MMAs take their operands from uniform
// registers: behind this predicate the compiler knows that one thread issues them, behind a
// comparison of lanes it has to issue them lane by lane (680 against 521 cycles a k-block of 8192^3, whose MMAs
// take 512).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// A bounded wait for an mbarrier (given by its shared-memory address) that costs the two threads
// feeding the tensor cores as little as a wait can: the clock and the error word (in host memory)
// are only looked at every 256th failed try. Each try may sleep in the hardware until the phase
// completes.
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_slow(uint32_t bar, uint32_t parity, int* err) {
  unsigned long long t0 = 0;
  for (uint32_t spin = 1;; ++spin) {
    if (try_wait(bar, parity)) return true;
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
  return try_wait(bar, parity) || wait_slow(bar, parity, err);
}
// The same without an error to report or heed: for copies and products that must have ended before
// their memory is given up.
__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity) { wait(bar, parity, nullptr); }

__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap* m, uint32_t bar_cluster, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, "
      "%4}], [%2];" ::"r"(dst),
      "l"(m), "r"(bar_cluster), "r"(c0), "r"(c1)
      : "memory");
}

// a(z) = z s(phi(z)) with the logistic s: phi = z (SiLU), or 2 sqrt(2/pi) (z + 0.044715 z^3), which
// is the tanh form of GELU since (1 + tanh y) / 2 = s(2 y). Beyond |z| = 64 s is 0 or 1 and phi's
// derivative no longer matters: z is held there inside phi so that no infinity meets a zero.
__device__ __forceinline__ void gate_of(int act, float z, float& a, float& da) {
  float phi = z, dphi = 1.0f;
  if (act == ZOPT_ACT_GELU) {
    const float c = 1.5957691216057308f;
    const float zc = fminf(fmaxf(z, -64.0f), 64.0f), z2 = zc * zc;
    phi = c * zc * (1.0f + 0.044715f * z2);
    dphi = c * (1.0f + 0.134145f * z2);
  }
  const float s = __fdividef(1.0f, 1.0f + ex2(-kLog2e * phi));
  a = z * s;
  da = s + a * (1.0f - s) * dphi;
}

// ---------------------------------------------------------------------- epilogues
//
// Each turns one warp's part of a tile into outputs: TMEM address `acc` (this warp's 32 lanes, the
// tile's column 0), row = the lane's row of D, row0 = the warp's first, h = which half of the
// tile's columns.

__device__ __forceinline__ void epi_store(const Job& j, const Unit& w, uint32_t acc, int row0, int lane, int h,
                                          Boxes& boxes) {
  const int row = row0 + lane;
  const float alpha = j.alpha != nullptr && j.splits == 1 ? __ldcg(j.alpha) : 1.0f;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    const int col = w.tj * kTileN + 128 * h + 32 * c;
    if (col >= j.N || row0 >= j.M) break;  // (warp-uniform)
    float o[32];
    ld32(acc + static_cast<uint32_t>(128 * h + 32 * c), o);
    if (j.add != nullptr && row < j.M) {
      const float* a = j.add + static_cast<long long>(row) * j.ld_add + col;
      if (col + 32 <= j.N) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float4 v = reinterpret_cast<const float4*>(a)[q];
          o[4 * q] += v.x, o[4 * q + 1] += v.y, o[4 * q + 2] += v.z, o[4 * q + 3] += v.w;
        }
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (col + k < j.N) o[k] += a[k];
      }
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) o[k] *= alpha;
    if (j.out_mode == kOutTma) {
      boxes.store(&j.D0, lane, o, col, row0);
    } else if (row < j.M) {
      const long long off = static_cast<long long>(row) * j.ld_out + col;
      if (j.out_mode == kOutBf16) {
        put_bf16(static_cast<__nv_bfloat16*>(j.out) + off, o, j.N - col);
      } else {
        float* p = static_cast<float*>(j.out) + w.split * j.split_stride + off;
        if (col + 32 <= j.N) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            reinterpret_cast<float4*>(p)[q] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (col + k < j.N) p[k] = o[k];
        }
      }
    }
  }
}

// The running maximum m and sum s = sum 2^(x - m) of the row's 128 logits times log2(e), one pass.
// Columns beyond the vocabulary take no part; an all -inf row keeps m = -inf, s = 0.
__device__ __forceinline__ void epi_ce_fwd(const Job& j, const Unit& w, uint32_t acc, int row0, int lane, int h) {
  const int row = row0 + lane;
  if (row0 >= j.M) return;
  const long long tgt = row < j.M ? j.target[row] : -1;
  float m = -INFINITY, s = 0.0f;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    const int col = w.tj * kTileN + 128 * h + 32 * c;
    if (col >= j.N) break;
    float o[32];
    ld32(acc + static_cast<uint32_t>(128 * h + 32 * c), o);
    if (tgt >= col && tgt < col + 32 && tgt < j.N) {
      float t = 0.0f;
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (col + k == tgt) t = o[k];
      j.tlogit[row] = t;
    }
    if (col + 32 > j.N) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (col + k >= j.N) o[k] = -INFINITY;
    }
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < 32; ++k) top = fmaxf(top, o[k]);
    const float mn = fmaxf(m, top * kLog2e);
    const float base = mn == -INFINITY ? 0.0f : mn;
    float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      t0 += ex2(fmaf(o[k], kLog2e, -base));
      t1 += ex2(fmaf(o[k + 1], kLog2e, -base));
    }
    s = fmaf(s, ex2(m - base), t0 + t1);
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
__device__ __forceinline__ void epi_ce_bwd(const Job& j, const Unit& w, uint32_t acc, int row0, int lane, int h,
                                           Boxes& boxes) {
  const int row = row0 + lane;
  if (row0 >= j.M) return;
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
  for (int c = 0; c < 4; ++c) {
    const int col = w.tj * kTileN + 128 * h + 32 * c;
    if (col >= j.N) break;
    float o[32];
    ld32(acc + static_cast<uint32_t>(128 * h + 32 * c), o);
#pragma unroll
    for (int k = 0; k < 32; ++k) o[k] = ex2(fmaf(o[k], kLog2e, -lse2));
    if (at >= col && at < col + 32) {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (col + k == at) o[k] -= 1.0f;
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) o[k] = live ? o[k] * dl : 0.0f;
    boxes.store(&j.D0, lane, o, col, row0);
  }
}

// TMEM columns 0 .. 127 hold the gate, 128 .. 255 the up product of the same 128 hidden columns.
// Warp half h makes h's columns 64 h .. 64 h + 63 and, where 8 bits are kept, the whole block of
// the gate (half 0) or of up (half 1): a tile is one block wide, so a block's largest magnitude is
// found within a lane.
__device__ __forceinline__ void epi_glu_fwd(const Job& j, const Unit& w, uint32_t acc, int row0, int lane, int h,
                                            Boxes& boxes) {
  const int row = row0 + lane;
  if (row0 >= j.M) return;
  const int n0 = w.tj * 128;
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    const int off = 64 * h + 32 * c, col = n0 + off;
    if (col >= j.N) break;
    float g[32], u[32];
    ld32(acc + static_cast<uint32_t>(off), g);
    ld32(acc + static_cast<uint32_t>(128 + off), u);
    if (j.kept_mode == kKeepTma) {
      boxes.store(&j.D1, lane, g, col, row0);
      boxes.store(&j.D2, lane, u, col, row0);
    } else if (j.kept_mode == kKeepBf16 && row < j.M) {
      __nv_bfloat16* p = static_cast<__nv_bfloat16*>(j.kept) + static_cast<long long>(row) * j.ld_kept + col;
      put_bf16(p, g, j.hidden - col);
      put_bf16(p + j.hidden, u, j.hidden - col);
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      float a, da;
      gate_of(j.act, g[k], a, da);
      u[k] *= a;
    }
    boxes.store(&j.D0, lane, u, col, row0);
  }
  if (j.kept_mode == kKeep8) {
    const int width = min(128, j.hidden - n0);
    float amax = 0.0f;
#pragma unroll 1
    for (int c = 0; 32 * c < width; ++c) {
      float o[32];
      ld32(acc + static_cast<uint32_t>(128 * h + 32 * c), o);
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (32 * c + k < width) amax = act8::amax_step(amax, o[k]);
    }
    const uint32_t e = act8::exponent_byte(amax);
    const float inv = act8::inv_scale(e);
    const long long nb = act8::blocks_of(j.hidden);
    if (row < j.M) j.kept_scale[static_cast<long long>(row) * 2 * nb + h * nb + w.tj] = static_cast<uint8_t>(e);
    uint8_t* p = static_cast<uint8_t*>(j.kept) + static_cast<long long>(row) * j.ld_kept + static_cast<long long>(h) * j.hidden + n0;
#pragma unroll 1
    for (int c = 0; 32 * c < width; ++c) {
      float o[32];
      ld32(acc + static_cast<uint32_t>(128 * h + 32 * c), o);
      if (row >= j.M) continue;
      uint32_t v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = act8::encode4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3], inv);
      uint8_t* d = p + 32 * c;
      if (32 * c + 32 <= width && (reinterpret_cast<uintptr_t>(d) & 15u) == 0) {
        reinterpret_cast<uint4*>(d)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4*>(d)[1] = make_uint4(v[4], v[5], v[6], v[7]);
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k)
          if (32 * c + k < width) d[k] = static_cast<uint8_t>(v[k >> 2] >> (8 * (k & 3)));
      }
    }
  }
}

// 32 kept values of one row (zero beyond n columns).
__device__ __forceinline__ void kept32(const Job& j, long long row, int col, int part, int n, float (&o)[32]) {
  if (j.kept_mode == kKeep8) {
    const uint8_t* p = static_cast<const uint8_t*>(j.kept) + row * j.ld_kept + static_cast<long long>(part) * j.hidden + col;
    const long long nb = act8::blocks_of(j.hidden);
    const float sc = act8::scale(j.kept_scale[row * 2 * nb + part * nb + (col >> 7)]);
    uint32_t v[8];
    if (n >= 32 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
      const uint4 a = __ldg(reinterpret_cast<const uint4*>(p)), b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        v[q] = 0;
#pragma unroll
        for (int t = 0; t < 4; ++t)
          if (4 * q + t < n) v[q] |= static_cast<uint32_t>(p[4 * q + t]) << (8 * t);
      }
    }
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const float2 f = act8::decode2(v[q >> 1] >> (16 * (q & 1)), sc);
      o[2 * q] = f.x;
      o[2 * q + 1] = f.y;
    }
  } else {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(j.kept) + row * j.ld_kept + static_cast<long long>(part) * j.hidden + col;
    if (n >= 32 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 a = __ldg(reinterpret_cast<const uint4*>(p) + q);
        const uint32_t x[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          o[8 * q + 2 * t] = __uint_as_float(x[t] << 16);
          o[8 * q + 2 * t + 1] = __uint_as_float(x[t] & 0xFFFF0000u);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < 32; ++k) o[k] = k < n ? __bfloat162float(p[k]) : 0.0f;
    }
  }
}

// dgate = dh up a'(gate), dup = dh a(gate), h = a(gate) up, each rounded to bf16 once: they are
// operands of the three products that follow.
__device__ __forceinline__ void epi_glu_bwd(const Job& j, const Unit& w, uint32_t acc, int row0, int lane, int h,
                                            Boxes& boxes) {
  const int row = row0 + lane;
  if (row0 >= j.M) return;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    const int col = w.tj * kTileN + 128 * h + 32 * c;
    if (col >= j.N) break;
    float g[32], u[32], d[32];
    const int n = row < j.M ? j.hidden - col : 0;
    kept32(j, row < j.M ? row : 0, col < j.hidden ? col : 0, 0, n, g);
    kept32(j, row < j.M ? row : 0, col < j.hidden ? col : 0, 1, n, u);
    ld32(acc + static_cast<uint32_t>(128 * h + 32 * c), d);
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      float a, da;
      gate_of(j.act, g[k], a, da);
      g[k] = d[k] * u[k] * da;
      d[k] *= a;
      u[k] *= a;
    }
    boxes.store(&j.D0, lane, g, col, row0);
    boxes.store(&j.D1, lane, d, col, row0);
    boxes.store(&j.D2, lane, u, col, row0);
  }
}

// ---------------------------------------------------------------------- the kernel

template <int kKinds>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    lm_gemm_kernel(const __grid_constant__ Batch B) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + kStages * kHalfBytes;
  uint8_t* sEpi = sB + kStages * kHalfBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(sEpi + kEpiWarps * kBoxes * kBoxBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drain + 1);

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
    tc::fence_mbar_init();
    for (int j = 0; j < B.n; ++j) {
      tc::prefetch_tmap(&B.job[j].P);
      tc::prefetch_tmap(&B.job[j].Q);
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
  if (warp == 0) {
    if (elect_one()) {
      // ---------------------------------------------------------------- TMA producer (both CTAs)
      // Every cycle of this loop counts: a k-block takes the MMAs 512 cycles, and the thread has to
      // wait for a stage, arm it and issue two to four loads in less. So everything that a job fixes
      // is in registers before its k-loop.
      const uint32_t a0 = tc::smem_u32(sA), b0 = tc::smem_u32(sB);
      const uint32_t lead0 = tc::map_to_rank(full0, 0);  // all loads complete on the leader's barriers
      uint32_t s = 0, ph = 1;
      long long done = 0;  // stages armed so far
      bool ok = true;
      for (int t = pair; ok && t < total; t += npairs) {
        const int ji = job_of(B, t);
        const Job& j = B.job[ji];
        const Unit w = unit_of(j, t - B.start[ji]);
        const CUtensorMap* const P = &j.P;
        const CUtensorMap* const Q = &j.Q;
        const bool amn = j.a_mn != 0, bmn = j.b_mn != 0;
        const int row0 = w.ti * kTileM + static_cast<int>(rank) * 128;  // this CTA's rows of P
        int col0 = w.tj * kTileN + static_cast<int>(rank) * 128;        // this CTA's columns of Q
        if ((kKinds & kGluFwd) && j.kind == kGluFwd) col0 = w.tj * 128 + (leader ? 0 : j.q_up);
        const int k_end = w.kb1 * kTileK;
        for (int k = w.kb0 * kTileK; k < k_end; k += kTileK) {
          if (!wait(empty0 + 8 * s, ph, err)) {
            ok = false;
            break;
          }
          if (leader) tc::mbar_arrive_expect_tx(full + s, 4 * kHalfBytes);  // both CTAs' halves of P and Q
          const uint32_t bar = lead0 + 8 * s, a = a0 + s * kHalfBytes, b = b0 + s * kHalfBytes;
          if (!amn) {
            load_box(a, P, bar, k, row0);
          } else {
            load_box(a, P, bar, row0, k);
            load_box(a + kMnBoxBytes, P, bar, row0 + 64, k);
          }
          if (!bmn) {
            load_box(b, Q, bar, k, col0);
          } else {
            load_box(b, Q, bar, col0, k);
            load_box(b + kMnBoxBytes, Q, bar, col0 + 64, k);
          }
          ++done;
          if (++s == kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok && leader) {  // the leader's stage barriers count both CTAs' copies: leave none in flight
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
      for (int t = pair; ok && t < total; t += npairs, ++it) {
        const int ji = job_of(B, t);
        const Job& j = B.job[ji];
        const Unit w = unit_of(j, t - B.start[ji]);
        const bool amn = j.a_mn != 0, bmn = j.b_mn != 0;
        const uint32_t idesc = tc::idesc_bf16_f32(kTileM, kTileN, amn, bmn);
        // a stage's descriptors differ in the address alone (16-byte units), and so do a stage's steps
        const uint64_t ad0 = tc::smem_desc_sw128(tc::smem_u32(sA), amn ? kMnBoxBytes : 16u, 1024u);
        const uint64_t bd0 = tc::smem_desc_sw128(tc::smem_u32(sB), bmn ? kMnBoxBytes : 16u, 1024u);
        const uint32_t astep = amn ? 128u : 2u, bstep = bmn ? 128u : 2u;
        const int b = it & 1;
        const uint32_t tph = static_cast<uint32_t>(it >> 1) & 1u;
        if (!wait(tempty0 + 8 * b, tph ^ 1u, err)) {
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
      tc::umma_commit_pair(drain, 1);
      wait_drain(tc::smem_u32(drain), 0);
    }
  } else {
    // ------------------------------------------------------------------ epilogue (warps 2..9)
    const int quad = warp & 3;          // this warp may read TMEM lanes [32 quad, 32 quad + 32)
    const int half = (warp - 2) >> 2;   // and takes this half of the columns
    const uint32_t tempty_leader[2] = {tc::map_to_rank(tc::smem_u32(tempty), 0),
                                       tc::map_to_rank(tc::smem_u32(tempty + 1), 0)};
    Boxes boxes{sEpi + (warp - 2) * kBoxes * kBoxBytes, 0};
    int it = 0;
    for (int t = pair; t < total; t += npairs, ++it) {
      const int b = it & 1;
      const uint32_t tph = static_cast<uint32_t>(it >> 1) & 1u;
      int ok = 1;
      if (lane == 0) ok = tc::mbar_wait_idle(tfull + b, tph, err) ? 1 : 0;
      if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) break;
      tc::fence_after_sync();
      const int ji = job_of(B, t);
      const Job& j = B.job[ji];
      const Unit w = unit_of(j, t - B.start[ji]);
      const uint32_t acc = tmem + (static_cast<uint32_t>(32 * quad) << 16) + static_cast<uint32_t>(b * kTileN);
      const int row0 = w.ti * kTileM + static_cast<int>(rank) * 128 + 32 * quad;
      if ((kKinds & kStore) && j.kind == kStore) epi_store(j, w, acc, row0, lane, half, boxes);
      if ((kKinds & kCeFwd) && j.kind == kCeFwd) epi_ce_fwd(j, w, acc, row0, lane, half);
      if ((kKinds & kCeBwd) && j.kind == kCeBwd) epi_ce_bwd(j, w, acc, row0, lane, half, boxes);
      if ((kKinds & kGluFwd) && j.kind == kGluFwd) epi_glu_fwd(j, w, acc, row0, lane, half, boxes);
      if ((kKinds & kGluBwd) && j.kind == kGluBwd) epi_glu_bwd(j, w, acc, row0, lane, half, boxes);
      tc::fence_before_sync();
      __syncwarp();  // every lane's TMEM reads are done: one arrival releases the warp's part
      if (lane == 0) tc::mbar_arrive_cluster(tempty_leader[b]);
    }
    if (lane == 0) tc::bulk_wait_all();  // every store has reached global memory
    __syncwarp();
  }
  tc::fence_before_sync();
  tc::cluster_sync();  // every MMA, copy and remote arrival of the pair is done
  if (warp == 1) {
    tc::fence_after_sync();
    tc::tmem_dealloc_pair(tmem, 2 * kTileN);
  }
}

// Partial sums added in split order, so a call's result does not depend on which pair ran when.
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

template <int kKinds>
zopt_status launch_kinds(Batch& b, dim3 grid, cudaStream_t s) {
  ZOPT_CUDA_TRY(once([] {
    return cudaFuncSetAttribute(lm_gemm_kernel<kKinds>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  }));
  return launch_pdl(lm_gemm_kernel<kKinds>, grid, dim3(kThreads), static_cast<size_t>(kSmemBytes), s, b);
}

}  // namespace

unsigned blocks_for(long long items, int sms) {
  const long long want = (items + 255) / 256, most = 8LL * sms;
  return static_cast<unsigned>(want < 1 ? 1 : (want < most ? want : most));
}

// ---------------------------------------------------------------------- host side

zopt_status make_map(const char* fn, CUtensorMap* m, const void* base, long long inner, long long outer,
                     long long pitch, int box_inner, int box_outer) {
  auto enc = ns::encode_fn();
  if (enc == nullptr) return fail(ZOPT_ECUDA, std::string(fn) + ": cuTensorMapEncodeTiled is unavailable");
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch) * 2};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_inner), static_cast<cuuint32_t>(box_outer)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                         CU_TENSOR_MAP_INTERLEAVE_NONE,
                         box_inner == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(ZOPT_ECUDA, std::string(fn) + ": cuTensorMapEncodeTiled failed (" + std::to_string(r) + ")");
  return ok();
}

zopt_status map_operand(const char* fn, CUtensorMap* m, const void* base, long long mn, long long k, long long pitch,
                        bool mn_major) {
  return mn_major ? make_map(fn, m, base, mn, k, pitch, 64, 64) : make_map(fn, m, base, k, mn, pitch, 64, 128);
}

zopt_status map_output(const char* fn, CUtensorMap* m, void* base, long long rows, long long cols, long long pitch) {
  return make_map(fn, m, base, cols, rows, pitch, 32, 32);
}

void set_tiles(Job& j) {
  const int width = j.kind == kGluFwd ? 128 : kTileN;
  j.tiles_m = (j.M + kTileM - 1) / kTileM;
  j.tiles_n = (j.N + width - 1) / width;
  j.nk = (j.K + kTileK - 1) / kTileK;
  j.kb_per_split = j.nk;
  j.splits = 1;
  // The larger operand is streamed once: tiles that run together share its rows (or columns) and
  // walk the smaller one, which stays in L2.
  j.rows_fast = j.N >= j.M ? 1 : 0;
}

void plan_splits(Job* jobs, int n) {
  // GB300's 76 CTA pairs. Fewer than four k-blocks a unit is not worth a partial sum.
  constexpr long long kPairs = 76, kLeast = 4;
  long long work = 0;
  for (int i = 0; i < n; ++i) work += static_cast<long long>(jobs[i].tiles_m) * jobs[i].tiles_n * jobs[i].nk;
  const long long share = (work + kPairs - 1) / kPairs;
  const long long run = share < kLeast ? kLeast : share;
  for (int i = 0; i < n; ++i) {
    Job& j = jobs[i];
    if (j.kind != kStore || j.whole || j.nk <= run) continue;
    j.kb_per_split = static_cast<int>(run);
    j.splits = (j.nk + j.kb_per_split - 1) / j.kb_per_split;
  }
}

zopt_status launch(const char* fn, Batch& b, int kinds, cudaStream_t s) {
  long long total = 0;
  for (int i = 0; i < b.n; ++i) {
    Job& j = b.job[i];
    const long long tiles = static_cast<long long>(j.tiles_m) * j.tiles_n;
    const long long units = tiles * j.splits;
    if (tiles < 1 || total + units > 0x7FFFFFFFLL) return fail(ZOPT_EINVAL, std::string(fn) + ": too many tiles");
    j.tiles = static_cast<int>(tiles);
    b.start[i] = static_cast<int>(total);
    total += units;
  }
  b.start[b.n] = static_cast<int>(total);
  const int sms = sm_count();
  if (sms < 2) return fail(ZOPT_ECUDA, std::string(fn) + ": no CUDA device");
  const long long pairs = total < sms / 2 ? total : sms / 2;
  const dim3 grid(static_cast<unsigned>(2 * pairs));
  switch (kinds) {
    case kStore: return launch_kinds<kStore>(b, grid, s);
    case kCeFwd: return launch_kinds<kCeFwd>(b, grid, s);
    case kStore | kCeBwd: return launch_kinds<kStore | kCeBwd>(b, grid, s);
    case kGluFwd: return launch_kinds<kGluFwd>(b, grid, s);
    case kGluBwd: return launch_kinds<kGluBwd>(b, grid, s);
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
