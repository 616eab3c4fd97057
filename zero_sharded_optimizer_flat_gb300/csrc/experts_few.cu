// The experts' forward for a few slots, bound by the bytes of the weights that they choose.
//
// As ffn_few.cu has it for a dense block, a slot in a token's place: nothing has to be sorted, each
// slot's products are sums of its expert's weight rows on the CUDA cores, in fp32 throughout.
//   1. gate and up:  partial[s][slot] = x[k in s] gate_up[k in s];
//   2. down: a CTA adds up the parts of its 128 hidden columns (one 8-bit block), forms h with the
//      slot's weight (and keeps what is to be kept), and writes partial[block][slot] = h[block] down[block];
//      its weights are on their way to L2 while it waits for the first launch;
//   3. y = the sum of a token's slots' parts.
// Everything is added in a fixed order. A slot without an expert reads and writes nothing. An expert that
// several slots name is read for each, from L2 as a rule.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "act8.cuh"
#include "experts_few.h"
#include "f2.cuh"
#include "few.cuh"
#include "launch.cuh"
#include "per_device.h"
#include "tc.cuh"

namespace zopt {
namespace few {
namespace {

struct Slots {
  const int32_t* index;
  const float* weight;
  int experts, top_k;
};

// slot's expert, or -1
__device__ __forceinline__ int expert_of(const Slots& s, int slot) {
  const int e = s.index[slot];
  return e >= 0 && e < s.experts ? e : -1;
}

__global__ void __launch_bounds__(kThreads, 2) expert_gate_up_kernel(Matrix m, long long stride, const Slots slots, const uint16_t* x,
                                                                     long long ld_x, int share, float* partial) {
  extern __shared__ float red[];  // [kWarps][kCols]
  __shared__ float xs[kRows];
  // Whatever wrote the weights, x or the routing has ended before the launch that follows may start.
  tc::pdl_wait();
  tc::pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slot = blockIdx.z;
  const int e = expert_of(slots, slot);
  if (e < 0) return;
  m.w += e * stride;
  const long long n0 = static_cast<long long>(blockIdx.x) * kCols, col = n0 + 8 * lane;
  const long long k0 = static_cast<long long>(blockIdx.y) * share, k1 = min(m.rows, k0 + share);
  const __nv_bfloat16* const row = reinterpret_cast<const __nv_bfloat16*>(x) + slot / slots.top_k * ld_x;
  F2 acc[1][4];
#pragma unroll
  for (int q = 0; q < 4; ++q) acc[0][q] = f2(0.0f, 0.0f);
  for (long long c = k0; c < k1; c += kRows) {
    const int n = static_cast<int>(min(static_cast<long long>(kRows), k1 - c));
    __syncthreads();
    for (int k = threadIdx.x; k < n; k += kThreads) xs[k] = __bfloat162float(row[c + k]);
    __syncthreads();
    add_rows<1>(m, c, n, col, xs, warp, acc);
  }
  join_warps<1>(acc, red, 1, n0, m.cols, partial + (static_cast<long long>(blockIdx.y) * gridDim.z + slot) * m.cols, warp, lane);
}

template <int kAct>
__global__ void __launch_bounds__(kThreads, 2) expert_down_kernel(Matrix m, long long stride, const Slots slots, const float* parts,
                                                                  int splits, const Keep keep, float* partial) {
  extern __shared__ float red[];  // [kWarps][kCols]
  __shared__ float hs[kBlock];
  __shared__ float top[2][4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slot = blockIdx.z;
  const int e = expert_of(slots, slot);  // (written before the launch before this one began its work)
  const long long n0 = static_cast<long long>(blockIdx.x) * kCols, col = n0 + 8 * lane;
  const long long F = m.rows, k0 = static_cast<long long>(blockIdx.y) * kBlock;
  const int n = static_cast<int>(min(static_cast<long long>(kBlock), F - k0));
  const int i = threadIdx.x & 127, group = threadIdx.x >> 7;
  if (e >= 0) m.w += e * stride;
  if (e >= 0 && i < n && n0 + 64 * group < m.cols)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(m.w + (k0 + i) * m.ld + n0 + 64 * group));
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  if (e < 0) return;
  const long long f = k0 + i, all = static_cast<long long>(gridDim.z) * 2 * F;
  if (group == 0) {
    const bool in = i < n;
    float g = 0.0f, u = 0.0f;
    if (in) {
      const float* p = parts + slot * 2 * F + f;
#pragma unroll 8
      for (int s = 0; s < splits; ++s) {
        g += __ldcg(p + s * all);
        u += __ldcg(p + s * all + F);
      }
    }
    if (blockIdx.x == 0 && keep.mode == 1 && in) {
      uint16_t* q = static_cast<uint16_t*>(keep.kept) + slot * keep.ld + f;
      q[0] = __bfloat16_as_ushort(__float2bfloat16_rn(g));
      q[F] = __bfloat16_as_ushort(__float2bfloat16_rn(u));
    }
    if (blockIdx.x == 0 && keep.mode == 2) {
      float a = act8::amax_step(0.0f, g), b = act8::amax_step(0.0f, u);
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) {
        a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, d));
        b = fmaxf(b, __shfl_xor_sync(0xFFFFFFFFu, b, d));
      }
      if (lane == 0) top[0][warp] = a, top[1][warp] = b;
      asm volatile("bar.sync 1, 128;" ::: "memory");  // (this group's four warps)
      const uint32_t eg = act8::exponent_byte(fmaxf(fmaxf(top[0][0], top[0][1]), fmaxf(top[0][2], top[0][3])));
      const uint32_t eu = act8::exponent_byte(fmaxf(fmaxf(top[1][0], top[1][1]), fmaxf(top[1][2], top[1][3])));
      if (in) {
        uint8_t* q = static_cast<uint8_t*>(keep.kept) + slot * keep.ld + f;
        q[0] = static_cast<uint8_t>(act8::encode2(g, 0.0f, act8::inv_scale(eg)) & 255u);
        q[F] = static_cast<uint8_t>(act8::encode2(u, 0.0f, act8::inv_scale(eu)) & 255u);
      }
      if (i == 0) {
        const long long nb = act8::blocks_of(F);
        keep.scale[slot * 2 * nb + blockIdx.y] = static_cast<uint8_t>(eg);
        keep.scale[slot * 2 * nb + nb + blockIdx.y] = static_cast<uint8_t>(eu);
      }
    }
    float phi = g;
    if (kAct == ZOPT_ACT_GELU) {
      const float z = fminf(fmaxf(g, -100.0f), 100.0f);
      phi = 1.5957691216057308f * z * fmaf(0.044715f * z, z, 1.0f);
    }
    hs[i] = in ? slots.weight[slot] * (g / (1.0f + __expf(-phi)) * u) : 0.0f;
  }
  __syncthreads();
  F2 acc[1][4];
#pragma unroll
  for (int q = 0; q < 4; ++q) acc[0][q] = f2(0.0f, 0.0f);
  add_rows<1>(m, k0, n, col, hs, warp, acc);
  join_warps<1>(acc, red, 1, n0, m.cols, partial + (static_cast<long long>(blockIdx.y) * gridDim.z + slot) * m.cols, warp, lane);
}

// y[t][c] = the sum of its slots' parts: 32 columns a CTA, its eight warps taking every eighth part.
__global__ void __launch_bounds__(256) expert_y_kernel(const float* partial, int blocks, const Slots slots, long long cols, uint16_t* y,
                                                       long long ld_y) {
  __shared__ float red[8][32];
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.y, first = t * slots.top_k, all = gridDim.y * slots.top_k;
  const long long c = static_cast<long long>(blockIdx.x) * 32 + lane;
  const int index = lane < slots.top_k ? slots.index[first + lane] : -1;
  const unsigned on = __ballot_sync(0xFFFFFFFFu, index >= 0 && index < slots.experts);
  const bool bad = __any_sync(0xFFFFFFFFu, index != -1 && !(index >= 0 && index < slots.experts));
  float s = 0.0f;
  if (c < cols) {
    for (int j = 0; j < slots.top_k; ++j) {
      if (((on >> j) & 1u) == 0) continue;
#pragma unroll 8
      for (int b = warp; b < blocks; b += 8) s += __ldcg(partial + (static_cast<long long>(b) * all + first + j) * cols + c);
    }
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= cols) return;
#pragma unroll
  for (int v = 1; v < 8; ++v) s += red[v][lane];
  if (bad) s = __uint_as_float(0x7FC00000u);
  y[t * ld_y + c] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
}

struct ExpertPlan {
  int slots, groups, splits, share, blocks, y_groups;
};
ExpertPlan plan_of(const zopt_experts_job& c) {
  ExpertPlan p;
  p.slots = static_cast<int>(c.tokens * c.top_k);
  p.groups = static_cast<int>((2 * c.hidden + kCols - 1) / kCols);
  // one wave of 152 SMs, two CTAs each, but not for fewer than two rows a warp
  const long long most = std::max<long long>(1, (c.dim + 31) / 32);
  const long long want = std::min<long long>(std::max<long long>(1, 304LL / (static_cast<long long>(p.groups) * p.slots)), most);
  p.share = static_cast<int>((c.dim + want - 1) / want);
  p.splits = static_cast<int>((c.dim + p.share - 1) / p.share);
  p.blocks = static_cast<int>((c.hidden + kBlock - 1) / kBlock);
  p.y_groups = static_cast<int>((c.dim + kCols - 1) / kCols);
  return p;
}

}  // namespace

bool takes(const zopt_experts_job& c) {
  if (c.tokens < 1 || c.tokens * c.top_k > 16) return false;
  const ExpertPlan p = plan_of(c);
  return p.splits <= 65535 && p.blocks <= 65535;  // (a grid's second dimension)
}

void partial_elems(const zopt_experts_job& c, long long* gate_up, long long* y) {
  const ExpertPlan p = plan_of(c);
  *gate_up = static_cast<long long>(p.splits) * p.slots * 2 * c.hidden;
  *y = static_cast<long long>(p.blocks) * p.slots * c.dim;
}

zopt_status experts_forward(const zopt_experts_job& c, float* gate_up, float* y, cudaStream_t s) {
  const ExpertPlan p = plan_of(c);
  constexpr size_t smem = static_cast<size_t>(kWarps) * kCols * 4;  // 16 KiB
  const Slots slots{c.index, c.weight, c.experts, c.top_k};
  const Matrix gu{c.w_gate_up, c.ld_gate_up, c.dim, 2 * c.hidden, c.ld_gate_up % 8 == 0 && (c.experts == 1 || c.stride_gate_up % 8 == 0)};
  zopt_status st = launch_pdl(expert_gate_up_kernel, dim3(p.groups, p.splits, p.slots), dim3(kThreads), smem, s, gu,
                              static_cast<long long>(c.stride_gate_up), slots, c.x, static_cast<long long>(c.ld_x), p.share, gate_up);
  if (st != ZOPT_OK) return st;
  Keep k{};
  if (c.kept8 != nullptr) {
    k = Keep{2, c.kept8->q, 2 * c.hidden, c.kept8->scale};
  } else if (c.kept != nullptr) {
    k = Keep{1, c.kept, c.ld_kept, nullptr};
  }
  const Matrix d{c.w_down, c.ld_down, c.hidden, c.dim, c.ld_down % 8 == 0 && (c.experts == 1 || c.stride_down % 8 == 0)};
  const auto kernel = c.act == ZOPT_ACT_GELU ? expert_down_kernel<ZOPT_ACT_GELU> : expert_down_kernel<ZOPT_ACT_SILU>;
  st = launch_pdl(kernel, dim3(p.y_groups, p.blocks, p.slots), dim3(kThreads), smem, s, d, static_cast<long long>(c.stride_down), slots,
                  static_cast<const float*>(gate_up), p.splits, k, y);
  if (st != ZOPT_OK) return st;
  return launch_pdl(expert_y_kernel, dim3(static_cast<unsigned>((c.dim + 31) / 32), static_cast<unsigned>(c.tokens)), dim3(256), 0, s,
                    static_cast<const float*>(y), p.blocks, slots, static_cast<long long>(c.dim), c.y, static_cast<long long>(c.ld_y));
}

}  // namespace few
}  // namespace zopt
