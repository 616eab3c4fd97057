// The experts' forward for a few slots, bound by the bytes of the weights that they choose.
//
// As ffn_few.cu has it for a dense block, a slot in a token's place: nothing has to be sorted, each
// slot's products are sums of its expert's weight rows on the CUDA cores, in fp32 throughout.
//   1. gate and up:  partial[s][slot] = x[k in s] gate_up[k in s]; its CTAs also bring the slots' down
//      matrices to L2, so that HBM has all the call's bytes to fetch from the start;
//   2. down: a CTA adds up the parts of its 256 hidden columns (two 8-bit blocks), forms h with the
//      slot's weight (and keeps what is to be kept), and writes partial[slot][part] = h[part] down[part];
//   3. y = the sum of a token's slots' parts.
// Everything is added in a fixed order. A slot without an expert reads and writes nothing. An expert that
// several slots name is read for each, from L2 as a rule.
//
// One token through six of 64 experts, 2048 x 1408 (104 MB): 25.5 us = 4.1 TB/s; the launches by themselves 18.5
// (4.9 TB/s with the prefetched matrices), 12.8 and 6.8. Without the prefetch and with CTAs of 128 hidden columns
// 33.4; on the tensor cores 45.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "act8.cuh"
#include "experts_few.h"
#include "f2.cuh"
#include "few.cuh"
#include "launch.cuh"
#include "tc.cuh"

namespace zopt {
namespace few {
namespace {

constexpr long long kFewSlots = 64;
constexpr int kParts = 2, kHidden = kParts * kBlock;  // of the hidden columns: a CTA's of the second launch

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

__global__ void __launch_bounds__(kThreads, 2) expert_gate_up_kernel(Matrix m, long long stride, const Matrix down, long long down_stride,
                                                                     const Slots slots, const uint16_t* x, long long ld_x, int share,
                                                                     float* partial) {
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
  {  // this CTA's share of the down matrix's 128-byte lines
    const long long lines = (down.cols + 63) / 64, all = down.rows * lines, ctas = static_cast<long long>(gridDim.x) * gridDim.y;
    const long long cta = static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x;
    for (long long i = cta * kThreads + threadIdx.x; i < all; i += ctas * kThreads)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(down.w + e * down_stride + i / lines * down.ld + i % lines * 64));
  }
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
  __shared__ float hs[kHidden];
  __shared__ float top[2][4 * kParts];
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, slot = blockIdx.z;
  const int e = expert_of(slots, slot);
  if (e < 0) return;
  m.w += e * stride;
  const long long n0 = static_cast<long long>(blockIdx.x) * kCols, col = n0 + 8 * lane;
  const long long F = m.rows, k0 = static_cast<long long>(blockIdx.y) * kHidden;
  const int n = static_cast<int>(min(static_cast<long long>(kHidden), F - k0));
  const int i = threadIdx.x, part = i / kBlock;  // a hidden column each; a block's 128 threads
  if (part < kParts) {
    const long long f = k0 + i, all = static_cast<long long>(gridDim.z) * 2 * F;
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
      asm volatile("bar.sync %0, 128;" ::"r"(1 + part) : "memory");  // (the block's four warps)
      const float *x = top[0] + 4 * part, *z = top[1] + 4 * part;
      const uint32_t eg = act8::exponent_byte(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
      const uint32_t eu = act8::exponent_byte(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])));
      if (in) {
        uint8_t* q = static_cast<uint8_t*>(keep.kept) + slot * keep.ld + f;
        q[0] = static_cast<uint8_t>(act8::encode2(g, 0.0f, act8::inv_scale(eg)) & 255u);
        q[F] = static_cast<uint8_t>(act8::encode2(u, 0.0f, act8::inv_scale(eu)) & 255u);
        if (i % kBlock == 0) {
          const long long nb = act8::blocks_of(F), block = blockIdx.y * kParts + part;
          keep.scale[slot * 2 * nb + block] = static_cast<uint8_t>(eg);
          keep.scale[slot * 2 * nb + nb + block] = static_cast<uint8_t>(eu);
        }
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
  join_warps<1>(acc, red, 1, n0, m.cols, partial + (static_cast<long long>(slot) * gridDim.y + blockIdx.y) * m.cols, warp, lane);
}

// y[t][c] = the sum of its slots' parts: 32 columns a CTA, its eight warps taking every eighth part.
__global__ void __launch_bounds__(256) expert_y_kernel(const float* partial, int parts, const Slots slots, long long cols, uint16_t* y,
                                                       long long ld_y) {
  __shared__ float red[8][32];
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.y, first = t * slots.top_k;
  const long long c = static_cast<long long>(blockIdx.x) * 32 + lane;
  const int index = lane < slots.top_k ? slots.index[first + lane] : -1;
  const unsigned on = __ballot_sync(0xFFFFFFFFu, index >= 0 && index < slots.experts);
  const bool bad = __any_sync(0xFFFFFFFFu, index != -1 && !(index >= 0 && index < slots.experts));
  float s = 0.0f;
  if (c < cols) {
    const float* const p = partial + static_cast<long long>(first) * parts * cols + c;
    const int all = slots.top_k * parts;
#pragma unroll 8
    for (int q = warp; q < all; q += 8)
      if ((on >> (q / parts)) & 1u) s += __ldcg(p + q * cols);
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
  int slots, groups, splits, share, parts, y_groups;
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
  p.parts = static_cast<int>((c.hidden + kHidden - 1) / kHidden);
  p.y_groups = static_cast<int>((c.dim + kCols - 1) / kCols);
  return p;
}

}  // namespace

// By an estimate of both paths' times, in us, the weights of a slot being W MB and `used` the experts that so
// many slots name where they choose at random: this path 17 + W (0.14 used + 0.08 slots), twice and more
// of that where the weights' rows do not start on 16 bytes; the tensor cores 40 + 0.18 W used, and 0.36 W
// for every expert that is copied because the TMA cannot read it in place. (This path against the other,
// from a cold L2: 2048 x 1408 of 64 experts, 6 slots 34 for 55, 24 82 for 106, 32 115 for 111, 64 200 for 142;
// 2048 x 5632 of 8, 8 slots 124 for 131, 12 153 for 129; 256 x 768 of 8, 64 slots 24 for 32; 1000 x 683 of 12,
// 24 slots 42 for 65, 64 108 for 66.)
bool takes(const zopt_experts_job& c) {
  const long long slots = c.tokens * c.top_k;
  if (c.tokens < 1 || slots > kFewSlots) return false;
  const ExpertPlan p = plan_of(c);
  if (p.splits > 65535 || p.parts > 65535) return false;  // (a grid's second dimension)
  const bool in_place = c.ld_gate_up % 8 == 0 && c.ld_down % 8 == 0 && c.hidden % 8 == 0 &&
                        (c.experts == 1 || (c.stride_gate_up % c.ld_gate_up == 0 && c.stride_down % c.ld_down == 0));
  const double mb = 6e-6 * static_cast<double>(c.dim) * static_cast<double>(c.hidden);
  double missed = 1.0;  // an expert's chance not to be named
  for (long long i = 0; i < slots; ++i) missed *= 1.0 - 1.0 / c.experts;
  const double used = std::max<double>(std::min(c.top_k, c.experts), c.experts * (1.0 - missed));
  return 17.0 + (in_place ? 1.0 : 2.2) * mb * (0.14 * used + 0.08 * static_cast<double>(slots)) <=
         40.0 + mb * (0.18 * used + (in_place ? 0.0 : 0.36 * c.experts));
}

void partial_elems(const zopt_experts_job& c, long long* gate_up, long long* y) {
  const ExpertPlan p = plan_of(c);
  *gate_up = static_cast<long long>(p.splits) * p.slots * 2 * c.hidden;
  *y = static_cast<long long>(p.parts) * p.slots * c.dim;
}

zopt_status experts_forward(const zopt_experts_job& c, float* gate_up, float* y, cudaStream_t s) {
  const ExpertPlan p = plan_of(c);
  constexpr size_t smem = static_cast<size_t>(kWarps) * kCols * 4;  // 16 KiB
  const Slots slots{c.index, c.weight, c.experts, c.top_k};
  const Matrix gu{c.w_gate_up, c.ld_gate_up, c.dim, 2 * c.hidden, c.ld_gate_up % 8 == 0 && (c.experts == 1 || c.stride_gate_up % 8 == 0)};
  const Matrix d{c.w_down, c.ld_down, c.hidden, c.dim, c.ld_down % 8 == 0 && (c.experts == 1 || c.stride_down % 8 == 0)};
  zopt_status st = launch_pdl(expert_gate_up_kernel, dim3(p.groups, p.splits, p.slots), dim3(kThreads), smem, s, gu,
                              static_cast<long long>(c.stride_gate_up), d, static_cast<long long>(c.stride_down), slots, c.x, static_cast<long long>(c.ld_x), p.share, gate_up);
  if (st != ZOPT_OK) return st;
  Keep k{};
  if (c.kept8 != nullptr) {
    k = Keep{2, c.kept8->q, 2 * c.hidden, c.kept8->scale};
  } else if (c.kept != nullptr) {
    k = Keep{1, c.kept, c.ld_kept, nullptr};
  }
  const auto kernel = c.act == ZOPT_ACT_GELU ? expert_down_kernel<ZOPT_ACT_GELU> : expert_down_kernel<ZOPT_ACT_SILU>;
  st = launch_pdl(kernel, dim3(p.y_groups, p.parts, p.slots), dim3(kThreads), smem, s, d, static_cast<long long>(c.stride_down), slots,
                  static_cast<const float*>(gate_up), p.splits, k, y);
  if (st != ZOPT_OK) return st;
  return launch_pdl(expert_y_kernel, dim3(static_cast<unsigned>((c.dim + 31) / 32), static_cast<unsigned>(c.tokens)), dim3(256), 0, s,
                    static_cast<const float*>(y), p.parts, slots, static_cast<long long>(c.dim), c.y, static_cast<long long>(c.ld_y));
}

}  // namespace few
}  // namespace zopt
