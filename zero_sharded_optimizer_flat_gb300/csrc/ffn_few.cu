// The feed-forward block's forward for a few tokens (at most kFewTokens), bound by the weights' bytes.
//
// With so few rows a tensor-core tile would be nearly empty, and tiles of 128 or 256 columns are too
// few to read the weights with every SM (one token, 2048 x 5632: 28 us for 69 MB on the tensor
// cores). So the products are sums of scaled weight rows on the CUDA cores: a warp owns 256 columns
// (16 bytes of a row a lane, 512 contiguous a warp) and some of the rows, reads kAhead rows at a time
// and adds them, scaled by the row's entry of every token, in fp32. A CTA's warps join in shared
// memory, the CTAs that share columns through partial sums in the workspace:
//   1. gate and up:  partial[s] = x[k in s] gate_up[k in s], the row ranges s chosen to give every SM
//      two CTAs;
//   2. down: a CTA adds up the gate's and up's parts of its 128 hidden columns (one 8-bit block),
//      forms h (and keeps what is to be kept), and writes partial[block] = h[block] down[block]; its
//      weights are on their way to L2 while it waits for the first launch;
//   3. y = the sum of those.
// Everything is added in a fixed order. One token, 2048 x 5632: 20 us = 3.4 TB/s (12 for the first
// launch by itself; the second's weights are mostly in L2 by then).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "act8.cuh"
#include "f2.cuh"
#include "few.cuh"
#include "ffn_few.h"
#include "launch.cuh"
#include "per_device.h"
#include "tc.cuh"

namespace zopt {
namespace few {
namespace {

// CTAs that share an SM: the sums of four tokens and more take the registers of both.
constexpr int ctas_per_sm(long long tokens) { return tokens <= 2 ? 2 : 1; }

template <int T>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(T)) gate_up_kernel(const Matrix m, const uint16_t* x, long long ld_x, int tokens,
                                                           int share, float* partial) {
  extern __shared__ float red[];  // [kWarps][T][kCols]
  __shared__ float xs[kRows * T];
  // Whatever wrote the weights or x has ended before the launch that follows may start.
  tc::pdl_wait();
  tc::pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long n0 = static_cast<long long>(blockIdx.x) * kCols, col = n0 + 8 * lane;
  const long long k0 = static_cast<long long>(blockIdx.y) * share, k1 = min(m.rows, k0 + share);
  F2 acc[T][4];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[t][q] = f2(0.0f, 0.0f);
  for (long long c = k0; c < k1; c += kRows) {
    const int n = static_cast<int>(min(static_cast<long long>(kRows), k1 - c));
    __syncthreads();
    for (int t = 0; t < T; ++t)
      for (int k = threadIdx.x; k < n; k += kThreads)
        xs[k * T + t] = t < tokens ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(x)[t * ld_x + c + k]) : 0.0f;
    __syncthreads();
    add_rows<T>(m, c, n, col, xs, warp, acc);
  }
  join_warps<T>(acc, red, tokens, n0, m.cols, partial + static_cast<long long>(blockIdx.y) * tokens * m.cols, warp, lane);
}

template <int T, int kAct>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(T)) down_kernel(const Matrix m, const float* parts, int splits, int tokens,
                                                        const Keep keep, float* partial) {
  extern __shared__ float red[];  // [kWarps][T][kCols]
  __shared__ float hs[kBlock * T];
  __shared__ float top[2][kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long n0 = static_cast<long long>(blockIdx.x) * kCols, col = n0 + 8 * lane;
  const long long F = m.rows, k0 = static_cast<long long>(blockIdx.y) * kBlock;
  const int n = static_cast<int>(min(static_cast<long long>(kBlock), F - k0));
  // 128 threads a token: a hidden column each (and, here, a quarter of a weight row)
  const int i = threadIdx.x & 127, group = threadIdx.x >> 7;
  // The launch before writes the partial sums alone: down may be read already.
  if (i < n && n0 + 64 * group < m.cols)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(m.w + (k0 + i) * m.ld + n0 + 64 * group));
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const bool in = i < n;
  const long long f = k0 + i;
#pragma unroll
  for (int t0 = 0; t0 < T; t0 += 4) {
    const int t = t0 + group;
    const bool live = t < tokens;
    float g = 0.0f, u = 0.0f;
    if (in && live) {
      const float* p = parts + t * 2 * F + f;
#pragma unroll 8
      for (int s = 0; s < splits; ++s) {
        g += __ldcg(p + s * tokens * 2 * F);
        u += __ldcg(p + s * tokens * 2 * F + F);
      }
    }
    if (blockIdx.x == 0 && keep.mode == 1 && in && live) {
      uint16_t* q = static_cast<uint16_t*>(keep.kept) + t * keep.ld + f;
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
      __syncthreads();
      if (lane == 0) top[0][warp] = a, top[1][warp] = b;
      __syncthreads();
      const float* x = top[0] + 4 * group;
      const float* z = top[1] + 4 * group;
      const uint32_t eg = act8::exponent_byte(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
      const uint32_t eu = act8::exponent_byte(fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])));
      if (in && live) {
        uint8_t* q = static_cast<uint8_t*>(keep.kept) + t * keep.ld + f;
        q[0] = static_cast<uint8_t>(act8::encode2(g, 0.0f, act8::inv_scale(eg)) & 255u);
        q[F] = static_cast<uint8_t>(act8::encode2(u, 0.0f, act8::inv_scale(eu)) & 255u);
      }
      if (i == 0 && live) {
        const long long nb = act8::blocks_of(F);
        keep.scale[t * 2 * nb + blockIdx.y] = static_cast<uint8_t>(eg);
        keep.scale[t * 2 * nb + nb + blockIdx.y] = static_cast<uint8_t>(eu);
      }
    }
    float phi = g;
    if (kAct == ZOPT_ACT_GELU) {
      const float z = fminf(fmaxf(g, -100.0f), 100.0f);
      phi = 1.5957691216057308f * z * fmaf(0.044715f * z, z, 1.0f);
    }
    const float h = in && live ? g / (1.0f + __expf(-phi)) * u : 0.0f;
    if (t < T) hs[i * T + t] = h;  // in fp32: nothing here needs the bf16 operand that the tensor cores do
  }
  __syncthreads();
  F2 acc[T][4];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[t][q] = f2(0.0f, 0.0f);
  add_rows<T>(m, k0, n, col, hs, warp, acc);
  join_warps<T>(acc, red, tokens, n0, m.cols, partial + static_cast<long long>(blockIdx.y) * tokens * m.cols, warp, lane);
}

// y[t][c] = the sum of `parts` partial sums: 32 columns a CTA, its eight warps taking every eighth.
__global__ void __launch_bounds__(256) y_kernel(const float* partial, int parts, int tokens, long long cols, uint16_t* y,
                                                long long ld_y) {
  __shared__ float red[8][32];
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.y;
  const long long c = static_cast<long long>(blockIdx.x) * 32 + lane;
  float s = 0.0f;
  if (c < cols) {
#pragma unroll 8
    for (int b = warp; b < parts; b += 8) s += __ldcg(partial + (static_cast<long long>(b) * tokens + t) * cols + c);
  }
  red[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || c >= cols) return;
#pragma unroll
  for (int v = 1; v < 8; ++v) s += red[v][lane];
  y[t * ld_y + c] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
}

struct Plan {
  int groups, splits, share, blocks, y_groups;
};
Plan plan(const zopt_ffn_job& c) {
  Plan p;
  p.groups = static_cast<int>((2 * c.hidden + kCols - 1) / kCols);
  // one wave of 152 SMs, but not for fewer than two rows a warp
  const long long most = std::max<long long>(1, (c.dim + 31) / 32);
  const long long want = std::min<long long>(std::max<long long>(1, 152 * ctas_per_sm(c.tokens) / p.groups), most);
  p.share = static_cast<int>((c.dim + want - 1) / want);
  p.splits = static_cast<int>((c.dim + p.share - 1) / p.share);
  p.blocks = static_cast<int>((c.hidden + kBlock - 1) / kBlock);
  p.y_groups = static_cast<int>((c.dim + kCols - 1) / kCols);
  return p;
}

template <int T>
zopt_status run(const zopt_ffn_job& c, const Plan& p, float* gate_up, float* y, cudaStream_t s) {
  const int tokens = static_cast<int>(c.tokens);
  constexpr size_t smem = static_cast<size_t>(kWarps) * T * kCols * 4;
  ZOPT_CUDA_TRY(once_per_device([] {
    cudaError_t e = cudaSuccess;
    for (const void* k : {reinterpret_cast<const void*>(gate_up_kernel<T>), reinterpret_cast<const void*>(down_kernel<T, ZOPT_ACT_SILU>),
                          reinterpret_cast<const void*>(down_kernel<T, ZOPT_ACT_GELU>)})
      if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    return e;
  }));
  const Matrix gu{c.w_gate_up, c.ld_gate_up, c.dim, 2 * c.hidden, c.ld_gate_up % 8 == 0};
  zopt_status st = launch_pdl(gate_up_kernel<T>, dim3(p.groups, p.splits), dim3(kThreads), smem, s, gu, c.x,
                              static_cast<long long>(c.ld_x), tokens, p.share, gate_up);
  if (st != ZOPT_OK) return st;
  Keep k{};
  if (c.kept8 != nullptr) {
    k = Keep{2, c.kept8->q, 2 * c.hidden, c.kept8->scale};
  } else if (c.kept != nullptr) {
    k = Keep{1, c.kept, c.ld_kept, nullptr};
  }
  const Matrix d{c.w_down, c.ld_down, c.hidden, c.dim, c.ld_down % 8 == 0};
  const auto kernel = c.act == ZOPT_ACT_GELU ? down_kernel<T, ZOPT_ACT_GELU> : down_kernel<T, ZOPT_ACT_SILU>;
  st = launch_pdl(kernel, dim3(p.y_groups, p.blocks), dim3(kThreads), smem, s, d, static_cast<const float*>(gate_up), p.splits,
                  tokens, k, y);
  if (st != ZOPT_OK) return st;
  return launch_pdl(y_kernel, dim3(static_cast<unsigned>((c.dim + 31) / 32), tokens), dim3(256), 0, s,
                    static_cast<const float*>(y), p.blocks, tokens, static_cast<long long>(c.dim), c.y,
                    static_cast<long long>(c.ld_y));
}

// With three and four tokens a CTA's sums take the registers of two, and this path's time grows faster
// with the weights' bytes (0.36 us a MB) than the tensor cores' (0.09, and 2.4 us for every 1024 of dim,
// which a tile walks alone, on 12 to start with); so it takes weights up to 16 MiB and 12 KiB for each of
// dim. Four tokens, this path against the other: 1000 x 2732 13.5 us for 19.6, 1024 x 4096 14.4 for 17.1,
// 1536 x 4096 20.5 for 19.5, 2048 x 5632 30.8 for 25.8, 4096 x 2048 22.2 for 26.3, 4096 x 4096 40.6 for 31.6,
// 8192 x 2048 38.6 for 41.7, 8192 x 4096 72.6 for 50.6. Weights that the TMA cannot read in place are
// read here once, there twice after a copy: 1999 x 4001 39.7 for 51.2, down alone copied 2047 x 5632 38.0
// for 37.4. One and two tokens (2048 x 5632 20.1 and 24.2 for 25.7) lose at 3000 x 8000 alone, of those
// measured (two tokens: 40.1 for 36.1).
bool few_bytes(const zopt_ffn_job& c) {
  const bool in_place = c.ld_gate_up % 8 == 0 && c.ld_down % 8 == 0 && c.hidden % 8 == 0;
  return c.tokens <= 2 || !in_place || 6 * c.dim * c.hidden <= (16LL << 20) + (12LL << 10) * c.dim;
}

}  // namespace

bool takes(const zopt_ffn_job& c) {
  const Plan p = plan(c);
  return c.tokens <= kFewTokens && few_bytes(c) && p.splits <= 65535 && p.blocks <= 65535;  // (a grid's second dimension)
}

void partial_elems(const zopt_ffn_job& c, long long* gate_up, long long* y) {
  const Plan p = plan(c);
  *gate_up = static_cast<long long>(p.splits) * c.tokens * 2 * c.hidden;
  *y = static_cast<long long>(p.blocks) * c.tokens * c.dim;
}

zopt_status ffn_forward(const zopt_ffn_job& c, float* gate_up, float* y, cudaStream_t s) {
  const Plan p = plan(c);
  return c.tokens <= 1   ? run<1>(c, p, gate_up, y, s)
         : c.tokens <= 2 ? run<2>(c, p, gate_up, y, s)
                         : run<4>(c, p, gate_up, y, s);
}

}  // namespace few
}  // namespace zopt
