// Linear cross entropy's forward for a few tokens (at most kFewTokens), bound by the weights' bytes.
//
// A tensor-core tile would be nearly empty, and the ring that feeds it reads the weights at 4.1 TB/s
// (one token, 2048 x 32000: 32 us). Here a warp takes kRows vocabulary entries at a time: its lanes
// share a row in pieces of 16 bytes (512 contiguous a load), add the products with every token's x in
// fp32, and exchange sums so that each lane ends with the logit of one entry and token, which it adds
// to a running maximum and sum (base 2). A CTA leaves one (maximum, sum) a token for the launch that
// joins them. Nothing is staged: rows that do not start on 16 bytes are read by single entries. One
// token, 2048 x 32000: 23 us for 131 MB (25.5 with the joining launch); 768 x 50304 16.4 us with it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "f2.cuh"
#include "launch.cuh"
#include "linear_ce_few.h"
#include "lm_gemm.cuh"
#include "tc.cuh"

namespace zopt {
namespace few {
namespace {

// Two CTAs of 128 registers a thread an SM: with three, whose 80 do not hold what is in flight, two
// tokens of 2048 x 32000 take 37 us for 30.
constexpr int kThreads = 256, kWarps = kThreads / 32, kCtasPerSm = 2;
// Vocabulary entries of a group, and pieces of each in flight. One token reads eight rows at a time
// (four, two pieces of each: 50000 x 100 19 us for 14.5, 50304 x 768 20.8 for 19.1); two tokens' sums
// leave registers for four (eight: 2048 x 32000 33 us for 30).
__host__ __device__ constexpr int rows_of(int tokens) { return tokens == 1 ? 8 : 4; }
__host__ __device__ constexpr int ahead_of(int tokens) { return tokens == 1 ? 1 : 2; }
// (Four tokens would be bound by their own arithmetic and loads of x: 2048 x 32000 40 us against the
// tensor cores' 32.)
constexpr long long kFewTokens = 2;

__device__ __forceinline__ F2 two(uint32_t w) { return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }

template <bool kWhole>
__device__ __forceinline__ uint4 piece(const uint16_t* p, long long left) {
  if constexpr (kWhole) return left > 0 ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
  return lm::row_piece8(p, left);
}

// (m, s) and (n, u) as one: m the larger maximum, s the sum of 2^(x - m).
__device__ __forceinline__ void join(float& m, float& s, float n, float u) {
  const float top = fmaxf(m, n), base = top == -INFINITY ? 0.0f : top;
  s = s * exp2f(m - base) + u * exp2f(n - base);
  m = top;
}

// kWhole: every row of x and w is whole 16-byte pieces.
template <int T, bool kWhole>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    ce_few_kernel(const uint16_t* x, long long ld_x, const uint16_t* w, long long ld_w, int tokens, long long dim,
                  long long vocab, const int64_t* target, float2* part, float* tlogit) {
  constexpr int kRows = rows_of(T), kAhead = ahead_of(T);
  constexpr int kValues = kRows * T, kCopies = 32 / kValues;  // logits of a group, lanes that end with the same one
  __shared__ float2 sh[kWarps][T];
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mine = lane / kCopies, mine_row = mine / T, mine_token = mine % T;
  const int64_t tgt = mine_token < tokens && lane % kCopies == 0 ? target[mine_token] : -1;
  float m = -INFINITY, s = 0.0f;
  const long long step = static_cast<long long>(gridDim.x) * kWarps * kRows;
  for (long long v0 = (static_cast<long long>(blockIdx.x) * kWarps + warp) * kRows; v0 < vocab; v0 += step) {
    F2 acc[kRows][T];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int t = 0; t < T; ++t) acc[r][t] = f2(0.0f, 0.0f);
    for (long long k0 = 8 * lane; k0 < dim; k0 += 256 * kAhead) {
      uint4 wv[kAhead][kRows], xv[kAhead][T];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const long long k = k0 + 256 * i;
        // (entries and tokens beyond the last repeat the last: nobody looks at their logits)
#pragma unroll
        for (int r = 0; r < kRows; ++r) wv[i][r] = piece<kWhole>(w + min(v0 + r, vocab - 1) * ld_w + k, dim - k);
#pragma unroll
        for (int t = 0; t < T; ++t) xv[i][t] = piece<kWhole>(x + min(t, tokens - 1) * ld_x + k, dim - k);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
          for (int t = 0; t < T; ++t) {
            acc[r][t] = fma2(two(wv[i][r].x), two(xv[i][t].x), acc[r][t]);
            acc[r][t] = fma2(two(wv[i][r].y), two(xv[i][t].y), acc[r][t]);
            acc[r][t] = fma2(two(wv[i][r].z), two(xv[i][t].z), acc[r][t]);
            acc[r][t] = fma2(two(wv[i][r].w), two(xv[i][t].w), acc[r][t]);
          }
    }
    float a[kValues];
#pragma unroll
    for (int i = 0; i < kValues; ++i) {
      const float2 q = f2(acc[i / T][i % T]);
      a[i] = q.x + q.y;
    }
    // each exchange halves the logits a lane still has a part of
    int d = 16;
#pragma unroll
    for (int n = kValues; n > 1; n >>= 1) {
#pragma unroll
      for (int i = 0; i < n / 2; ++i) {
        const bool up = (lane & d) != 0;
        const float give = up ? a[i] : a[i + n / 2], keep = up ? a[i + n / 2] : a[i];
        a[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, d);
      }
      d >>= 1;
    }
#pragma unroll
    for (int c = kCopies / 2; c >= 1; c >>= 1) a[0] += __shfl_xor_sync(0xFFFFFFFFu, a[0], c);
    const long long row = v0 + mine_row;
    if (row < vocab) {
      const float top = fmaxf(m, a[0] * lm::kLog2e), base = top == -INFINITY ? 0.0f : top;
      s = s * exp2f(m - base) + exp2f(fmaf(a[0], lm::kLog2e, -base));
      m = top;
      if (row == tgt) tlogit[mine_token] = a[0];
    }
  }
  // over the lanes of one token, then over the warps
#pragma unroll
  for (int c = 16; c >= kCopies * T; c >>= 1) {
    const float n = __shfl_xor_sync(0xFFFFFFFFu, m, c), u = __shfl_xor_sync(0xFFFFFFFFu, s, c);
    join(m, s, n, u);
  }
  if (mine_row == 0 && lane % kCopies == 0) sh[warp][mine_token] = make_float2(m, s);
  __syncthreads();
  if (static_cast<int>(threadIdx.x) < tokens) {
    const int t = threadIdx.x;
    m = sh[0][t].x, s = sh[0][t].y;
    for (int v = 1; v < kWarps; ++v) join(m, s, sh[v][t].x, sh[v][t].y);
    part[static_cast<long long>(blockIdx.x) * tokens + t] = make_float2(m, s);
  }
}

template <int T>
zopt_status run(const zopt_linear_ce_job& c, float2* part, float* tlogit, cudaStream_t s) {
  const bool whole = c.dim % 8 == 0 && c.ld_x % 8 == 0 && c.ld_w % 8 == 0;
  const auto kernel = whole ? ce_few_kernel<T, true> : ce_few_kernel<T, false>;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(ce_parts(c))), dim3(kThreads), 0, s, c.x, static_cast<long long>(c.ld_x),
                    c.w, static_cast<long long>(c.ld_w), static_cast<int>(c.tokens), static_cast<long long>(c.dim),
                    static_cast<long long>(c.vocab), c.target, part, tlogit);
}

}  // namespace

bool takes(const zopt_linear_ce_job& c) { return c.tokens >= 1 && c.tokens <= kFewTokens; }

int ce_parts(const zopt_linear_ce_job& c) {
  const long long per_cta = kWarps * rows_of(static_cast<int>(c.tokens));
  return static_cast<int>(std::min<long long>((c.vocab + per_cta - 1) / per_cta, 152 * kCtasPerSm));
}

zopt_status ce_logits(const zopt_linear_ce_job& c, float2* part, float* tlogit, cudaStream_t s) {
  return c.tokens <= 1 ? run<1>(c, part, tlogit, s) : run<2>(c, part, tlogit, s);
}

}  // namespace few
}  // namespace zopt
