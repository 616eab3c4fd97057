// Sums of scaled weight rows on the CUDA cores, for a few tokens (ffn_few.cu, experts_few.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "act8.cuh"
#include "f2.cuh"

namespace zopt {
namespace few {
namespace {

// 16 warps: a row takes a warp about 40 instructions, and with four warps, twice the rows in flight
// each, two CTAs an SM were bound by their latency (gate and up of one token, 2048 x 5632: 16 us).
constexpr int kThreads = 512, kWarps = 16, kCols = 256, kBlock = act8::kBlock;
constexpr int kRows = 512;  // rows of the inner length whose x a CTA holds at a time
constexpr int kAhead = 8;   // weight rows a warp has in flight
__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

struct Matrix {
  const uint16_t* w;  // [rows][cols]
  long long ld, rows, cols;
  int vec;  // rows start on 16 bytes
};

// acc[t] += sum over the CTA's rows first .. first + n - 1 (at most kRows, xs[row][token] beside them)
// of the lane's eight columns from col on; the warp takes every 16th row.
template <int T>
__device__ __forceinline__ void add_rows(const Matrix& m, long long first, int n, long long col, const float* xs, int warp,
                                         F2 (&acc)[T][4]) {
  const long long left = m.cols - col;
  const uint16_t* w = m.w + first * m.ld + col;
  for (int r0 = warp; r0 < n; r0 += kWarps * kAhead) {
    uint4 v[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + i * kWarps;
      v[i] = make_uint4(0, 0, 0, 0);
      if (r < n && left > 0) {
        const uint16_t* p = w + r * m.ld;
        if (m.vec && left >= 8) {
          v[i] = __ldcs(reinterpret_cast<const uint4*>(p));
        } else {
          uint32_t x[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) x[q] = q < left ? p[q] : 0u;
          v[i] = make_uint4(x[0] | (x[1] << 16), x[2] | (x[3] << 16), x[4] | (x[5] << 16), x[6] | (x[7] << 16));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + i * kWarps;
      if (r >= n) break;
      const F2 f[4] = {f2(lo(v[i].x), hi(v[i].x)), f2(lo(v[i].y), hi(v[i].y)), f2(lo(v[i].z), hi(v[i].z)),
                       f2(lo(v[i].w), hi(v[i].w))};
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const float x = xs[r * T + t];
        const F2 xx = f2(x, x);
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[t][q] = fma2(xx, f[q], acc[t][q]);
      }
    }
  }
}

// The warps' sums added and written to out[t][column], rows of `cols` fp32.
template <int T>
__device__ __forceinline__ void join_warps(const F2 (&acc)[T][4], float* red, int tokens, long long n0, long long cols,
                                           float* out, int warp, int lane) {
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 two = f2(acc[t][q]);
      *reinterpret_cast<float2*>(red + (warp * T + t) * kCols + 8 * lane + 2 * q) = two;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < T * kCols; i += kThreads) {
    const int t = i / kCols, c = i % kCols;
    float s = red[i];
#pragma unroll
    for (int v = 1; v < kWarps; ++v) s += red[v * T * kCols + i];
    if (t < tokens && n0 + c < cols) out[t * cols + n0 + c] = s;
  }
}

struct Keep {
  int mode;  // 0 nothing, 1 bf16, 2 8 bits
  void* kept;
  long long ld;
  uint8_t* scale;
};

}  // namespace
}  // namespace few
}  // namespace zopt
