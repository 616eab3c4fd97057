// Packing activations into 8-bit checkpoints and unpacking them (the format: act8.cuh).
//
// Both are one pass, bound by HBM: 3 bytes an entry, plus a byte per block of 128. A block belongs to
// eight lanes, each with pieces of eight columns (16-byte loads, three shuffles for the block's
// largest magnitude) or, where rows or parts do not start on such pieces, of four columns, to 16
// lanes with pieces of two or 32 with single ones. A lane's loads for kSteps blocks are in flight
// before it works on the first. Both directions, 16384 x 2048: 31.7 us = 6.4 TB/s; 4099 x 11240 in two
// parts of 5620 (pieces of four) 47.5 us = 5.8 TB/s.
#include <cuda_runtime.h>

#include <string>

#include "act8.cuh"
#include "act8_host.h"
#include "divisor.cuh"
#include "guarded.h"
#include "launch.cuh"
#include "tc.cuh"

namespace zopt {
namespace act8 {
namespace {

struct Args {
  uint16_t* x;  // pack: read; unpack: written
  long long ld;
  uint8_t* q;
  uint8_t* scale;
  long long cols;
  uint32_t blocks;  // of all rows
  int width;        // a part's columns
  Divisor per_row, per_part;
};

template <int V>
struct Pieces;  // V bf16 values and V bytes
template <>
struct Pieces<8> {
  using X = uint4;
  using Q = uint2;
};
template <>
struct Pieces<4> {
  using X = uint2;
  using Q = uint32_t;
};
template <>
struct Pieces<2> {
  using X = uint32_t;
  using Q = uint16_t;
};
template <>
struct Pieces<1> {
  using X = uint16_t;
  using Q = uint8_t;
};

// The largest magnitude bits of the bf16 values in `w` (two a word), as bf16 bits in both halves.
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// V: the columns of a piece; a lane has kMine columns of a block, in pieces V * kLanes apart.
template <bool kPack, int V>
__global__ void __launch_bounds__(256) act8_kernel(const Args a) {
  using X = typename Pieces<V>::X;
  using Q = typename Pieces<V>::Q;
  constexpr int kMine = V >= 4 ? 16 : 4 * V, kPieces = kMine / V, kLanes = kBlock / kMine, kPerWarp = 32 / kLanes;
  constexpr int kSteps = V >= 4 ? 2 : 4;
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int sub = threadIdx.x % kLanes, lane_block = (threadIdx.x & 31) / kLanes;
  const uint32_t warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, warps = (gridDim.x * blockDim.x) >> 5;
  // (the bound is warp-uniform: the shuffles name every lane)
  for (uint32_t b0 = warp * kPerWarp; b0 < a.blocks; b0 += kSteps * warps * kPerWarp) {
    union {
      X x[kPieces];
      uint32_t w[(kMine + 1) / 2];
    } xv[kSteps];
    union {
      Q q[kPieces];
      uint32_t w[kMine / 4];
    } qv[kSteps];
    long long xo[kSteps], qo[kSteps];  // the lane's first piece
    int n[kSteps];                     // its columns from there to the part's end
    uint32_t e[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const uint32_t b = b0 + i * warps * kPerWarp + lane_block;
      n[i] = 0;
      e[i] = 1;
      if (b < a.blocks && b >= b0) {
        const uint32_t row = a.per_row(b), r = b - row * a.per_row.d, part = a.per_part(r), k = r - part * a.per_part.d;
        const int c = static_cast<int>(k) * kBlock + V * sub;
        n[i] = a.width - c;
        const long long col = static_cast<long long>(part) * a.width + c;
        xo[i] = row * a.ld + col;
        qo[i] = row * a.cols + col;
        if (!kPack) e[i] = __ldg(a.scale + b);
      }
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const int at = p * V * kLanes;
        if (kPack) {
          xv[i].x[p] = X{};
          if (at + V <= n[i]) xv[i].x[p] = __ldcs(reinterpret_cast<const X*>(a.x + xo[i] + at));
        } else {
          qv[i].q[p] = Q{};
          if (at + V <= n[i]) qv[i].q[p] = __ldcs(reinterpret_cast<const Q*>(a.q + qo[i] + at));
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (kPack) {
        // magnitudes compare as integers; a block that has an inf or NaN (bits from 0x7F80 on) is
        // gone through again without them
        uint32_t top = 0;
#pragma unroll
        for (int t = 0; t < kMine / 2; ++t) top = max2(top, xv[i].w[t] & 0x7FFF7FFFu);
        top = max2(top, (top >> 16) | (top << 16));
        const bool odd = (top & 0xFFFFu) >= 0x7F80u;
        if (odd) {
          top = 0;
#pragma unroll
          for (int t = 0; t < kMine; ++t) {
            const uint32_t m = (xv[i].w[t / 2] >> (16 * (t & 1))) & 0x7FFFu;
            if (m < 0x7F80u && m > top) top = m;
          }
          top |= top << 16;
        }
#pragma unroll
        for (int d = kLanes / 2; d >= 1; d >>= 1) top = max2(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        e[i] = exponent_byte(__uint_as_float(top << 16));
        const float inv = inv_scale(e[i]);
#pragma unroll
        for (int t = 0; t < kMine / 4; ++t) {
          const uint32_t lo = xv[i].w[2 * t], hi = xv[i].w[2 * t + 1];
          const float x0 = __uint_as_float(lo << 16), x1 = __uint_as_float(lo & 0xFFFF0000u);
          const float x2 = __uint_as_float(hi << 16), x3 = __uint_as_float(hi & 0xFFFF0000u);
          qv[i].w[t] = odd ? encode4(x0, x1, x2, x3, inv)
                           : encode_finite2(x0 * inv, x1 * inv) | (encode_finite2(x2 * inv, x3 * inv) << 16);
        }
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          const int at = p * V * kLanes;
          if (at + V <= n[i]) *reinterpret_cast<Q*>(a.q + qo[i] + at) = qv[i].q[p];
        }
        const uint32_t b = b0 + i * warps * kPerWarp + lane_block;
        if (sub == 0 && b < a.blocks && b >= b0) a.scale[b] = static_cast<uint8_t>(e[i]);
      } else {
        const float sc = scale(e[i]);
#pragma unroll
        for (int t = 0; t < kMine / 2; ++t) {
          const float2 f = decode2(qv[i].w[t >> 1] >> (16 * (t & 1)));
          const __nv_bfloat162 h = __floats2bfloat162_rn(f.x * sc, f.y * sc);
          xv[i].w[t] = *reinterpret_cast<const uint32_t*>(&h);
        }
#pragma unroll
        for (int p = 0; p < kPieces; ++p) {
          const int at = p * V * kLanes;
          if (at + V <= n[i]) *reinterpret_cast<X*>(a.x + xo[i] + at) = xv[i].x[p];
        }
      }
    }
  }
}

template <int V>
zopt_status launch(bool pack, const Args& a, int sms, cudaStream_t s) {
  constexpr long long kPerCta = 8 * (V >= 4 ? 4 * 2 : V * 4);  // blocks a CTA takes at a time
  const long long want = (a.blocks + kPerCta - 1) / kPerCta, most = 8LL * sms;
  const dim3 grid(static_cast<unsigned>(want < most ? want : most));
  return pack ? launch_pdl(act8_kernel<true, V>, grid, dim3(256), 0, s, a)
              : launch_pdl(act8_kernel<false, V>, grid, dim3(256), 0, s, a);
}

zopt_status run(const char* fn, bool pack, const uint16_t* x, long long ld, const zopt_act8& c, cudaStream_t s) {
  const int sms = sm_count();
  if (sms < 1) return fail(ZOPT_ECUDA, std::string(fn) + ": no CUDA device");
  const long long width = c.cols / c.parts, nb = blocks_of(width), per_row = c.parts * nb;
  const unsigned mis = static_cast<unsigned>(ld | c.cols | width);  // (x and q start on 16 bytes)
  const long long most_rows = (1LL << 30) / per_row;                // block numbers of a launch stay below 2^30
  for (long long r0 = 0; r0 < c.rows; r0 += most_rows) {
    const long long rows = c.rows - r0 < most_rows ? c.rows - r0 : most_rows;
    Args a{const_cast<uint16_t*>(x) + r0 * ld, ld, c.q + r0 * c.cols, c.scale + r0 * per_row, c.cols,
           static_cast<uint32_t>(rows * per_row), static_cast<int>(width), Divisor(static_cast<uint32_t>(per_row)),
           Divisor(static_cast<uint32_t>(nb))};
    const zopt_status st = mis % 8 == 0   ? launch<8>(pack, a, sms, s)
                           : mis % 4 == 0 ? launch<4>(pack, a, sms, s)
                           : mis % 2 == 0 ? launch<2>(pack, a, sms, s)
                                          : launch<1>(pack, a, sms, s);
    if (st != ZOPT_OK) return st;
  }
  return ok();
}

zopt_status call(const char* fn, bool pack, const uint16_t* x, int64_t ld, const zopt_act8* c, zopt_stream stream) {
  const std::string f(fn);
  if (c == nullptr || (x == nullptr && c->rows != 0)) return fail(ZOPT_EINVAL, f + ": NULL argument");
  zopt_status st = check(fn, *c);
  if (st != ZOPT_OK) return st;
  if (!aligned16(x)) return fail(ZOPT_EINVAL, f + ": the bf16 matrix must be 16-byte aligned");
  if (ld < c->cols || ld > (1LL << 32)) return fail(ZOPT_EINVAL, f + ": row distance below cols or above 2^32");
  if (c->rows == 0) return ok();
  return run(fn, pack, x, ld, *c, stream);
}

}  // namespace

size_t scale_bytes(long long rows, long long cols, int parts) {
  if (rows < 0 || cols < 1 || parts < 1 || parts > 2 || cols % parts != 0 || rows > kMaxDim || cols > kMaxDim) return 0;
  return static_cast<size_t>(rows) * parts * blocks_of(cols / parts);
}

zopt_status check(const char* fn, const zopt_act8& c) {
  const std::string f(fn);
  if (c.rows < 0 || c.cols < 1 || c.rows > kMaxDim || c.cols > kMaxDim)
    return fail(ZOPT_EINVAL, f + ": a checkpoint's rows must be in [0, 2^30], its cols in [1, 2^30]");
  if (c.parts < 1 || c.parts > 2 || c.cols % c.parts != 0)
    return fail(ZOPT_EINVAL, f + ": a checkpoint's parts must be 1 or 2 and divide its cols");
  if (c.rows > 0 && (c.q == nullptr || c.scale == nullptr)) return fail(ZOPT_EINVAL, f + ": NULL checkpoint");
  if (!aligned16(c.q)) return fail(ZOPT_EINVAL, f + ": a checkpoint's q must be 16-byte aligned");
  return ok();
}

zopt_status unpack(const char* fn, const zopt_act8& c, uint16_t* out, long long ld, cudaStream_t s) {
  return run(fn, false, out, ld, c, s);
}

}  // namespace act8
}  // namespace zopt

extern "C" size_t zopt_act8_scale_bytes(int64_t rows, int64_t cols, int32_t parts) {
  return zopt::act8::scale_bytes(rows, cols, parts);
}

extern "C" zopt_status zopt_act_pack(const uint16_t* x, int64_t ld_x, const zopt_act8* out, zopt_stream stream) {
  return zopt::guarded([&] { return zopt::act8::call("zopt_act_pack", true, x, ld_x, out, stream); });
}

extern "C" zopt_status zopt_act_unpack(const zopt_act8* in, uint16_t* out, int64_t ld_out, zopt_stream stream) {
  return zopt::guarded([&] { return zopt::act8::call("zopt_act_unpack", false, out, ld_out, in, stream); });
}
