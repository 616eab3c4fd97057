// Packing activations into 8-bit checkpoints and unpacking them (the format: act8.cuh).
//
// Both are one pass at HBM's rate: 3 bytes an entry, plus a byte per block of 128. Sixteen lanes
// own a block, eight columns each: one 16-byte load, the block's largest magnitude by four
// shuffles, one 8-byte store. A warp takes two blocks side by side.
#include <cuda_runtime.h>

#include <string>

#include "act8.cuh"
#include "act8_host.h"
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
  long long rows, cols, width;  // width: a part's columns
  int parts;
  long long nb;  // blocks per part
  int vec;       // every block of a row starts on 16 bytes of x and 8 of q
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <bool kPack>
__global__ void __launch_bounds__(256) act8_kernel(const Args a) {
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const long long per_row = a.parts * a.nb, blocks = a.rows * per_row;
  const int sub = threadIdx.x & 15;
  const long long step = static_cast<long long>(gridDim.x) * (blockDim.x / 16);
  // both halves of a warp run the same number of rounds (the shuffles name every lane)
  long long b = static_cast<long long>(blockIdx.x) * (blockDim.x / 16) + (threadIdx.x >> 4);
  const long long first = b - ((threadIdx.x >> 4) & 1);
  for (long long f = first; f < blocks; f += step, b += step) {
    const bool live = b < blocks;
    const long long row = live ? b / per_row : 0, r = live ? b - row * per_row : 0;
    const long long part = r / a.nb, k = r - part * a.nb;
    const long long c = k * kBlock + 8 * sub;  // the lane's first column within the part
    const int n = live ? static_cast<int>(min(8LL, max(0LL, a.width - c))) : 0;
    uint16_t* x = a.x + row * a.ld + part * a.width + c;
    uint8_t* q = a.q + row * a.cols + part * a.width + c;
    if (kPack) {
      float v[8];
      if (n == 8 && a.vec) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4*>(x));
        v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
        v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
      } else {
#pragma unroll
        for (int t = 0; t < 8; ++t) v[t] = t < n ? __uint_as_float(static_cast<uint32_t>(x[t]) << 16) : 0.0f;
      }
      float amax = 0.0f;
#pragma unroll
      for (int t = 0; t < 8; ++t) amax = amax_step(amax, v[t]);
#pragma unroll
      for (int d = 8; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
      const uint32_t e = exponent_byte(amax);
      const float inv = inv_scale(e);
      const uint32_t lo = encode4(v[0], v[1], v[2], v[3], inv), hi = encode4(v[4], v[5], v[6], v[7], inv);
      if (n == 8 && a.vec) {
        *reinterpret_cast<uint2*>(q) = make_uint2(lo, hi);
      } else {
#pragma unroll
        for (int t = 0; t < 8; ++t)
          if (t < n) q[t] = static_cast<uint8_t>((t < 4 ? lo : hi) >> (8 * (t & 3)));
      }
      if (live && sub == 0) a.scale[b] = static_cast<uint8_t>(e);
    } else {
      const float sc = scale(live ? a.scale[b] : 1u);
      uint32_t w[2] = {0, 0};
      if (n == 8 && a.vec) {
        const uint2 u = __ldcs(reinterpret_cast<const uint2*>(q));
        w[0] = u.x, w[1] = u.y;
      } else {
#pragma unroll
        for (int t = 0; t < 8; ++t)
          if (t < n) w[t >> 2] |= static_cast<uint32_t>(q[t]) << (8 * (t & 3));
      }
      uint32_t o[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float2 f = decode2(w[t >> 1] >> (16 * (t & 1)));
        const __nv_bfloat162 h = __floats2bfloat162_rn(f.x * sc, f.y * sc);
        o[t] = *reinterpret_cast<const uint32_t*>(&h);
      }
      if (n == 8 && a.vec) {
        *reinterpret_cast<uint4*>(x) = make_uint4(o[0], o[1], o[2], o[3]);
      } else {
#pragma unroll
        for (int t = 0; t < 8; ++t)
          if (t < n) x[t] = static_cast<uint16_t>(o[t >> 1] >> (16 * (t & 1)));
      }
    }
  }
}

zopt_status run(const char* fn, bool pack, const uint16_t* x, long long ld, const zopt_act8& c, cudaStream_t s) {
  Args a;
  a.x = const_cast<uint16_t*>(x);
  a.ld = ld;
  a.q = c.q;
  a.scale = c.scale;
  a.rows = c.rows;
  a.cols = c.cols;
  a.parts = c.parts;
  a.width = c.cols / c.parts;
  a.nb = blocks_of(a.width);
  a.vec = ld % 8 == 0 && c.cols % 8 == 0 && a.width % 8 == 0;
  const int sms = sm_count();
  if (sms < 1) return fail(ZOPT_ECUDA, std::string(fn) + ": no CUDA device");
  const long long want = (a.rows * a.parts * a.nb + 15) / 16, most = 16LL * sms;
  const dim3 grid(static_cast<unsigned>(want < most ? want : most));
  return pack ? launch_pdl(act8_kernel<true>, grid, dim3(256), 0, s, a)
              : launch_pdl(act8_kernel<false>, grid, dim3(256), 0, s, a);
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
