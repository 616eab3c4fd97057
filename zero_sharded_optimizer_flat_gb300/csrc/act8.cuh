// The 8-bit activation checkpoint: its block, its power of two, and the conversions that the pack
// and unpack kernels and the feed-forward block's epilogues share.
//
// A block is 128 consecutive columns of a row (a part's last block may be shorter). With amax its
// largest finite magnitude, m 2^k (1 <= m < 2), the block's power is 2^e, e = k - 8, or k - 7 where
// m > 1.75, so that amax 2^-e <= 448, the largest e4m3 value; e is held at -126 at least and stored
// as the byte e + 127. An entry x is stored as e4m3(x 2^-e), rounded to nearest even; inf and NaN
// are both stored as NaN, so that a checkpoint of a non-finite activation still ends in a
// non-finite gradient. 2^e being a power of two, scaling is exact both ways, and what an entry
// stands for (four significant bits times 2^e) is a bf16 value exactly: products read it unrounded.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace zopt {
namespace act8 {

constexpr int kBlock = 128;

__host__ __device__ inline long long blocks_of(long long cols) { return (cols + kBlock - 1) / kBlock; }

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.402823466e38f; }
// The running largest finite magnitude (NaN fails the comparison).
__device__ __forceinline__ float amax_step(float amax, float x) {
  const float a = fabsf(x);
  return (a <= 3.402823466e38f && a > amax) ? a : amax;
}
// The block's stored byte, e + 127 (1 .. 247).
__device__ __forceinline__ uint32_t exponent_byte(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int b = static_cast<int>(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(b < 1 ? 1 : b);
}
// 2^-e and 2^e of a stored byte (normal fp32 values for bytes 1 .. 253).
__device__ __forceinline__ float inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
__device__ __forceinline__ float scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Two finite entries, already scaled, as e4m3, the first in the low byte.
__device__ __forceinline__ uint32_t encode_finite2(float a, float b) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}
// Two entries as e4m3, inf and NaN as NaN.
__device__ __forceinline__ uint32_t encode2(float a, float b, float inv) {
  const float nan = __uint_as_float(0x7FC00000u);
  const float2 v = make_float2(finite(a) ? a * inv : nan, finite(b) ? b * inv : nan);
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv) {
  return encode2(a, b, inv) | (encode2(c, d, inv) << 16);
}
// Two stored bytes' e4m3 values (without the block's power).
__device__ __forceinline__ float2 decode2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xFFFFu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace act8
}  // namespace zopt
