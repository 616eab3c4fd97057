// Routing tokens to experts, forward and backward.
//
// A warp takes a token's row, a lane V experts that follow one another. Ranking is in exact order (of the
// score plus the bias as real numbers, the lowest index first among equal ones), so that a choice never
// depends on how an exponential rounds. An expert is one word: 22 bits that do not decrease with its
// rank's number, above 10 that fall with its index. A lane sorts its words once (a fixed network); the
// warp's largest word, an integer maximum, is the next choice, and its lane moves its words up. Without a
// bias the 22 bits are the logit's own leading ones (a bf16 logit's are all of it), with one, or with
// groups, the score's and the bias's sum in fixed point over the row's range. Neighbours in the
// order that come closer than those bits and the score's error tell apart, if they are not the same
// numbers, are told apart in fp64, together with what the border of the choice may have left out (one
// row in some hundreds).
//
// Bound by the instructions of a row, some 200 for eight of 256 experts.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "divisor.cuh"
#include "guarded.h"
#include "launch.cuh"
#include "tc.cuh"

namespace zopt {
namespace route {
namespace {

constexpr int kMaxExperts = 1024, kMaxTopK = 32, kMaxGroups = 32;
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr unsigned kAll = 0xFFFFFFFFu;

struct Args {
  const void* logits;
  long long ld;
  const float* bias;
  const uint8_t* live;
  int32_t* index;
  float* weight;
  int32_t* counts;
  const float* dweight;
  void* dlogits;
  long long ld_d;
  long long tokens;
  int experts, top_k, groups, top_groups;
  Divisor per_group;
  int bf16, renormalise, alone;  // alone: one block has all rows, counts need no sum over blocks
  int vec, vec_d;                // a lane's experts can be loaded (stored) at once
  int lanes_per_group;           // where a group is a power of two of whole lanes' experts, else 0
  float scale;
};

__device__ __forceinline__ float load(const Args& a, long long row, int i) {
  const long long at = row * a.ld + i;
  return a.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[at]) : static_cast<const float*>(a.logits)[at];
}
// The lane's V logits, -inf behind the last expert.
template <int V>
__device__ __forceinline__ void load_row(const Args& a, long long row, int first, float (&l)[V]) {
  if (V >= 2 && a.vec && first + V <= a.experts) {
    if (a.bf16) {
      const uint16_t* const p = static_cast<const uint16_t*>(a.logits) + row * a.ld + first;
      if constexpr (V >= 8) {
#pragma unroll
        for (int q = 0; q < V / 8; ++q) {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(p) + q);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) l[8 * q + 2 * k] = __uint_as_float(w[k] << 16), l[8 * q + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
      } else if constexpr (V == 4) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
        l[0] = __uint_as_float(x.x << 16), l[1] = __uint_as_float(x.x & 0xFFFF0000u);
        l[2] = __uint_as_float(x.y << 16), l[3] = __uint_as_float(x.y & 0xFFFF0000u);
      } else if constexpr (V == 2) {
        const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(p));
        l[0] = __uint_as_float(x << 16), l[1] = __uint_as_float(x & 0xFFFF0000u);
      }
    } else {
      const float* const p = static_cast<const float*>(a.logits) + row * a.ld + first;
      if constexpr (V >= 4) {
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
          const float4 x = __ldg(reinterpret_cast<const float4*>(p) + q);
          l[4 * q] = x.x, l[4 * q + 1] = x.y, l[4 * q + 2] = x.z, l[4 * q + 3] = x.w;
        }
      } else if constexpr (V == 2) {
        const float2 x = __ldg(reinterpret_cast<const float2*>(p));
        l[0] = x.x, l[1] = x.y;
      }
    }
    return;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = first + v < a.experts ? load(a, row, first + v) : -INFINITY;
}

template <int V>
__device__ __forceinline__ void store_row(const Args& a, long long row, int first, const float (&x)[V]) {
  const long long at = row * a.ld_d + first;
  if (V >= 2 && a.vec_d && first + V <= a.experts) {
    if (a.bf16) {
      uint16_t* const p = static_cast<uint16_t*>(a.dlogits) + at;
      uint32_t w[V / 2 > 0 ? V / 2 : 1];
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      }
      if constexpr (V >= 8) {
#pragma unroll
        for (int q = 0; q < V / 8; ++q) reinterpret_cast<uint4*>(p)[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
      } else if constexpr (V == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
      } else if constexpr (V == 2) {
        *reinterpret_cast<uint32_t*>(p) = w[0];
      }
    } else {
      float* const p = static_cast<float*>(a.dlogits) + at;
      if constexpr (V >= 4) {
#pragma unroll
        for (int q = 0; q < V / 4; ++q) reinterpret_cast<float4*>(p)[q] = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
      } else if constexpr (V == 2) {
        *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
      }
    }
    return;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (first + v >= a.experts) continue;
    if (a.bf16) {
      static_cast<__nv_bfloat16*>(a.dlogits)[at + v] = __float2bfloat16_rn(x[v]);
    } else {
      static_cast<float*>(a.dlogits)[at + v] = x[v];
    }
  }
}

// Unsigned integers in the order of the numbers, NaN above them all; 0, below them all, is no number's.
__device__ __forceinline__ uint32_t key_of(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 is 0
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ (static_cast<uint32_t>(static_cast<int32_t>(~k) >> 31) | 0x80000000u));
}
__device__ __forceinline__ uint64_t key_of(double x) {
  if (x != x) return ~0ull;
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return u ^ (static_cast<uint64_t>(static_cast<int64_t>(u) >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double of_key(uint64_t k) {
  return __longlong_as_double(static_cast<long long>(k ^ (static_cast<uint64_t>(static_cast<int64_t>(~k) >> 63) | 0x8000000000000000ull)));
}
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
  const uint32_t hi = static_cast<uint32_t>(k >> 32), top = __reduce_max_sync(kAll, hi);
  const uint32_t lo = __reduce_max_sync(kAll, hi == top ? static_cast<uint32_t>(k) : 0u);
  return (static_cast<uint64_t>(top) << 32) | lo;
}
// (NaN: the others' largest)
__device__ __forceinline__ float warp_max(float x) {
  return of_key(__reduce_max_sync(kAll, x != x ? 0x007FFFFFu : key_of(x)));  // 0x007FFFFF: -inf's
}
template <typename T>
__device__ __forceinline__ T warp_sum(T x) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
  return x;
}

// ---------------------------------------------------------------------- in fp64

// What an expert is ranked by: the score and the bias, or without a bias the logit.
template <bool kSoftmax>
__device__ __forceinline__ double rank64(const Args& a, float l, int i, double top, double z) {
  if (a.bias == nullptr) return static_cast<double>(l);
  const double s = kSoftmax ? exp(static_cast<double>(l) - top) / z : 1.0 / (1.0 + exp(-static_cast<double>(l)));
  return s + static_cast<double>(a.bias[i]);
}
__device__ __forceinline__ void softmax64(const Args& a, long long row, int lane, double& top, double& z) {
  float m = -INFINITY;
  for (int i = lane; i < a.experts; i += 32) m = fmaxf(m, load(a, row, i));
  top = static_cast<double>(warp_max(m));
  double part = 0.0;
  for (int i = lane; i < a.experts; i += 32) part += exp(static_cast<double>(load(a, row, i)) - top);
  z = warp_sum(part);
}

// The best `most` of the candidates, one a lane (key 0: none), the lowest index first among equal ones.
__device__ __forceinline__ int best64(uint64_t key, int i, int most, int lane) {
  int mine = -1;
  for (int j = 0; j < most; ++j) {
    const uint64_t top = warp_max(key);
    if (top == 0) break;
    const int at = static_cast<int>(__reduce_min_sync(kAll, key == top ? static_cast<uint32_t>(i) : kAll));
    if (lane == j) mine = at;
    if (key == top && i == at) key = 0;
  }
  return mine;
}

// The row's choice among `i` of every lane (-1: none).
template <bool kSoftmax>
__device__ __noinline__ int among(const Args& a, long long row, int i, int lane) {
  double top = 0.0, z = 1.0;
  if (kSoftmax && a.bias != nullptr) softmax64(a, row, lane, top, z);
  return best64(i >= 0 ? key_of(rank64<kSoftmax>(a, load(a, row, i), i, top, z)) : 0ull, i, a.top_k, lane);
}

// The row's choice among all experts, its groups' scores in fp64 as well. Experts a lane at a time: lane l
// looks at l, l + 32, ...; those taken are marked in `gone`.
template <bool kSoftmax>
__device__ __noinline__ int among_all(const Args& a, long long row, int lane) {
  double top = 0.0, z = 1.0;
  if (kSoftmax) softmax64(a, row, lane, top, z);
  uint32_t gone = 0, groups = kAll;
  if (a.groups > 1) {
    uint64_t mine = 0;
    for (int g = 0; g < a.groups; ++g) {
      uint64_t first = 0, second = 0;
      for (int i = g * static_cast<int>(a.per_group.d) + lane; i < (g + 1) * static_cast<int>(a.per_group.d); i += 32) {
        const float l = load(a, row, i);
        if (l == -INFINITY) continue;
        double c = kSoftmax ? exp(static_cast<double>(l) - top) / z : 1.0 / (1.0 + exp(-static_cast<double>(l)));
        if (a.bias != nullptr) c += static_cast<double>(a.bias[i]);
        const uint64_t k = key_of(c);
        second = k > first ? first : k > second ? k : second;
        first = k > first ? k : first;
      }
      const uint64_t one = warp_max(first);
      const int owner = __ffs(__ballot_sync(kAll, first == one)) - 1;
      const uint64_t two = warp_max(lane == owner ? second : first);
      if (lane == g) mine = one == 0 ? 0 : two == 0 ? one : key_of(of_key(one) + of_key(two));
    }
    const int g = best64(mine, lane, a.top_groups, lane);
    groups = __reduce_or_sync(kAll, g >= 0 ? 1u << g : 0u);
  }
  int mine = -1;
  for (int j = 0; j < a.top_k; ++j) {
    uint64_t best = 0;
    int at = -1;
    for (int i = lane, v = 0; i < a.experts; i += 32, ++v) {
      const float l = load(a, row, i);
      if (l == -INFINITY || ((gone >> v) & 1u) != 0) continue;
      if (a.groups > 1 && ((groups >> a.per_group(static_cast<uint32_t>(i))) & 1u) == 0) continue;
      const uint64_t k = key_of(rank64<kSoftmax>(a, l, i, top, z));
      if (k > best) best = k, at = i;
    }
    const uint64_t win = warp_max(best);
    if (win == 0) break;
    const int i = static_cast<int>(__reduce_min_sync(kAll, best == win ? static_cast<uint32_t>(at) : kAll));
    if (lane == j) mine = i;
    if (best == win && at == i) gone |= 1u << (i >> 5);
  }
  return mine;
}

// ---------------------------------------------------------------------- by words

constexpr int kIndexBits = 10;
constexpr uint32_t kIndexMask = (1u << kIndexBits) - 1u, kTopRank = (1u << (32 - kIndexBits)) - 1u;

// Largest first: Batcher's odd-even merges.
template <int V>
__device__ __forceinline__ void sort_words(uint32_t (&w)[V]) {
#pragma unroll
  for (int p = 1; p < V; p <<= 1)
#pragma unroll
    for (int k = p; k >= 1; k >>= 1)
#pragma unroll
      for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t x = w[i + j], y = w[i + j + k];
            w[i + j] = max(x, y), w[i + j + k] = min(x, y);
          }
}
template <int V>
__device__ __forceinline__ void drop_first(uint32_t (&w)[V], bool mine) {
#pragma unroll
  for (int v = 0; v + 1 < V; ++v) w[v] = mine ? w[v + 1] : w[v];
  w[V - 1] = mine ? 0u : w[V - 1];
}

// What is reckoned with, in units of 2^-24: for a score in fp32, of the row's largest, an exponential
// and divisions (8), and for the softmax a sum of V terms a lane over the warp as well; for the sum
// with a bias, and what is taken from it, 2 of their terms.
constexpr float kUnit = 1.0f / (1 << 24);

// What the biases of a warp's lanes have in common for every row.
template <int V>
struct Bias {
  float b[V], lo, hi;
  __device__ __forceinline__ Bias(const Args& a, int first) {
    lo = 0.0f, hi = 0.0f;
    if (a.bias == nullptr) return;
    lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      b[v] = first + v < a.experts ? __ldg(a.bias + first + v) : 0.0f;
      if (first + v < a.experts) lo = fminf(lo, b[v]), hi = fmaxf(hi, b[v]);
    }
    lo = -warp_max(-lo), hi = warp_max(hi);
  }
};

template <int V, bool kSoftmax>
__device__ __forceinline__ int choose(const Args& a, long long row, const float (&l)[V], const Bias<V>& bias, int lane) {
  const int first = lane * V;
  uint32_t w[V];
  int near = 0;  // ranks this close or closer need a second look
  if (a.bias == nullptr && a.groups == 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint32_t name = kIndexMask - static_cast<uint32_t>(first + v);
      w[v] = l[v] == -INFINITY ? 0u : (key_of(l[v]) & ~kIndexMask) | name;
    }
    if (a.bf16) near = -1;  // (16 bits are all there is)
    sort_words<V>(w);
  } else {
    float m = 0.0f, rz = 1.0f, c[V];
    if (kSoftmax) {
      m = l[0];
#pragma unroll
      for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
      m = warp_max(m);
      float z = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = expf(l[v] - m), z += c[v];
      rz = 1.0f / warp_sum(z);
    }
    const float range = (kSoftmax ? rz : 1.0f) + (bias.hi - bias.lo), scale = (kTopRank - 3) / range;
    bool bad = !(range < INFINITY);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      c[v] = kSoftmax ? c[v] * rz : 1.0f / (1.0f + expf(-l[v]));
      if (a.bias != nullptr) c[v] += bias.b[v];
      bad = bad || c[v] != c[v];
      const uint32_t q = min(1u + static_cast<uint32_t>(fmaxf((c[v] - bias.lo) * scale, 0.0f)), kTopRank - 1u);
      w[v] = l[v] == -INFINITY ? 0u : (q << kIndexBits) | (kIndexMask - static_cast<uint32_t>(first + v));
    }
    if (__any_sync(kAll, bad)) return among_all<kSoftmax>(a, row, lane);
    const float off = kUnit * (2.0f * (kSoftmax ? (V + 16) * rz : 8.0f) + 4.0f * (fabsf(bias.lo) + fabsf(bias.hi) + range));
    near = static_cast<int>(off * scale) + 3;  // (and a unit of each of the two, and of the product)
    if (a.groups > 1) {
      const float unit = range / (kTopRank - 3);
      auto value = [&](uint32_t word) { return bias.lo + unit * static_cast<float>(word >> kIndexBits); };
      uint32_t one, two;
      int group;  // whose two best words the lane has
      bool in_lane = a.lanes_per_group > 0;
      if (in_lane) {  // a group is a power of two of lanes: their first two words are merged
        sort_words<V>(w);
        one = w[0], two = V > 1 ? w[V > 1 ? 1 : 0] : 0u;
        for (int d = 1; d < a.lanes_per_group; d <<= 1) {
          const uint32_t x = __shfl_xor_sync(kAll, one, d), y = __shfl_xor_sync(kAll, two, d);
          two = max(min(one, x), max(two, y));
          one = max(one, x);
        }
        group = lane / a.lanes_per_group;
      } else {
        one = two = 0;
        for (int g = 0; g < a.groups; ++g) {
          uint32_t x = 0, y = 0;
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const uint32_t k = static_cast<int>(a.per_group(static_cast<uint32_t>(first + v))) == g ? w[v] : 0u;
            y = max(y, min(x, k));
            x = max(x, k);
          }
          const uint32_t best = __reduce_max_sync(kAll, x), next = __reduce_max_sync(kAll, x == best ? y : x);
          if (lane == g) one = best, two = next;
        }
        group = lane;
      }
      const bool speaks = in_lane ? lane % a.lanes_per_group == 0 && group < a.groups : group < a.groups;
      uint32_t sum = !speaks || one == 0 ? 0u : key_of(two == 0 ? value(one) : value(one) + value(two));
      uint32_t mask = 0, worst = 0;
      for (int j = 0; j < a.top_groups; ++j) {
        const uint32_t top = __reduce_max_sync(kAll, sum);
        if (top == 0) break;
        const int owner = __ffs(__ballot_sync(kAll, sum == top)) - 1;
        worst = top;
        mask |= 1u << __shfl_sync(kAll, group, owner);
        if (lane == owner) sum = 0;
      }
      const uint32_t left = __reduce_max_sync(kAll, sum);
      if (left != 0 && !(of_key(worst) - of_key(left) > 2.0f * (near + 1) * unit + 8.0f * kUnit * (fabsf(of_key(worst)) + fabsf(of_key(left)))))
        return among_all<kSoftmax>(a, row, lane);
      if (in_lane) {
        if (((mask >> group) & 1u) == 0 || group >= a.groups) {
#pragma unroll
          for (int v = 0; v < V; ++v) w[v] = 0;
        }
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (first + v < a.experts && ((mask >> a.per_group(static_cast<uint32_t>(first + v))) & 1u) == 0) w[v] = 0;
        sort_words<V>(w);
      }
    } else {
      sort_words<V>(w);
    }
  }
  uint32_t mine = 0, top = 0;
  int n = 0;
  for (; n < a.top_k; ++n) {
    top = __reduce_max_sync(kAll, w[0]);
    if (top == 0) break;
    if (lane == n) mine = top;
    drop_first<V>(w, w[0] == top);
  }
  const int chosen = mine == 0 ? -1 : static_cast<int>(kIndexMask - (mine & kIndexMask));
  if (near < 0) return chosen;
  // neighbours in the order
  const int rank = static_cast<int>(mine >> kIndexBits), next = __shfl_down_sync(kAll, rank, 1);
  const bool close = lane + 1 < n && rank - next <= near;
  uint32_t left = n == a.top_k ? __reduce_max_sync(kAll, w[0]) : 0u;
  const int last = __shfl_sync(kAll, rank, n > 0 ? n - 1 : 0);
  const bool border = left != 0 && last - static_cast<int>(left >> kIndexBits) <= near;
  if (!__any_sync(kAll, close) && !border) return chosen;
  // the same numbers (their order is the index's), or others
  float ml = 0.0f, mb = 0.0f;
  if (chosen >= 0) ml = load(a, row, chosen), mb = a.bias != nullptr ? a.bias[chosen] : 0.0f;
  const float nl = __shfl_down_sync(kAll, ml, 1), nb = __shfl_down_sync(kAll, mb, 1);
  bool again = __any_sync(kAll, close && !(ml == nl && mb == nb));
  const float ll = __shfl_sync(kAll, ml, n > 0 ? n - 1 : 0), lb = __shfl_sync(kAll, mb, n > 0 ? n - 1 : 0);
  int candidate = chosen, found = n;
  while (left != 0 && last - static_cast<int>(left >> kIndexBits) <= near) {
    const int i = static_cast<int>(kIndexMask - (left & kIndexMask));
    if (!(load(a, row, i) == ll && (a.bias == nullptr || a.bias[i] == lb))) again = true;
    if (lane == found) candidate = i;
    ++found;
    drop_first<V>(w, w[0] == left);
    left = __reduce_max_sync(kAll, w[0]);
  }
  if (!again) return chosen;
  if (found > 32) return among_all<kSoftmax>(a, row, lane);
  return among<kSoftmax>(a, row, candidate, lane);
}

template <int V, bool kSoftmax>
__global__ void __launch_bounds__(kThreads) forward_kernel(const Args a) {
  __shared__ int count[kMaxExperts];
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  if (a.counts != nullptr) {
    for (int i = threadIdx.x; i < a.experts; i += kThreads) count[i] = 0;
    __syncthreads();
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Bias<V> bias(a, lane * V);
  for (long long row = static_cast<long long>(blockIdx.x) * kWarps + warp; row < a.tokens;
       row += static_cast<long long>(gridDim.x) * kWarps) {
    int mine = -1;
    float w = 0.0f;
    if (a.live == nullptr || a.live[row] != 0) {
      float l[V];
      load_row<V>(a, row, lane * V, l);
      mine = choose<V, kSoftmax>(a, row, l, bias, lane);
      const bool on = mine >= 0;
      const float ml = on ? load(a, row, mine) : -INFINITY;
      if (kSoftmax) {
        // relative to the largest logit: of the chosen ones where the weights are renormalised (the other
        // terms cancel), else of all. A row with a NaN or +inf has no softmax.
        bool bad = false;
#pragma unroll
        for (int v = 0; v < V; ++v) bad = bad || !(l[v] < INFINITY);
        float m, z;
        if (a.renormalise) {
          m = warp_max(ml);
          w = on ? expf(ml - m) : 0.0f;
          z = warp_sum(w);
        } else {
          m = l[0];
#pragma unroll
          for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
          m = warp_max(m);
          w = on ? expf(ml - m) : 0.0f;
          float part = 0.0f;
#pragma unroll
          for (int v = 0; v < V; ++v) part += l[v] == -INFINITY ? 0.0f : expf(l[v] - m);
          z = warp_sum(part);
        }
        w = on ? w / z * a.scale : 0.0f;
        if (__any_sync(kAll, bad) && on) w = __uint_as_float(0x7FC00000u);
      } else {
        // s = e^l / (1 + e^l); where all chosen logits are negative, e^(l - max) in its place where the
        // weights are renormalised: the quotients stay what they are and nothing underflows.
        const float top = a.renormalise ? fminf(0.0f, warp_max(ml)) : 0.0f;
        w = !on ? 0.0f : ml >= 0.0f ? 1.0f / (1.0f + expf(-ml)) : expf(ml - top) / (1.0f + expf(ml));
        if (a.renormalise) w = w / warp_sum(w);
        w = on ? w * a.scale : 0.0f;
      }
    }
    if (lane < a.top_k) {
      a.index[row * a.top_k + lane] = mine;
      a.weight[row * a.top_k + lane] = w;
      if (a.counts != nullptr && mine >= 0) atomicAdd(count + mine, 1);
    }
  }
  if (a.counts == nullptr) return;
  __syncthreads();
  for (int i = threadIdx.x; i < a.experts; i += kThreads) {  // (sums of integers: in any order the same)
    if (a.alone) {
      a.counts[i] = count[i];
    } else if (count[i] != 0) {
      atomicAdd(a.counts + i, count[i]);
    }
  }
}

// With q the chosen scores over their sum (renormalised) or the scores, and w = scale q as the forward
// gave it:
//   softmax, renormalised:  dl_j = w_j (dw_j - sum_k dw_k q_k)            for chosen j, 0 elsewhere
//   softmax:                dl_i = scale p_i ([i chosen] dw_i - sum_k dw_k p_k)
//   logistic:               as the first with a factor 1 - s_j; without the sum where not renormalised.
//
// A warp writes its row whole, with what the chosen experts' entries would be if they had not been
// chosen, and then the chosen ones' again, a lane each. Bound by what it writes.
template <int V, bool kSoftmax>
__global__ void __launch_bounds__(kThreads) backward_kernel(const Args a) {
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, first = lane * V;
  const float nan = __uint_as_float(0x7FC00000u);
  for (long long row = static_cast<long long>(blockIdx.x) * kWarps + warp; row < a.tokens;
       row += static_cast<long long>(gridDim.x) * kWarps) {
    int mine = -1;
    float w = 0.0f, g = 0.0f;
    if (lane < a.top_k) mine = a.index[row * a.top_k + lane];
    const bool on = mine >= 0 && mine < a.experts, bad = __any_sync(kAll, mine != -1 && !on);
    float ml = 0.0f;
    if (on) {
      w = a.weight[row * a.top_k + lane];
      g = a.dweight[row * a.top_k + lane];
      if (!kSoftmax) ml = load(a, row, mine);
    }
    const float mean = warp_sum(g * w) / a.scale;
    float d = (a.renormalise ? g - mean : g) * w;
    if (!kSoftmax) d *= 1.0f / (1.0f + expf(ml));  // 1 - s
    float out[V];
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = 0.0f;
    float rest = 0.0f;  // what the lane's expert would have if it were not chosen
    if (kSoftmax && !a.renormalise && __any_sync(kAll, on)) {
      float m, z = 0.0f;
      load_row<V>(a, row, first, out);
      m = out[0];
#pragma unroll
      for (int v = 1; v < V; ++v) m = fmaxf(m, out[v]);
      m = warp_max(m);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        out[v] = out[v] == -INFINITY ? 0.0f : expf(out[v] - m);
        z += out[v];
      }
      const float f = -mean * a.scale / warp_sum(z);
#pragma unroll
      for (int v = 0; v < V; ++v) out[v] *= f;
      if (on) rest = expf(load(a, row, mine) - m) * f;
    }
    if (bad) {
#pragma unroll
      for (int v = 0; v < V; ++v) out[v] = nan;
    }
    store_row<V>(a, row, first, out);
    if (bad) continue;
    // an expert that the row names more than once takes all its slots' parts, in their order
    const unsigned same = __match_any_sync(kAll, on ? mine : -1 - lane);
    float sum = d;
    if (__any_sync(kAll, __popc(same) > 1)) {
      sum = 0.0f;
      for (int j = 0; j < a.top_k; ++j) {
        const float x = __shfl_sync(kAll, d, j);
        if ((same >> j) & 1u) sum += x;
      }
    }
    __syncwarp();  // (orders the two stores to one address)
    if (on && (same & ((1u << lane) - 1u)) == 0) {
      const long long at = row * a.ld_d + mine;
      if (a.bf16) {
        static_cast<__nv_bfloat16*>(a.dlogits)[at] = __float2bfloat16_rn(rest + sum);
      } else {
        static_cast<float*>(a.dlogits)[at] = rest + sum;
      }
    }
  }
}

zopt_status check(const char* fn, const zopt_route_job* c, bool backward) {
  const std::string f(fn);
  auto bad = [&](const char* what) { return fail(ZOPT_EINVAL, f + ": " + what); };
  if (c == nullptr) return bad("NULL job");
  if (c->dtype != ZOPT_F32 && c->dtype != ZOPT_BF16) return fail(ZOPT_EUNSUPPORTED, f + ": dtype must be ZOPT_F32 or ZOPT_BF16");
  if (c->score != ZOPT_SCORE_SOFTMAX && c->score != ZOPT_SCORE_SIGMOID)
    return bad("score must be ZOPT_SCORE_SOFTMAX or ZOPT_SCORE_SIGMOID");
  if (c->tokens < 0 || c->tokens > (1LL << 30)) return bad("tokens < 0 or above 2^30");
  if (c->experts < 1 || c->experts > kMaxExperts) return bad("experts outside 1 .. 1024");
  if (c->groups < 1 || c->groups > kMaxGroups || c->experts % c->groups != 0) return bad("groups outside 1 .. 32 or not dividing experts");
  if (c->top_groups < 1 || c->top_groups > c->groups) return bad("top_groups outside 1 .. groups");
  if (c->top_k < 1 || c->top_k > kMaxTopK || c->top_k > c->experts / c->groups * c->top_groups)
    return bad("top_k outside 1 .. 32 or above the experts that take part");
  if (c->renormalise != 0 && c->renormalise != 1) return bad("renormalise must be 0 or 1");
  if (!(c->scale > 0.0f && c->scale <= 3.402823466e38f)) return bad("scale must be positive and finite");
  if (c->reserved[0] != 0 || c->reserved[1] != 0) return bad("reserved must be 0");
  if (c->ld_logits < c->experts || c->ld_logits > (1LL << 32)) return bad("logits: a row distance below experts or above 2^32");
  const uintptr_t size = c->dtype == ZOPT_BF16 ? 2 : 4;
  auto off = [](const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
  if (off(c->bias, 4) || off(c->counts, 4) || off(c->index, 4) || off(c->weight, 4) || off(c->dweight, 4) ||
      off(c->logits, size) || off(c->dlogits, size))
    return bad("a pointer is not aligned to its element");
  if (c->tokens == 0) return ok();
  if (c->logits == nullptr || c->index == nullptr || c->weight == nullptr) return bad("NULL logits, index or weight");
  if (backward) {
    if (c->dweight == nullptr || c->dlogits == nullptr) return bad("NULL dweight or dlogits");
    if (c->ld_dlogits < c->experts || c->ld_dlogits > (1LL << 32)) return bad("dlogits: a row distance below experts or above 2^32");
  }
  return ok();
}

Args args_of(const zopt_route_job& c) {
  Args a{};
  a.logits = c.logits, a.ld = c.ld_logits;
  a.bias = c.bias, a.live = c.live;
  a.index = c.index, a.weight = c.weight, a.counts = c.counts, a.dweight = c.dweight;
  a.dlogits = c.dlogits, a.ld_d = c.ld_dlogits;
  a.tokens = c.tokens;
  a.experts = c.experts, a.top_k = c.top_k, a.groups = c.groups, a.top_groups = c.top_groups;
  a.per_group = Divisor(static_cast<uint32_t>(c.experts / c.groups));
  a.bf16 = c.dtype == ZOPT_BF16, a.renormalise = c.renormalise;
  a.scale = c.scale;
  return a;
}

template <int V>
zopt_status launch(Args& a, bool softmax, bool backward, unsigned blocks, cudaStream_t s) {
  const uintptr_t size = a.bf16 ? 2 : 4, piece = std::min<uintptr_t>(16, V * size);
  a.vec = reinterpret_cast<uintptr_t>(a.logits) % piece == 0 && a.ld * size % piece == 0;
  a.vec_d = reinterpret_cast<uintptr_t>(a.dlogits) % piece == 0 && a.ld_d * size % piece == 0;
  const int per = static_cast<int>(a.per_group.d), lanes = per / V;
  a.lanes_per_group = per % V == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
  const auto kernel = backward ? (softmax ? backward_kernel<V, true> : backward_kernel<V, false>)
                               : (softmax ? forward_kernel<V, true> : forward_kernel<V, false>);
  return launch_pdl(kernel, dim3(blocks), dim3(kThreads), 0, s, a);
}

zopt_status run(const char* fn, const zopt_route_job* cp, bool backward, cudaStream_t s) {
  const zopt_status st = check(fn, cp, backward);
  if (st != ZOPT_OK) return st;
  const zopt_route_job& c = *cp;
  Args a = args_of(c);
  if (c.tokens == 0) {
    if (!backward && c.counts != nullptr) ZOPT_CUDA_TRY(cudaMemsetAsync(c.counts, 0, sizeof(int32_t) * c.experts, s));
    return ok();
  }
  const int sms = sm_count();
  if (sms < 1) return fail(ZOPT_ECUDA, std::string(fn) + ": no CUDA device");
  const unsigned blocks = static_cast<unsigned>(std::min<long long>((c.tokens + kWarps - 1) / kWarps, 8LL * sms));
  a.alone = blocks == 1;
  if (!backward && c.counts != nullptr && !a.alone) ZOPT_CUDA_TRY(cudaMemsetAsync(c.counts, 0, sizeof(int32_t) * c.experts, s));
  const bool softmax = c.score == ZOPT_SCORE_SOFTMAX;
  const int v = (c.experts + 31) / 32;
  return v <= 1   ? launch<1>(a, softmax, backward, blocks, s)
         : v <= 2 ? launch<2>(a, softmax, backward, blocks, s)
         : v <= 4 ? launch<4>(a, softmax, backward, blocks, s)
         : v <= 8 ? launch<8>(a, softmax, backward, blocks, s)
         : v <= 16 ? launch<16>(a, softmax, backward, blocks, s)
                   : launch<32>(a, softmax, backward, blocks, s);
}

}  // namespace
}  // namespace route
}  // namespace zopt

extern "C" zopt_status zopt_route_forward(const zopt_route_job* job, zopt_stream stream) {
  return zopt::guarded([&] { return zopt::route::run("zopt_route_forward", job, false, stream); });
}

extern "C" zopt_status zopt_route_backward(const zopt_route_job* job, zopt_stream stream) {
  return zopt::guarded([&] { return zopt::route::run("zopt_route_backward", job, true, stream); });
}
