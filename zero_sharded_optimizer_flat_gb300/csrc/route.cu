// Routing tokens to experts, forward and backward.
//
// A warp takes a few tokens' rows one after another, a lane V experts that follow one another. Ranking is
// in exact order (of the score plus the bias as real numbers, the lowest index first among equal ones), so
// that a choice never depends on how an exponential rounds. An expert is one word: 22 bits that do not
// decrease with its rank's number, above 10 that fall with its index. A lane sorts its words once (a
// fixed network); the warp's largest word, an integer maximum, is the next choice, and its lane moves its
// words up. Without a bias the 22 bits are the logit's own leading ones (a bf16 logit's are all of
// it), with one, or with groups, the score's and the bias's sum in fixed point over the row's range.
// Neighbours in the order that come closer than those bits and the score's error tell apart have the
// warp rank their row again in fp64, and where fp64 is too coarse by sums of two parts. How many rows that are
// depends on the numbers (8192 rows of 256 experts): two in a thousand for logits of deviation 1 and biases of
// 0.02, 20 us; nearly all where scores crowd at 0 and 1 and the biases are equal (deviation 8, zeros), 80 us;
// biases that spread far (100: 23 us, 1e3: 35, 1e6 or the lowest value: 550) leave no word a meaning, every row is
// ranked from all its experts. Without a bias 15 us whatever the logits.
//
// The choices of the rows lie side by side in the warp's lanes, so that weights, checks and stores are
// done once for all of them, and two rows take turns, since a choice waits for the one before it.
//
// Bound by latency: a row's instructions (310 for eight of 128 experts, 18 of them a choice; 530 with a bias for
// eight of 256) hang on chains of choices, two rows' at a time, and fill 40 to 49 % of the issue slots while an SM
// has warps, 23 to 38 % of the whole time: 32768 x 128 in bf16 20.5 us, 0.4 TB/s; 8192 x 256 in eight groups with a
// bias 22 us, 16384 x 256 with a bias 25 (and 10 for the backward, which writes 17 MB in it). Tried: a row to eight
// or sixteen lanes, with 16 words each (a fifth fewer instructions, half the warps: 25 and 50 us), scores in fp64
// for whole rows (38 us: a close row took as long as the rest).
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
  int softmax, bf16, renormalise, alone;  // alone: one block has all rows, counts need no sum over blocks
  int width, rows;               // lanes for a row's choices (a power of two), rows of a warp at a time
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
          const uint4 x = reinterpret_cast<const uint4*>(p)[q];
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) l[8 * q + 2 * k] = __uint_as_float(w[k] << 16), l[8 * q + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
      } else if constexpr (V == 4) {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        l[0] = __uint_as_float(x.x << 16), l[1] = __uint_as_float(x.x & 0xFFFF0000u);
        l[2] = __uint_as_float(x.y << 16), l[3] = __uint_as_float(x.y & 0xFFFF0000u);
      } else if constexpr (V == 2) {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(p);
        l[0] = __uint_as_float(x << 16), l[1] = __uint_as_float(x & 0xFFFF0000u);
      }
    } else {
      const float* const p = static_cast<const float*>(a.logits) + row * a.ld + first;
      if constexpr (V >= 4) {
#pragma unroll
        for (int q = 0; q < V / 4; ++q) {
          const float4 x = reinterpret_cast<const float4*>(p)[q];
          l[4 * q] = x.x, l[4 * q + 1] = x.y, l[4 * q + 2] = x.z, l[4 * q + 3] = x.w;
        }
      } else if constexpr (V == 2) {
        const float2 x = *reinterpret_cast<const float2*>(p);
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
__device__ __forceinline__ float warp_max(float x) {  // (NaN: the others' largest)
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, d));
  return x;
}
template <typename T>
__device__ __forceinline__ T warp_sum(T x) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
  return x;
}
// Over `width` (a power of two) lanes side by side.
__device__ __forceinline__ float lanes_max(float x, int width) {
  for (int d = width >> 1; d >= 1; d >>= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, d));
  return x;
}
__device__ __forceinline__ float lanes_sum(float x, int width) {
  for (int d = width >> 1; d >= 1; d >>= 1) x += __shfl_xor_sync(kAll, x, d);
  return x;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// ---------------------------------------------------------------------- in fp64

// e^x, x at most 700, to some 2^-50: x = k ln 2 + r with |r| <= ln 2 / 2 (ln 2 in two parts, as Cody and Waite take
// it) and r's Taylor series. (The fp64 pipe is narrow, and this need not be exact to the last bit.)
__device__ __forceinline__ double exp64(double x) {
  x = x < -700.0 ? -700.0 : x > 700.0 ? 700.0 : x;  // (NaN stays)
  const double k = rint(x * 1.4426950408889634);
  const double r = fma(-k, 1.9082149292705877e-10, fma(-k, 0.693147180369123816490, x));
  double p = 1.0 / 479001600.0;
#pragma unroll
  for (int n = 11; n >= 0; --n) {
    constexpr double c[12] = {1.0,         1.0,          1.0 / 2.0,     1.0 / 6.0,      1.0 / 24.0,      1.0 / 120.0,
                              1.0 / 720.0, 1.0 / 5040.0, 1.0 / 40320.0, 1.0 / 362880.0, 1.0 / 3628800.0, 1.0 / 39916800.0};
    p = fma(p, r, c[n]);
  }
  return p * __longlong_as_double(static_cast<long long>(static_cast<uint64_t>(1023 + static_cast<int>(k)) << 52));
}

// A number in two parts, the second what the first's rounding left out: neither a score beside a bias of 1e10 nor
// the 1e-18 that a logistic score lacks of 1 is lost.
struct Sum {
  double hi, lo;
};
__device__ __forceinline__ Sum sum_of(double a, double b) {  // (Knuth's two-sum)
  const double s = a + b, v = s - a;
  return Sum{s, (a - (s - v)) + (b - v)};
}
__device__ __forceinline__ bool finite(double x) { return x - x == 0.0; }
// a and a small part more (Dekker's: the first is the larger one).
__device__ __forceinline__ Sum with(const Sum& a, double lo) {
  if (!finite(a.hi)) return Sum{a.hi, 0.0};
  const double l = a.lo + lo, s = a.hi + l;
  return Sum{s, l - (s - a.hi)};
}
__device__ __forceinline__ Sum operator+(const Sum& a, const Sum& b) { return with(sum_of(a.hi, b.hi), a.lo + b.lo); }

// What an expert (or a group) is ranked by: the parts of s + bias in turn, then the logit, in which s grows: what 53
// bits a part and exp64's range do not tell apart, it does where the biases are equal. hi 0: none.
struct Rank {
  uint64_t hi = 0, lo = 0;
  uint32_t l = 0;
};
__device__ __forceinline__ Rank rank_of(const Sum& c, float l) {
  Rank r;
  r.hi = key_of(c.hi);
  if (c.hi == c.hi) r.lo = finite(c.hi) ? key_of(c.lo) : 0, r.l = key_of(l);  // (NaN: equal to any other)
  return r;
}
__device__ __forceinline__ Sum of_rank(const Rank& r, int lane) {  // lane's, in every lane
  return Sum{of_key(__shfl_sync(kAll, r.hi, lane)), of_key(__shfl_sync(kAll, r.lo, lane))};
}
__device__ __forceinline__ bool above(const Rank& x, const Rank& y) {
  return x.hi != y.hi ? x.hi > y.hi : x.lo != y.lo ? x.lo > y.lo : x.l > y.l;
}
// The lanes that hold the warp's largest; 0: there is none.
__device__ __forceinline__ unsigned best_lanes(const Rank& r) {
  const uint64_t top = warp_max(r.hi);
  bool on = top != 0 && r.hi == top;
  unsigned who = __ballot_sync(kAll, on);
  if (__popc(who) > 1) {  // (the whole warp's)
    const uint64_t lo = warp_max(on ? r.lo : uint64_t{0});
    on = on && r.lo == lo;
    const uint32_t l = __reduce_max_sync(kAll, on ? r.l : 0u);
    on = on && r.l == l;
    who = __ballot_sync(kAll, on);
  }
  return who;
}

// The best `most` of the candidates, one a lane, the lowest index first among equal ones.
__device__ __forceinline__ int best_ranks(Rank r, int i, int most, int lane) {
  int mine = -1;
  for (int j = 0; j < most; ++j) {
    const unsigned who = best_lanes(r);
    if (who == 0) break;
    const bool on = ((who >> lane) & 1u) != 0;
    const int at = static_cast<int>(__reduce_min_sync(kAll, on ? static_cast<uint32_t>(i) : kAll));
    if (lane == j) mine = at;
    if (on && i == at) r = Rank{};
  }
  return mine;
}
// The same by single fp64 numbers, which is quicker; -2 in every lane where two neighbours in the order, from place
// `from` on and as far as the best one left out, are no further apart than such a number may be off (`off` of 1 and
// of the number itself; negative: they are exact).
__device__ __forceinline__ int best_keys(uint64_t key, int i, int most, int lane, int from, double off) {
  int mine = -1;
  uint64_t mine_key = 0;
  for (int j = 0; j < most; ++j) {
    const uint64_t top = warp_max(key);
    if (top == 0) break;
    const int at = static_cast<int>(__reduce_min_sync(kAll, key == top ? static_cast<uint32_t>(i) : kAll));
    if (lane == j) mine = at, mine_key = top;
    if (key == top && i == at) key = 0;
  }
  if (off < 0.0) return mine;
  const uint64_t left = warp_max(key), below = __shfl_down_sync(kAll, mine_key, 1), next = lane + 1 == most ? left : below;
  const double v = of_key(mine_key);
  const bool close = lane + 1 >= from && mine >= 0 && next != 0 && !(v - of_key(next) > off * (1.0 + fabs(v)));
  return __any_sync(kAll, close) ? -2 : mine;
}

// An expert's rank: its score and the bias, without a bias (but for groups' sums) its logit.
struct Rank64 {
  double m = 0.0, z = 1.0;
  __device__ __forceinline__ Sum score(const Args& a, float l, int i) const {
    const double x = static_cast<double>(l), b = a.bias != nullptr ? static_cast<double>(a.bias[i]) : 0.0;
    const double e = exp64(a.softmax ? x - m : -fabs(x));
    if (a.softmax) return sum_of(b, e / z);
    const double t = e / (1.0 + e);  // s, or where that is above 1/2 what it lacks of 1
    const Sum one = sum_of(l > 0.0f ? 1.0 : 0.0, b);
    return with(sum_of(one.hi, l > 0.0f ? -t : t), one.lo);
  }
  // The first part, to 2^-50 of 1 and 2^-52 of itself.
  __device__ __forceinline__ double about(const Args& a, float l, int i) const {
    const double x = static_cast<double>(l), e = exp64(a.softmax ? x - m : -x);
    const double s = a.softmax ? e / z : 1.0 / (1.0 + e);
    return a.bias != nullptr ? s + static_cast<double>(a.bias[i]) : s;
  }
  __device__ __forceinline__ Rank rank(const Args& a, float l, int i) const {
    return a.bias == nullptr ? rank_of(Sum{static_cast<double>(l), 0.0}, 0.0f) : rank_of(score(a, l, i), l);
  }
};

// What the sum of two of `about` may be off, of 1 and of itself; `most` is the largest bias.
__device__ __forceinline__ double group_off(float most) { return 0x1p-47 * (1.0 + static_cast<double>(most)); }

// A row's choice once more, from those alone whose word is `least` or more, in the groups given: lane j gets
// the j-th. They are few as a rule; they are listed, a lane takes each (the fp64 pipe being narrow), and more
// than 32 are left to choose_all.
// (kPlain: no bias, no groups: by the logits alone.)
template <int V, bool kPlain>
__device__ __noinline__ int choose_near(const Args& a, long long row, float lo, float scale, uint32_t least, uint32_t groups,
                                        uint16_t* list) {
  const int lane = threadIdx.x & 31, first = lane * V;
  float l[V];
  load_row<V>(a, row, first, l);
  Rank64 r;
  float m = 0.0f, rz = 1.0f;
  if (!kPlain && a.softmax) {
    m = l[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
    m = warp_max(m);
    double z = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) z += l[v] == -INFINITY ? 0.0 : exp64(static_cast<double>(l[v]) - static_cast<double>(m));
    r.m = static_cast<double>(m), r.z = warp_sum(z);
    rz = 1.0f / static_cast<float>(r.z);
  }
  int n = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = first + v;
    bool in = l[v] != -INFINITY && (kPlain || a.groups == 1 || ((groups >> a.per_group(static_cast<uint32_t>(i))) & 1u) != 0);
    if (!kPlain) {  // (as Chooser::words has it, but for the last bits)
      const float s = (a.softmax ? __expf(l[v] - m) * rz : 1.0f / (1.0f + __expf(-l[v]))) + (a.bias != nullptr && i < a.experts ? a.bias[i] : 0.0f);
      in = in && (s - lo) * scale + 16.0f >= static_cast<float>(least);
    } else {
      in = in && (key_of(l[v]) >> 10) >= least;
    }
    const unsigned who = __ballot_sync(kAll, in);
    const int at = n + __popc(who & ((1u << lane) - 1u));
    if (in && at < 32) list[at] = static_cast<uint16_t>(i);
    n += __popc(who);
  }
  __syncwarp();
  if (n > 32) return -2;
  const int i = lane < n ? list[lane] : -1;
  __syncwarp();
  const float li = i >= 0 ? load(a, row, i) : 0.0f;
  const bool exact = kPlain || a.bias == nullptr;
  const double c = exact ? static_cast<double>(li) : i >= 0 ? r.about(a, li, i) : 0.0;
  const int got = best_keys(i >= 0 ? key_of(c) : 0, i, a.top_k, lane, 1, exact ? -1.0 : 0x1p-48);
  if (kPlain || got != -2) return got;  // (-2: the whole warp's)
  return best_ranks(i >= 0 ? r.rank(a, li, i) : Rank{}, i, a.top_k, lane);
}

// A row's choice once more, from all its experts, the groups ranked again as well. Lane l looks at experts l,
// l + 32, ....
template <bool kPlain>
__device__ __noinline__ int choose_all(const Args& a, long long row) {
  const int lane = threadIdx.x & 31;
  Rank64 r;
  if (!kPlain && a.softmax && (a.bias != nullptr || a.groups > 1)) {
    float m = -INFINITY;
    for (int i = lane; i < a.experts; i += 32) m = fmaxf(m, load(a, row, i));
    m = warp_max(m);
    double part = 0.0;
    for (int i = lane; i < a.experts; i += 32) part += exp64(static_cast<double>(load(a, row, i)) - static_cast<double>(m));
    r.m = static_cast<double>(m), r.z = warp_sum(part);
    if (!(m < INFINITY)) r.z = __longlong_as_double(0x7FF8000000000000ll);
  }
  uint32_t groups = kAll, gone = 0;
  if (!kPlain && a.groups > 1) {
    const int per = static_cast<int>(a.per_group.d);
    uint64_t sum_key = 0;
    float most = 0.0f;  // the largest bias
    for (int i = lane; a.bias != nullptr && i < a.experts; i += 32) most = fmaxf(most, fabsf(a.bias[i]));
    most = warp_max(most);
    for (int g = 0; g < a.groups; ++g) {
      uint64_t first = 0, second = 0;
      for (int i = g * per + lane; i < (g + 1) * per; i += 32) {
        const float l = load(a, row, i);
        if (l == -INFINITY) continue;
        const uint64_t k = key_of(r.about(a, l, i));
        second = k > first ? first : k > second ? k : second;
        first = k > first ? k : first;
      }
      const uint64_t one = warp_max(first);
      const int owner = __ffs(__ballot_sync(kAll, first == one)) - 1;
      const uint64_t two = warp_max(lane == owner ? second : first);
      if (lane == g) sum_key = one == 0 ? 0 : two == 0 ? one : key_of(of_key(one) + of_key(two));
    }
    int best_group = best_keys(sum_key, lane, a.top_groups, lane, a.top_groups, group_off(most));
    if (best_group == -2) {  // (in every lane: the same by two-part sums)
      Rank mine;
      for (int g = 0; g < a.groups; ++g) {
        Rank first, second;
        for (int i = g * per + lane; i < (g + 1) * per; i += 32) {
          const float l = load(a, row, i);
          if (l == -INFINITY) continue;
          const Rank k = rank_of(r.score(a, l, i), l);
          if (above(k, first)) {
            second = first, first = k;
          } else if (above(k, second)) {
            second = k;
          }
        }
        const unsigned one = best_lanes(first);
        if (one == 0) continue;  // (the whole warp's)
        const int owner = __ffs(one) - 1;
        Sum sum = of_rank(first, owner);
        if (lane == owner) first = second;
        const unsigned two = best_lanes(first);
        if (two != 0) sum = sum + of_rank(first, __ffs(two) - 1);
        if (lane == g) mine = rank_of(sum, 0.0f);
      }
      best_group = best_ranks(mine, lane, a.top_groups, lane);
    }
    groups = __reduce_or_sync(kAll, best_group >= 0 ? 1u << best_group : 0u);
  }
  // A lane keeps its two best: it looks through its experts again when both have been taken.
  Rank best, next;
  int mine = -1, at = -1, at_next = -1;
  bool more = true;
  for (int j = 0; j < a.top_k; ++j) {
    if (__any_sync(kAll, at < 0 && more)) {
      best = next = Rank{};
      at = at_next = -1;
      more = false;
      for (int i = lane, v = 0; i < a.experts; i += 32, ++v) {
        const float l = load(a, row, i);
        if (((gone >> v) & 1u) != 0 || l == -INFINITY) continue;
        if (!kPlain && a.groups > 1 && ((groups >> a.per_group(static_cast<uint32_t>(i))) & 1u) == 0) continue;
        const Rank k = kPlain ? rank_of(Sum{static_cast<double>(l), 0.0}, 0.0f) : r.rank(a, l, i);
        more = at_next >= 0;
        if (above(k, best)) {
          next = best, at_next = at;
          best = k, at = i;
        } else if (above(k, next)) {
          next = k, at_next = i;
        }
      }
    }
    const unsigned who = best_lanes(best);
    if (who == 0) break;
    const bool on = ((who >> lane) & 1u) != 0;
    const int i = static_cast<int>(__reduce_min_sync(kAll, on ? static_cast<uint32_t>(at) : kAll));
    if (lane == j) mine = i;
    if (on && at == i) {
      gone |= 1u << (i >> 5);
      best = next, at = at_next;
      next = Rank{}, at_next = -1;
    }
  }
  return mine;
}

// The groups that take part, from the two best experts of each (lane g: group g's; -1: there is none), in fp64; 0:
// it does not tell. Logistic scores; `most` is the largest bias. (Called amid a row's words: its registers are theirs.)
__device__ __noinline__ uint32_t groups64(const Args& a, long long row, int one, int two, float most) {
  const Rank64 r;
  const int lane = threadIdx.x & 31;
  double sum = 0.0;
  if (one >= 0) sum = r.about(a, load(a, row, one), one);
  if (two >= 0) sum += r.about(a, load(a, row, two), two);
  const int g = best_keys(one >= 0 ? key_of(sum) : 0, lane, a.top_groups, lane, a.top_groups, group_off(most));
  return g == -2 ? 0u : __reduce_or_sync(kAll, g >= 0 ? 1u << g : 0u);
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

// What a rank in fp32 may be off, in units of 2^-24. A logistic score: its exponential's 2^-22 and its
// argument's rounding weigh at most a quarter, the sum and the reciprocal are 2^-24 and 2^-23: 5. A
// softmax score, of the row's largest: an exponential (5), the sum of V terms a lane over the warp's
// lanes (V + 5) and the reciprocal and products (5). What is made of it and the bias: 2 of their terms.
constexpr float kUnit = 1.0f / (1 << 24);
// 2^23, what brings a number below 2^22 into the low bits of its fp32 pattern.
constexpr float kMagic = 8388608.0f;

// What a batch of rows has in its lanes: lane r W + j row r's j-th choice, and in all of a row's W lanes
// what else is known of the row.
struct Batch {
  uint32_t mine = 0;       // the choice's word
  uint32_t left = 0;       // the best word that was left out
  int near = -1;           // ranks this close or closer need a second look
  float scale = 0.0f;      // of fixed point (0: the words are of logits)
  uint32_t groups = kAll;  // those that take part
  bool all = false;        // its groups may be others, or a number was none: choose_all
  bool bad = false;        // softmax: a NaN or +inf
  float m = 0.0f, z = 1.0f;  // softmax: the largest logit and the sum relative to it
};

template <int V, bool kPlain>
struct Chooser {
  const Args& a;
  int lane, first;
  float b[V], lo = 0.0f, hi = 0.0f;

  __device__ __forceinline__ explicit Chooser(const Args& args) : a(args), lane(threadIdx.x & 31), first(lane * V) {
#pragma unroll
    for (int v = 0; v < V; ++v) b[v] = 0.0f;
    if (kPlain || a.bias == nullptr) return;
    lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (first + v >= a.experts) continue;
      b[v] = a.bias[first + v];
      lo = fminf(lo, b[v]), hi = fmaxf(hi, b[v]);
    }
    lo = -warp_max(-lo), hi = warp_max(hi);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (first + v >= a.experts) b[v] = lo;  // (behind the last one: within the range, as the check in words() wants it)
  }
  __device__ __forceinline__ uint32_t name(int v) const { return kIndexMask - static_cast<uint32_t>(first + v); }

  // The words of the groups that take part, sorted; what the row's lanes have to know goes to r.
  __device__ __forceinline__ void choose_groups(uint32_t (&w)[V], long long row, float unit, int near, Batch& r) const {
    auto value = [&](uint32_t word) { return lo + unit * static_cast<float>(word >> kIndexBits); };
    // a group's sum, its name (the lowest first among equal sums) in the low bits
    auto sum_of = [&](uint32_t one, uint32_t two, int g) {
      return one == 0 ? 0u : (key_of(two == 0 ? value(one) : value(one) + value(two)) & ~31u) | (31u - static_cast<uint32_t>(g));
    };
    uint32_t sum = 0, one = 0, two = 0;  // (in_lane: of the lane's group; else of group `lane`)
    const bool in_lane = a.lanes_per_group > 0;
    if (in_lane) {  // a group is a power of two of lanes: their first two words are merged
      sort_words<V>(w);
      one = w[0], two = V > 1 ? w[V > 1 ? 1 : 0] : 0u;
      for (int d = 1; d < a.lanes_per_group; d <<= 1) {
        const uint32_t x = __shfl_xor_sync(kAll, one, d), y = __shfl_xor_sync(kAll, two, d);
        two = max(min(one, x), max(two, y));
        one = max(one, x);
      }
      const int g = lane / a.lanes_per_group;
      if (lane % a.lanes_per_group == 0 && g < a.groups) sum = sum_of(one, two, g);
    } else {  // one group after another
      for (int g = 0; g < a.groups; ++g) {
        uint32_t x = 0, y = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const uint32_t k = static_cast<int>(a.per_group(static_cast<uint32_t>(first + v))) == g ? w[v] : 0u;
          y = max(y, min(x, k));
          x = max(x, k);
        }
        const uint32_t top = __reduce_max_sync(kAll, x), next = __reduce_max_sync(kAll, x == top ? y : x);
        if (lane == g) one = top, two = next, sum = sum_of(top, next, g);
      }
    }
    uint32_t mask = 0, worst = 0;
    for (int j = 0; j < a.top_groups; ++j) {
      const uint32_t top = __reduce_max_sync(kAll, sum);
      if (top == 0) break;  // (the whole warp's)
      worst = top;
      mask |= 1u << (31u - (top & 31u));
      if (sum == top) sum = 0;
    }
    const uint32_t left = __reduce_max_sync(kAll, sum);
    const float in = of_key(worst & ~31u), out = of_key(left & ~31u);
    // (32 ulp of each go with their names)
    if (left != 0 && !(in - out > 2.0f * (near + 1) * unit + 80.0f * kUnit * (fabsf(in) + fabsf(out)))) {
      // The sums again in fp64, if it is clear which two experts they are of and (softmax) no sum is needed.
      bool third = false;
      if (in_lane) {
#pragma unroll
        for (int v = 0; v < V; ++v)
          third = third || (w[v] != 0 && w[v] < two && static_cast<int>((two >> kIndexBits) - (w[v] >> kIndexBits)) <= near);
      }
      if (!in_lane || a.softmax || __any_sync(kAll, third)) {
        r.all = true;
      } else {
        const int from = min(lane * a.lanes_per_group, 31);
        const uint32_t x = __shfl_sync(kAll, one, from), y = __shfl_sync(kAll, two, from);
        auto expert = [&](uint32_t word) { return lane < a.groups && word != 0 ? static_cast<int>(kIndexMask - (word & kIndexMask)) : -1; };
        mask = groups64(a, row, expert(x), expert(y), fmaxf(fabsf(lo), fabsf(hi)));
        r.all = r.all || mask == 0;
      }
    }
    r.groups = mask;
    if (in_lane) {
      const int g = lane / a.lanes_per_group;
      if (g >= a.groups || ((mask >> g) & 1u) == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) w[v] = 0;
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (first + v < a.experts && ((mask >> a.per_group(static_cast<uint32_t>(first + v))) & 1u) == 0) w[v] = 0;
      sort_words<V>(w);
    }
  }

  // A row's words, sorted, and what else its lanes have to know of it.
  __device__ __forceinline__ void words(const float (&l)[V], long long at, uint32_t (&w)[V], Batch& r) const {
    // (of a 1024th of each: no sum of finite ones overflows)
    float size = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) size = fmaf(l[v], 1.0f / 1024.0f, size);
    r.bad = __any_sync(kAll, !(size < INFINITY));
    if (a.softmax && !(kPlain && a.renormalise)) {
      r.m = l[0];
#pragma unroll
      for (int v = 1; v < V; ++v) r.m = fmaxf(r.m, l[v]);
      r.m = warp_max(r.m);
    }
    if constexpr (kPlain) {
      if (a.softmax && !a.renormalise) {
        float z = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) z += l[v] == -INFINITY ? 0.0f : ex2((l[v] - r.m) * kLog2e);
        r.z = warp_sum(z);
      }
      r.near = a.bf16 ? -1 : 0;  // (of a bf16 logit 16 bits are all there is)
      r.all = r.bad;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint32_t u = __float_as_uint(l[v] + 0.0f);  // -0 is 0
        const uint32_t key = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
        w[v] = l[v] == -INFINITY ? 0u : (key & ~kIndexMask) | name(v);
      }
      sort_words<V>(w);
    } else {
      float s[V], rz = 1.0f;
      if (a.softmax) {
        float z = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = ex2((l[v] - r.m) * kLog2e), z += s[v];
        r.z = warp_sum(z);
        rz = rcp(r.z);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) s[v] = rcp(1.0f + ex2(l[v] * -kLog2e));
      }
      const float range = rz + (hi - lo), scale = (kTopRank - 3) * rcp(range), from = rz * scale;
      uint32_t seen = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) {  // rank = 1 + (s + b - lo) scale, rounded into the low bits
        const uint32_t u = __float_as_uint(fmaf(s[v], from, fmaf(b[v] - lo, scale, kMagic + 1.0f)));
        seen |= u;
        w[v] = l[v] == -INFINITY ? 0u : (u << kIndexBits) | name(v);
      }
      // (a number that is none has other leading bits than 2^23's; a range from 2^104 on leaves no word a meaning:
      // its reciprocal flushes to 0 from 2^126 on)
      r.all = __any_sync(kAll, (seen >> 23) != (__float_as_uint(kMagic) >> 23)) || !(range < 0x1p104f);
      const float off = kUnit * (2.0f * (a.softmax ? (V + 15) * rz : 5.0f) + 4.0f * (fabsf(lo) + fabsf(hi) + range));
      // (and two units of each of the two; biases may be so much larger than the range that every rank is this near)
      r.near = static_cast<int>(fminf(off * scale, static_cast<float>(kTopRank))) + 4;
      r.scale = scale;
      if (a.groups > 1) {
        choose_groups(w, at, range * (1.0f / (kTopRank - 3)), r.near, r);
      } else {
        sort_words<V>(w);
      }
    }
  }

  // kRows rows' choices, the k-th row's into the `width` lanes from (k0 + k) width on. Rows that take turns hide
  // one another's latencies; a choice that there is not is 0, and so is any after it.
  template <int kRows>
  __device__ __forceinline__ void rows(const float (&l)[kRows][V], long long at, int k0, Batch& batch) const {
    uint32_t w[kRows][V];
    Batch r[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) words(l[k], at + k, w[k], r[k]);
    const int slot = lane - k0 * a.width;
#pragma unroll 2
    for (int n = 0; n < a.top_k; ++n) {
      uint32_t top[kRows];
#pragma unroll
      for (int k = 0; k < kRows; ++k) top[k] = __reduce_max_sync(kAll, w[k][0]);
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        if (slot - k * a.width == n) batch.mine = top[k];
        drop_first<V>(w[k], w[k][0] == top[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      r[k].left = __reduce_max_sync(kAll, w[k][0]);
      if (slot >= k * a.width && slot < (k + 1) * a.width) {
        r[k].mine = batch.mine;
        batch = r[k];
      }
    }
  }
};

template <int V, bool kPlain>
__global__ void __launch_bounds__(kThreads, V >= 16 ? 2 : V >= 8 ? 3 : 4) forward_kernel(const Args a) {
  __shared__ int count[kMaxExperts];
  __shared__ uint16_t list[kWarps][32];
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  if (a.counts != nullptr) {
    for (int i = threadIdx.x; i < a.experts; i += kThreads) count[i] = 0;
    __syncthreads();
  }
  const Chooser<V, kPlain> chooser(a);
  const int lane = threadIdx.x & 31, W = a.width, j = lane & (W - 1), which = lane / W;
  const long long step = static_cast<long long>(gridDim.x) * kWarps * a.rows;
  for (long long row0 = (static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * a.rows; row0 < a.tokens; row0 += step) {
    const int n = static_cast<int>(min(static_cast<long long>(a.rows), a.tokens - row0));
    // bit r: row row0 + r is no padding
    const uint32_t live = __ballot_sync(kAll, lane < n && (a.live == nullptr || a.live[row0 + lane] != 0));
    Batch r;
    // (the next rows are on their way while some are worked on; padding has none)
    constexpr int kRows = V <= 8 ? 2 : 1;
    float next[kRows][V];
    auto fetch = [&](int k) {
#pragma unroll
      for (int q = 0; q < kRows; ++q) {
#pragma unroll
        for (int v = 0; v < V; ++v) next[q][v] = -INFINITY;
        if (k + q < n && ((live >> (k + q)) & 1u)) load_row<V>(a, row0 + k + q, chooser.first, next[q]);
      }
    };
    fetch(0);
    for (int k = 0; k < n; k += kRows) {
      float l[kRows][V];
#pragma unroll
      for (int q = 0; q < kRows; ++q)
#pragma unroll
        for (int v = 0; v < V; ++v) l[q][v] = next[q][v];
      if (k + kRows < n) fetch(k + kRows);
      if ((live >> k) == 0) break;
      if (kRows == 2 && ((live >> k) & 2u) != 0) {
        chooser.template rows<kRows>(l, row0 + k, k, r);
      } else if ((live >> k) & 1u) {
        const float (&one)[1][V] = reinterpret_cast<const float (&)[1][V]>(l);
        chooser.template rows<1>(one, row0 + k, k, r);
      }
    }
    const long long row = row0 + which;
    const bool there = which < n && ((live >> which) & 1u) != 0;
    int mine = r.mine == 0 ? -1 : static_cast<int>(kIndexMask - (r.mine & kIndexMask));
    // neighbours in the order, and the last one against the best that was left out
    const int rank = static_cast<int>(r.mine >> kIndexBits), below = static_cast<int>(r.left >> kIndexBits);
    const int after = __shfl_down_sync(kAll, rank, 1);
    const bool close = j + 1 < a.top_k ? after > 0 && rank - after <= r.near : j + 1 == a.top_k && rank > 0 && below > 0 && rank - below <= r.near;
    unsigned todo = __ballot_sync(kAll, there && (close || r.all));
    while (todo != 0) {
      const int from = (__ffs(todo) - 1) / W * W;  // the row's first lane
      const int least = __shfl_sync(kAll, rank, from + a.top_k - 1) - __shfl_sync(kAll, r.near, from);
      const bool all = __shfl_sync(kAll, r.all ? 1 : 0, from) != 0;
      int got = -2;
      if (!all)
        got = choose_near<V, kPlain>(a, row0 + from / W, chooser.lo, __shfl_sync(kAll, r.scale, from), static_cast<uint32_t>(max(least, 1)),
                             __shfl_sync(kAll, r.groups, from), list[threadIdx.x >> 5]);
      if (got == -2) got = choose_all<kPlain>(a, row0 + from / W);  // (-2 in every lane)
      const int here = __shfl_sync(kAll, got, j);
      if (lane - j == from) mine = j < a.top_k ? here : -1;
      todo &= ~((W == 32 ? kAll : (1u << W) - 1u) << from);
    }
    const bool on = there && mine >= 0;
    const float ml = on ? load(a, row, mine) : -INFINITY;
    float w;
    if (a.softmax) {
      // relative to the largest logit: of the chosen ones where the weights are renormalised (the other
      // terms cancel), else of all. A row with a NaN or +inf has no softmax.
      const float top = a.renormalise ? lanes_max(ml, W) : r.m;
      w = on ? ex2((ml - top) * kLog2e) : 0.0f;
      const float z = a.renormalise ? lanes_sum(w, W) : r.z;
      w = on ? __fdividef(w, z) * a.scale : 0.0f;
      if (r.bad && on) w = __uint_as_float(0x7FC00000u);
    } else {
      // s = e^l / (1 + e^l); where all chosen logits are negative, e^(l - max) in its place where the
      // weights are renormalised: the quotients stay what they are and nothing underflows.
      const float top = a.renormalise ? fminf(0.0f, lanes_max(ml, W)) : 0.0f;
      const float e = ex2(-fabsf(ml) * kLog2e);
      w = !on ? 0.0f : __fdividef(ml >= 0.0f ? 1.0f : top < 0.0f ? ex2((ml - top) * kLog2e) : e, 1.0f + e);
      if (a.renormalise) w = __fdividef(w, lanes_sum(w, W));
      w = on ? w * a.scale : 0.0f;
    }
    if (j < a.top_k && which < n) {
      a.index[row * a.top_k + j] = on ? mine : -1;
      a.weight[row * a.top_k + j] = w;
      if (a.counts != nullptr && on) atomicAdd(count + mine, 1);
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
// As in the forward the slots of a warp's rows lie side by side in its lanes. A row is written whole, with
// what the chosen experts' entries would be if they had not been chosen, and then all the chosen ones' again,
// a lane each. Bound by what it writes.
template <int V>
__global__ void __launch_bounds__(kThreads) backward_kernel(const Args a) {
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int lane = threadIdx.x & 31, first = lane * V, W = a.width, j = lane & (W - 1), which = lane / W;
  const float nan = __uint_as_float(0x7FC00000u);
  const bool dense = a.softmax && !a.renormalise;
  const long long step = static_cast<long long>(gridDim.x) * kWarps * a.rows;
  for (long long row0 = (static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * a.rows; row0 < a.tokens; row0 += step) {
    const int n = static_cast<int>(min(static_cast<long long>(a.rows), a.tokens - row0));
    const long long row = row0 + which, slot = row * a.top_k + j;
    int mine = -1;
    float w = 0.0f, g = 0.0f, ml = 0.0f;
    if (which < n && j < a.top_k) mine = a.index[slot];
    const bool on = mine >= 0 && mine < a.experts;
    const unsigned none = __ballot_sync(kAll, mine != -1 && !on), some = __ballot_sync(kAll, on);
    if (on) {
      w = a.weight[slot];
      g = a.dweight[slot];
      if (a.softmax ? dense : true) ml = load(a, row, mine);
    }
    const float mean = lanes_sum(g * w, W) / a.scale;
    float d = (a.renormalise ? g - mean : g) * w;
    if (!a.softmax) d *= 1.0f / (1.0f + expf(ml));  // 1 - s
    float rest = 0.0f;  // what the lane's expert would have if it were not chosen
    const unsigned lanes = W == 32 ? kAll : (1u << W) - 1u;  // a row's
    for (int k = 0; k < n; ++k) {
      const bool bad = ((none >> (k * W)) & lanes) != 0;
      float out[V];
#pragma unroll
      for (int v = 0; v < V; ++v) out[v] = bad ? nan : 0.0f;
      if (dense && !bad && ((some >> (k * W)) & lanes) != 0) {
        load_row<V>(a, row0 + k, first, out);
        float m = out[0], z = 0.0f;
#pragma unroll
        for (int v = 1; v < V; ++v) m = fmaxf(m, out[v]);
        m = warp_max(m);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          out[v] = out[v] == -INFINITY ? 0.0f : expf(out[v] - m);
          z += out[v];
        }
        const float f = -__shfl_sync(kAll, mean, k * W) * a.scale / warp_sum(z);
#pragma unroll
        for (int v = 0; v < V; ++v) out[v] *= f;
        if (which == k && on) rest = expf(ml - m) * f;
      }
      store_row<V>(a, row0 + k, first, out);
    }
    // an expert that a row names more than once takes all its slots' parts, in their order
    const unsigned same = __match_any_sync(kAll, on ? which * kMaxExperts + mine : -1 - lane);
    float sum = d;
    if (__any_sync(kAll, __popc(same) > 1)) {
      sum = 0.0f;
      for (int q = 0; q < 32; ++q) {
        const float x = __shfl_sync(kAll, d, q);
        if ((same >> q) & 1u) sum += x;
      }
    }
    __syncwarp();  // (orders the two stores to one address)
    if (on && (same & ((1u << lane) - 1u)) == 0 && ((none >> (which * W)) & lanes) == 0) {
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
  a.softmax = c.score == ZOPT_SCORE_SOFTMAX;
  a.bf16 = c.dtype == ZOPT_BF16, a.renormalise = c.renormalise;
  a.scale = c.scale;
  return a;
}

// Rows of a warp at a time: as many as its lanes hold the choices of, but not so many that fewer than 16
// warps an SM have some.
void set_rows(Args& a, int sms) {
  for (a.width = 1; a.width < a.top_k;) a.width *= 2;
  a.rows = static_cast<int>(std::max<long long>(1, std::min<long long>(32 / a.width, a.tokens / (16LL * sms))));
}

template <int V>
zopt_status launch_forward(Args a, int sms, cudaStream_t s) {
  const uintptr_t size = a.bf16 ? 2 : 4, piece = std::min<uintptr_t>(16, V * size);
  a.vec = reinterpret_cast<uintptr_t>(a.logits) % piece == 0 && a.ld * size % piece == 0;
  const int per = static_cast<int>(a.per_group.d), lanes = per / V;
  a.lanes_per_group = per % V == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
  set_rows(a, sms);
  const auto kernel = a.bias == nullptr && a.groups == 1 ? forward_kernel<V, true> : forward_kernel<V, false>;
  const long long rows = static_cast<long long>(kWarps) * a.rows;
  const unsigned blocks = static_cast<unsigned>(std::min<long long>((a.tokens + rows - 1) / rows, 8LL * sms));
  a.alone = blocks == 1;
  if (a.counts != nullptr && !a.alone) ZOPT_CUDA_TRY(cudaMemsetAsync(a.counts, 0, sizeof(int32_t) * a.experts, s));
  return launch_pdl(kernel, dim3(blocks), dim3(kThreads), 0, s, a);
}
template <int V>
zopt_status launch_backward(Args a, int sms, cudaStream_t s) {
  const uintptr_t size = a.bf16 ? 2 : 4, piece = std::min<uintptr_t>(16, V * size);
  a.vec = reinterpret_cast<uintptr_t>(a.logits) % piece == 0 && a.ld * size % piece == 0;
  a.vec_d = reinterpret_cast<uintptr_t>(a.dlogits) % piece == 0 && a.ld_d * size % piece == 0;
  set_rows(a, sms);
  const long long rows = static_cast<long long>(kWarps) * a.rows;
  const unsigned blocks = static_cast<unsigned>(std::min<long long>((a.tokens + rows - 1) / rows, 8LL * sms));
  return launch_pdl(backward_kernel<V>, dim3(blocks), dim3(kThreads), 0, s, a);
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
  const int e = c.experts;
  if (backward) {
    return e <= 32    ? launch_backward<1>(a, sms, s)
           : e <= 64  ? launch_backward<2>(a, sms, s)
           : e <= 128 ? launch_backward<4>(a, sms, s)
           : e <= 256 ? launch_backward<8>(a, sms, s)
                      : launch_backward<32>(a, sms, s);
  }
  return e <= 32    ? launch_forward<1>(a, sms, s)
         : e <= 64  ? launch_forward<2>(a, sms, s)
         : e <= 128 ? launch_forward<4>(a, sms, s)
         : e <= 256 ? launch_forward<8>(a, sms, s)
         : e <= 512 ? launch_forward<16>(a, sms, s)
                    : launch_forward<32>(a, sms, s);
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
