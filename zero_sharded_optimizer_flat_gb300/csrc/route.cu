// Routing tokens to experts, forward and backward.
//
// A warp takes a token's row: lane l holds experts l, l + 32, ... in registers. Ranking is in exact
// order (of the score plus the bias as real numbers, the lowest index first among equal ones), so that
// a choice never depends on how an exponential rounds. Without a bias that is the logits' own order.
// With one, or with groups, scores are formed in fp32 and every comparison that decides something is
// held against their error; a row that has a closer one is ranked again in fp64 (one row in some
// thousands).
//
// The largest of a row is found by an integer maximum over the warp of an order-preserving key, its
// index by a minimum, top_k times.
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
  float scale;
};

__device__ __forceinline__ float load(const Args& a, long long row, int i) {
  const long long at = row * a.ld + i;
  return a.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[at]) : static_cast<const float*>(a.logits)[at];
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
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(kAll, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
  const uint32_t hi = static_cast<uint32_t>(k >> 32), top = __reduce_max_sync(kAll, hi);
  const uint32_t lo = __reduce_max_sync(kAll, hi == top ? static_cast<uint32_t>(k) : 0u);
  return (static_cast<uint64_t>(top) << 32) | lo;
}
__device__ __forceinline__ float warp_max(float x) {
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

// The first register (lowest index) that holds the lane's largest key.
template <int V, typename K>
__device__ __forceinline__ K lane_max(const K (&key)[V], int& at) {
  K best = key[0];
  at = 0;
#pragma unroll
  for (int v = 1; v < V; ++v)
    if (key[v] > best) best = key[v], at = v;
  return best;
}
template <int V, typename K>
__device__ __forceinline__ void clear(K (&key)[V], int v) {
#pragma unroll
  for (int q = 0; q < V; ++q)
    if (q == v) key[q] = 0;
}

// The `most` best, one after another: lane j gets the j-th one's index (-1: there is none), and the
// keys of those taken become 0.
template <int V, typename K>
__device__ __forceinline__ int take_best(K (&key)[V], int most, int lane) {
  int mine = -1;
  for (int j = 0; j < most; ++j) {
    int at;
    const K best = lane_max<V>(key, at);
    const K top = warp_max(best);
    if (top == 0) break;
    const uint32_t i = __reduce_min_sync(kAll, best == top ? static_cast<uint32_t>(lane + 32 * at) : kAll);
    if (lane == j) mine = static_cast<int>(i);
    if ((i & 31u) == static_cast<uint32_t>(lane)) clear<V>(key, static_cast<int>(i >> 5));
  }
  return mine;
}

// Lane g's key of the sum of group g's two largest (the largest alone where there is one; 0: none).
template <int V, typename K>
__device__ __forceinline__ K group_keys(const K (&key)[V], const Args& a, int lane) {
  K mine = 0;
  for (int g = 0; g < a.groups; ++g) {
    K in[V];
#pragma unroll
    for (int v = 0; v < V; ++v) in[v] = static_cast<int>(a.per_group(static_cast<uint32_t>(lane + 32 * v))) == g ? key[v] : 0;
    int at;
    K best = lane_max<V>(in, at);
    const K first = warp_max(best);
    const uint32_t i = __reduce_min_sync(kAll, best == first ? static_cast<uint32_t>(lane + 32 * at) : kAll);
    if ((i & 31u) == static_cast<uint32_t>(lane)) clear<V>(in, static_cast<int>(i >> 5));
    best = lane_max<V>(in, at);
    const K second = warp_max(best);
    if (lane == g) mine = first == 0 ? 0 : second == 0 ? first : key_of(of_key(first) + of_key(second));
  }
  return mine;
}

// The mask of the groups that take part, from lane g's key of group g.
template <typename K>
__device__ __forceinline__ uint32_t best_groups(K key, const Args& a, int lane) {
  K k[1] = {key};
  const int g = take_best<1>(k, a.top_groups, lane);
  return __reduce_or_sync(kAll, g >= 0 ? 1u << g : 0u);
}

template <int V, typename K>
__device__ __forceinline__ void drop_groups(K (&key)[V], uint32_t mask, const Args& a, int lane) {
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (lane + 32 * v < a.experts && ((mask >> a.per_group(static_cast<uint32_t>(lane + 32 * v))) & 1u) == 0) key[v] = 0;
}

// A row's choice with everything in fp64.
template <int V, bool kSoftmax>
__device__ __noinline__ int choose64(const Args& a, long long row, int lane) {
  uint64_t key[V];
  double top = 0.0, rz = 1.0;
  if (kSoftmax) {
    float m = -INFINITY;
    for (int i = lane; i < a.experts; i += 32) m = fmaxf(m, load(a, row, i));
    top = static_cast<double>(warp_max(m));
    double z = 0.0;
    for (int i = lane; i < a.experts; i += 32) z += exp(static_cast<double>(load(a, row, i)) - top);
    rz = warp_sum(z);
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = lane + 32 * v;
    key[v] = 0;
    if (i >= a.experts) continue;
    const double l = static_cast<double>(load(a, row, i));
    const double s = kSoftmax ? exp(l - top) / rz : 1.0 / (1.0 + exp(-l));
    if (l != -INFINITY) key[v] = key_of(a.bias != nullptr ? s + static_cast<double>(a.bias[i]) : s);
  }
  if (a.groups > 1) {
    drop_groups<V>(key, best_groups(group_keys<V>(key, a, lane), a, lane), a, lane);
    if (a.bias == nullptr) {  // within the groups the logits' own order, as everywhere without a bias
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (key[v] != 0) key[v] = key_of(static_cast<double>(load(a, row, lane + 32 * v)));
    }
  }
  return take_best<V>(key, a.top_k, lane);
}

// What is reckoned with, in units of 2^-24: for a score in fp32, of the row's largest, an exponential
// and divisions (8), and for the softmax a sum of V terms a lane over the warp as well; for sums with a
// bias or of two scores, of their terms, 4.
constexpr float kUnit = 1.0f / (1 << 24), kSumError = 4.0f * kUnit;

template <int V, bool kSoftmax>
__device__ __forceinline__ int choose(const Args& a, long long row, const float (&l)[V], int lane) {
  uint32_t key[V];
  if (a.bias == nullptr && a.groups == 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = l[v] == -INFINITY ? 0u : key_of(l[v]);
    return take_best<V>(key, a.top_k, lane);
  }
  float m = 0.0f, rz = 1.0f;
  if (kSoftmax) {
    m = l[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = fmaxf(m, l[v]);
    m = warp_max(m);
    float z = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) z += expf(l[v] - m);
    rz = 1.0f / warp_sum(z);
  }
  float c[V], b[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = lane + 32 * v;
    b[v] = a.bias != nullptr && i < a.experts ? a.bias[i] : 0.0f;
    c[v] = (kSoftmax ? expf(l[v] - m) * rz : 1.0f / (1.0f + expf(-l[v]))) + b[v];
    key[v] = l[v] == -INFINITY ? 0u : key_of(c[v]);
  }
  // what two of them may be off together
  const float off = 2.0f * kUnit * (kSoftmax ? (V + 16) * rz : 8.0f);
  auto near = [&](float x, float y) { return !(x - y > off + kSumError * (fabsf(x) + fabsf(y))); };
  bool again = false;
  if (a.groups > 1) {
    const uint32_t mine = group_keys<V>(key, a, lane);
    const uint32_t mask = best_groups(mine, a, lane);
    const bool in = (mask >> lane) & 1u;
    // the worst group in and the best one out
    const uint32_t worst = ~warp_max(in ? ~mine : 0u), best = warp_max(in || lane >= a.groups ? 0u : mine);
    again = best != 0 && (near(of_key(worst), of_key(best) + off));
    drop_groups<V>(key, mask, a, lane);
    if (a.bias == nullptr) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (key[v] != 0) key[v] = key_of(l[v]);
    }
  }
  int mine = -1;
  if (!again) {
    mine = take_best<V>(key, a.top_k, lane);
    if (a.bias != nullptr) {
      // neighbours in the order, and the last one against the best that was left
      const int n = __popc(__ballot_sync(kAll, mine >= 0));
      const float ml = mine >= 0 ? load(a, row, mine) : 0.0f, mb = mine >= 0 ? a.bias[mine] : 0.0f;
      const float mc = (kSoftmax ? expf(ml - m) * rz : 1.0f / (1.0f + expf(-ml))) + mb;
      const float nl = __shfl_down_sync(kAll, ml, 1), nb = __shfl_down_sync(kAll, mb, 1), nc = __shfl_down_sync(kAll, mc, 1);
      again = lane + 1 < n && near(mc, nc) && !(ml == nl && mb == nb);
      const int last = n > 0 ? n - 1 : 0;
      const float ll = __shfl_sync(kAll, ml, last), lb = __shfl_sync(kAll, mb, last), lc = __shfl_sync(kAll, mc, last);
      float left = -INFINITY;
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (key[v] != 0 && !(l[v] == ll && b[v] == lb)) left = fmaxf(left, c[v]);
      again = again || (n == a.top_k && left != -INFINITY && near(lc, left));
    }
  }
  if (__any_sync(kAll, again)) mine = choose64<V, kSoftmax>(a, row, lane);
  return mine;
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
  for (long long row = static_cast<long long>(blockIdx.x) * kWarps + warp; row < a.tokens;
       row += static_cast<long long>(gridDim.x) * kWarps) {
    int mine = -1;
    float w = 0.0f;
    if (a.live == nullptr || a.live[row] != 0) {
      float l[V];
#pragma unroll
      for (int v = 0; v < V; ++v) l[v] = lane + 32 * v < a.experts ? load(a, row, lane + 32 * v) : -INFINITY;
      mine = choose<V, kSoftmax>(a, row, l, lane);
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
template <int V, bool kSoftmax>
__global__ void __launch_bounds__(kThreads) backward_kernel(const Args a) {
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (long long row = static_cast<long long>(blockIdx.x) * kWarps + warp; row < a.tokens;
       row += static_cast<long long>(gridDim.x) * kWarps) {
    int mine = -1;
    float w = 0.0f, g = 0.0f;
    if (lane < a.top_k) {
      mine = a.index[row * a.top_k + lane];
      if (mine >= 0 && mine < a.experts) {
        w = a.weight[row * a.top_k + lane];
        g = a.dweight[row * a.top_k + lane];
      } else {
        mine = mine == -1 ? -1 : a.experts;
      }
    }
    const bool on = mine >= 0 && mine < a.experts;
    const bool bad = __any_sync(kAll, mine >= a.experts), any = __any_sync(kAll, on);
    const float mean = warp_sum(g * w) / a.scale;
    float d = (a.renormalise ? g - mean : g) * w;
    if (!kSoftmax && on) {
      const float ml = load(a, row, mine);
      d *= 1.0f / (1.0f + expf(ml));  // 1 - s
    }
    float out[V];
#pragma unroll
    for (int v = 0; v < V; ++v) out[v] = 0.0f;
    if (kSoftmax && !a.renormalise && any) {
      float l[V], m = -INFINITY, z = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        l[v] = lane + 32 * v < a.experts ? load(a, row, lane + 32 * v) : -INFINITY;
        m = fmaxf(m, l[v]);
      }
      m = warp_max(m);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        out[v] = l[v] == -INFINITY ? 0.0f : expf(l[v] - m);
        z += out[v];
      }
      const float f = -mean * a.scale / warp_sum(z);
#pragma unroll
      for (int v = 0; v < V; ++v) out[v] *= f;
    }
    for (int j = 0; j < a.top_k; ++j) {
      const int i = __shfl_sync(kAll, mine, j);
      const float x = __shfl_sync(kAll, d, j);
      if (i >= 0 && (i & 31) == lane) {
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (v == i >> 5) out[v] += x;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = lane + 32 * v;
      if (i >= a.experts) continue;
      if (bad) out[v] = __uint_as_float(0x7FC00000u);
      const long long at = row * a.ld_d + i;
      if (a.bf16) {
        static_cast<__nv_bfloat16*>(a.dlogits)[at] = __float2bfloat16_rn(out[v]);
      } else {
        static_cast<float*>(a.dlogits)[at] = out[v];
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
zopt_status launch(const Args& a, bool softmax, bool backward, unsigned blocks, cudaStream_t s) {
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
