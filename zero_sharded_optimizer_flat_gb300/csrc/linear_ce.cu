// Linear cross entropy over a vocabulary, forward and backward, without keeping the logits.
//
// Forward: one product launch whose epilogue turns 128 of a row's logits (64 in narrow tiles) into a
// maximum and a sum (base 2), and one launch that joins a row's pieces: 2 T V D flops, and 8 bytes a row
// and 128 (64) logits of partial results instead of the logits' 2 to 4 bytes each. One or two tokens take
// linear_ce_few.cu in place of the first launch.
//
// Backward: dl needs each row's whole lse, so the logits are computed a second time: 6 T V D flops in
// all. The vocabulary is walked in pieces: piece i's dl is written to a workspace buffer in bf16
// (its kernel also computes p from lse and subtracts the target), then one launch computes
// dw_i = dl_i' x, dx (+)= dl_i w_i, and piece i+1's dl into the other buffer, so that the three
// products' last waves overlap. dx is summed over the pieces in fp32 in the workspace and rounded
// once, with the last piece. A call whose dl fits one piece needs neither the second buffer nor the
// fp32 sum.
//
// Measured (GB300): forward 4096 x 768 x 50304 187 us = 1.69 PFLOP/s, the rate of a large bf16 product
// under the power cap; backward 8192 x 2048 x 32000 1.98 ms = 1.63 PFLOP/s.
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "act8_host.h"
#include "guarded.h"
#include "launch.cuh"
#include "linear_ce_few.h"
#include "lm_gemm.cuh"
#include "ns_internal.h"
#include "tc.cuh"

namespace zopt {
namespace lm {
namespace {

constexpr long long kMaxDim = 1LL << 30, kMaxLd = 1LL << 32;
constexpr long long kMaxElems = 1LL << 44;  // of any matrix, the logits too: tile numbers stay well below 2^31
// dl of one piece: about 128 MiB (bf16), so that a piece is written and read once each while the
// products over it run for a few hundred microseconds; at least 4096 entries, below which the dx
// sum's 8 bytes per row and feature would be noticed.
constexpr long long kPieceBytes = 128LL << 20, kPieceLeast = 4096;

struct CePlan {
  bool few;  // the forward on the CUDA cores
  bool stage_x, stage_w;
  long long pitch;  // staged rows: dim rounded up to 8
  long long piece;  // vocabulary entries per piece, a multiple of 256
  int pieces;
  size_t xs, ws, xm, unit, dl[2], acc, part, tlogit, slab;  // offsets
  size_t total;
};

size_t take(size_t& at, long long bytes) {
  const size_t here = at;
  at += static_cast<size_t>(round_up(bytes, 1024));
  return here;
}

bool sizes_ok(const zopt_linear_ce_job& c) {
  return c.tokens <= kMaxDim && c.dim <= kMaxDim && c.vocab <= kMaxDim && c.tokens * c.dim <= kMaxElems &&
         c.vocab * c.dim <= kMaxElems && c.tokens * c.vocab <= kMaxElems;
}

// The inner lengths of the products: dim, the backward's tokens, and a piece of the vocabulary (2^26
// entries at most: kPieceBytes).
bool inner_ok(const zopt_linear_ce_job& c, bool backward) {
  return c.dim <= kMaxInner && (!backward || c.tokens <= kMaxInner);
}
static_assert(kPieceBytes / 2 <= kMaxInner, "a piece is dx's inner length");

bool shape_ok(const zopt_linear_ce_job& c, bool backward) {
  return c.tokens >= 0 && c.dim >= 1 && c.vocab >= 1 && sizes_ok(c) && inner_ok(c, backward) &&
         c.ld_x >= c.dim && c.ld_w >= c.dim && c.ld_x <= kMaxLd && c.ld_w <= kMaxLd;
}

// dx and dw of one piece of vc entries (without splits, maps and pointers).
void piece_jobs(const zopt_linear_ce_job& c, long long vc, Job& dx, Job& dw) {
  dx = Job{};
  dx.kind = kStore;
  dx.M = static_cast<int>(c.tokens), dx.N = static_cast<int>(c.dim), dx.K = static_cast<int>(vc);
  dx.b_mn = 1;
  set_tiles(dx);
  dw = Job{};
  dw.kind = kStore;
  dw.M = static_cast<int>(vc), dw.N = static_cast<int>(c.dim), dw.K = static_cast<int>(c.tokens);
  dw.a_mn = dw.b_mn = 1;
  set_tiles(dw);
}

CePlan plan(const zopt_linear_ce_job& c, bool backward) {
  CePlan p{};
  const long long T = c.tokens, D = c.dim, V = c.vocab;
  p.pitch = round_up(D, 8);
  if (!backward && few::takes(c)) {
    p.few = true;
    p.part = take(p.total, few::ce_parts(c) * T * 8);
    p.tlogit = take(p.total, T * 4);
    return p;
  }
  p.stage_x = c.ld_x % 8 != 0;
  p.stage_w = c.ld_w % 8 != 0;
  size_t at = 0;
  if (p.stage_x) p.xs = take(at, T * p.pitch * 2);
  if (p.stage_w) p.ws = take(at, V * p.pitch * 2);
  const size_t shared = at;
  p.part = take(at, 2 * ((V + 127) / 128) * T * 8);  // (of tiles of 128 columns)
  p.tlogit = take(at, T * 4);
  p.total = at;
  if (!backward) return p;
  at = shared;
  p.xm = take(at, T * p.pitch * 2);
  p.unit = take(at, 4);
  const long long most = std::max(kPieceLeast, kPieceBytes / (2 * std::max<long long>(T, 1)) / kTileN * kTileN);
  p.pieces = static_cast<int>((V + most - 1) / most);
  p.piece = round_up((V + p.pieces - 1) / p.pieces, kTileN);
  p.pieces = static_cast<int>((V + p.piece - 1) / p.piece);
  p.dl[0] = take(at, T * p.piece * 2);
  p.dl[1] = p.pieces > 1 ? take(at, T * p.piece * 2) : p.dl[0];
  if (p.pieces > 1) p.acc = take(at, T * split_pitch(D) * 4);
  // partial sums: those of a whole piece or of the last one, whichever takes more
  long long slab = 0;
  for (const long long vc : {std::min(p.piece, V), V - (p.pieces - 1) * p.piece}) {
    if (T == 0) break;  // (nothing is multiplied)
    for (int both = 0; both < 3; ++both) {  // dx and dw, or one of them alone
      Job j[2];
      piece_jobs(c, vc, j[0], j[1]);
      j[0].whole = p.pieces > 1;  // a dx summed over the pieces is not cut as well
      Job* first = both == 2 ? j + 1 : j;
      const int n = both == 0 ? 2 : 1;
      plan_splits(first, n);
      long long e = 0;
      for (int i = 0; i < n; ++i) e += round_up(split_elems(first[i]), 256);
      slab = std::max(slab, e);
    }
  }
  if (slab) p.slab = take(at, slab * 4);
  p.total = std::max(p.total, at);
  return p;
}

// What the backward's products need beside the logits' gradient (12.5 us for 8192 x 2048, of 1.98 ms).
// Block 0: *unit = the largest finite |dloss| of a counted row (1 if there is none). The others: xm =
// x with its ignored rows zero, the operand of dw, which must not meet whatever such rows hold (0
// times inf is not 0): 4 bytes an entry of x beside 6 V flops.
__global__ void __launch_bounds__(256)
    ce_prep_kernel(float* unit, const float* dloss, const int64_t* target, int64_t ignore, long long tokens,
                   uint16_t* xm, long long pitch, const uint16_t* x, long long ld_x, long long rows, long long dim) {
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  if (blockIdx.x == 0) {
    __shared__ float top[8];
    float m = 0.0f;
    for (long long t = threadIdx.x; t < tokens; t += blockDim.x) {
      const float a = fabsf(dloss[t]);
      if (target[t] != ignore && a <= 3.402823466e38f) m = fmaxf(m, a);
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
    if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < 8; ++w) m = fmaxf(m, top[w]);
      *unit = m > 0.0f ? m : 1.0f;
    }
    return;
  }
  const long long per_row = pitch / 8, n = rows * per_row;
  const long long stride = static_cast<long long>(gridDim.x - 1) * blockDim.x;
  for (long long g = static_cast<long long>(blockIdx.x - 1) * blockDim.x + threadIdx.x; g < n; g += stride) {
    const long long row = g / per_row, col = (g - row * per_row) * 8;
    *reinterpret_cast<uint4*>(xm + row * pitch + col) =
        target[row] != ignore ? row_piece8(x + row * ld_x + col, dim - col) : make_uint4(0, 0, 0, 0);
  }
}

// A row's pieces joined: lse = (M + log2 sum_p s_p 2^(m_p - M)) / kLog2e. Lanes are rows and the block's
// warps share the pieces; or, up to as many rows as such blocks make one wave (kJoinOneRow, four an
// SM), a block's threads share one row's: one token and 304 pieces 8.2 us for 4.1, cross entropy
// forward of 300 x 768 x 50304 33.7 us for 31.0, of 600 x 256 x 4096 11.1 for 11.3.
// The last sum is in fp64, once a row: in fp32 the sum of a maximum near 15 and a logarithm is rounded
// by 1e-6, which a loss much smaller than lse shows (1.3e-6 against the 1e-7 of the rest; the logarithm
// itself is then small, and its own fp32 rounding with it); dividing by the very constant that scaled
// the logits undoes its rounding. Bound by its loads' latency, so a warp has kJoinAhead pieces in
// flight (one at a time: 12 us for the 13 MB of 4096 rows and 393 pieces, for 7.6).
constexpr int kJoinWarps = 16, kJoinAhead = 8, kJoinOneRow = 608;
template <bool kOneRow>
__global__ void __launch_bounds__(32 * kJoinWarps)
    ce_join_kernel(const float2* part, int parts, long long tokens, const int64_t* target, int64_t ignore,
                   int64_t vocab, const float* tlogit, float* loss, float* lse) {
  __shared__ float2 sh[kJoinWarps][32];
  tc::pdl_launch_dependents();
  tc::pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = kOneRow ? blockIdx.x : static_cast<long long>(blockIdx.x) * 32 + lane;
  constexpr int kStep = kOneRow ? 32 * kJoinWarps : kJoinWarps;
  float m = -INFINITY, s = 0.0f;
  if (row < tokens) {
    for (int p0 = kOneRow ? static_cast<int>(threadIdx.x) : warp; p0 < parts; p0 += kJoinAhead * kStep) {
      float2 v[kJoinAhead];
      float mn = m;
#pragma unroll
      for (int i = 0; i < kJoinAhead; ++i) {
        const int p = p0 + i * kStep;
        v[i] = p < parts ? part[static_cast<long long>(p) * tokens + row] : make_float2(-INFINITY, 0.0f);
      }
#pragma unroll
      for (int i = 0; i < kJoinAhead; ++i) mn = fmaxf(mn, v[i].x);
      const float base = mn == -INFINITY ? 0.0f : mn;
      s *= exp2f(m - base);
#pragma unroll
      for (int i = 0; i < kJoinAhead; ++i) s = fmaf(v[i].y, exp2f(v[i].x - base), s);
      m = mn;
    }
  }
  if (kOneRow) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
      const float n = __shfl_xor_sync(0xFFFFFFFFu, m, d), u = __shfl_xor_sync(0xFFFFFFFFu, s, d), mn = fmaxf(m, n);
      const float base = mn == -INFINITY ? 0.0f : mn;
      s = s * exp2f(m - base) + u * exp2f(n - base);
      m = mn;
    }
  }
  sh[warp][lane] = make_float2(m, s);
  __syncthreads();
  if (warp != 0 || row >= tokens || (kOneRow && lane != 0)) return;
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) m = fmaxf(m, sh[w][lane].x);
  const float base = m == -INFINITY ? 0.0f : m;
  s = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) s = fmaf(sh[w][lane].y, exp2f(sh[w][lane].x - base), s);
  const int64_t t = target[row];
  if (t == ignore) {
    loss[row] = 0.0f;
    lse[row] = 0.0f;
    return;
  }
  constexpr double kLn2 = 1.0 / static_cast<double>(kLog2e);
  const double l = (static_cast<double>(m) + static_cast<double>(log2f(s))) * kLn2;
  lse[row] = static_cast<float>(l);
  loss[row] = t >= 0 && t < vocab ? static_cast<float>(l - static_cast<double>(tlogit[row])) : __uint_as_float(0x7FC00000u);
}

zopt_status check(const char* fn, const zopt_linear_ce_job* c, bool backward, void* d_ws, size_t ws_bytes) {
  const std::string f(fn);
  if (c == nullptr) return fail(ZOPT_EINVAL, f + ": NULL job");
  if (c->dtype != ZOPT_BF16) return fail(ZOPT_EUNSUPPORTED, f + ": dtype must be ZOPT_BF16");
  if (c->tokens < 0 || c->dim < 1 || c->vocab < 1) return fail(ZOPT_EINVAL, f + ": tokens < 0, dim < 1 or vocab < 1");
  if (!sizes_ok(*c)) return fail(ZOPT_EINVAL, f + ": tokens, dim or vocab above 2^30, or a matrix above 2^44 elements");
  if (!inner_ok(*c, backward)) return fail(ZOPT_EINVAL, f + ": dim above 2^26 or, in the backward, tokens above 2^26");
  auto ld_bad = [&](int64_t ld) { return ld < c->dim || ld > kMaxLd; };
  if (ld_bad(c->ld_x) || ld_bad(c->ld_w) || (backward && c->dx && ld_bad(c->ld_dx)) || (backward && c->dw && ld_bad(c->ld_dw)))
    return fail(ZOPT_EINVAL, f + ": row distance below dim or above 2^32");
  if (backward && c->dx == nullptr && c->dw == nullptr && c->tokens > 0) return fail(ZOPT_EINVAL, f + ": neither dx nor dw is wanted");
  if (backward && c->dw != nullptr && !aligned16(c->dw)) return fail(ZOPT_EINVAL, f + ": matrices must be 16-byte aligned");
  if (c->tokens == 0) return ok();
  if (c->x == nullptr || c->w == nullptr || c->target == nullptr || c->lse == nullptr)
    return fail(ZOPT_EINVAL, f + ": NULL x, w, target or lse");
  if (backward ? c->dloss == nullptr : c->loss == nullptr) return fail(ZOPT_EINVAL, f + ": NULL loss or dloss");
  if (!aligned16(c->x) || !aligned16(c->w) || (backward && c->dx != nullptr && !aligned16(c->dx)))
    return fail(ZOPT_EINVAL, f + ": matrices must be 16-byte aligned");
  auto off = [](const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; };
  if (off(c->target, 8) || off(c->lse, 4) || off(backward ? static_cast<const void*>(c->dloss) : c->loss, 4))
    return fail(ZOPT_EINVAL, f + ": a vector is not aligned to its element");
  if (d_ws == nullptr || !aligned16(d_ws)) return fail(ZOPT_EINVAL, f + ": the workspace must be 16-byte aligned");
  if (ws_bytes < plan(*c, backward).total) return fail(ZOPT_EINVAL, f + ": workspace too small");
  return ok();
}

#define TRY(expr)                                \
  do {                                           \
    const zopt_status st_ = (expr);              \
    if (st_ != ZOPT_OK) return st_;              \
  } while (0)

// x and w as the TMA reads them: in place, or copied into the workspace.
zopt_status stage_inputs(const char* fn, const zopt_linear_ce_job& c, const CePlan& p, uint8_t* ws, const uint16_t** x,
                         long long* px, const uint16_t** w, long long* pw, cudaStream_t s) {
  *x = c.x, *px = c.ld_x, *w = c.w, *pw = c.ld_w;
  if (p.stage_x) {
    uint16_t* d = reinterpret_cast<uint16_t*>(ws + p.xs);
    TRY(launch_stage(fn, d, p.pitch, p.pitch, c.x, c.ld_x, c.tokens, c.dim, s));
    *x = d, *px = p.pitch;
  }
  if (p.stage_w) {
    uint16_t* d = reinterpret_cast<uint16_t*>(ws + p.ws);
    TRY(launch_stage(fn, d, p.pitch, p.pitch, c.w, c.ld_w, c.vocab, c.dim, s));
    *w = d, *pw = p.pitch;
  }
  return ok();
}

void ce_fields(Job& j, const zopt_linear_ce_job& c) {
  j.target = c.target;
  j.ignore = c.ignore_index;
  j.vocab = c.vocab;
  j.lse = c.lse;
  j.dloss = c.dloss;
}

zopt_status forward(const zopt_linear_ce_job* cp, void* d_ws, size_t ws_bytes, cudaStream_t s) {
  const char* fn = "zopt_linear_ce_forward";
  TRY(check(fn, cp, false, d_ws, ws_bytes));
  const zopt_linear_ce_job& c = *cp;
  if (c.tokens == 0) return ok();
  Batch b{};
  TRY(ns::take_error_word(fn, &b.err));
  const CePlan p = plan(c, false);
  uint8_t* ws = static_cast<uint8_t*>(d_ws);
  float2* part = reinterpret_cast<float2*>(ws + p.part);
  float* tlogit = reinterpret_cast<float*>(ws + p.tlogit);
  int parts;
  if (p.few) {
    TRY(few::ce_logits(c, part, tlogit, s));
    parts = few::ce_parts(c);
  } else {
    const uint16_t *x, *w;
    long long px, pw;
    TRY(stage_inputs(fn, c, p, ws, &x, &px, &w, &pw, s));
    b.n = 1;
    Job& j = b.job[0];
    j.kind = kCeFwd;
    j.M = static_cast<int>(c.tokens), j.N = static_cast<int>(c.vocab), j.K = static_cast<int>(c.dim);
    set_tiles(j);
    ce_fields(j, c);
    j.part = part;
    j.tlogit = tlogit;
    TRY(map_p(fn, j, x, px));
    TRY(map_q(fn, j, w, c.vocab, pw));
    TRY(launch(fn, b, kCeFwd, s));
    parts = static_cast<int>((c.vocab + j.tile_n / 2 - 1) / (j.tile_n / 2));
  }
  const bool one_row = c.tokens <= kJoinOneRow;
  return launch_pdl(one_row ? ce_join_kernel<true> : ce_join_kernel<false>,
                    dim3(static_cast<unsigned>(one_row ? c.tokens : (c.tokens + 31) / 32)), dim3(32 * kJoinWarps), 0, s,
                    static_cast<const float2*>(part), parts, static_cast<long long>(c.tokens), c.target,
                    c.ignore_index, c.vocab, static_cast<const float*>(tlogit), c.loss, c.lse);
}

zopt_status backward(const zopt_linear_ce_job* cp, void* d_ws, size_t ws_bytes, cudaStream_t s) {
  const char* fn = "zopt_linear_ce_backward";
  TRY(check(fn, cp, true, d_ws, ws_bytes));
  const zopt_linear_ce_job& c = *cp;
  if (c.tokens == 0) {
    if (c.dw != nullptr) ZOPT_CUDA_TRY(cudaMemset2DAsync(c.dw, c.ld_dw * 2, 0, c.dim * 2, c.vocab, s));
    return ok();
  }
  int* err = nullptr;
  TRY(ns::take_error_word(fn, &err));
  const CePlan p = plan(c, true);
  uint8_t* ws = static_cast<uint8_t*>(d_ws);
  const uint16_t *x, *w;
  long long px, pw;
  TRY(stage_inputs(fn, c, p, ws, &x, &px, &w, &pw, s));
  uint16_t* xm = reinterpret_cast<uint16_t*>(ws + p.xm);
  float* unit = reinterpret_cast<float*>(ws + p.unit);
  {
    const int sms = sm_count();
    if (sms < 1) return fail(ZOPT_ECUDA, std::string(fn) + ": no CUDA device");
    const long long rows = c.dw != nullptr ? c.tokens : 0;
    TRY(launch_pdl(ce_prep_kernel, dim3(1 + blocks_for(rows * (p.pitch / 8), sms)), dim3(256), 0, s, unit, c.dloss,
                   c.target, c.ignore_index, static_cast<long long>(c.tokens), xm, p.pitch, c.x,
                   static_cast<long long>(c.ld_x), rows, static_cast<long long>(c.dim)));
  }

  auto entries = [&](int i) { return std::min<long long>(p.piece, c.vocab - i * p.piece); };
  auto dl_of = [&](int i) { return reinterpret_cast<uint16_t*>(ws + p.dl[i & 1]); };
  auto dl_job = [&](Job& j, int i) -> zopt_status {
    const long long v0 = i * p.piece, vc = entries(i);
    j.kind = kCeBwd;
    j.M = static_cast<int>(c.tokens), j.N = static_cast<int>(vc), j.K = static_cast<int>(c.dim);
    set_tiles(j);
    ce_fields(j, c);
    j.col0 = v0;
    j.unit = unit;
    TRY(map_p(fn, j, x, px));
    TRY(map_q(fn, j, w + v0 * pw, vc, pw));
    j.out = dl_of(i);
    j.ld_out = p.piece;
    return ok();
  };
  {
    Batch b{};
    b.err = err;
    b.n = 1;
    TRY(dl_job(b.job[0], 0));
    TRY(launch(fn, b, kStore | kCeBwd, s));
  }
  float* acc = reinterpret_cast<float*>(ws + p.acc);
  const long long acc_pitch = split_pitch(c.dim);
  for (int i = 0; i < p.pieces; ++i) {
    const long long v0 = i * p.piece, vc = entries(i);
    Batch b{};
    b.err = err;
    Job dx, dw;
    piece_jobs(c, vc, dx, dw);
    dx.whole = p.pieces > 1;
    if (i > 0) dx.add = acc, dx.ld_add = acc_pitch;
    const bool partial = i + 1 < p.pieces;  // dx stays an fp32 sum
    // The longest units first: the launch's end is then made of short ones.
    const bool dx_first = dx.nk >= dw.nk;
    for (int k = 0; k < 2; ++k) {
      if ((k == 0) == dx_first) {
        if (c.dx != nullptr) b.job[b.n++] = dx;
      } else if (c.dw != nullptr) {
        b.job[b.n++] = dw;
      }
    }
    plan_splits(b.job, b.n);
    SumBatch sums{};
    float* slab = reinterpret_cast<float*>(ws + p.slab);
    const int products = b.n;
    for (int k = 0; k < products; ++k) {
      Job& j = b.job[k];
      const bool is_dw = j.a_mn != 0;
      if (is_dw || !partial) j.alpha = unit;
      uint16_t* out = is_dw ? c.dw + v0 * c.ld_dw : c.dx;
      const long long ld = is_dw ? c.ld_dw : c.ld_dx;
      if (is_dw) {
        TRY(map_p(fn, j, dl_of(i), p.piece));
        TRY(map_q(fn, j, xm, c.dim, p.pitch));
      } else {
        TRY(map_p(fn, j, dl_of(i), p.piece));
        TRY(map_q(fn, j, w + v0 * pw, c.dim, pw));
      }
      if (j.splits > 1) {
        j.out_mode = kOutF32;
        j.out = slab;
        j.ld_out = split_pitch(j.N);
        j.split_stride = j.M * j.ld_out;
        SumJob& q = sums.job[sums.n];
        q = SumJob{slab, j.split_stride, j.ld_out, j.splits, j.M, j.N, out, ld, unit};
        j.alpha = nullptr;
        sums.start[sums.n + 1] = sums.start[sums.n] + q.M * (q.pitch / 4);
        ++sums.n;
        slab += round_up(split_elems(j), 256);
      } else if (!is_dw && partial) {
        j.out_mode = kOutF32;
        j.out = acc;
        j.ld_out = acc_pitch;
      } else {
        j.out_mode = kOutBf16;
        j.out = out;
        j.ld_out = ld;
      }
    }
    if (partial) TRY(dl_job(b.job[b.n++], i + 1));
    TRY(launch(fn, b, kStore | kCeBwd, s));
    if (sums.n > 0) TRY(launch_sums(fn, sums, s));
  }
  return ok();
}

}  // namespace
}  // namespace lm
}  // namespace zopt

extern "C" size_t zopt_linear_ce_workspace(const zopt_linear_ce_job* job, int32_t backward) {
  if (job == nullptr || !zopt::lm::shape_ok(*job, backward != 0)) return 0;
  const size_t n = zopt::lm::plan(*job, backward != 0).total;
  return n < 16 ? 16 : n;
}

extern "C" zopt_status zopt_linear_ce_forward(const zopt_linear_ce_job* job, void* d_ws, size_t ws_bytes,
                                              zopt_stream stream) {
  return zopt::guarded([&] { return zopt::lm::forward(job, d_ws, ws_bytes, stream); });
}

extern "C" zopt_status zopt_linear_ce_backward(const zopt_linear_ce_job* job, void* d_ws, size_t ws_bytes,
                                               zopt_stream stream) {
  return zopt::guarded([&] { return zopt::lm::backward(job, d_ws, ws_bytes, stream); });
}
