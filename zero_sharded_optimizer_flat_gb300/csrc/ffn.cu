// The gated feed-forward block, forward and backward.
//
// Forward, two products: gate and up in one kernel whose epilogue applies the activation and the
// product (and keeps gate and up, in bf16 or in 8 bits), then y = h down. h takes one pass through
// memory in bf16; the gate and up themselves only where they are kept. (A few tokens take ffn_few.cu,
// where h stays in fp32.)
//
// Backward, four products in two launches: dh = dy down', whose epilogue reads the kept gate and up
// and writes dgate, dup and h; then dx, dgate_up and ddown in one launch, longest units first, so
// that only one launch's last wave runs short. 18 T D F flops for both directions.
//
// Measured (GB300, 8192 x 2048 x 5632): forward 361 us = 1.57 PFLOP/s (gate and up 200, y 109 by
// themselves); both directions with 8-bit checkpoints 1.10 ms = 1.55 PFLOP/s (the backward's two
// launches 139 and 495 by themselves), at the power cap, where a plain bf16 product runs at 1.70.
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "act8_host.h"
#include "ffn_few.h"
#include "guarded.h"
#include "launch.cuh"
#include "lm_gemm.cuh"
#include "ns_internal.h"

namespace zopt {
namespace lm {
namespace {

constexpr long long kMaxDim = 1LL << 30, kMaxLd = 1LL << 32;
constexpr long long kMaxElems = 1LL << 44;  // of any matrix: tile numbers stay well below 2^31

struct FfnPlan {
  long long dp, fp, gp;  // dim, hidden and 2 hidden rounded up to 8: row distances in the workspace
  bool stage_x, stage_dy, stage_gate, stage_up, stage_down, few;
  size_t xs, dys, gate, up, down, h, dgu, slab, few_gate_up, few_y, total;
};

size_t take(size_t& at, long long bytes) {
  const size_t here = at;
  at += static_cast<size_t>(round_up(bytes, 1024));
  return here;
}

bool sizes_ok(const zopt_ffn_job& c) {
  return c.tokens <= kMaxDim && c.dim <= kMaxDim && c.hidden <= kMaxDim / 2 && c.tokens * c.dim <= kMaxElems &&
         c.tokens * 2 * c.hidden <= kMaxElems && c.dim * 2 * c.hidden <= kMaxElems;
}

// The inner lengths of the products: dim and hidden, the backward's 2 hidden and tokens too.
bool inner_ok(const zopt_ffn_job& c, bool backward) {
  return c.dim <= kMaxInner && c.hidden <= kMaxInner / 2 && (!backward || c.tokens <= kMaxInner);
}

bool shape_ok(const zopt_ffn_job& c, bool backward) {
  auto ld = [](int64_t v, int64_t least) { return v >= least && v <= kMaxLd; };
  return c.tokens >= 0 && c.dim >= 1 && c.hidden >= 1 && sizes_ok(c) && inner_ok(c, backward) &&
         ld(c.ld_gate_up, 2 * c.hidden) && ld(c.ld_down, c.dim) && (c.x8 != nullptr || ld(c.ld_x, c.dim)) &&
         (!backward || ld(c.ld_dy, c.dim));
}

void y_job(const zopt_ffn_job& c, Job& j) {
  j = Job{};
  j.kind = kStore;
  j.M = static_cast<int>(c.tokens), j.N = static_cast<int>(c.dim), j.K = static_cast<int>(c.hidden);
  j.b_mn = 1;
  set_tiles(j);
}

// The backward's second launch: dx, dgate_up and ddown.
int grad_jobs(const zopt_ffn_job& c, Job* j) {
  const int T = static_cast<int>(c.tokens), D = static_cast<int>(c.dim), F = static_cast<int>(c.hidden);
  const int shape[3][3] = {{T, D, 2 * F}, {D, 2 * F, T}, {F, D, T}};
  for (int k = 0; k < 3; ++k) {
    j[k] = Job{};
    j[k].kind = kStore;
    j[k].M = shape[k][0], j[k].N = shape[k][1], j[k].K = shape[k][2];
    j[k].a_mn = j[k].b_mn = k > 0;
    set_tiles(j[k]);
  }
  return 3;
}

long long slab_elems(Job* j, int n) {
  plan_splits(j, n);
  long long e = 0;
  for (int i = 0; i < n; ++i) e += round_up(split_elems(j[i]), 256);
  return e;
}

FfnPlan plan(const zopt_ffn_job& c, bool backward) {
  FfnPlan p{};
  const long long T = c.tokens, D = c.dim, F = c.hidden;
  p.dp = round_up(D, 8), p.fp = round_up(F, 8), p.gp = round_up(2 * F, 8);
  p.stage_x = (backward && c.x8 != nullptr) || c.ld_x % 8 != 0;
  p.stage_dy = backward && c.ld_dy % 8 != 0;
  p.stage_gate = c.ld_gate_up % 8 != 0;
  p.stage_up = p.stage_gate || F % 8 != 0;  // (the forward reads up's columns from column hidden on)
  p.stage_down = c.ld_down % 8 != 0;
  size_t at = 0;
  if (p.stage_gate) p.gate = take(at, D * p.gp * 2);
  if (p.stage_up) p.up = take(at, D * p.fp * 2);
  if (p.stage_down) p.down = take(at, F * p.dp * 2);
  if (p.stage_x) p.xs = take(at, T * p.dp * 2);
  p.h = take(at, T * p.fp * 2);
  const size_t shared = at;
  Job j[kMaxJobs];
  y_job(c, j[0]);
  p.few = T > 0 && few::takes(c);
  if (p.few) {
    long long gate_up, y;
    few::partial_elems(c, &gate_up, &y);
    p.few_gate_up = take(at, gate_up * 4);
    p.few_y = take(at, y * 4);
  } else if (T > 0) {
    const long long e = slab_elems(j, 1);
    if (e) p.slab = take(at, e * 4);
  }
  p.total = at;
  if (!backward) return p;
  at = shared;
  if (p.stage_dy) p.dys = take(at, T * p.dp * 2);
  p.dgu = take(at, T * p.gp * 2);
  p.slab = at;
  if (T > 0) {
    const long long e = slab_elems(j, grad_jobs(c, j));
    if (e) take(at, e * 4);
  }
  p.total = std::max(p.total, at);
  return p;
}

zopt_status check(const char* fn, const zopt_ffn_job* c, bool backward, void* d_ws, size_t ws_bytes) {
  const std::string f(fn);
  auto bad = [&](const char* what) { return fail(ZOPT_EINVAL, f + ": " + what); };
  if (c == nullptr) return bad("NULL job");
  if (c->dtype != ZOPT_BF16) return fail(ZOPT_EUNSUPPORTED, f + ": dtype must be ZOPT_BF16");
  if (c->act != ZOPT_ACT_SILU && c->act != ZOPT_ACT_GELU) return bad("act must be ZOPT_ACT_SILU or ZOPT_ACT_GELU");
  if (c->tokens < 0 || c->dim < 1 || c->hidden < 1) return bad("tokens < 0, dim < 1 or hidden < 1");
  if (!sizes_ok(*c)) return bad("tokens or dim above 2^30, hidden above 2^29 or a matrix above 2^44 elements");
  if (!inner_ok(*c, backward)) return bad("dim above 2^26, hidden above 2^25 or, in the backward, tokens above 2^26");
  const int64_t T = c->tokens, D = c->dim, F = c->hidden;
  auto ld_bad = [](int64_t ld, int64_t least) { return ld < least || ld > kMaxLd; };
  if (ld_bad(c->ld_gate_up, 2 * F) || ld_bad(c->ld_down, D)) return bad("a weight's row distance below its row or above 2^32");
  if (c->w_gate_up == nullptr || c->w_down == nullptr) return bad("NULL weight");
  if (!aligned16(c->w_gate_up) || !aligned16(c->w_down)) return bad("matrices must be 16-byte aligned");
  if (c->kept != nullptr && c->kept8 != nullptr) return bad("both kept and kept8");
  if (c->kept != nullptr && (ld_bad(c->ld_kept, 2 * F) || !aligned16(c->kept))) return bad("kept: row distance or alignment");
  if (c->kept8 != nullptr) {
    const zopt_status st = act8::check(fn, *c->kept8);
    if (st != ZOPT_OK) return st;
    if (c->kept8->rows != T || c->kept8->cols != 2 * F || c->kept8->parts != 2)
      return bad("kept8 must be tokens x 2 hidden in two parts");
  }
  if (backward) {
    if ((c->dx == nullptr && T > 0) || c->dw_gate_up == nullptr || c->dw_down == nullptr) return bad("NULL dx, dw_gate_up or dw_down");
    if (ld_bad(c->ld_dx, D) || ld_bad(c->ld_dw_gate_up, 2 * F) || ld_bad(c->ld_dw_down, D))
      return bad("a gradient's row distance below its row or above 2^32");
    if (!aligned16(c->dx) || !aligned16(c->dw_gate_up) || !aligned16(c->dw_down)) return bad("matrices must be 16-byte aligned");
  }
  if (!backward && c->x8 != nullptr) return bad("the forward takes x in bf16");
  if ((c->x != nullptr) == (backward && c->x8 != nullptr) && T > 0) return bad("exactly one of x and x8 is wanted");
  if (T == 0) return ok();
  if (c->x8 != nullptr) {
    const zopt_status st = act8::check(fn, *c->x8);
    if (st != ZOPT_OK) return st;
    if (c->x8->rows != T || c->x8->cols != D || c->x8->parts != 1) return bad("x8 must be tokens x dim in one part");
  } else if (ld_bad(c->ld_x, D) || !aligned16(c->x)) {
    return bad("x: row distance or alignment");
  }
  if (backward) {
    if (c->kept == nullptr && c->kept8 == nullptr) return bad("the backward needs kept or kept8");
    if (c->dy == nullptr || ld_bad(c->ld_dy, D) || !aligned16(c->dy)) return bad("dy: NULL, row distance or alignment");
  } else {
    if (c->y == nullptr || ld_bad(c->ld_y, D) || !aligned16(c->y)) return bad("y: NULL, row distance or alignment");
  }
  if (d_ws == nullptr || !aligned16(d_ws)) return bad("the workspace must be 16-byte aligned");
  if (ws_bytes < plan(*c, backward).total) return bad("workspace too small");
  return ok();
}

#define TRY(expr)                   \
  do {                              \
    const zopt_status st_ = (expr); \
    if (st_ != ZOPT_OK) return st_; \
  } while (0)

// The operands as the TMA reads them: in place, or copied (or unpacked) into the workspace. The
// backward reads gate_up's rows whole, the forward its gate and up columns.
struct Inputs {
  const uint16_t *x, *gate_up, *up, *down, *dy;
  long long px, pgu, pup, pdown, pdy;
};
zopt_status stage_inputs(const char* fn, const zopt_ffn_job& c, const FfnPlan& p, bool backward, uint8_t* ws, Inputs& in,
                         cudaStream_t s) {
  in = Inputs{c.x, c.w_gate_up, c.w_gate_up + c.hidden, c.w_down, c.dy, c.ld_x, c.ld_gate_up, c.ld_gate_up, c.ld_down, c.ld_dy};
  auto copy = [&](size_t off, long long pitch, const uint16_t* src, long long ld, long long rows, long long cols,
                  const uint16_t** to, long long* pitch_to) {
    uint16_t* d = reinterpret_cast<uint16_t*>(ws + off);
    *to = d, *pitch_to = pitch;
    return launch_stage(fn, d, pitch, pitch, src, ld, rows, cols, s);
  };
  if (p.stage_gate)
    TRY(copy(p.gate, p.gp, c.w_gate_up, c.ld_gate_up, c.dim, backward ? 2 * c.hidden : c.hidden, &in.gate_up, &in.pgu));
  if (p.stage_up && !backward) TRY(copy(p.up, p.fp, c.w_gate_up + c.hidden, c.ld_gate_up, c.dim, c.hidden, &in.up, &in.pup));
  if (p.stage_down) TRY(copy(p.down, p.dp, c.w_down, c.ld_down, c.hidden, c.dim, &in.down, &in.pdown));
  if (p.stage_x && c.x8 != nullptr) {
    in.x = reinterpret_cast<uint16_t*>(ws + p.xs), in.px = p.dp;
    TRY(act8::unpack(fn, *c.x8, reinterpret_cast<uint16_t*>(ws + p.xs), p.dp, s));
  } else if (p.stage_x) {
    TRY(copy(p.xs, p.dp, c.x, c.ld_x, c.tokens, c.dim, &in.x, &in.px));
  }
  if (p.stage_dy) TRY(copy(p.dys, p.dp, c.dy, c.ld_dy, c.tokens, c.dim, &in.dy, &in.pdy));
  return ok();
}

void glu_fields(Job& j, const zopt_ffn_job& c) {
  j.act = c.act;
  j.hidden = static_cast<int>(c.hidden);
  if (c.kept8 != nullptr) {
    j.kept_mode = kKeep8;
    j.kept = c.kept8->q;
    j.ld_kept = 2 * c.hidden;
    j.kept_scale = c.kept8->scale;
  } else if (c.kept != nullptr) {
    j.kept_mode = kKeepBf16;
    j.kept = c.kept;
    j.ld_kept = c.ld_kept;
  }
}

// Where a kStore job's result goes: its partial sums' slab, or the caller's matrix.
void finish(Job& j, uint16_t* out, long long ld, float*& slab, SumBatch& sums) {
  if (j.splits > 1) {
    j.out_mode = kOutF32;
    j.out = slab;
    j.ld_out = split_pitch(j.N);
    j.split_stride = j.M * j.ld_out;
    SumJob& q = sums.job[sums.n];
    q = SumJob{slab, j.split_stride, j.ld_out, j.splits, j.M, j.N, out, ld, nullptr};
    sums.start[sums.n + 1] = sums.start[sums.n] + q.M * (q.pitch / 4);
    ++sums.n;
    slab += round_up(split_elems(j), 256);
    return;
  }
  j.out_mode = kOutBf16;
  j.out = out;
  j.ld_out = ld;
}

zopt_status forward(const zopt_ffn_job* cp, void* d_ws, size_t ws_bytes, cudaStream_t s) {
  const char* fn = "zopt_ffn_forward";
  TRY(check(fn, cp, false, d_ws, ws_bytes));
  const zopt_ffn_job& c = *cp;
  if (c.tokens == 0) return ok();
  int* err = nullptr;
  TRY(ns::take_error_word(fn, &err));
  const FfnPlan p = plan(c, false);
  uint8_t* ws = static_cast<uint8_t*>(d_ws);
  uint16_t* h = reinterpret_cast<uint16_t*>(ws + p.h);
  if (p.few) return few::ffn_forward(c, reinterpret_cast<float*>(ws + p.few_gate_up), reinterpret_cast<float*>(ws + p.few_y), s);
  Inputs in;
  TRY(stage_inputs(fn, c, p, false, ws, in, s));
  {
    Batch b{};
    b.err = err;
    b.n = 1;
    Job& j = b.job[0];
    j.kind = kGluFwd;
    j.M = static_cast<int>(c.tokens), j.N = static_cast<int>(c.hidden), j.K = static_cast<int>(c.dim);
    j.b_mn = 1;
    glu_fields(j, c);
    set_tiles(j);
    TRY(map_p(fn, j, in.x, in.px));
    TRY(map_q(fn, j, in.gate_up, c.hidden, in.pgu));
    TRY(map_up(fn, j, in.up, c.hidden, in.pup));
    j.out = h;
    j.ld_out = p.fp;
    TRY(launch(fn, b, kGluFwd, s));
  }
  Batch b{};
  b.err = err;
  b.n = 1;
  y_job(c, b.job[0]);
  plan_splits(b.job, 1);
  TRY(map_p(fn, b.job[0], h, p.fp));
  TRY(map_q(fn, b.job[0], in.down, c.dim, in.pdown));
  SumBatch sums{};
  float* slab = reinterpret_cast<float*>(ws + p.slab);
  finish(b.job[0], c.y, c.ld_y, slab, sums);
  TRY(launch(fn, b, kStore, s));
  return sums.n > 0 ? launch_sums(fn, sums, s) : ok();
}

zopt_status backward(const zopt_ffn_job* cp, void* d_ws, size_t ws_bytes, cudaStream_t s) {
  const char* fn = "zopt_ffn_backward";
  TRY(check(fn, cp, true, d_ws, ws_bytes));
  const zopt_ffn_job& c = *cp;
  if (c.tokens == 0) {
    ZOPT_CUDA_TRY(cudaMemset2DAsync(c.dw_gate_up, c.ld_dw_gate_up * 2, 0, 2 * c.hidden * 2, c.dim, s));
    ZOPT_CUDA_TRY(cudaMemset2DAsync(c.dw_down, c.ld_dw_down * 2, 0, c.dim * 2, c.hidden, s));
    return ok();
  }
  int* err = nullptr;
  TRY(ns::take_error_word(fn, &err));
  const FfnPlan p = plan(c, true);
  uint8_t* ws = static_cast<uint8_t*>(d_ws);
  Inputs in;
  TRY(stage_inputs(fn, c, p, true, ws, in, s));
  uint16_t* h = reinterpret_cast<uint16_t*>(ws + p.h);
  uint16_t* dgu = reinterpret_cast<uint16_t*>(ws + p.dgu);
  {
    Batch b{};
    b.err = err;
    b.n = 1;
    Job& j = b.job[0];
    j.kind = kGluBwd;
    j.M = static_cast<int>(c.tokens), j.N = static_cast<int>(c.hidden), j.K = static_cast<int>(c.dim);
    glu_fields(j, c);
    set_tiles(j);
    TRY(map_p(fn, j, in.dy, in.pdy));
    TRY(map_q(fn, j, in.down, c.hidden, in.pdown));
    j.out = dgu;
    j.ld_out = p.gp;
    j.out_h = h;
    j.ld_h = p.fp;
    TRY(launch(fn, b, kGluBwd, s));
  }
  Batch b{};
  b.err = err;
  Job jobs[kMaxJobs];
  const int n = grad_jobs(c, jobs);
  plan_splits(jobs, n);
  SumBatch sums{};
  float* slab = reinterpret_cast<float*>(ws + p.slab);
  TRY(map_p(fn, jobs[0], dgu, p.gp));
  TRY(map_q(fn, jobs[0], in.gate_up, c.dim, in.pgu));
  finish(jobs[0], c.dx, c.ld_dx, slab, sums);
  TRY(map_p(fn, jobs[1], in.x, in.px));
  TRY(map_q(fn, jobs[1], dgu, 2 * c.hidden, p.gp));
  finish(jobs[1], c.dw_gate_up, c.ld_dw_gate_up, slab, sums);
  TRY(map_p(fn, jobs[2], h, p.fp));
  TRY(map_q(fn, jobs[2], in.dy, c.dim, in.pdy));
  finish(jobs[2], c.dw_down, c.ld_dw_down, slab, sums);
  // The longest units first: the launch's end is then made of short ones.
  const bool dx_first = jobs[0].kb_per_split >= jobs[1].kb_per_split;
  b.n = n;
  for (int k = 0; k < n; ++k) b.job[k] = jobs[dx_first ? k : (k + 1) % n];
  TRY(launch(fn, b, kStore, s));
  return sums.n > 0 ? launch_sums(fn, sums, s) : ok();
}

}  // namespace
}  // namespace lm
}  // namespace zopt

extern "C" size_t zopt_ffn_workspace(const zopt_ffn_job* job, int32_t backward) {
  if (job == nullptr || !zopt::lm::shape_ok(*job, backward != 0)) return 0;
  const size_t n = zopt::lm::plan(*job, backward != 0).total;
  return n < 16 ? 16 : n;
}

extern "C" zopt_status zopt_ffn_forward(const zopt_ffn_job* job, void* d_ws, size_t ws_bytes, zopt_stream stream) {
  return zopt::guarded([&] { return zopt::lm::forward(job, d_ws, ws_bytes, stream); });
}

extern "C" zopt_status zopt_ffn_backward(const zopt_ffn_job* job, void* d_ws, size_t ws_bytes, zopt_stream stream) {
  return zopt::guarded([&] { return zopt::lm::backward(job, d_ws, ws_bytes, stream); });
}
