// hybrid_api.cpp -- the C ABI of a hybrid's training and residual operators
// (declared in include/gdn_hybrid.h).  As in gdn_api.cpp every argument is
// validated on the host before anything is enqueued.
#include "gdn_hybrid.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>

#include "attn_checks.hpp"
#include "hybrid_kernels.hpp"

namespace {

using gdn::Span;
using gdn::aligned;
using gdn::aligned16;
using gdn::apart;
using gdn::check_head;
using gdn::check_rope;
using gdn::check_rows;
using gdn::dtype_bytes;
using gdn::kMaxElems;
using gdn::kMaxThreads;
using gdn::overlaps;
using gdn::rows_span;
using gdn::span;
using gdn::to_dtype;

gdn_status launched(hipError_t e) {
  if (e != hipSuccess) return GDN_ERR_HIP;
#ifdef GDN_CHECK
  const unsigned long long v = (unsigned long long)gdn::check_violations_attn_prefill() +
                               gdn::check_violations_attn_bwd() + gdn::check_violations_norm_ops() +
                               gdn::check_violations_rope_bwd();
  if (v != 0) {
    fprintf(stderr, "libgdn_check: %llu LDS accesses outside the layout\n", v);
    return GDN_ERR_CHECK;
  }
#endif
  return GDN_OK;
}

// A type of its own beside io_dtype: the same or fp32.
gdn_status check_second(int32_t io, int32_t other) {
  if (io != GDN_F32 && io != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (other != GDN_F32 && other != GDN_BF16) return GDN_ERR_INVALID_ARG;
  return other == io || other == GDN_F32 ? GDN_OK : GDN_ERR_UNSUPPORTED;
}

gdn_status check_width(int64_t rows, int32_t C, int64_t ld) {
  if (rows < 0 || C < 1 || C % 8 != 0 || ld < C || ld % 8 != 0 || ld > (int64_t(1) << 24))
    return GDN_ERR_INVALID_ARG;
  if (C > 16384) return GDN_ERR_UNSUPPORTED;
  if ((double)rows * (double)ld > kMaxElems) return GDN_ERR_INVALID_ARG;
  return (double)rows * 256.0 > kMaxThreads ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

// Outputs that may stand exactly where an input does.
struct Same {
  Span out, in;
  bool exactly;       // the same rows of the same type
};
bool only_exactly(const Same& s) { return !overlaps(s.out, s.in) || s.exactly; }

bool workspace_ok(const void* ws, size_t bytes, int64_t need) {
  return need == 0 || (ws && aligned16(ws) && bytes >= (size_t)need);
}

gdn_status check_prefill(const gdn_attn_prefill_desc* d) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (d->N < 0 || d->total_T < 0 || d->window < 0 || d->H_q < 1 || d->H_k < 1 ||
      d->H_q % d->H_k != 0)
    return GDN_ERR_INVALID_ARG;
  if (!std::isfinite(d->scale) || d->scale == 0.f) return GDN_ERR_INVALID_ARG;
  gdn_status st = check_head(d->d, d->io_dtype);
  if (st != GDN_OK) return st;
  if ((st = check_rows(d->total_T, d->ld_q, d->H_q, d->d)) != GDN_OK) return st;
  if ((st = check_rows(d->total_T, d->ld_k, d->H_k, d->d)) != GDN_OK) return st;
  return check_rows(d->total_T, d->ld_v, d->H_k, d->d);
}

gdn_status check_attn_bwd(const gdn_attn_bwd_desc* d) {
  if (!d) return GDN_ERR_INVALID_ARG;
  const gdn_attn_prefill_desc f{d->N, d->total_T, d->ld_q, d->ld_k, d->ld_v, d->window, d->H_q, d->H_k,
                                d->d, d->io_dtype, d->scale};
  gdn_status st = check_prefill(&f);
  if (st != GDN_OK) return st;
  if ((st = check_second(d->io_dtype, d->grad_dtype)) != GDN_OK) return st;
  if ((st = check_rows(d->total_T, d->ld_dq, d->H_q, d->d)) != GDN_OK) return st;
  if ((st = check_rows(d->total_T, d->ld_dk, d->H_k, d->d)) != GDN_OK) return st;
  if ((st = check_rows(d->total_T, d->ld_dv, d->H_k, d->d)) != GDN_OK) return st;
  const float s = std::fabs(d->scale);
  if (!(s >= 0x1p-60f && s <= 0x1p60f)) return GDN_ERR_UNSUPPORTED;
  return (double)d->total_T > 2.0e9 || (double)d->N > 2.0e9 ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

gdn::AttnBwdPlan bwd_plan(const gdn_attn_bwd_desc* d) {
  return gdn::attn_bwd_plan(d->N, d->total_T, d->window, d->H_q, d->H_k, d->d, to_dtype(d->io_dtype));
}

gdn_status check_qk_bwd(const gdn_qk_bwd_desc* d) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (d->rows < 0 || d->H_q < 0 || d->H_k < 0 || (d->H_q == 0 && d->H_k == 0))
    return GDN_ERR_INVALID_ARG;
  gdn_status st = check_head(d->d, d->io_dtype);
  if (st != GDN_OK) return st;
  if ((st = check_second(d->io_dtype, d->grad_dtype)) != GDN_OK) return st;
  st = check_rope(d->rope_dim, d->rope_mode, d->rope_scale, d->eps, d->d);
  if (st != GDN_OK) return st;
  if (d->H_q) {
    if ((st = check_rows(d->rows, d->ld_q, d->H_q, d->d)) != GDN_OK) return st;
    if ((st = check_rows(d->rows, d->ld_dq, d->H_q, d->d)) != GDN_OK) return st;
  }
  if (d->H_k) {
    if ((st = check_rows(d->rows, d->ld_k, d->H_k, d->d)) != GDN_OK) return st;
    if ((st = check_rows(d->rows, d->ld_dk, d->H_k, d->d)) != GDN_OK) return st;
  }
  return (double)d->rows > 2.0e9 ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

gdn_status check_add_norm_bwd(const gdn_add_norm_bwd_desc* d) {
  if (!d) return GDN_ERR_INVALID_ARG;
  gdn_status st = check_second(d->io_dtype, d->res_dtype);
  if (st != GDN_OK) return st;
  if (!std::isfinite(d->eps) || d->eps < 0.f) return GDN_ERR_INVALID_ARG;
  return check_width(d->rows, d->C, d->ld_dx);
}

}  // namespace

extern "C" {

gdn_status gdn_attn_prefill_save(const gdn_attn_prefill_desc* d, const int64_t* cu_seqlens,
                                 const void* q, const void* k, const void* v, void* o,
                                 float* stats, void* stream) {
  gdn_status st = check_prefill(d);
  if (st != GDN_OK) return st;
  if (d->N == 0) return GDN_OK;
  if (!cu_seqlens && d->total_T % d->N != 0) return GDN_ERR_INVALID_ARG;
  if (d->total_T == 0) return GDN_OK;
  const int64_t Tseq = cu_seqlens ? 0 : d->total_T / d->N;
  if ((double)d->total_T > 2.0e9 || (double)d->N > 2.0e9 ||
      (double)gdn::prefill_blocks(d->N, d->total_T, Tseq, cu_seqlens != nullptr, d->H_q,
                                  to_dtype(d->io_dtype)) * 256.0 > kMaxThreads)
    return GDN_ERR_UNSUPPORTED;
  if (!q || !k || !v || !o || !stats || !aligned16(q) || !aligned16(k) || !aligned16(v) ||
      !aligned16(o) || !aligned16(stats) || !aligned(cu_seqlens, 8))
    return GDN_ERR_INVALID_ARG;
  const Span ins[] = {rows_span(q, d->total_T, d->ld_q, d->H_q, d->d, d->io_dtype),
                      rows_span(k, d->total_T, d->ld_k, d->H_k, d->d, d->io_dtype),
                      rows_span(v, d->total_T, d->ld_v, d->H_k, d->d, d->io_dtype),
                      span(cu_seqlens, d->N + 1, 8)};
  const Span outs[] = {span(o, d->total_T * d->H_q * d->d, dtype_bytes(d->io_dtype)),
                       span(stats, d->total_T * d->H_q * gdn::stats_width(to_dtype(d->io_dtype), d->d), 4)};
  if (!apart(ins, outs)) return GDN_ERR_INVALID_ARG;

  gdn::PrefillArgs a;
  a.N = d->N; a.total_T = d->total_T; a.Tseq = Tseq; a.cu_seqlens = cu_seqlens;
  a.ld_q = d->ld_q; a.ld_k = d->ld_k; a.ld_v = d->ld_v; a.window = d->window;
  a.Hq = d->H_q; a.Hk = d->H_k; a.d = d->d; a.io = to_dtype(d->io_dtype); a.scale = d->scale;
  a.q = q; a.k = k; a.v = v; a.o = o; a.stats = stats;
  return launched(gdn::launch_attn_prefill(a, static_cast<hipStream_t>(stream)));
}

size_t gdn_attn_backward_workspace_size(const gdn_attn_bwd_desc* d) {
  if (check_attn_bwd(d) != GDN_OK || d->N == 0 || d->total_T == 0) return 0;
  return (size_t)bwd_plan(d).ws_floats * 4;
}

gdn_status gdn_attn_backward(const gdn_attn_bwd_desc* d, const int64_t* cu_seqlens,
                             const void* q, const void* k, const void* v, const void* o,
                             const void* d_o, const float* stats, void* workspace,
                             size_t workspace_bytes, void* dq, void* dk, void* dv, void* stream) {
  gdn_status st = check_attn_bwd(d);
  if (st != GDN_OK) return st;
  if (d->N == 0) return GDN_OK;
  if (!cu_seqlens && d->total_T % d->N != 0) return GDN_ERR_INVALID_ARG;
  if (d->total_T == 0) return GDN_OK;
  const int64_t Tseq = cu_seqlens ? 0 : d->total_T / d->N;
  const gdn::AttnBwdPlan plan = bwd_plan(d);
  if ((double)gdn::attn_bwd_blocks(d->N, d->total_T, Tseq, cu_seqlens != nullptr, d->H_q,
                                   to_dtype(d->io_dtype)) * 256.0 > kMaxThreads)
    return GDN_ERR_UNSUPPORTED;
  const void* all[] = {q, k, v, o, d_o, stats, dq, dk, dv};
  for (const void* p : all)
    if (!p || !aligned16(p)) return GDN_ERR_INVALID_ARG;
  if (!aligned(cu_seqlens, 8)) return GDN_ERR_INVALID_ARG;
  const int64_t need = plan.ws_floats * 4;
  if (!workspace_ok(workspace, workspace_bytes, need)) return GDN_ERR_INVALID_ARG;

  const int64_t T = d->total_T, n = T * d->H_q * d->d, eb = dtype_bytes(d->io_dtype);
  const Span ins[] = {rows_span(q, T, d->ld_q, d->H_q, d->d, d->io_dtype),
                      rows_span(k, T, d->ld_k, d->H_k, d->d, d->io_dtype),
                      rows_span(v, T, d->ld_v, d->H_k, d->d, d->io_dtype), span(o, n, eb),
                      span(d_o, n, eb),
                      span(stats, T * d->H_q * gdn::stats_width(to_dtype(d->io_dtype), d->d), 4),
                      span(cu_seqlens, d->N + 1, 8)};
  // dq, dk and dv may be column blocks of one buffer: rows apart, not spans
  const Span sdq = rows_span(dq, T, d->ld_dq, d->H_q, d->d, d->grad_dtype);
  const Span sdk = rows_span(dk, T, d->ld_dk, d->H_k, d->d, d->grad_dtype);
  const Span sdv = rows_span(dv, T, d->ld_dv, d->H_k, d->d, d->grad_dtype);
  const Span ws[] = {span(workspace, need, 1)};
  const Span outs[] = {sdq, sdk, sdv};
  for (const Span& s : outs) {
    const Span one[] = {s};
    if (!apart(ins, one) || !apart(outs, ws)) return GDN_ERR_INVALID_ARG;
  }
  if (!apart(ins, ws)) return GDN_ERR_INVALID_ARG;
  const int64_t gb = dtype_bytes(d->grad_dtype), wq = (int64_t)d->H_q * d->d * gb, wk = (int64_t)d->H_k * d->d * gb;
  if (!gdn::blocks_apart(sdq, d->ld_dq * gb, wq, sdk, d->ld_dk * gb, wk) ||
      !gdn::blocks_apart(sdq, d->ld_dq * gb, wq, sdv, d->ld_dv * gb, wk) ||
      !gdn::blocks_apart(sdk, d->ld_dk * gb, wk, sdv, d->ld_dv * gb, wk))
    return GDN_ERR_INVALID_ARG;

  gdn::AttnBwdArgs a;
  a.N = d->N; a.total_T = T; a.Tseq = Tseq; a.cu_seqlens = cu_seqlens;
  a.ld_q = d->ld_q; a.ld_k = d->ld_k; a.ld_v = d->ld_v;
  a.ld_dq = d->ld_dq; a.ld_dk = d->ld_dk; a.ld_dv = d->ld_dv; a.window = d->window;
  a.Hq = d->H_q; a.Hk = d->H_k; a.d = d->d;
  a.io = to_dtype(d->io_dtype); a.grad = to_dtype(d->grad_dtype); a.scale = d->scale;
  a.q = q; a.k = k; a.v = v; a.o = o; a.d_o = d_o; a.stats = stats;
  a.dq = dq; a.dk = dk; a.dv = dv; a.ws = static_cast<float*>(workspace);
  return launched(gdn::launch_attn_bwd(a, plan, static_cast<hipStream_t>(stream)));
}

size_t gdn_qk_norm_rope_backward_workspace_size(const gdn_qk_bwd_desc* d) {
  if (check_qk_bwd(d) != GDN_OK) return 0;
  return (size_t)gdn::qk_bwd_ws_floats(d->rows, d->H_q, d->H_k, d->d) * 4;
}

gdn_status gdn_qk_norm_rope_backward(const gdn_qk_bwd_desc* d, const void* dq, const void* dk,
                                     const void* q_raw, const void* k_raw,
                                     const float* q_weight, const float* k_weight,
                                     const int64_t* positions, const float* inv_freq,
                                     void* workspace, size_t workspace_bytes, void* dq_raw,
                                     void* dk_raw, float* dq_weight, float* dk_weight,
                                     void* stream) {
  gdn_status st = check_qk_bwd(d);
  if (st != GDN_OK) return st;
  const bool has_q = d->H_q > 0, has_k = d->H_k > 0;
  if ((!has_q && (dq || dq_raw || q_raw || q_weight || dq_weight)) ||
      (!has_k && (dk || dk_raw || k_raw || k_weight || dk_weight)))
    return GDN_ERR_INVALID_ARG;
  if ((dq_weight && !q_weight) || (dk_weight && !k_weight)) return GDN_ERR_INVALID_ARG;
  if (d->rows > 0) {
    if (has_q != (dq != nullptr) || has_q != (dq_raw != nullptr) || has_k != (dk != nullptr) ||
        has_k != (dk_raw != nullptr) || (q_weight && !q_raw) || (k_weight && !k_raw))
      return GDN_ERR_INVALID_ARG;
    if ((d->rope_dim > 0) != (positions != nullptr) || (d->rope_dim > 0) != (inv_freq != nullptr))
      return GDN_ERR_INVALID_ARG;
  }
  const void* all[] = {dq, dk, q_raw, k_raw, q_weight, k_weight, dq_raw, dk_raw, dq_weight, dk_weight};
  for (const void* p : all)
    if (!aligned16(p)) return GDN_ERR_INVALID_ARG;
  if (!aligned(positions, 8) || !aligned(inv_freq, 4)) return GDN_ERR_INVALID_ARG;
  const int64_t need = dq_weight || dk_weight ? gdn::qk_bwd_ws_floats(d->rows, d->H_q, d->H_k, d->d) * 4 : 0;
  if (!workspace_ok(workspace, workspace_bytes, need)) return GDN_ERR_INVALID_ARG;
  if (d->rows == 0 && !dq_weight && !dk_weight) return GDN_OK;

  const int64_t R = d->rows, gb = dtype_bytes(d->grad_dtype);
  const int64_t nq = (int64_t)d->H_q * d->d, nk = (int64_t)d->H_k * d->d;
  const Span ins[] = {rows_span(q_raw, has_q ? R : 0, d->ld_q, d->H_q, d->d, d->io_dtype),
                      rows_span(k_raw, has_k ? R : 0, d->ld_k, d->H_k, d->d, d->io_dtype),
                      span(q_weight, d->d, 4), span(k_weight, d->d, 4), span(positions, R, 8),
                      span(inv_freq, d->rope_dim / 2, 4)};
  const Span sq = span(dq, R * nq, gb), sk = span(dk, R * nk, gb);
  const Span oq = rows_span(dq_raw, has_q ? R : 0, d->ld_dq, d->H_q, d->d, d->grad_dtype);
  const Span ok = rows_span(dk_raw, has_k ? R : 0, d->ld_dk, d->H_k, d->d, d->grad_dtype);
  const Span rows_out[] = {oq, ok};
  const Span rest[] = {span(dq_weight, d->d, 4), span(dk_weight, d->d, 4), span(workspace, need, 1)};
  const Span ups[] = {sq, sk};
  for (const Span& s : rows_out) {
    const Span one[] = {s};
    if (!apart(ins, one)) return GDN_ERR_INVALID_ARG;
  }
  if (!apart(ins, rest) || !apart(ups, rest) || !apart(rows_out, rest)) return GDN_ERR_INVALID_ARG;
  if (!gdn::blocks_apart(oq, d->ld_dq * gb, nq * gb, ok, d->ld_dk * gb, nk * gb)) return GDN_ERR_INVALID_ARG;
  // in place only where gradient and output are the same rows
  if (overlaps(oq, sk) || overlaps(ok, sq) ||
      !only_exactly(Same{oq, sq, dq == dq_raw && d->ld_dq == nq}) ||
      !only_exactly(Same{ok, sk, dk == dk_raw && d->ld_dk == nk}))
    return GDN_ERR_INVALID_ARG;

  gdn::QkNormRopeBwdArgs a;
  a.rows = R; a.ld_q = d->ld_q; a.ld_k = d->ld_k; a.ld_dq = d->ld_dq; a.ld_dk = d->ld_dk;
  a.Hq = d->H_q; a.Hk = d->H_k; a.d = d->d;
  a.io = to_dtype(d->io_dtype); a.grad = to_dtype(d->grad_dtype);
  a.rope = gdn::RopeArgs{d->rope_dim, d->rope_mode == GDN_ROPE_INTERLEAVED, d->rope_scale, d->eps,
                         inv_freq};
  a.dq = dq; a.dk = dk; a.q_raw = q_raw; a.k_raw = k_raw; a.q_weight = q_weight;
  a.k_weight = k_weight; a.positions = positions; a.dq_raw = dq_raw; a.dk_raw = dk_raw;
  a.dq_weight = dq_weight; a.dk_weight = dk_weight; a.ws = static_cast<float*>(workspace);
  return launched(gdn::launch_qk_norm_rope_bwd(a, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_add_norm(const gdn_add_norm_desc* d, const void* x, const void* res,
                        const float* weight, void* res_out, void* y, float* y_scale,
                        void* stream) {
  if (!d) return GDN_ERR_INVALID_ARG;
  gdn_status st = check_second(d->io_dtype, d->res_dtype);
  if (st != GDN_OK) return st;
  if (!std::isfinite(d->eps) || d->eps < 0.f) return GDN_ERR_INVALID_ARG;
  if ((st = check_width(d->rows, d->C, d->ld_x)) != GDN_OK) return st;
  if (d->group < -1) return GDN_ERR_INVALID_ARG;
  if (d->group > 0) {
    if (d->group != 32 && d->group != 64 && d->group != 128) return GDN_ERR_UNSUPPORTED;
    if (d->C % d->group != 0) return GDN_ERR_INVALID_ARG;
  }
  if (d->rows == 0) return GDN_OK;
  if (!x || !y || (d->group >= 0) != (y_scale != nullptr)) return GDN_ERR_INVALID_ARG;
  const void* all[] = {x, res, weight, res_out, y};
  for (const void* p : all)
    if (!aligned16(p)) return GDN_ERR_INVALID_ARG;
  if (!aligned(y_scale, 4)) return GDN_ERR_INVALID_ARG;

  const int64_t n = d->rows * d->C, eb = dtype_bytes(d->io_dtype), rb = dtype_bytes(d->res_dtype);
  const bool dense = d->ld_x == d->C;
  const Span sx = rows_span(x, d->rows, d->ld_x, 1, d->C, d->io_dtype), sr = span(res, n, rb);
  const Span so = span(res_out, n, rb), sy = span(y, n, d->group < 0 ? eb : 1);
  const Span ss = span(y_scale, d->rows * (d->group > 0 ? d->C / d->group : 1), 4);
  const Span w[] = {span(weight, d->C, 4)};
  const Span outs[] = {so, sy, ss};
  if (!apart(w, outs)) return GDN_ERR_INVALID_ARG;
  if (!only_exactly(Same{so, sr, res_out == res}) ||
      !only_exactly(Same{so, sx, res_out == x && dense && eb == rb}) ||
      !only_exactly(Same{sy, sx, y == x && dense && d->group < 0}) || overlaps(sy, sr) ||
      overlaps(ss, sx) || overlaps(ss, sr))
    return GDN_ERR_INVALID_ARG;

  gdn::AddNormArgs a;
  a.rows = d->rows; a.ld_x = d->ld_x; a.C = d->C; a.group = d->group;
  a.io = to_dtype(d->io_dtype); a.res_type = to_dtype(d->res_dtype); a.eps = d->eps;
  a.x = x; a.res = res; a.weight = weight; a.res_out = res_out; a.y = y; a.y_scale = y_scale;
  return launched(gdn::launch_add_norm(a, static_cast<hipStream_t>(stream)));
}

size_t gdn_add_norm_backward_workspace_size(const gdn_add_norm_bwd_desc* d) {
  if (check_add_norm_bwd(d) != GDN_OK) return 0;
  return (size_t)gdn::add_norm_bwd_ws_floats(d->rows, d->C) * 4;
}

gdn_status gdn_add_norm_backward(const gdn_add_norm_bwd_desc* d, const void* dy, const void* r,
                                 const float* weight, const void* d_res_out, void* workspace,
                                 size_t workspace_bytes, void* dx, void* d_res, float* d_weight,
                                 void* stream) {
  gdn_status st = check_add_norm_bwd(d);
  if (st != GDN_OK) return st;
  if (d->rows > 0 && (!dy || !r)) return GDN_ERR_INVALID_ARG;
  const void* all[] = {dy, r, weight, d_res_out, dx, d_res, d_weight};
  for (const void* p : all)
    if (!aligned16(p)) return GDN_ERR_INVALID_ARG;
  const int64_t need = d_weight ? gdn::add_norm_bwd_ws_floats(d->rows, d->C) * 4 : 0;
  if (!workspace_ok(workspace, workspace_bytes, need)) return GDN_ERR_INVALID_ARG;
  if ((d->rows == 0 || (!dx && !d_res)) && !d_weight) return GDN_OK;

  const int64_t n = d->rows * d->C, eb = dtype_bytes(d->io_dtype), rb = dtype_bytes(d->res_dtype);
  const Span sy = span(dy, n, eb), sd = span(d_res_out, n, rb);
  const Span ox = rows_span(dx, d->rows, d->ld_dx, 1, d->C, d->io_dtype), od = span(d_res, n, rb);
  const Span ins[] = {span(r, n, rb), span(weight, d->C, 4)};
  const Span outs[] = {ox, od, span(d_weight, d->C, 4), span(workspace, need, 1)};
  if (!apart(ins, outs)) return GDN_ERR_INVALID_ARG;
  const Span ups[] = {sy, sd}, rest[] = {outs[2], outs[3]};
  if (!apart(ups, rest) || !only_exactly(Same{ox, sy, dx == dy && d->ld_dx == d->C}) ||
      !only_exactly(Same{od, sd, d_res == d_res_out}) || overlaps(ox, sd) || overlaps(od, sy))
    return GDN_ERR_INVALID_ARG;

  gdn::AddNormBwdArgs a;
  a.rows = d->rows; a.ld_dx = d->ld_dx; a.C = d->C;
  a.io = to_dtype(d->io_dtype); a.res_type = to_dtype(d->res_dtype); a.eps = d->eps;
  a.dy = dy; a.r = r; a.d_res_out = d_res_out; a.weight = weight; a.dx = dx; a.d_res = d_res;
  a.d_weight = d_weight; a.ws = static_cast<float*>(workspace);
  return launched(gdn::launch_add_norm_bwd(a, static_cast<hipStream_t>(stream)));
}

int gdn_hybrid_abi_version(void) { return GDN_HYBRID_ABI_VERSION; }

}  // extern "C"
