// attn_api.cpp -- the C ABI of the attention operators (declared in
// include/gdn_attn.h).  As in gdn_api.cpp every argument is validated on the
// host before anything is enqueued.
#include "gdn_attn.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>

#include "attn_checks.hpp"
#include "attn_kernels.hpp"

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
  const unsigned long long v = (unsigned long long)gdn::check_violations_attn_rope() +
                               gdn::check_violations_attn_prefill() +
                               gdn::check_violations_attn_decode();
  if (v != 0) {
    fprintf(stderr, "libgdn_check: %llu LDS accesses outside the layout\n", v);
    return GDN_ERR_CHECK;
  }
#endif
  return GDN_OK;
}

// Shape of a paged cache and its table.
gdn_status check_cache(int64_t N, int64_t num_pages, int64_t max_pages, int32_t page_size,
                       int32_t Hk, int32_t d) {
  if (num_pages < 1 || num_pages >= (int64_t(1) << 31) || max_pages < 1) return GDN_ERR_INVALID_ARG;
  if (page_size < 1) return GDN_ERR_INVALID_ARG;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128)
    return GDN_ERR_UNSUPPORTED;
  if ((double)N * (double)max_pages > kMaxElems || (double)max_pages * page_size > kMaxElems ||
      (double)num_pages * page_size * (double)Hk * d > kMaxElems)
    return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

struct CachePtrs {
  const void *k, *v;
  const float *ks, *vs;
  const int32_t* table;
  const int64_t* lens;
};
gdn_status check_cache_ptrs(const CachePtrs& c) {
  if (!c.k || !c.v || !c.ks || !c.vs || !c.table || !c.lens) return GDN_ERR_INVALID_ARG;
  if (!aligned16(c.k) || !aligned16(c.v) || !aligned16(c.ks) || !aligned16(c.vs) ||
      !aligned(c.table, 4) || !aligned(c.lens, 8))
    return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

gdn_status check_decode_desc(const gdn_attn_decode_desc* d) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (d->N < 0 || d->window < 0 || d->H_q < 1 || d->H_k < 1 || d->H_q % d->H_k != 0)
    return GDN_ERR_INVALID_ARG;
  if (!std::isfinite(d->scale) || d->scale == 0.f) return GDN_ERR_INVALID_ARG;
  gdn_status st = check_head(d->d, d->io_dtype);
  if (st != GDN_OK) return st;
  st = check_cache(d->N, d->num_pages, d->max_pages, d->page_size, d->H_k, d->d);
  if (st != GDN_OK) return st;
  if ((int64_t)d->H_q * d->d > (int64_t(1) << 22)) return GDN_ERR_UNSUPPORTED;
  if ((double)d->N * d->H_q * d->d > kMaxElems) return GDN_ERR_INVALID_ARG;
  // segments are counted in 32 bits, and so are their rounds of 128 tokens
  if ((double)d->N * d->H_q * 256.0 > kMaxThreads ||
      (double)d->N * d->H_q * ((double)d->max_pages * d->page_size / 128.0 + 1.0) > 2.0e9)
    return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

gdn::AttnDecodePlan decode_plan(const gdn_attn_decode_desc* d) {
  return gdn::attn_decode_plan(d->N, d->max_pages * d->page_size, d->window, d->H_q, d->H_k, d->d);
}

}  // namespace

extern "C" {

gdn_status gdn_qk_norm_rope(const gdn_qk_desc* d, const void* q_raw, const void* k_raw,
                            const float* q_weight, const float* k_weight,
                            const int64_t* positions, const float* inv_freq, void* q, void* k,
                            void* stream) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (d->rows < 0 || d->H_q < 0 || d->H_k < 0 || (d->H_q == 0 && d->H_k == 0))
    return GDN_ERR_INVALID_ARG;
  gdn_status st = check_head(d->d, d->io_dtype);
  if (st != GDN_OK) return st;
  st = check_rope(d->rope_dim, d->rope_mode, d->rope_scale, d->eps, d->d);
  if (st != GDN_OK) return st;
  if (d->H_q && (st = check_rows(d->rows, d->ld_q, d->H_q, d->d)) != GDN_OK) return st;
  if (d->H_k && (st = check_rows(d->rows, d->ld_k, d->H_k, d->d)) != GDN_OK) return st;
  if (d->rows == 0) return GDN_OK;
  if ((double)d->rows > 2.0e9 ||
      (double)gdn::qk_norm_rope_blocks(d->rows, d->H_q, d->H_k, d->d) * 256.0 > kMaxThreads)
    return GDN_ERR_UNSUPPORTED;
  if ((d->H_q > 0) != (q_raw != nullptr) || (d->H_q > 0) != (q != nullptr) ||
      (d->H_k > 0) != (k_raw != nullptr) || (d->H_k > 0) != (k != nullptr))
    return GDN_ERR_INVALID_ARG;
  if ((d->rope_dim > 0) != (positions != nullptr) || (d->rope_dim > 0) != (inv_freq != nullptr))
    return GDN_ERR_INVALID_ARG;
  const void* all[] = {q_raw, k_raw, q_weight, k_weight, q, k};
  for (const void* p : all)
    if (!aligned16(p)) return GDN_ERR_INVALID_ARG;
  if (!aligned(positions, 8) || !aligned(inv_freq, 4)) return GDN_ERR_INVALID_ARG;

  const int64_t R = d->rows, eb = dtype_bytes(d->io_dtype);
  const int64_t nq = (int64_t)d->H_q * d->d, nk = (int64_t)d->H_k * d->d;
  const Span sqr = rows_span(q_raw, d->H_q ? R : 0, d->ld_q, d->H_q, d->d, d->io_dtype);
  const Span skr = rows_span(k_raw, d->H_k ? R : 0, d->ld_k, d->H_k, d->d, d->io_dtype);
  const Span sq = span(q, R * nq, eb), sk = span(k, R * nk, eb);
  const Span rest[] = {span(q_weight, d->d, 4), span(k_weight, d->d, 4), span(positions, R, 8),
                       span(inv_freq, d->rope_dim / 2, 4)};
  const Span outs[] = {sq, sk};
  if (!apart(rest, outs)) return GDN_ERR_INVALID_ARG;
  // in place only where input and output are the same rows
  const bool q_same = q == q_raw && d->ld_q == nq, k_same = k == k_raw && d->ld_k == nk;
  if ((overlaps(sq, sqr) && !q_same) || (overlaps(sk, skr) && !k_same) || overlaps(sq, skr) ||
      overlaps(sk, sqr))
    return GDN_ERR_INVALID_ARG;

  gdn::QkNormRopeArgs a;
  a.rows = R; a.ld_q = d->ld_q; a.ld_k = d->ld_k;
  a.Hq = d->H_q; a.Hk = d->H_k; a.d = d->d; a.io = to_dtype(d->io_dtype);
  a.rope = gdn::RopeArgs{d->rope_dim, d->rope_mode == GDN_ROPE_INTERLEAVED, d->rope_scale, d->eps,
                         inv_freq};
  a.q_raw = q_raw; a.k_raw = k_raw; a.q_weight = q_weight; a.k_weight = k_weight;
  a.positions = positions; a.q = q; a.k = k;
  return launched(gdn::launch_qk_norm_rope(a, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_kv_append(const gdn_kv_append_desc* d, const int64_t* cu_seqlens,
                         const int64_t* seq_lens, const int32_t* page_table, const void* k_raw,
                         const void* v_raw, const float* k_weight, const float* inv_freq,
                         void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                         void* stream) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (d->N < 0 || d->total_T < 0 || d->H_k < 1) return GDN_ERR_INVALID_ARG;
  gdn_status st = check_head(d->d, d->io_dtype);
  if (st != GDN_OK) return st;
  st = check_rope(d->rope_dim, d->rope_mode, d->rope_scale, d->eps, d->d);
  if (st != GDN_OK) return st;
  st = check_cache(d->N, d->num_pages, d->max_pages, d->page_size, d->H_k, d->d);
  if (st != GDN_OK) return st;
  if ((st = check_rows(d->total_T, d->ld_k, d->H_k, d->d)) != GDN_OK) return st;
  if ((st = check_rows(d->total_T, d->ld_v, d->H_k, d->d)) != GDN_OK) return st;
  if (d->N == 0) return GDN_OK;
  if (!cu_seqlens && d->total_T % d->N != 0) return GDN_ERR_INVALID_ARG;
  if (d->total_T == 0) return GDN_OK;
  const int64_t Tseq = cu_seqlens ? 0 : d->total_T / d->N;
  if ((double)d->total_T > 2.0e9 || (double)d->N > 2.0e9 || d->H_k > 65535 ||
      (double)gdn::kv_append_slots(d->N, d->total_T, Tseq, cu_seqlens != nullptr, d->page_size) *
              4.0 * d->page_size > kMaxThreads)   // a wave for 16 rows of a page
    return GDN_ERR_UNSUPPORTED;
  if (!k_raw || !v_raw || !aligned16(k_raw) || !aligned16(v_raw) || !aligned16(k_weight) ||
      !aligned(inv_freq, 4) || !aligned(cu_seqlens, 8))
    return GDN_ERR_INVALID_ARG;
  if ((d->rope_dim > 0) != (inv_freq != nullptr)) return GDN_ERR_INVALID_ARG;
  st = check_cache_ptrs(CachePtrs{k_cache, v_cache, k_scale, v_scale, page_table, seq_lens});
  if (st != GDN_OK) return st;

  const int64_t per = (int64_t)d->page_size * d->H_k * d->d;
  const Span ins[] = {rows_span(k_raw, d->total_T, d->ld_k, d->H_k, d->d, d->io_dtype),
                      rows_span(v_raw, d->total_T, d->ld_v, d->H_k, d->d, d->io_dtype),
                      span(cu_seqlens, d->N + 1, 8), span(seq_lens, d->N, 8),
                      span(page_table, d->N * d->max_pages, 4), span(k_weight, d->d, 4),
                      span(inv_freq, d->rope_dim / 2, 4)};
  const Span outs[] = {span(k_cache, d->num_pages * per, 1), span(v_cache, d->num_pages * per, 1),
                       span(k_scale, d->num_pages * d->H_k, 4),
                       span(v_scale, d->num_pages * d->H_k, 4)};
  if (!apart(ins, outs)) return GDN_ERR_INVALID_ARG;

  gdn::KvAppendArgs a;
  a.N = d->N; a.total_T = d->total_T; a.Tseq = Tseq; a.cu_seqlens = cu_seqlens;
  a.ld_k = d->ld_k; a.ld_v = d->ld_v; a.Hk = d->H_k; a.d = d->d; a.io = to_dtype(d->io_dtype);
  a.rope = gdn::RopeArgs{d->rope_dim, d->rope_mode == GDN_ROPE_INTERLEAVED, d->rope_scale, d->eps,
                         inv_freq};
  a.k_raw = k_raw; a.v_raw = v_raw; a.k_weight = k_weight;
  a.cache = gdn::PagedCache{d->num_pages, d->max_pages, d->page_size, page_table, seq_lens,
                            static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache),
                            k_scale, v_scale};
  return launched(gdn::launch_kv_append(a, static_cast<hipStream_t>(stream)));
}

gdn_status gdn_attn_prefill(const gdn_attn_prefill_desc* d, const int64_t* cu_seqlens,
                            const void* q, const void* k, const void* v, void* o, void* stream) {
  if (!d) return GDN_ERR_INVALID_ARG;
  if (d->N < 0 || d->total_T < 0 || d->window < 0 || d->H_q < 1 || d->H_k < 1 ||
      d->H_q % d->H_k != 0)
    return GDN_ERR_INVALID_ARG;
  if (!std::isfinite(d->scale) || d->scale == 0.f) return GDN_ERR_INVALID_ARG;
  gdn_status st = check_head(d->d, d->io_dtype);
  if (st != GDN_OK) return st;
  if ((st = check_rows(d->total_T, d->ld_q, d->H_q, d->d)) != GDN_OK) return st;
  if ((st = check_rows(d->total_T, d->ld_k, d->H_k, d->d)) != GDN_OK) return st;
  if ((st = check_rows(d->total_T, d->ld_v, d->H_k, d->d)) != GDN_OK) return st;
  if (d->N == 0) return GDN_OK;
  if (!cu_seqlens && d->total_T % d->N != 0) return GDN_ERR_INVALID_ARG;
  if (d->total_T == 0) return GDN_OK;
  const int64_t Tseq = cu_seqlens ? 0 : d->total_T / d->N;
  if ((double)d->total_T > 2.0e9 || (double)d->N > 2.0e9 ||
      (double)gdn::prefill_blocks(d->N, d->total_T, Tseq, cu_seqlens != nullptr, d->H_q,
                                  to_dtype(d->io_dtype)) * 256.0 > kMaxThreads)
    return GDN_ERR_UNSUPPORTED;
  if (!q || !k || !v || !o || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) ||
      !aligned(cu_seqlens, 8))
    return GDN_ERR_INVALID_ARG;
  const Span ins[] = {rows_span(q, d->total_T, d->ld_q, d->H_q, d->d, d->io_dtype),
                      rows_span(k, d->total_T, d->ld_k, d->H_k, d->d, d->io_dtype),
                      rows_span(v, d->total_T, d->ld_v, d->H_k, d->d, d->io_dtype),
                      span(cu_seqlens, d->N + 1, 8)};
  const Span outs[] = {span(o, d->total_T * d->H_q * d->d, dtype_bytes(d->io_dtype))};
  if (!apart(ins, outs)) return GDN_ERR_INVALID_ARG;

  gdn::PrefillArgs a;
  a.N = d->N; a.total_T = d->total_T; a.Tseq = Tseq; a.cu_seqlens = cu_seqlens;
  a.ld_q = d->ld_q; a.ld_k = d->ld_k; a.ld_v = d->ld_v; a.window = d->window;
  a.Hq = d->H_q; a.Hk = d->H_k; a.d = d->d; a.io = to_dtype(d->io_dtype); a.scale = d->scale;
  a.q = q; a.k = k; a.v = v; a.o = o;
  return launched(gdn::launch_attn_prefill(a, static_cast<hipStream_t>(stream)));
}

size_t gdn_attn_decode_workspace_size(const gdn_attn_decode_desc* d) {
  if (check_decode_desc(d) != GDN_OK || d->N == 0) return 0;
  return (size_t)decode_plan(d).ws_floats * 4;
}

gdn_status gdn_attn_decode(const gdn_attn_decode_desc* d, const void* q, const void* k_cache,
                           const void* v_cache, const float* k_scale, const float* v_scale,
                           const int32_t* page_table, const int64_t* seq_lens, void* o,
                           void* workspace, size_t workspace_bytes, void* stream) {
  gdn_status st = check_decode_desc(d);
  if (st != GDN_OK) return st;
  if (d->N == 0) return GDN_OK;
  const gdn::AttnDecodePlan plan = decode_plan(d);
  if (!q || !o || !aligned16(q) || !aligned16(o)) return GDN_ERR_INVALID_ARG;
  st = check_cache_ptrs(CachePtrs{k_cache, v_cache, k_scale, v_scale, page_table, seq_lens});
  if (st != GDN_OK) return st;
  const int64_t need = plan.ws_floats * 4;
  if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < (size_t)need))
    return GDN_ERR_INVALID_ARG;

  const int64_t n = d->N * d->H_q * d->d, eb = dtype_bytes(d->io_dtype);
  const int64_t per = (int64_t)d->page_size * d->H_k * d->d;
  const Span ins[] = {span(q, n, eb), span(k_cache, d->num_pages * per, 1),
                      span(v_cache, d->num_pages * per, 1), span(k_scale, d->num_pages * d->H_k, 4),
                      span(v_scale, d->num_pages * d->H_k, 4),
                      span(page_table, d->N * d->max_pages, 4), span(seq_lens, d->N, 8)};
  const Span outs[] = {span(o, n, eb), span(workspace, need, 1)};
  if (!apart(ins, outs)) return GDN_ERR_INVALID_ARG;

  gdn::AttnDecodeArgs a;
  a.N = d->N; a.window = d->window; a.Hq = d->H_q; a.Hk = d->H_k; a.d = d->d;
  a.io = to_dtype(d->io_dtype); a.scale = d->scale; a.q = q;
  a.cache = gdn::PagedCache{d->num_pages, d->max_pages, d->page_size, page_table, seq_lens,
                            static_cast<uint8_t*>(const_cast<void*>(k_cache)),
                            static_cast<uint8_t*>(const_cast<void*>(v_cache)),
                            const_cast<float*>(k_scale), const_cast<float*>(v_scale)};
  a.o = o;
  a.ws = static_cast<float*>(workspace);
  return launched(gdn::launch_attn_decode(a, static_cast<hipStream_t>(stream)));
}

int gdn_attn_abi_version(void) { return GDN_ATTN_ABI_VERSION; }

}  // extern "C"
