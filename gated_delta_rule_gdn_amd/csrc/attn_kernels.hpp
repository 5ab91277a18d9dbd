// attn_kernels.hpp -- host-side launch interface between the C ABI layer of
// the attention operators (attn_api.cpp) and their kernels.  Arguments arrive
// already validated; each launcher picks the template instantiation and
// launches on the given stream, returning the launch status.
#pragma once

#include "gdn_kernels.hpp"

namespace gdn {

// Rotary position and norm of a head's row.
struct RopeArgs {
  int dim;                            // channels rotated, % 16 == 0 (0: none)
  bool inter;                         // pairs (2 i, 2 i + 1), else (i, i + dim / 2)
  float factor;                       // on cos and sin
  float eps;
  const float* inv_freq;              // [dim / 2]
};

struct QkNormRopeArgs {
  int64_t rows, ld_q, ld_k;
  int Hq, Hk, d;
  DType io;
  RopeArgs rope;
  const void *q_raw, *k_raw;
  const float *q_weight, *k_weight;   // [d] or NULL (no norm)
  const int64_t* positions;           // [rows]
  void *q, *k;
};

// A paged cache of e4m3 codes with one fp32 scale for each page and head.
struct PagedCache {
  int64_t num_pages, max_pages;
  int page_size;
  const int32_t* table;               // [N, max_pages]
  const int64_t* seq_lens;            // [N]
  uint8_t *k, *v;                     // [num_pages, Hk, page_size, d]
  float *k_scale, *v_scale;           // [num_pages, Hk]
};

struct KvAppendArgs {
  int64_t N, total_T, Tseq;           // Tseq: tokens per sequence when cu_seqlens is NULL
  const int64_t* cu_seqlens;          // device [N + 1] or NULL
  int64_t ld_k, ld_v;
  int Hk, d;
  DType io;
  RopeArgs rope;
  const void *k_raw, *v_raw;
  const float* k_weight;              // [d] or NULL (no norm)
  PagedCache cache;
};

struct PrefillArgs {
  int64_t N, total_T, Tseq;           // Tseq: tokens per sequence when cu_seqlens is NULL
  const int64_t* cu_seqlens;          // device [N + 1] or NULL
  int64_t ld_q, ld_k, ld_v, window;   // window 0: none
  int Hq, Hk, d;
  DType io;
  float scale;
  const void *q, *k, *v;
  void* o;
};

struct AttnDecodeArgs {
  int64_t N, window;                  // window 0: none
  int Hq, Hk, d;
  DType io;
  float scale;
  const void* q;
  PagedCache cache;                   // read only
  void* o;
  float* ws;                          // attn_decode_plan(...).ws_floats
};

// How a decode call divides the caches: its workgroups, the most rounds of
// work there can be (fits in 32 bits, checked by the caller) and the workspace.
struct AttnDecodePlan {
  int64_t blocks, rounds, ws_floats;
};
AttnDecodePlan attn_decode_plan(int64_t N, int64_t max_tokens, int64_t window, int Hq, int Hk,
                                int d);

// Workgroups of a launch (checked against the grid limit by the caller).
int64_t qk_norm_rope_blocks(int64_t rows, int Hq, int Hk, int d);
int64_t kv_append_slots(int64_t N, int64_t total_T, int64_t Tseq, bool packed, int page_size);
int64_t prefill_blocks(int64_t N, int64_t total_T, int64_t Tseq, bool packed, int Hq, DType io);

hipError_t launch_qk_norm_rope(const QkNormRopeArgs& a, hipStream_t stream);
hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t stream);
hipError_t launch_attn_prefill(const PrefillArgs& a, hipStream_t stream);
hipError_t launch_attn_decode(const AttnDecodeArgs& a, hipStream_t stream);

#ifdef GDN_CHECK
unsigned check_violations_attn_rope();
unsigned check_violations_attn_prefill();
unsigned check_violations_attn_decode();
#endif

}  // namespace gdn
