// hybrid_kernels.hpp -- host-side launch interface between the C ABI layer of a
// hybrid's training and residual operators (hybrid_api.cpp) and their kernels.
// Arguments arrive already validated; each launcher picks the template
// instantiation and launches on the given stream, returning the launch status.
#pragma once

#include "attn_kernels.hpp"

namespace gdn {

struct AttnBwdArgs {
  int64_t N, total_T, Tseq;           // Tseq: tokens per sequence when cu_seqlens is NULL
  const int64_t* cu_seqlens;          // device [N + 1] or NULL
  int64_t ld_q, ld_k, ld_v, ld_dq, ld_dk, ld_dv, window;
  int Hq, Hk, d;
  DType io, grad;
  float scale;
  const void *q, *k, *v, *o, *d_o;
  const float* stats;                 // total_T Hq stats_width words
  void *dq, *dk, *dv;
  float* ws;                          // attn_bwd_plan(...).ws_floats
};

// To how many workgroups a backward call may deal its key tiles' walks in equal shares (0:
// each tile has a workgroup of its own), and the workspace.
struct AttnBwdPlan {
  int workers;
  int64_t ws_floats;
};
AttnBwdPlan attn_bwd_plan(int64_t N, int64_t total_T, int64_t window, int Hq, int Hk, int d,
                          DType io);
// The most workgroups of any launch (checked against the grid limit by the caller).
int64_t attn_bwd_blocks(int64_t N, int64_t total_T, int64_t Tseq, bool packed, int Hq, DType io);

struct QkNormRopeBwdArgs {
  int64_t rows, ld_q, ld_k, ld_dq, ld_dk;
  int Hq, Hk, d;
  DType io, grad;
  RopeArgs rope;
  const void *dq, *dk, *q_raw, *k_raw;
  const float *q_weight, *k_weight;   // [d] or NULL (no norm)
  const int64_t* positions;           // [rows]
  void *dq_raw, *dk_raw;
  float *dq_weight, *dk_weight;       // [d] or NULL
  float* ws;                          // qk_bwd_ws_floats(...)
};
int64_t qk_bwd_ws_floats(int64_t rows, int Hq, int Hk, int d);

struct AddNormArgs {
  int64_t rows, ld_x;
  int C, group;                       // group < 0: y in io; 0: one scale for a row; else channels of a scale
  DType io, res_type;
  float eps;
  const void *x, *res;                // res or NULL
  const float* weight;                // [C] or NULL
  void *res_out, *y;                  // res_out or NULL
  float* y_scale;
};

struct AddNormBwdArgs {
  int64_t rows, ld_dx;
  int C;
  DType io, res_type;
  float eps;
  const void *dy, *r, *d_res_out;     // d_res_out or NULL
  const float* weight;                // [C] or NULL
  void *dx, *d_res;                   // each or NULL
  float* d_weight;                    // [C] or NULL
  float* ws;                          // add_norm_bwd_ws_floats(...)
};
int64_t add_norm_bwd_ws_floats(int64_t rows, int C);

hipError_t launch_attn_bwd(const AttnBwdArgs& a, const AttnBwdPlan& plan, hipStream_t stream);
hipError_t launch_qk_norm_rope_bwd(const QkNormRopeBwdArgs& a, hipStream_t stream);
hipError_t launch_add_norm(const AddNormArgs& a, hipStream_t stream);
hipError_t launch_add_norm_bwd(const AddNormBwdArgs& a, hipStream_t stream);

#ifdef GDN_CHECK
unsigned check_violations_attn_bwd();
unsigned check_violations_norm_ops();
unsigned check_violations_rope_bwd();
#endif

}  // namespace gdn
