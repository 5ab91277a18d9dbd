/*
 * gdn_hybrid.h -- C ABI of libgdn.so for what a hybrid model needs besides its
 * delta-rule layers (gdn.h) and the serving of its softmax-attention layers
 * (gdn_attn.h) on AMD Instinct MI355X (gfx950): the residual stream between all
 * of its layers, and the training of the attention layers ("Gated DeltaNet",
 * §Architecture et versions hybrides).  The pages leave the arithmetic of both
 * to the literature; what is computed here is stated with each entry point.
 *
 * A training step of an attention layer is gdn_add_norm, the projection,
 * gdn_qk_norm_rope (gdn_attn.h) and gdn_attn_prefill_save forward, and
 * gdn_attn_backward, gdn_qk_norm_rope_backward, the projection's gradient and
 * gdn_add_norm_backward back.
 *
 * The conventions of gdn.h and gdn_attn.h hold (memory, row strides, head
 * groups, asynchrony, errors, status codes, nothing allocated, no mutable
 * state), with these additions:
 *  - grad_dtype and res_dtype equal io_dtype, or are GDN_F32 (GDN_ERR_UNSUPPORTED
 *    otherwise).
 *  - Sums have a fixed order: the same call on the same inputs gives the same
 *    bits.
 *  - A workspace needs no initial contents, its contents are unspecified on
 *    return, and calls that may overlap in time need one each.
 *  - Gradients of weights are sums over all rows; with rows == 0 they are zero.
 */
#ifndef GDN_HYBRID_H
#define GDN_HYBRID_H

#include "gdn_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_HYBRID_ABI_VERSION 1

/*
 * gdn_attn_prefill_save -- gdn_attn_prefill (same descriptor, arguments and
 * result) that also leaves, for gdn_attn_backward, each query's statistics.
 *
 *   stats (output) 16-byte aligned.  [total_T, H_q, 2] fp32: m, the maximum score
 *         (times log2 e) or a number at most 8 below it, and the sum of 2^(score - m).
 *         With bf16 io, behind those, [total_T, H_q, d] bytes b: what o was, to 16 bits,
 *         before it was rounded, its bits as fp32's + 2^8 b - 2^15 + 2^7.  Rows that no
 *         range covers are kept
 */
gdn_status gdn_attn_prefill_save(const gdn_attn_prefill_desc* desc, const int64_t* cu_seqlens,
                                 const void* q, const void* k, const void* v, void* o,
                                 float* stats, void* stream);

/* Gradients of causal attention. */
typedef struct gdn_attn_bwd_desc {
  int64_t N;          /* sequences, >= 0 (0: nothing to do)                      */
  int64_t total_T;    /* packed tokens, >= 0, < 2^31                             */
  int64_t ld_q, ld_k, ld_v;    /* row strides of q, k, v (elements)              */
  int64_t ld_dq, ld_dk, ld_dv; /* row strides of dq, dk, dv (elements)           */
  int64_t window;     /* as in gdn_attn_prefill_desc                             */
  int32_t H_q, H_k;   /* >= 1, H_q % H_k == 0                                    */
  int32_t d;          /* 64 or 128                                               */
  int32_t io_dtype;   /* gdn_dtype of q, k, v, o, d_o                            */
  int32_t grad_dtype; /* gdn_dtype of dq, dk, dv                                 */
  float scale;        /* the forward's; 2^-60 <= |scale| <= 2^60                 */
} gdn_attn_bwd_desc;

/*
 * gdn_attn_backward_workspace_size -- bytes of device workspace gdn_attn_backward
 * needs for this descriptor (0 for an invalid one or when there is no token):
 * 16 for each token and query head, and where several workgroups may share a key
 * tile their partial sums.
 */
size_t gdn_attn_backward_workspace_size(const gdn_attn_bwd_desc* desc);

/*
 * gdn_attn_backward -- gradients of L = sum(o * d_o) with o of gdn_attn_prefill:
 * with p_ts its weights, formed again from q, k and stats,
 *
 *   D_t = d_o_t . o_t,   e_ts = p_ts (d_o_t . v_s - D_t)
 *   dq_t = scale sum_s e_ts k_s
 *   dk_s = scale sum_t e_ts q_t,   dv_s = sum_t p_ts d_o_t     (over the query
 *                                                     heads of the key head too)
 *
 * Sums in fp32; with bf16 io, p and e are rounded to bf16 for the products that
 * use them, and o is the forward's to 16 bits (see stats).  p carries the rounding of scores
 * and of m in fp32, relative 2^-23 times the larger of them: scores (times
 * log2 e) of 2^20 and more have no meaningful gradients.
 * Non-finite inputs: what is not finite in a token makes gradients of its own
 * sequence, in the heads concerned, unspecified; other sequences and heads, and
 * tokens further than the window and 256 more from it, are not touched by it.
 *
 *   cu_seqlens, q, k, v  as for gdn_attn_prefill_save
 *   o, d_o     [total_T, H_q, d] io_dtype, dense: the forward's output and the
 *              upstream gradient
 *   stats      of gdn_attn_prefill_save for the same arguments (others give
 *              meaningless gradients, never an access outside the arguments)
 *   workspace  >= gdn_attn_backward_workspace_size(desc) bytes, 16-byte aligned
 *   dq [total_T, H_q, d], dk, dv [total_T, H_k, d] grad_dtype, row strides
 *              (outputs); may be column blocks of one buffer.  Rows before the
 *              first range and behind the last are kept; offsets that fall give
 *              unspecified gradients, never an access outside the arguments.
 */
gdn_status gdn_attn_backward(const gdn_attn_bwd_desc* desc, const int64_t* cu_seqlens,
                             const void* q, const void* k, const void* v, const void* o,
                             const void* d_o, const float* stats, void* workspace,
                             size_t workspace_bytes, void* dq, void* dk, void* dv, void* stream);

/* Gradient of the norm and rotation of query and key rows. */
typedef struct gdn_qk_bwd_desc {
  int64_t rows;         /* tokens, >= 0                                          */
  int64_t ld_q, ld_k;   /* row strides of q_raw and k_raw (elements)             */
  int64_t ld_dq, ld_dk; /* row strides of dq_raw and dk_raw (elements)           */
  int32_t H_q, H_k;     /* >= 0, not both 0 (0: that operand is absent)          */
  int32_t d;            /* 64 or 128                                             */
  int32_t rope_dim;     /* as in gdn_qk_desc                                     */
  int32_t rope_mode;    /* gdn_rope_mode                                         */
  int32_t io_dtype;     /* gdn_dtype of q_raw, k_raw                             */
  int32_t grad_dtype;   /* gdn_dtype of dq, dk, dq_raw, dk_raw                   */
  float rope_scale;     /* finite                                                */
  float eps;            /* finite, >= 0                                          */
} gdn_qk_bwd_desc;

/* Bytes of device workspace gdn_qk_norm_rope_backward needs (0 for an invalid
 * descriptor or when there is no row). */
size_t gdn_qk_norm_rope_backward_workspace_size(const gdn_qk_bwd_desc* desc);

/*
 * gdn_qk_norm_rope_backward -- gradients of gdn_qk_norm_rope for upstream
 * gradients dq, dk: with g = dy turned back by the row's angles (times
 * rope_scale), n = x / sqrt(mean(x^2) + eps),
 *
 *   d_weight = sum over rows and heads of g n
 *   dx = (g weight - n mean(n g weight)) / sqrt(mean(x^2) + eps)
 *
 * and dx = g for an operand that is not normed.  Accuracy and ranges as
 * gdn_qk_norm_rope.
 *
 *   dq, dk     [rows, H, d] grad_dtype, dense (NULL when H is 0)
 *   q_raw, k_raw, q_weight, k_weight, positions, inv_freq  the forward's inputs
 *              (q_raw and k_raw are not read, and may be NULL, where that operand
 *              is not normed)
 *   workspace  as its size function says; NULL where no gradient of a weight is
 *              asked for
 *   dq_raw, dk_raw [rows, H, d] grad_dtype, row strides (outputs); may equal dq,
 *              dk exactly where they are dense too
 *   dq_weight, dk_weight [d] fp32 (outputs), or NULL; NULL where not normed
 */
gdn_status gdn_qk_norm_rope_backward(const gdn_qk_bwd_desc* desc, const void* dq, const void* dk,
                                     const void* q_raw, const void* k_raw,
                                     const float* q_weight, const float* k_weight,
                                     const int64_t* positions, const float* inv_freq,
                                     void* workspace, size_t workspace_bytes, void* dq_raw,
                                     void* dk_raw, float* dq_weight, float* dk_weight,
                                     void* stream);

/* The residual's addition and the norm behind it. */
typedef struct gdn_add_norm_desc {
  int64_t rows;       /* tokens, >= 0 (0: nothing to do)                         */
  int64_t ld_x;       /* row stride of x: C <= ld_x <= 2^24, % 8 == 0            */
  int32_t C;          /* channels: 8 .. 16384, % 8 == 0                          */
  int32_t io_dtype;   /* gdn_dtype of x, and of y where group < 0                */
  int32_t res_dtype;  /* gdn_dtype of res, res_out                               */
  int32_t group;      /* -1: y in io_dtype; 0: e4m3, one scale for a row; 32, 64
                         or 128: e4m3, a scale for so many channels (C % group == 0) */
  float eps;          /* finite, >= 0                                            */
} gdn_add_norm_desc;

/*
 * gdn_add_norm --
 *
 *   r = x + res                               (res NULL: r = x)
 *   y = r / sqrt(mean(r^2) + eps) * weight    (weight NULL: 1)
 *
 * with r in fp32 throughout: res_out is its rounding, y is formed from r itself.
 * The 8-bit output is for a projection in 8 bits:
 *
 *   y_scale = max(2^-100, max|y| over the scale's channels) / 448
 *   y       = code of OCP e4m3 of y / y_scale, rounded to nearest even
 *
 * (infinities do not count towards max|y| and are written as +-448, NaN as NaN).
 * |r| < 2^60; where eps is 0 the mean of a row's squares must be a normal number.
 *
 *   x          [rows, C] io_dtype, row stride ld_x
 *   res        [rows, C] res_dtype, dense, or NULL
 *   weight     [C] fp32, or NULL
 *   res_out    [rows, C] res_dtype, dense (output), or NULL; may equal res exactly,
 *              or x where that is dense and of res_dtype
 *   y          [rows, C] io_dtype or codes, dense (output); in io_dtype it may equal
 *              x exactly where that is dense
 *   y_scale    [rows, C / group] or [rows] fp32, 4-byte aligned (output; NULL where
 *              group < 0)
 */
gdn_status gdn_add_norm(const gdn_add_norm_desc* desc, const void* x, const void* res,
                        const float* weight, void* res_out, void* y, float* y_scale,
                        void* stream);

/* Its gradient. */
typedef struct gdn_add_norm_bwd_desc {
  int64_t rows;       /* tokens, >= 0                                            */
  int64_t ld_dx;      /* row stride of dx: C <= ld_dx <= 2^24, % 8 == 0          */
  int32_t C;          /* channels: 8 .. 16384, % 8 == 0                          */
  int32_t io_dtype;   /* gdn_dtype of dy, dx                                     */
  int32_t res_dtype;  /* gdn_dtype of r, d_res_out, d_res                        */
  float eps;          /* finite, >= 0                                            */
} gdn_add_norm_bwd_desc;

/* Bytes of device workspace gdn_add_norm_backward needs (0 for an invalid
 * descriptor or when there is no row). */
size_t gdn_add_norm_backward_workspace_size(const gdn_add_norm_bwd_desc* desc);

/*
 * gdn_add_norm_backward -- gradients of gdn_add_norm at the r that it left in
 * res_out (or at x, where it had no res), for upstream gradients dy of y and
 * d_res_out of r: with n = r / sqrt(mean(r^2) + eps),
 *
 *   d_r = d_res_out + (dy weight - n mean(n dy weight)) / sqrt(mean(r^2) + eps)
 *   d_weight = sum over rows of dy n
 *
 * d_r is the gradient of x and of res alike; it is written in either type.
 * |r|, |dy| and |dy weight| < 2^60, and where eps is 0 as gdn_add_norm.
 *
 *   dy         [rows, C] io_dtype, dense
 *   r          [rows, C] res_dtype, dense
 *   weight     [C] fp32, or NULL (1)
 *   d_res_out  [rows, C] res_dtype, dense, or NULL (0)
 *   workspace  as its size function says; NULL where d_weight is
 *   dx         [rows, C] io_dtype, row stride ld_dx (output), or NULL; may equal dy
 *              exactly where it is dense
 *   d_res      [rows, C] res_dtype, dense (output), or NULL; may equal d_res_out
 *              exactly
 *   d_weight   [C] fp32 (output), or NULL
 */
gdn_status gdn_add_norm_backward(const gdn_add_norm_bwd_desc* desc, const void* dy, const void* r,
                                 const float* weight, const void* d_res_out, void* workspace,
                                 size_t workspace_bytes, void* dx, void* d_res, float* d_weight,
                                 void* stream);

/* Returns GDN_HYBRID_ABI_VERSION of the loaded library. */
int gdn_hybrid_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_HYBRID_H */
