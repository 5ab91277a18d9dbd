/*
 * gdn_attn.h -- C ABI of libgdn.so for the softmax-attention layers of a
 * hybrid model on AMD Instinct MI355X (gfx950): the layers that stand between
 * the gated delta-rule layers of gdn.h ("Gated DeltaNet", §Architecture et
 * versions hybrides: hybrids that alternate the delta rule with sliding-window
 * attention; the architecture notes' hybrid has full attention layers).  The
 * pages name those layers and leave their arithmetic to the literature; what
 * is computed here is stated with each entry point.
 *
 * A prompt goes through gdn_qk_norm_rope and gdn_attn_prefill, and its keys
 * and values into a paged cache of 8-bit floats with gdn_kv_append; a decode
 * step is gdn_qk_norm_rope (queries only), gdn_kv_append with one token for
 * each sequence, and gdn_attn_decode over the cache.
 *
 * The conventions of gdn.h hold (memory, asynchrony, errors, status codes,
 * nothing allocated, no mutable state), with these additions:
 *  - Row strides: an input of shape [rows, H, d] has its H d elements of a row
 *    together and `ld` elements from one row to the next, so it may be a
 *    column block of a projection output.  ld % 8 == 0, H d <= ld <= 2^24.
 *    Pointers are 16-byte aligned unless stated otherwise.
 *  - Query head h reads key/value head h / (H_q / H_k).
 *  - Paged cache: k_cache, v_cache [num_pages, H_k, page_size, d] are codes of
 *    OCP e4m3 (largest 448), k_scale, v_scale [num_pages, H_k] fp32 powers of
 *    two; an element stands for code * scale.  page_table [N, max_pages] int32
 *    maps token t of sequence n to row t % page_size of page
 *    page_table[n][t / page_size].  An entry outside [0, num_pages) is no page:
 *    nothing is written there, and its tokens are not attended to.  seq_lens
 *    [N] int64 is clamped into [0, max_pages * page_size] on the device.  So
 *    neither a bad table nor a bad length makes a kernel touch memory outside
 *    the arguments.
 *  - Non-finite inputs: a token's non-finite q spoils its own output, its k and
 *    v the outputs of the queries that see it, and nothing else.  The weights
 *    of a sum are below 2^9 before it is divided by theirs, so values are
 *    summed without overflow while 2^9 sum |v| over the seen tokens (in a cache,
 *    and 2^9 times its pages' scales) is finite in fp32.
 *  - Scores are formed in fp32 as (q . k) (scale log2 e) and may be of any size
 *    there: both factors and the score below 2^127.  (gdn_attn_prefill in bf16
 *    computes rows whose scores reach 2^24 one after another, which is slow.)
 */
#ifndef GDN_ATTN_H
#define GDN_ATTN_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_ATTN_ABI_VERSION 1

typedef enum gdn_rope_mode {
  GDN_ROPE_HALF = 0,        /* channel i turns with channel i + rope_dim / 2  */
  GDN_ROPE_INTERLEAVED = 1  /* channel 2 i turns with channel 2 i + 1         */
} gdn_rope_mode;

/* Norm and rotation of query and key rows. */
typedef struct gdn_qk_desc {
  int64_t rows;       /* tokens, >= 0 (0: nothing to do)                         */
  int64_t ld_q, ld_k; /* row strides of q_raw and k_raw (elements)               */
  int32_t H_q, H_k;   /* >= 0, not both 0 (0: that operand is absent)            */
  int32_t d;          /* 64 or 128                                               */
  int32_t rope_dim;   /* channels rotated: 0 (none) .. d, % 16 == 0              */
  int32_t rope_mode;  /* gdn_rope_mode                                           */
  int32_t io_dtype;   /* gdn_dtype of q_raw, k_raw, q, k                         */
  float rope_scale;   /* factor on cos and sin (long-context scaling), finite    */
  float eps;          /* finite, >= 0                                            */
} gdn_qk_desc;

/*
 * gdn_qk_norm_rope -- RMS norm of each query and key head, then the rotary
 * position, in one pass:
 *
 *   y = x / sqrt(mean(x^2) + eps) * weight            (weight NULL: y = x)
 *   (a, b) -> (f (a cos t - b sin t), f (b cos t + a sin t)),
 *       t = positions[r] * inv_freq[i],  f = rope_scale,  i < rope_dim / 2
 *
 * for the channel pairs (a, b) of rope_mode; channels from rope_dim on are
 * not rotated.  The angle is formed and reduced to 2^-25 of a turn at every
 * position up to +-2^53 and frequency up to 2^24, so far ones lose nothing;
 * frequencies scaled for long contexts come in through inv_freq and rope_scale.
 * The rest is fp32, rounded once at the end: x^2 is formed in it, so |x| < 2^60,
 * and eps plus the mean of a row's squares must be a normal number (2^-126 or
 * more: a row of zeros needs such an eps).
 *
 *   q_raw     [rows, H_q, d] io_dtype, row stride ld_q (NULL when H_q == 0)
 *   k_raw     [rows, H_k, d] io_dtype, row stride ld_k (NULL when H_k == 0)
 *   q_weight, k_weight [d] fp32, or NULL: that operand is not normed
 *   positions [rows] int64, 8-byte aligned (NULL when rope_dim == 0)
 *   inv_freq  [rope_dim / 2] fp32 (NULL when rope_dim == 0)
 *   q, k      [rows, H, d] io_dtype, dense (outputs); may equal q_raw, k_raw
 *             exactly where that is dense too
 */
gdn_status gdn_qk_norm_rope(const gdn_qk_desc* desc, const void* q_raw, const void* k_raw,
                            const float* q_weight, const float* k_weight,
                            const int64_t* positions, const float* inv_freq, void* q, void* k,
                            void* stream);

/* New tokens of a paged cache. */
typedef struct gdn_kv_append_desc {
  int64_t N;          /* sequences, >= 0 (0: nothing to do)                      */
  int64_t total_T;    /* new tokens of all sequences, >= 0                       */
  int64_t ld_k, ld_v; /* row strides of k_raw and v_raw (elements)               */
  int64_t num_pages;  /* pages of the cache, >= 1, < 2^31                        */
  int64_t max_pages;  /* columns of page_table, >= 1                             */
  int32_t H_k;        /* >= 1                                                    */
  int32_t d;          /* 64 or 128                                               */
  int32_t page_size;  /* tokens of a page: 16, 32, 64 or 128                     */
  int32_t rope_dim;   /* as in gdn_qk_desc                                       */
  int32_t rope_mode;  /* gdn_rope_mode                                           */
  int32_t io_dtype;   /* gdn_dtype of k_raw, v_raw                               */
  float rope_scale;   /* finite                                                  */
  float eps;          /* finite, >= 0                                            */
} gdn_kv_append_desc;

/*
 * gdn_kv_append -- writes each sequence's new keys and values into its pages
 * at positions seq_lens[n], seq_lens[n] + 1, ...: keys normed and rotated for
 * their position as gdn_qk_norm_rope does (from fp32, not rounded to io_dtype
 * in between), values as they come.  For every page and head that gets new
 * tokens
 *
 *   scale = max(the least 2^e >= max|x| / 448 over the new tokens, e >= -100;
 *               the page's old scale, where it holds older tokens of the
 *               sequence)
 *   code  = x / scale rounded to nearest even
 *
 * and where the scale grows, the older tokens' codes are rounded again at the
 * new one (a shift of the exponent: exact but for codes that become
 * subnormal).  A page whose first row is new is taken as empty, whatever it
 * held.  Infinities do not count towards max|x| and are written as +-448, NaN
 * as NaN.  Rows of a page behind the last token keep their bytes.  seq_lens is
 * not changed; tokens that would lie behind the page table are dropped.  A page
 * written by the call must stand once in the table (else its contents are
 * unspecified).
 *
 *   cu_seqlens [N + 1] int64 offsets of the new tokens (clamped on the device
 *              as in gdn_chunk_fwd_varlen), or NULL for total_T / N tokens
 *              each (total_T % N == 0)
 *   seq_lens   [N] int64: tokens held before the call, 8-byte aligned
 *   page_table [N, max_pages] int32, 4-byte aligned
 *   k_raw, v_raw [total_T, H_k, d] io_dtype, row strides ld_k, ld_v
 *   k_weight   [d] fp32 or NULL (keys not normed)
 *   inv_freq   [rope_dim / 2] fp32 (NULL when rope_dim == 0)
 *   k_cache, v_cache, k_scale, v_scale   the cache (read and written)
 */
gdn_status gdn_kv_append(const gdn_kv_append_desc* desc, const int64_t* cu_seqlens,
                         const int64_t* seq_lens, const int32_t* page_table, const void* k_raw,
                         const void* v_raw, const float* k_weight, const float* inv_freq,
                         void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                         void* stream);

/* Causal attention over whole prompts. */
typedef struct gdn_attn_prefill_desc {
  int64_t N;          /* sequences, >= 0 (0: nothing to do)                      */
  int64_t total_T;    /* packed tokens, >= 0, < 2^31                             */
  int64_t ld_q, ld_k, ld_v; /* row strides (elements)                            */
  int64_t window;     /* >= 0: a token sees itself and the window - 1 before it; 0: all */
  int32_t H_q, H_k;   /* >= 1, H_q % H_k == 0                                    */
  int32_t d;          /* 64 or 128                                               */
  int32_t io_dtype;   /* gdn_dtype of q, k, v, o                                 */
  float scale;        /* finite, not 0; usually 1 / sqrt(d)                      */
} gdn_attn_prefill_desc;

/*
 * gdn_attn_prefill -- o_t = sum_s p_ts v_s with p_ts = softmax over s of
 * scale * q_t . k_s, s running over the tokens of t's own sequence up to t
 * (the last `window` of them).  Statistics and sums in fp32; with bf16 io the
 * weights are rounded to bf16 for the product with v (and summed before that).
 * Tokens that t does not see have no part in o_t, infinite and NaN keys and
 * values included.  (For that the rows near a value that is not finite, up to 200
 * on either side of what sees it, are computed one after another: 114 ms instead
 * of 4 where 32768 tokens hold one.)
 *
 *   cu_seqlens [N + 1] int64 offsets (clamped on the device as in
 *              gdn_chunk_fwd_varlen), or NULL for total_T / N tokens each
 *              (total_T % N == 0); rows of o that no range covers are kept
 *   q          [total_T, H_q, d], k, v [total_T, H_k, d] io_dtype, row strides
 *   o          [total_T, H_q, d] io_dtype, dense (output)
 */
gdn_status gdn_attn_prefill(const gdn_attn_prefill_desc* desc, const int64_t* cu_seqlens,
                            const void* q, const void* k, const void* v, void* o, void* stream);

/* Attention of one new token per sequence over the paged cache. */
typedef struct gdn_attn_decode_desc {
  int64_t N;          /* sequences, >= 0 (0: nothing to do)                      */
  int64_t num_pages;  /* pages of the cache, >= 1, < 2^31                        */
  int64_t max_pages;  /* columns of page_table, >= 1                             */
  int64_t window;     /* >= 0: the last `window` tokens are seen; 0: all         */
  int32_t H_q, H_k;   /* >= 1, H_q % H_k == 0                                    */
  int32_t d;          /* 64 or 128                                               */
  int32_t page_size;  /* 16, 32, 64 or 128                                       */
  int32_t io_dtype;   /* gdn_dtype of q, o                                       */
  float scale;        /* finite, not 0                                           */
} gdn_attn_decode_desc;

/*
 * gdn_attn_decode_workspace_size -- bytes of device workspace gdn_attn_decode
 * needs for this descriptor (0 where none is needed, and for an invalid
 * descriptor): the partial results of the splits of a long cache.
 */
size_t gdn_attn_decode_workspace_size(const gdn_attn_decode_desc* desc);

/*
 * gdn_attn_decode -- the attention of gdn_attn_prefill for the newest token of
 * each sequence over the seq_lens[n] tokens that its pages hold (the new one
 * among them).  A sequence that sees no token gives o = 0.  Statistics and sums
 * in fp32, codes exact; the weights times their page's v_scale are rounded to
 * bf16 with bf16 io (and summed before that), to 24 bits with fp32.
 *
 *   q          [N, H_q, d] io_dtype, dense
 *   k_cache, v_cache, k_scale, v_scale, page_table, seq_lens   the cache (read)
 *   o          [N, H_q, d] io_dtype (output)
 *   workspace  >= gdn_attn_decode_workspace_size(desc) bytes, 16-byte aligned
 *              (NULL when that is 0); needs no initial contents, and calls
 *              that may overlap in time need one each
 */
gdn_status gdn_attn_decode(const gdn_attn_decode_desc* desc, const void* q, const void* k_cache,
                           const void* v_cache, const float* k_scale, const float* v_scale,
                           const int32_t* page_table, const int64_t* seq_lens, void* o,
                           void* workspace, size_t workspace_bytes, void* stream);

/* Returns GDN_ATTN_ABI_VERSION of the loaded library. */
int gdn_attn_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_ATTN_H */
