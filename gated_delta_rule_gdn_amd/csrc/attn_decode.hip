// attn_decode.hip -- attention of one query token per sequence over a paged
// cache of e4m3 codes on gfx950:
//
//   o = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale * q . k_t - m),
//
// t over the tokens that the sequence's pages hold (the last `window` of
// them).  Every code is read once; a token's 2 d bytes take 4 d flops for
// each of the group's query heads, so the kernel is bound by HBM.
//
// A workgroup has one sequence, one key head, up to 16 query heads of its
// group and one span of tokens.  Its 4 waves take steps of 32 tokens in turn,
// each with a running maximum and sum of its own, and join through LDS at the
// end.  Products run on v_mfma_f32_16x16x32_bf16 with the queries as columns:
//
//   S^T [16 tokens x 16 queries] = K Q^T     twice, tokens 0-15 and 16-31
//   O^T [d x 16 queries]        += V^T P^T   over the 32 tokens
//
// e4m3 is exact in bf16, so K and V lose nothing.  Lane 16 g + j holds query
// j's scores of tokens 4 g .. 4 g + 3 of each tile, and these 8 weights are
// the very k-values that lane supplies to the second product: the weights
// never leave their lane.  V's 8 tokens x D/16 columns of a lane are
// transposed in registers by byte permutes.  A page's scales multiply the
// scores and the weights, not the elements.  fp32 queries and weights go
// through the same products as three bf16 terms each (24 bits).
#include "attn_device.hpp"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kStep = 32;                 // tokens of a wave's step
constexpr int kRound = kWaves * kStep;    // tokens of a workgroup's step
constexpr float kNone = -1e30f;           // running maximum (log2 units) before any token

// Two e4m3 codes (low or high half of a dword) as bf16.
template <bool HI>
__device__ __forceinline__ bf16x2 cvt2(uint32_t c) {
  return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.f, HI);
}
__device__ __forceinline__ bf16x8 cvt8(uint32_t lo, uint32_t hi) {
  const bf16x2 a = cvt2<false>(lo), b = cvt2<true>(lo), c = cvt2<false>(hi), d = cvt2<true>(hi);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// 4 x 4 bytes transposed: out[i] byte j = in[j] byte i.
__device__ __forceinline__ void transpose4(const uint32_t* in, uint32_t* out) {
  const uint32_t a = __builtin_amdgcn_perm(in[1], in[0], 0x05010400);  // 0.0 1.0 0.1 1.1
  const uint32_t b = __builtin_amdgcn_perm(in[1], in[0], 0x07030602);  // 0.2 1.2 0.3 1.3
  const uint32_t c = __builtin_amdgcn_perm(in[3], in[2], 0x05010400);
  const uint32_t d = __builtin_amdgcn_perm(in[3], in[2], 0x07030602);
  out[0] = __builtin_amdgcn_perm(c, a, 0x05040100);
  out[1] = __builtin_amdgcn_perm(c, a, 0x07060302);
  out[2] = __builtin_amdgcn_perm(d, b, 0x05040100);
  out[3] = __builtin_amdgcn_perm(d, b, 0x07060302);
}

// x as NT bf16 terms: one (rounded) for bf16 io, three that sum to x for fp32.
template <int NT>
__device__ __forceinline__ void split_terms(float x, bf16* t) {
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    t[i] = (bf16)x;
    x -= (float)t[i];
  }
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Codes of one step in this lane.
template <int D>
struct StepCodes {
  uint32_t k[2][D / 16];      // tile, D/4 bytes of token j of the tile
  uint32_t v[8][D / 64];      // token 4 g + i (tile i / 4), D/16 columns
  float ks[2], vs[2];         // the tiles' scales; ks < 0: no page
};

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_decode_kernel(AttnDecodeArgs p, int qgroups,
                                                               int splits, int64_t span) {
  constexpr int NT = std::is_same<T, float>::value ? 3 : 1;   // bf16 terms of q and of a weight
  constexpr int KB = D / 32;              // k-blocks of the score product
  constexpr int MT = D / 16;              // 16-column tiles of the output
  __shared__ float s_o[kWaves][16][D + 4];
  __shared__ float s_m[kWaves][16], s_l[kWaves][16];
  lds_nan_fill(s_o, sizeof s_o);
  lds_nan_fill(s_m, sizeof s_m);
  lds_nan_fill(s_l, sizeof s_l);

  const int G = p.Hq / p.Hk;
  const int split = blockIdx.x % splits;
  const int64_t rest = blockIdx.x / splits;
  const int qg = (int)(rest % qgroups);
  const int64_t nh = rest / qgroups;
  const int64_t n = nh / p.Hk;
  const int hk = (int)(nh - n * p.Hk);
  const int g0 = 16 * qg;                 // first query head of the group here
  const int gn = G - g0 < 16 ? G - g0 : 16;

  const PagedCache& kv = p.cache;
  const int P = kv.page_size;
  const DecodeSpan sp = decode_span(kv.seq_lens[n], kv.max_pages, P, p.window, split, span, kStep);
  const int64_t len = sp.len, lo = sp.lo, begin = sp.begin, end = sp.end;
  const bool only = sp.only;
  if (begin >= end && !(only && split == 0)) return;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, j = lane & 15;

  // queries: lane holds query j's channels [g D/4, +D/4), as B operands
  bf16x8 q[NT][KB];
  {
    const T* qp = static_cast<const T*>(p.q) +
                  ((n * p.Hq) + hk * G + g0 + (j < gn ? j : 0)) * (int64_t)D + g * (D / 4);
    const float flip = p.scale < 0.f ? -1.f : 1.f;            // the scale below is positive
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      float x[8];
      load_f32<8, T>(qp + 8 * kb, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        bf16 t[NT];
        split_terms<NT>(j < gn ? x[i] * flip : 0.f, t);
#pragma unroll
        for (int c = 0; c < NT; ++c) q[c][kb][i] = t[c];
      }
    }
  }
  const float c_scale = fabsf(p.scale) * kLog2e;

  f32x4 o[MT];
#pragma unroll
  for (int c = 0; c < MT; ++c) o[c] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = kNone, l = 0.f;

  const int32_t* __restrict__ table = kv.table + n * kv.max_pages;
  auto load_step = [&](int64_t t0, StepCodes<D>& s) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int64_t tok = t0 + 16 * t;
      const int64_t pi = tok / P;
      int64_t page = tok < len ? table[pi] : -1;
      const bool there = page >= 0 && page < kv.num_pages;
      if (!there) page = 0;
      const int64_t at = page * p.Hk + hk;
      const int64_t row = at * P + (tok - pi * P);            // first row of the tile
      s.ks[t] = there ? kv.k_scale[at] : -1.f;
      s.vs[t] = there ? kv.v_scale[at] : 0.f;
      const uint8_t* kp = kv.k + (row + j) * D + g * (D / 4);
      const uint8_t* vp = kv.v + (row + 4 * g) * D + j * (D / 16);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const uint4 u = reinterpret_cast<const uint4*>(kp)[i];
        s.k[t][4 * i] = u.x; s.k[t][4 * i + 1] = u.y;
        s.k[t][4 * i + 2] = u.z; s.k[t][4 * i + 3] = u.w;
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
          s.v[4 * t + r][i] = reinterpret_cast<const uint32_t*>(vp + r * D)[i];
    }
  };

  for (int64_t t0 = begin + wave * kStep; t0 < end; t0 += kRound) {
    StepCodes<D> s;
    load_step(t0, s);
    const bool edge = t0 < lo || t0 + kStep > len || s.ks[0] < 0.f || s.ks[1] < 0.f;

    // scores of query j: x[4 t + r] is token t0 + 16 t + 4 g + r, in log2 units
    float x[8];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const bf16x8 a = cvt8(s.k[t][2 * kb], s.k[t][2 * kb + 1]);
#pragma unroll
        for (int c = NT - 1; c >= 0; --c) acc = mfma(a, q[c][kb], acc);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) x[4 * t + r] = acc[r] * (s.ks[t] * c_scale);
    }
    if (edge) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t tok = t0 + 16 * (i / 4) + 4 * g + i % 4;
        const bool seen = tok >= lo && tok < len && s.ks[i / 4] >= 0.f;
        if (!seen) {
          x[i] = -__builtin_huge_valf();
#pragma unroll
          for (int c = 0; c < D / 64; ++c) s.v[i][c] = 0;     // a code behind the end may be NaN
        }
      }
    }
    float mx = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])),
                     fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float m_new = fmaxf(m, mx);
    const float alpha = exp2_fast(m - m_new);
    m = m_new;
    l *= alpha;
#pragma unroll
    for (int c = 0; c < MT; ++c)
#pragma unroll
      for (int r = 0; r < 4; ++r) o[c][r] *= alpha;

    bf16x8 w[NT];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float e = exp2_fast(x[i] - m);
      l += e;
      bf16 t[NT];
      split_terms<NT>(e * s.vs[i / 4], t);
#pragma unroll
      for (int c = 0; c < NT; ++c) w[c][i] = t[c];
    }
    // V^T: columns j D/16 + c of 8 tokens
#pragma unroll
    for (int cc = 0; cc < D / 64; ++cc) {
      uint32_t in0[4], in1[4], a[4], b[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) { in0[r] = s.v[r][cc]; in1[r] = s.v[4 + r][cc]; }
      transpose4(in0, a);
      transpose4(in1, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bf16x8 va = cvt8(a[i], b[i]);
#pragma unroll
        for (int c = NT - 1; c >= 0; --c) o[4 * cc + i] = mfma(va, w[c], o[4 * cc + i]);
      }
    }
  }

  // join the waves: o[c][r] is column (4 g + r) D/16 + c of query j
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < MT; c += 4) {
      float* dst = &s_o[wave][j][(4 * g + r) * MT + c];
      lds_check(dst, 16);
      *reinterpret_cast<float4*>(dst) = make_float4(o[c][r], o[c + 1][r], o[c + 2][r], o[c + 3][r]);
    }
  if (g == 0) { s_m[wave][j] = m; s_l[wave][j] = l; }
  __syncthreads();
  constexpr int LPQ = D / 4;              // threads of a query, 4 columns each
  for (int qi = tid / LPQ; qi < gn; qi += kThreads / LPQ) {
    const int col = 4 * (tid % LPQ);
    float mm = kNone, ll = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) mm = fmaxf(mm, s_m[w][qi]);
    float r[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float f = exp2_fast(s_m[w][qi] - mm);
      ll += f * s_l[w][qi];
      const float4 u = *reinterpret_cast<const float4*>(&s_o[w][qi][col]);
      r[0] += f * u.x; r[1] += f * u.y; r[2] += f * u.z; r[3] += f * u.w;
    }
    const int64_t row = n * p.Hq + hk * G + g0 + qi;
    if (only) {
      const float inv = ll > 0.f ? 1.f / ll : 0.f;            // no token seen: o = 0
      store4<T>(static_cast<T*>(p.o) + row * D + col, r[0] * inv, r[1] * inv, r[2] * inv, r[3] * inv);
    } else {
      float* part = p.ws + (row * splits + split) * (D + 4);
      *reinterpret_cast<float4*>(part + col) = make_float4(r[0], r[1], r[2], r[3]);
      if (col == 0) { part[D] = mm; part[D + 1] = ll; }
    }
  }
}

// Joins the partial results of a sequence's splits: one workgroup for each
// query row, its threads over (split mod groups, 4 columns).
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(AttnDecodeArgs p, int splits,
                                                             int64_t span) {
  constexpr int LPQ = D / 4, GR = kThreads / LPQ;
  __shared__ float s_o[GR][D];
  __shared__ float s_l[GR], s_m[GR];
  const int64_t row = blockIdx.x;
  const int64_t n = row / p.Hq;
  const PagedCache& kv = p.cache;
  const DecodeSpan sp =
      decode_span(kv.seq_lens[n], kv.max_pages, kv.page_size, p.window, 0, span, kStep);
  if (sp.only) return;                    // written whole by its one split
  const int ns = (int)((sp.len - sp.begin + span - 1) / span);
  const int gr = threadIdx.x / LPQ, col = 4 * (threadIdx.x % LPQ);
  const float* part = p.ws + row * splits * (D + 4);
  float mm = kNone, ll = 0.f, r[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = gr; s < ns; s += GR) {
    const float ms = part[s * (D + 4) + D], ls = part[s * (D + 4) + D + 1];
    const float4 u = *reinterpret_cast<const float4*>(part + s * (D + 4) + col);
    const float m2 = fmaxf(mm, ms);
    const float f0 = exp2_fast(mm - m2), f1 = exp2_fast(ms - m2);
    mm = m2;
    ll = ll * f0 + ls * f1;
    r[0] = r[0] * f0 + u.x * f1; r[1] = r[1] * f0 + u.y * f1;
    r[2] = r[2] * f0 + u.z * f1; r[3] = r[3] * f0 + u.w * f1;
  }
  *reinterpret_cast<float4*>(&s_o[gr][col]) = make_float4(r[0], r[1], r[2], r[3]);
  if (col == 0) { s_m[gr] = mm; s_l[gr] = ll; }
  __syncthreads();
  if (gr != 0) return;
  for (int w = 0; w < GR; ++w) mm = fmaxf(mm, s_m[w]);
  ll = 0.f;
  r[0] = r[1] = r[2] = r[3] = 0.f;
  for (int w = 0; w < GR; ++w) {
    const float f = exp2_fast(s_m[w] - mm);
    ll += f * s_l[w];
    const float4 u = *reinterpret_cast<const float4*>(&s_o[w][col]);
    r[0] += f * u.x; r[1] += f * u.y; r[2] += f * u.z; r[3] += f * u.w;
  }
  const float inv = ll > 0.f ? 1.f / ll : 0.f;
  store4<T>(static_cast<T*>(p.o) + row * D + col, r[0] * inv, r[1] * inv, r[2] * inv, r[3] * inv);
}

template <typename T, int D>
hipError_t launch_t(const AttnDecodeArgs& a, hipStream_t stream) {
  const AttnDecodeSplit sp = attn_decode_split(a.N, a.cache.max_pages * a.cache.page_size, a.window,
                                               a.Hq, a.Hk, D);
  const int qgroups = (a.Hq / a.Hk + 15) / 16;
  const int64_t blocks = a.N * a.Hk * qgroups * sp.splits;
  attn_decode_kernel<T, D><<<dim3((unsigned)blocks), kThreads, 0, stream>>>(
      a, qgroups, (int)sp.splits, sp.span);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || sp.splits == 1) return e;
  attn_join_kernel<T, D><<<dim3((unsigned)(a.N * a.Hq)), kThreads, 0, stream>>>(
      a, (int)sp.splits, sp.span);
  return hipGetLastError();
}

}  // namespace

// The tokens that a sequence can hold are known on the host (the width of the
// page table), its length is not.  Spans are as long as leaves kTarget
// workgroups if all sequences are full, and at least kLeast tokens: a span's
// partial result costs 2 (D + 4) 4 bytes for each query head against
// 2 D bytes for each token.
AttnDecodeSplit attn_decode_split(int64_t N, int64_t max_tokens, int64_t window, int Hq, int Hk,
                                  int d) {
  constexpr int64_t kTarget = 2048, kLeast = 512;
  if (window > 0 && window + kStep < max_tokens) max_tokens = window + kStep;
  const int64_t groups = N * Hk * ((Hq / Hk + 15) / 16);
  int64_t want = groups > 0 ? kTarget / groups : 1;
  if (want < 1) want = 1;
  int64_t span = (max_tokens + want - 1) / want;
  if (span < kLeast) span = kLeast;
  span = (span + kRound - 1) / kRound * kRound;
  AttnDecodeSplit s;
  s.splits = (max_tokens + span - 1) / span;
  s.span = span;
  s.ws_floats = s.splits > 1 ? N * Hq * s.splits * (d + 4) : 0;
  return s;
}

hipError_t launch_attn_decode(const AttnDecodeArgs& a, hipStream_t stream) {
  if (a.io == DType::F32)
    return a.d == 128 ? launch_t<float, 128>(a, stream) : launch_t<float, 64>(a, stream);
  return a.d == 128 ? launch_t<bf16, 128>(a, stream) : launch_t<bf16, 64>(a, stream);
}

#ifdef GDN_CHECK
unsigned check_violations_attn_decode() { return take_check_violations(); }
#endif

}  // namespace gdn
