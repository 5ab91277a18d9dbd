// attn_decode.hip -- attention of one query token per sequence over a paged
// cache of e4m3 codes on gfx950:
//
//   o = sum_t p_t v_t / sum_t p_t,   p_t = exp(scale * q . k_t - m),
//
// t over the tokens that the sequence's pages hold (the last `window` of
// them).  Every code is read once; a token's 2 d bytes take 4 d flops for
// each of the group's query heads, so the kernel is bound by HBM (256 caches,
// 730 MB, in 148 to 161 us with the join, by the card: 4.5 to 4.9 TB/s; one of 128K
// tokens, 134 MB, in 26 us, 35.5 with the join and its launch).
//
// The work is cut into rounds of 128 tokens of one segment: a sequence, a key
// head and up to 16 query heads of its group.  The rounds of all segments, in
// order, are dealt to the workgroups in equal shares (to within one: 14 caches,
// 110000 tokens, 64 heads over 4: 39.4 us; in equal shares but the last 44.1),
// so lengths need not be alike and one long cache fills the chip; a share begins
// and ends anywhere.
// What a workgroup has of a segment is written straight to the output if that
// is all of it, else as a partial result, and a second kernel joins those.
// (Where no cache can be longer than kDecodeDirect tokens each workgroup has one
// whole segment, and nothing is joined: a round costs a workgroup 1.2 us (fp32
// 1.6), the second kernel about 5.  32 heads over 4, bf16 / fp32: 64 sequences of
// 768 tokens 15.4 / 18.0 us so, joined 18.9 / 20.6; 2 sequences of 768 tokens 11.6 /
// 14.7, joined 10.8 / 11.8; of 1024 tokens, 64 sequences 18.9 / 22.3, joined 21.4 /
// 23.3, 2 sequences 15.1 / 18.7, joined 11.0 / 11.9.)
//
// The 4 waves of a workgroup take 32 tokens of a round each, with a running
// maximum and sum of their own, and join through LDS when the segment ends.
// Products run on v_mfma_f32_16x16x32_bf16 with the queries as columns:
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
// through the same products as three bf16 terms each (24 bits).  With bf16 io a
// weight times its page's scale is rounded to bf16, as a prompt's weights are: half
// a step, 2^-8 of each, against the 2^-8 that the output is rounded by (error
// against 64 bits 1.8e-3 for 256 caches, 1.5e-3 with fp32 weights throughout), and a
// third of the products.
#include "attn_device.hpp"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kStep = kDecodeStep;
constexpr int kRound = kDecodeRound;
constexpr int64_t kBlocks = kDecodeBlocks;
static_assert(kRound == kWaves * kStep, "a step for each wave");

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

// Codes of one step in this lane, and the tiles' scales.
template <int D>
struct StepCodes {
  uint32_t k[2][D / 16];      // tile, bytes [16 g, +16) of each 64 of token j
  uint32_t v[8][D / 64];      // token 4 g + i (tile i / 4), D/16 columns
  float ks[2], vs[2];
  bool there[2];
};

// A segment's round: tokens [token, token + 128) of those in [lo, len).
struct Round {
  int n, hk, qg;      // the segment
  int r, rounds;      // number within the segment, and how many it has
  int64_t token, lo, len;
};

// Partial results in the workspace: two for each workgroup, of gn <= 16 rows of
// D + 4 floats (sums, maximum, sum of weights): [0] of a segment that began in
// an earlier workgroup, [1] of one that goes on in the next.  Then for each
// workgroup the segment of [1] (-1: none) and the last workgroup that has a
// part of it.
template <int D>
__device__ __forceinline__ float* part_at(float* ws, int rows, int64_t block, int which, int row) {
  return ws + ((block * 2 + which) * rows + row) * (D + 4);
}
__device__ __forceinline__ int2* chain_at(float* ws, int rows, int D, int64_t blocks, int64_t block) {
  return reinterpret_cast<int2*>(ws + blocks * 2 * rows * (D + 4)) + block;
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads, 2) void attn_decode_kernel(AttnDecodeArgs p, int qgroups,
                                                                  bool direct) {
  constexpr int NT = std::is_same<T, float>::value ? 3 : 1;   // bf16 terms of q and of a weight
  constexpr int KB = D / 32;              // k-blocks of the score product
  constexpr int MT = D / 16;              // 16-column tiles of the output
  __shared__ float s_o[kWaves][16][D + 4];
  __shared__ float s_m[kWaves][16], s_l[kWaves][16];
  lds_nan_fill(s_o, sizeof s_o);
  lds_nan_fill(s_m, sizeof s_m);
  lds_nan_fill(s_l, sizeof s_l);

  const int G = p.Hq / p.Hk;
  const int prows = G < 16 ? G : 16;      // rows of a partial result
  const PagedCache& kv = p.cache;
  const int P = kv.page_size;
  const int N = (int)p.N;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, j = lane & 15;
  const uint32_t per_seq = (uint32_t)(p.Hk * qgroups);

  // this workgroup's share, and the segment it begins in
  auto rounds_of = [&](int64_t seq_len) {
    return decode_rounds(seq_len, kv.max_pages, P, p.window, kRound, kStep);
  };
  auto begin_round = [&](int n, uint32_t seg_in_seq, int r, int64_t seq_len) {
    const DecodeSpan sp = decode_span(seq_len, kv.max_pages, P, p.window, kStep);
    Round u;
    u.n = n;
    u.hk = (int)(seg_in_seq / (uint32_t)qgroups);
    u.qg = (int)(seg_in_seq - (uint32_t)u.hk * qgroups);
    u.rounds = sp.rounds(kRound);
    u.r = r;
    u.lo = sp.lo;
    u.len = sp.len;
    u.token = sp.first + (int64_t)r * kRound;
    return u;
  };
  Round cur;
  int count;                              // rounds of this workgroup
  int total = 0, at = 0;                  // rounds of all; first round here
  if (direct) {
    const int n = (int)(blockIdx.x / per_seq);
    cur = begin_round(n, blockIdx.x - (uint32_t)n * per_seq, 0, kv.seq_lens[n]);
    count = cur.rounds;
  } else {
    // the lengths of 64 sequences, a lane each; of the first 64 read once
    const int64_t first_lens = lane < N ? kv.seq_lens[lane] : 0;
    auto lens_from = [&](int n0) {
      return n0 == 0 ? first_lens : n0 + lane < N ? kv.seq_lens[n0 + lane] : 0;
    };
    for (int n0 = 0; n0 < N; n0 += 64) total += n0 + lane < N ? rounds_of(lens_from(n0)) : 0;
    total = wave_sum(total) * (int)per_seq;
    const DecodeShare share = decode_share(total, (int)gridDim.x, (int)blockIdx.x);
    at = share.at;
    count = share.count;
    if (count <= 0) {
      if (tid == 0) *chain_at(p.ws, prows, D, gridDim.x, blockIdx.x) = make_int2(-1, 0);
      return;
    }
    int before = 0;                       // rounds of the sequences before n
    for (int n0 = 0;; n0 += 64) {
      const int64_t lens = lens_from(n0);
      const int mine = (n0 + lane < N ? rounds_of(lens) : 0) * (int)per_seq;
      const int all = wave_sum(mine);
      if (before + all <= at && n0 + 64 < N) { before += all; continue; }
      int upto = mine;                    // inclusive scan over the lanes
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int v = __shfl_up(upto, off);
        if (lane >= off) upto += v;
      }
      const uint64_t past = __ballot(before + upto > at);   // some lane: at < total
      const int i = past ? __ffsll((unsigned long long)past) - 1 : 0;
      const int n = n0 + i;
      before += __builtin_amdgcn_readlane(upto, i) - __builtin_amdgcn_readlane(mine, i);
      const int64_t seq_len = read_lane(lens, i);
      const int rn = rounds_of(seq_len);
      int seg = (at - before) / rn;
      if (seg > (int)per_seq - 1) seg = (int)per_seq - 1;   // (lengths that change meanwhile)
      cur = begin_round(n, (uint32_t)seg, at - before - seg * rn, seq_len);
      break;
    }
  }
  auto advance = [&](const Round& u) {
    Round v = u;
    v.r++;
    v.token += kRound;
    if (v.r < v.rounds) return v;
    uint32_t seg = (uint32_t)(u.hk * qgroups + u.qg) + 1;
    int n = u.n;
    if (seg == per_seq) { seg = 0; n = n + 1 < N ? n + 1 : n; }
    return begin_round(n, seg, 0, kv.seq_lens[n]);
  };

  // queries: lane holds query j's channels [16 g, +16) of each 64, as B operands
  bf16x8 q[NT][KB];
  Chunk8<T> raw[KB];
  auto ask_queries = [&](const Round& u) {
    const int gn = G - 16 * u.qg < 16 ? G - 16 * u.qg : 16;
    const T* qp = static_cast<const T*>(p.q) +
                  ((int64_t)u.n * p.Hq + u.hk * G + 16 * u.qg + (j < gn ? j : 0)) * (int64_t)D +
                  16 * g;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) raw[kb].load(qp + 64 * (kb / 2) + 8 * (kb % 2));
  };
  auto take_queries = [&](const Round& u) {
    const int gn = G - 16 * u.qg < 16 ? G - 16 * u.qg : 16;
    const float flip = p.scale < 0.f ? -1.f : 1.f;            // the scale below is positive
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      float x[8];
      raw[kb].unpack(x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        bf16 t[NT];
        split_terms<NT>(j < gn ? x[i] * flip : 0.f, t);
#pragma unroll
        for (int c = 0; c < NT; ++c) q[c][kb][i] = t[c];
      }
    }
  };
  const float c_scale = fabsf(p.scale) * kLog2e;

  f32x4 o[MT];
  float m, l;
  auto reset = [&]() {
#pragma unroll
    for (int c = 0; c < MT; ++c) o[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    m = kNone;
    l = 0.f;
  };

  // The loop runs two loads ahead: the table entries of round i + 2 and the
  // codes of round i + 1 are on their way while round i is computed.
  const int shift = __builtin_ctz(P);     // P is a power of two
  const float* __restrict__ kscale = kv.k_scale;
  const float* __restrict__ vscale = kv.v_scale;
  const uint32_t k_lane = (uint32_t)(j * D + 16 * g);
  const uint32_t v_lane = (uint32_t)(4 * g * D + j * (D / 16));
  auto entries = [&](const Round& u, int* e) {
    const int32_t* __restrict__ table = kv.table + u.n * kv.max_pages;
    const int64_t t0 = u.token + wave * kStep;
#pragma unroll
    for (int t = 0; t < 2; ++t) e[t] = t0 + 16 * t < u.len ? table[(t0 + 16 * t) >> shift] : -1;
  };
  auto load_step = [&](const Round& u, const int* e, StepCodes<D>& s) {
    const int64_t t0 = u.token + wave * kStep;
    if (t0 >= u.len) return;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int page = __builtin_amdgcn_readfirstlane(e[t]);
      s.there[t] = page >= 0 && page < kv.num_pages;
      const int64_t at = s.there[t] ? (int64_t)page * p.Hk + u.hk : u.hk;   // else any page
      const int64_t row = (at << shift) + ((t0 + 16 * t) & (P - 1));
      s.ks[t] = kscale[at];
      s.vs[t] = s.there[t] ? vscale[at] : 0.f;   // (0 weight times a stray NaN)
      const uint8_t* kp = kv.k + row * D;
      const uint8_t* vp = kv.v + row * D;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const uint4 w = *reinterpret_cast<const uint4*>(kp + k_lane + 64 * i);
        s.k[t][4 * i] = w.x; s.k[t][4 * i + 1] = w.y;
        s.k[t][4 * i + 2] = w.z; s.k[t][4 * i + 3] = w.w;
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int i = 0; i < D / 64; ++i)
          s.v[4 * t + r][i] = reinterpret_cast<const uint32_t*>(vp + v_lane + r * D)[i];
    }
  };

  auto compute = [&](const Round& u, StepCodes<D>& s) {
    const int64_t t0 = u.token + wave * kStep, lo = u.lo, len = u.len;
    if (t0 >= len) return;                  // (the wave has no token of this round)
    const bool edge = t0 < lo || t0 + kStep > len || !s.there[0] || !s.there[1];

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
      // a first tile wholly before the window may be a page of its own, whose scale may be no
      // number: 0 times it is not 0 (a second tile never is: steps begin at multiples of 32)
      if (t0 + 16 <= lo) s.vs[0] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t tok = t0 + 16 * (i / 4) + 4 * g + i % 4;
        const bool seen = tok >= lo && tok < len && s.there[i / 4];
        if (!seen) {
          x[i] = -__builtin_huge_valf();
#pragma unroll
          for (int c = 0; c < D / 64; ++c) s.v[i][c] = 0;     // a code behind the end may be NaN
        }
      }
    }
    float mx = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])),
                     fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
    mx = over_halves(over_rows(mx));
    // The sums are kept relative to m, which need not be the maximum: it is
    // moved only when a score passes it by 2^8.
    if (__any(mx > m + 8.f)) {
      const float m_new = fmaxf(m, mx);
      const float alpha = exp2_fast(m - m_new);
      m = m_new;
      l *= alpha;
#pragma unroll
      for (int c = 0; c < MT; ++c)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[c][r] *= alpha;
    }

    bf16x8 w[NT];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float e = weight_of(x[i], m);
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
  };

  // Joins the waves and writes this workgroup's part of a segment that `u` ends
  // here.  o[c][r] is column (4 g + r) D/16 + c of query j.
  auto flush = [&](const Round& u, bool from_start) {
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    __syncthreads();                        // the last flush has been read
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < MT; c += 4) {
        float* dst = &s_o[wave][j][(4 * g + r) * MT + c];
        lds_check(dst, 16);
        *reinterpret_cast<float4*>(dst) =
            make_float4(o[c][r], o[c + 1][r], o[c + 2][r], o[c + 3][r]);
      }
    if (g == 0) { s_m[wave][j] = m; s_l[wave][j] = l; }
    __syncthreads();
    const bool to_end = u.r == u.rounds - 1;
    const int gn = G - 16 * u.qg < 16 ? G - 16 * u.qg : 16;
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
        const float4 x = *reinterpret_cast<const float4*>(&s_o[w][qi][col]);
        r[0] += f * x.x; r[1] += f * x.y; r[2] += f * x.z; r[3] += f * x.w;
      }
      if (from_start && to_end) {
        const int64_t row = (int64_t)u.n * p.Hq + u.hk * G + 16 * u.qg + qi;
        const float inv = ll > 0.f ? 1.f / ll : 0.f;          // no token seen: o = 0
        store4<T>(static_cast<T*>(p.o) + row * D + col, r[0] * inv, r[1] * inv, r[2] * inv,
                  r[3] * inv);
      } else {
        float* part = part_at<D>(p.ws, prows, blockIdx.x, from_start ? 1 : 0, qi);
        *reinterpret_cast<float4*>(part + col) = make_float4(r[0], r[1], r[2], r[3]);
        if (col == 0) { part[D] = mm; part[D + 1] = ll; }
      }
    }
  };

  int e[2];
  StepCodes<D> sa, sb;
  entries(cur, e);
  ask_queries(cur);
  take_queries(cur);
  reset();
  load_step(cur, e, sa);
  Round next = cur;
  if (count > 1) { next = advance(cur); entries(next, e); }
  bool from_start = cur.r == 0;
  bool chained = false;                     // the last segment goes on in the next workgroup
  auto step = [&](int i, StepCodes<D>& s, StepCodes<D>& sn) {
    Round after = next;
    if (i + 1 < count) {
      load_step(next, e, sn);
      if (i + 2 < count) { after = advance(next); entries(after, e); }
    }
    compute(cur, s);
    const bool ends = cur.r == cur.rounds - 1;
    if (ends || i + 1 == count) {
      if (i + 1 < count) ask_queries(next);   // on their way during the flush
      flush(cur, from_start);
      chained = !ends && from_start;
      if (i + 1 < count) {
        take_queries(next);
        reset();
        from_start = true;
      }
    }
    if (i + 1 < count) cur = next;
    next = after;
  };
  for (int i = 0; i < count; i += 2) {
    step(i, sa, sb);
    if (i + 1 < count) step(i + 1, sb, sa);
  }
  if (!direct && tid == 0) {
    const int last = at + count - 1 + (cur.rounds - 1 - cur.r);   // the segment's, of all rounds
    const int seg = cur.n * (int)per_seq + cur.hk * qgroups + cur.qg;
    *chain_at(p.ws, prows, D, gridDim.x, blockIdx.x) =
        chained ? make_int2(seg, decode_owner(total, (int)gridDim.x, last)) : make_int2(-1, 0);
  }
}

// Joins the parts of the segments that lie in several workgroups.  Every
// workgroup reads which of the first kernel's begin such a segment, and they
// share the work.  Few segments (of many parts): a workgroup takes 32 columns
// of one query, 8 lanes for each of 32 parts at a time.  More of those than
// workgroups (segments of few parts): a wave takes a query, D/4 lanes for each
// part.  (56 segments of 16 queries, with the first kernel: 41 us so, 44 by
// columns; 32 of 8 queries, by columns 15.0, by queries 16.4.)  Bound by latency: the launch,
// the chains, the parts.  (128K tokens of one sequence, 4 segments of 128
// parts: 10.9 us with a workgroup to a query, 6.3 us so, 5.2 us with the 32
// sums joined across lanes first.)
constexpr int kJoinBlocks = 1024;

template <int D>
struct JoinSum {
  float m = kNone, l = 0.f, r[4] = {0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ void add(float m1, float l1, float4 u) {
    const float m2 = fmaxf(m, m1);
    const float f0 = exp2_fast(m - m2), f1 = exp2_fast(m1 - m2);
    m = m2;
    l = l * f0 + l1 * f1;
    r[0] = r[0] * f0 + u.x * f1; r[1] = r[1] * f0 + u.y * f1;
    r[2] = r[2] * f0 + u.z * f1; r[3] = r[3] * f0 + u.w * f1;
  }
  // parts first, first + by, ... of the chain that begins in `block`
  __device__ __forceinline__ void gather(float* ws, int rows, int block, int parts, int qi, int col,
                                         int first, int by) {
#pragma unroll 4
    for (int i = first; i < parts; i += by) {
      const float* part = part_at<D>(ws, rows, block + i, i == 0 ? 1 : 0, qi);
      add(part[D], part[D + 1], *reinterpret_cast<const float4*>(part + col));
    }
  }
  // over the lanes of the wave that hold the same columns: `apart` lanes apart
  __device__ __forceinline__ void over_lanes(int apart) {
#pragma unroll
    for (int off = 32; off >= apart; off >>= 1) {
      const float4 u = make_float4(__shfl_xor(r[0], off), __shfl_xor(r[1], off),
                                   __shfl_xor(r[2], off), __shfl_xor(r[3], off));
      const float m1 = __shfl_xor(m, off), l1 = __shfl_xor(l, off);
      add(m1, l1, u);
    }
  }
};

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_join_kernel(AttnDecodeArgs p, int qgroups,
                                                             int rows, int blocks) {
  __shared__ int s_start[kBlocks], s_end[kBlocks], s_seg[kBlocks], s_count[kBlocks / 64];
  __shared__ __align__(16) float s_o[kWaves][32];
  __shared__ float s_m[kWaves], s_l[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // the workgroups that begin a segment others go on with, in order
  int2 chain[kBlocks / kThreads];
#pragma unroll
  for (int i = 0; i < kBlocks / kThreads; ++i) {
    const int b = i * kThreads + tid;
    chain[i] = b < blocks ? *chain_at(p.ws, rows, D, blocks, b) : make_int2(-1, 0);
    const uint64_t m = __ballot(chain[i].x >= 0);
    if (lane == 0) s_count[i * kWaves + wave] = __popcll(m);
  }
  __syncthreads();
  int chains = 0;
#pragma unroll
  for (int i = 0; i < kBlocks / kThreads; ++i) {
    const uint64_t m = __ballot(chain[i].x >= 0);
    int before = 0;
    for (int w = 0; w < i * kWaves + wave; ++w) before += s_count[w];
    if (chain[i].x >= 0) {
      const int k = before + __popcll(m & ((1ull << lane) - 1));
      s_start[k] = i * kThreads + tid;
      s_end[k] = chain[i].y < blocks ? chain[i].y : blocks - 1;
      s_seg[k] = chain[i].x;
    }
  }
  for (int w = 0; w < kBlocks / 64; ++w) chains += s_count[w];
  __syncthreads();

  const int G = p.Hq / p.Hk, per_seq = p.Hk * qgroups;
  auto out_row = [&](int seg, int qi) -> int64_t {   // -1: not a query of the group
    const int n = seg / per_seq, hk = (seg - n * per_seq) / qgroups, qg = seg % qgroups;
    return 16 * qg + qi < G ? (int64_t)n * p.Hq + hk * G + 16 * qg + qi : -1;
  };
  auto write = [&](int64_t row, int col, const JoinSum<D>& a) {
    const float inv = a.l > 0.f ? 1.f / a.l : 0.f;
    store4<T>(static_cast<T*>(p.o) + row * D + col, a.r[0] * inv, a.r[1] * inv, a.r[2] * inv,
              a.r[3] * inv);
  };
  constexpr int CP = D / 32;                // column parts
  if (chains * rows * CP > (int)gridDim.x) {
    constexpr int LPQ = D / 4;
    const int col = 4 * (lane % LPQ);
    for (int it = blockIdx.x * kWaves + wave; it < chains * rows; it += gridDim.x * kWaves) {
      const int k = it / rows, qi = it - k * rows;
      const int64_t row = out_row(s_seg[k], qi);
      if (row < 0) continue;
      JoinSum<D> a;
      a.gather(p.ws, rows, s_start[k], s_end[k] - s_start[k] + 1, qi, col, lane / LPQ, 64 / LPQ);
      a.over_lanes(LPQ);
      if (lane < LPQ) write(row, col, a);
    }
    return;
  }
  const int gr = tid / 8, c4 = 4 * (tid % 8);
  for (int it = blockIdx.x; it < chains * rows * CP; it += gridDim.x) {
    const int k = it / (rows * CP), qi = it / CP % rows, col = 32 * (it % CP) + c4;
    const int64_t row = out_row(s_seg[k], qi);
    JoinSum<D> a;
    if (row >= 0) a.gather(p.ws, rows, s_start[k], s_end[k] - s_start[k] + 1, qi, col, gr, 32);
    a.over_lanes(8);
    if (lane < 8) *reinterpret_cast<float4*>(&s_o[wave][c4]) = make_float4(a.r[0], a.r[1], a.r[2], a.r[3]);
    if (lane == 0) { s_m[wave] = a.m; s_l[wave] = a.l; }
    __syncthreads();
    if (tid < 8 && row >= 0) {
#pragma unroll
      for (int w = 1; w < kWaves; ++w) a.add(s_m[w], s_l[w], *reinterpret_cast<const float4*>(&s_o[w][c4]));
      write(row, col, a);
    }
    __syncthreads();
  }
}

template <typename T, int D>
hipError_t launch_t(const AttnDecodeArgs& a, hipStream_t stream) {
  const AttnDecodePlan plan = attn_decode_plan(a.N, a.cache.max_pages * a.cache.page_size, a.window,
                                               a.Hq, a.Hk, D);
  const int G = a.Hq / a.Hk, qgroups = (G + 15) / 16, rows = G < 16 ? G : 16;
  attn_decode_kernel<T, D><<<dim3((unsigned)plan.blocks), kThreads, 0, stream>>>(
      a, qgroups, plan.ws_floats == 0);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || plan.ws_floats == 0) return e;
  attn_join_kernel<T, D><<<dim3(kJoinBlocks), kThreads, 0, stream>>>(a, qgroups, rows,
                                                                     (int)plan.blocks);
  return hipGetLastError();
}

}  // namespace

AttnDecodePlan attn_decode_plan(int64_t N, int64_t max_tokens, int64_t window, int Hq, int Hk,
                                int d) {
  const DecodePlan p = decode_plan(N, max_tokens, window, Hq, Hk);
  return AttnDecodePlan{p.blocks, p.rounds,
                        p.part_rows ? p.blocks * (2 * p.part_rows * (d + 4) + 2) : 0};
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
