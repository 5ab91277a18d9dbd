// attn_rope.hip -- what happens to query, key and value rows between the
// projection and the attention of a hybrid model's softmax-attention layers:
//
//   qk_norm_rope : RMS norm of each head and the rotary position, rows in and
//                  rows out.
//   kv_append    : the same on keys, and the codes and scales of the new keys
//                  and values into a paged cache of e4m3 codes.
//
// Both read their rows once and write once, at about ten flops per element:
// HBM-bound for many rows, launch latency for few.
//
// A head of D channels is held by D/16 lanes with 16 channels each, in two
// chunks of 8.  Which chunks makes both members of every rotary pair meet in
// one lane, so no value crosses lanes but the row's sum of squares.  Lanes l <
// dim/16 turn, and hold
//   half pairs    [8 l, +8) and [dim/2 + 8 l, +8), frequencies 8 l .. 8 l + 7;
//   interleaved   norm_rope: the same chunks, so that neighbours have
//                 neighbouring ones, frequencies 4 l .. 4 l + 3 and dim/4 + 4 l
//                 .. dim/4 + 4 l + 3; append: [16 l, +16), as half pairs.
// The others share the rest: norm_rope [8 l', +8) and the same behind half of
// it, append [16 l, +16).  (norm_rope, 32768 fp32 rows of 18 heads of 128, with
// 16 neighbouring channels to a lane / spread: interleaved 132 / 109 us, not
// turned 153 / 108; bf16 57.8 / 54.7, 57.3 / 54.6.  append, whose codes of 16
// channels are one piece: no difference, 32768 bf16 tokens of 4 heads 25.9 / 25.6.
// These times and those below are on inputs that the caches do not hold.)
#include "attn_device.hpp"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// Chunk offsets of lane l, whether it turns, and its frequencies: f0 .. f0 + 3
// and f0 + gap .. f0 + gap + 3 (some that exist where it does not turn).
// SPREAD: neighbours have neighbouring chunks.
struct LaneMap {
  int c0, c1, f0, gap;
  bool turns;
};
template <int D, bool INTER, bool SPREAD>
__device__ __forceinline__ LaneMap lane_map(int l, const RopeArgs& r) {
  LaneMap m;
  m.turns = 16 * l < r.dim;
  const bool whole = !SPREAD && (INTER || !m.turns);
  m.c0 = whole ? 16 * l : (m.turns ? 0 : r.dim / 2) + 8 * l;
  m.c1 = m.c0 + (whole ? 8 : (m.turns ? r.dim : D - r.dim) / 2);
  m.f0 = m.turns ? (INTER && SPREAD ? 4 : 8) * l : 0;
  m.gap = INTER && SPREAD && m.turns ? r.dim / 4 : 4;
  return m;
}

// cos and sin of pos * inv_freq[8 l ..], times the factor.  The angle is needed
// in turns, reduced; pos * freq alone would lose 2^-24 of a far position's
// angle.  Positions below 2^24 are exact in fp32, and the frequency in turns is
// kept as two fp32 terms: the leading product's error comes back by an fma, its
// whole turns leave exactly, and the rest is added: an error of 2^-25 turns up
// to 2^22 turns, which frequencies of at most 1 stay below.  Other angles go
// the same way in two 64-bit terms (positions are exact there up to 2^53), whose
// conversions and products are slow (an append of 32768 tokens, 4 heads: 32.9 us
// with them for all, 25.9 us so).  Results that
// are rounded to bf16 or e4m3 take the hardware's sine, whose error (about
// 2^-20) is far below their half step of 2^-8 or 2^-4; fp32 results take the
// exact routine.  (UNROLL is the far angles' loop: rolled it leaves append
// registers; 32768 rows of far positions in norm_rope, rolled / unrolled: bf16 70 /
// 55 us, fp32 121 / 111.)
struct Freqs {
  float hi[8], lo[8];                       // inv_freq / 2 pi
  float most;                               // largest of |hi|
};
__device__ __forceinline__ void load_freqs(const RopeArgs& r, const LaneMap& m, Freqs& f) {
#pragma clang fp contract(off)             // the products below are meant to be rounded
  constexpr float kHi = 0.15915494f, kLo = (float)(0.15915494309189533577 - (double)kHi);
  float x[8];
  const float* src = r.inv_freq + m.f0;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = src[i < 4 ? i : m.gap + i - 4];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f.hi[i] = x[i] * kHi;
    f.lo[i] = __builtin_fmaf(x[i], kLo, __builtin_fmaf(x[i], kHi, -f.hi[i]));
    f.most = i ? fmaxf(f.most, fabsf(f.hi[i])) : fabsf(f.hi[i]);
  }
}

template <bool EXACT, int UNROLL>
__device__ __forceinline__ void turn(int64_t pos, const Freqs& f, const RopeArgs& rope,
                                     const LaneMap& m, float* c, float* s) {
#pragma clang fp contract(off)
  float r[8];                               // turns in [-1/2, 1/2]
  const float x = (float)(int)pos;          // (of near positions)
  if (pos < (1 << 24) && pos > -(1 << 24) && fabsf(x) * f.most < 0x1p22f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = x * f.hi[i];
      const float e = __builtin_fmaf(x, f.hi[i], -p);
      r[i] = (p - __builtin_rintf(p)) + __builtin_fmaf(x, f.lo[i], e);
    }
  } else {
    const float* src = rope.inv_freq + m.f0;
#pragma unroll UNROLL
    for (int i = 0; i < 8; ++i) {
      constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;   // 1 / 2 pi
      const double w = src[i < 4 ? i : m.gap + i - 4], at = (double)pos;
      const double c1 = w * kHi, c2 = __builtin_fma(w, kHi, -c1) + w * kLo;
      const double p = at * c1, e = __builtin_fma(at, c1, -p);
      const double t = (p - __builtin_rint(p)) + __builtin_fma(at, c2, e);
      r[i] = (float)(t - __builtin_rint(t));
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (EXACT) {
      sincospif(2.f * r[i], &s[i], &c[i]);
    } else {
      s[i] = __builtin_amdgcn_sinf(r[i]);   // of r turns
      c[i] = __builtin_amdgcn_cosf(r[i]);
    }
    c[i] *= rope.factor;
    s[i] *= rope.factor;
  }
}

// Norm (when normed) and rotation of one row's 16 channels in this lane.
// `w` are the norm's weights of those channels.
template <int LPR, bool INTER>
__device__ __forceinline__ void norm_turn(float* x, bool normed, const float* w, float eps,
                                          bool turns, const float* c, const float* s) {
  if (normed) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss += x[i] * x[i];
    ss = lanes_sum<LPR>(ss);
    const float inv = __builtin_amdgcn_rsqf(ss * (1.f / (16 * LPR)) + eps);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] *= inv * w[i];
  }
  if (turns) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int ia = INTER ? 2 * i : i, ib = INTER ? 2 * i + 1 : 8 + i;
      const float a = x[ia], b = x[ib];
      x[ia] = a * c[i] - b * s[i];
      x[ib] = b * c[i] + a * s[i];
    }
  }
}

__device__ __forceinline__ void load_weights(const float* weight, const LaneMap& m, float* w) {
  if (!weight) return;
  load_f32<8, float>(weight + m.c0, w);
  load_f32<8, float>(weight + m.c1, w + 8);
}

// ---------------------------------------------------------------------------
// qk_norm_rope.  A thread keeps its lane of one token for kHeads heads of one
// operand, so the angles are computed once for them and every load is issued
// before the first value is used.  Blocks run over head groups first, so that
// a token's whole row is read by workgroups that run together.  HBM-bound:
// 32768 tokens of 18 heads of 128, bf16, 302 MB: 54.6 us, 5.5 TB/s (4 heads to a
// thread 61.2, one 55.5); fp32 109 us (117, 118).
// ---------------------------------------------------------------------------
constexpr int kHeads = 2;

template <typename T, int D, bool INTER>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(QkNormRopeArgs p) {
  constexpr int LPR = D / 16;
  constexpr int TB = kThreads / LPR;          // tokens of a workgroup
  const int gq = (p.Hq + kHeads - 1) / kHeads, gk = (p.Hk + kHeads - 1) / kHeads;
  const int64_t tb = blockIdx.x / (gq + gk);
  const int grp = (int)(blockIdx.x - tb * (gq + gk));
  const bool is_q = grp < gq;
  const int H = is_q ? p.Hq : p.Hk;
  const int h0 = (is_q ? grp : grp - gq) * kHeads;
  const int64_t ld = is_q ? p.ld_q : p.ld_k;
  const float* weight = is_q ? p.q_weight : p.k_weight;
  const int l = threadIdx.x % LPR;
  const int64_t r = tb * TB + threadIdx.x / LPR;
  if (r >= p.rows) return;                    // whole rows of lanes leave together
  const LaneMap m = lane_map<D, INTER, true>(l, p.rope);
  const T* __restrict__ in = static_cast<const T*>(is_q ? p.q_raw : p.k_raw) + r * ld;
  T* out = static_cast<T*>(is_q ? p.q : p.k) + r * (int64_t)H * D;

  Chunk8<T> a[kHeads], b[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = h0 + i < H ? h0 + i : H - 1;
    a[i].load(in + h * D + m.c0);
    b[i].load(in + h * D + m.c1);
  }
  float w[16], c[8], s[8];
  load_weights(weight, m, w);
  if (p.rope.dim) {
    Freqs f;
    load_freqs(p.rope, m, f);
    turn<std::is_same<T, float>::value, 8>(p.positions[r], f, p.rope, m, c, s);
  }
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    float x[16];
    a[i].unpack(x);
    b[i].unpack(x + 8);
    norm_turn<LPR, INTER>(x, weight != nullptr, w, p.rope.eps, m.turns, c, s);
    if (h0 + i < H) {
      store8(out + (h0 + i) * D + m.c0, x);
      store8(out + (h0 + i) * D + m.c1, x + 8);
    }
  }
}

// ---------------------------------------------------------------------------
// kv_append.  One workgroup for each (page that may get new tokens, head, key
// or value): it holds the page's new rows in registers, finds their largest
// magnitude, and writes their codes; where the scale of a page that holds older
// tokens grows it also rounds those again.  So a row is read once though its scale
// is known only after the page's last row.  HBM-bound for many tokens (32768
// tokens of 4 heads of 128, bf16, pages of 64: 101 MB in 24 us, 4.2 TB/s; fp32
// 168 MB in 41 us), by latency and the waves that fit where pages are partly filled
// (213 sequences of 40 tokens, 8 heads of 64, pages of 128: 24 us for 26 MB), and
// by the launch for a token to a sequence (256: 4.3 us).
//
// A wave takes two passes of 1024 / D rows: as many registers as 5 waves to a
// SIMD leave.  (One pass at D 64: 32.3 us for the 213 sequences; four at D 128
// spill, 32768 tokens in pages of 128: 56.6 us instead of 29.8.)
//
// Which pages get tokens is known on the device only.  L new tokens behind a
// length s touch at most floor(L / P) + 2 pages, so packed sequences own the
// slots floor(cu[n] / P) + 2 n onwards and slots past a sequence's last page
// leave at once.
// ---------------------------------------------------------------------------
constexpr int append_rows_per_wave(int P, int D) { return P < 2048 / D ? P : 2048 / D; }

__device__ __forceinline__ float pow2_scale(float amax) {
  // least 2^e with amax <= 448 2^e: amax = m 2^x, m in [1, 2), and 448 = 1.75 2^8
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  if (e < -100) e = -100;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Four e4m3 codes of x * inv, rounded to nearest even; NaN stays NaN.  Where
// there may be infinities (clamp), they become the largest code.
__device__ __forceinline__ uint32_t codes4(const float* x, float inv, bool clamp) {
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[i] = x[i] * inv;
    if (clamp && y[i] == y[i]) y[i] = __builtin_amdgcn_fmed3f(y[i], -448.f, 448.f);
  }
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
}

__device__ __forceinline__ uint32_t recode4(uint32_t c, float factor) {
  float x[4] = {__builtin_amdgcn_cvt_f32_fp8(c, 0), __builtin_amdgcn_cvt_f32_fp8(c, 1),
                __builtin_amdgcn_cvt_f32_fp8(c, 2), __builtin_amdgcn_cvt_f32_fp8(c, 3)};
  return codes4(x, factor, false);          // codes hold no infinities
}

// The rows of one wave.  FULL: the page's rows are all new; otherwise passes without a
// new row are skipped (a single token's page has one).
template <typename T, int D, bool INTER, int P, bool FULL>
__device__ __forceinline__ void append_rows(const KvAppendArgs& p, const RopeArgs& rope,
                                            const LaneMap& m, const T* __restrict__ in, int64_t ld,
                                            const AppendPage& ap, int64_t page, int head,
                                            bool is_k, int wrow, int row0, int l) {
  constexpr int LPR = D / 16;
  constexpr int RPW = 64 / LPR;               // rows of a wave's pass
  constexpr int ROWS = append_rows_per_wave(P, D);
  constexpr int PASSES = ROWS / RPW;
  constexpr int WAVES = P / ROWS;
  const PagedCache& kv = p.cache;
  const int kept = ap.kept, stop = ap.stop;
  auto has = [&](int i) { return FULL || (wrow + i * RPW < stop && wrow + (i + 1) * RPW > kept); };

  Chunk8<T> ca[PASSES], cb[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    if (!has(i)) continue;
    int row = row0 + i * RPW;
    row = row < kept ? kept : (row >= stop ? stop - 1 : row);   // loads stay on new rows
    ca[i].load(in + (ap.tok0 + row) * ld + m.c0);
    cb[i].load(in + (ap.tok0 + row) * ld + m.c1);
  }
  float w[16];
  const bool normed = is_k && p.k_weight;
  load_weights(is_k ? p.k_weight : nullptr, m, w);
  Freqs f;
  if (rope.dim) load_freqs(rope, m, f);

  float x[PASSES][16];
  float top = 0.f;                            // of |x|; NaN does not count
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    if (!has(i)) continue;
    const int row = row0 + i * RPW;
    ca[i].unpack(x[i]);
    cb[i].unpack(x[i] + 8);
    if (is_k) {
      float c[8], sn[8];
      if (rope.dim) turn<false, 1>(ap.pi * P + row, f, rope, m, c, sn);
      norm_turn<LPR, INTER>(x[i], normed, w, rope.eps, m.turns, c, sn);
    }
    if (FULL || (row >= kept && row < stop))
#pragma unroll
      for (int t = 0; t < 16; ++t) top = fmaxf(top, fabsf(x[i][t]));
  }
  // the table entry, asked for before the rows, is first needed here
  if (page < 0 || page >= kv.num_pages) return;     // (the same for the workgroup)
  const int64_t at = page * p.Hk + head;
  uint8_t* __restrict__ codes = (is_k ? kv.k : kv.v) + at * (int64_t)(P * D);
  float* scale = (is_k ? kv.k_scale : kv.v_scale) + at;
  const float old_scale = kept ? *scale : 0.f;
  bool infinite = __any(top == __builtin_huge_valf());
  if (infinite) {                             // again without the infinities
    top = 0.f;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int row = row0 + i * RPW;
      if (has(i) && row >= kept && row < stop)
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          const float a = fabsf(x[i][t]);
          top = fmaxf(top, a < __builtin_huge_valf() ? a : 0.f);
        }
    }
  }
  top = wave_max(top);
  if constexpr (WAVES > 1) {
    __shared__ float s_top[WAVES];
    if ((threadIdx.x & 63) == 0) s_top[threadIdx.x >> 6] = top;
    __syncthreads();                          // (and every wave has read the old scale)
#pragma unroll
    for (int i = 0; i < WAVES; ++i) top = fmaxf(top, s_top[i]);
  }
  const float sc = fmaxf(pow2_scale(top), old_scale);
  const float inv = 1.f / sc;                 // exact: a power of two
  if (threadIdx.x == 0) *scale = sc;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int row = row0 + i * RPW;
    uint8_t* dst = codes + row * D;
    if (FULL || (has(i) && row >= kept && row < stop)) {
      *reinterpret_cast<uint2*>(dst + m.c0) =
          make_uint2(codes4(x[i], inv, infinite), codes4(x[i] + 4, inv, infinite));
      *reinterpret_cast<uint2*>(dst + m.c1) =
          make_uint2(codes4(x[i] + 8, inv, infinite), codes4(x[i] + 12, inv, infinite));
    } else if (row < kept && sc > old_scale) {
      const float factor = old_scale * inv;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint2* q = reinterpret_cast<uint2*>(dst + (h ? m.c1 : m.c0));
        const uint2 u = *q;
        *q = make_uint2(recode4(u.x, factor), recode4(u.y, factor));
      }
    }
  }
}

template <typename T, int D, bool INTER, int P>
__global__ __launch_bounds__(64 * P / append_rows_per_wave(P, D), sizeof(T) == 2 ? 5 : 4) void kv_append_kernel(KvAppendArgs p) {
  constexpr int LPR = D / 16;
  const int head = blockIdx.y;
  const bool is_k = blockIdx.z == 0;

  // which sequence and page; the table entry is needed only where the codes go
  const PagedCache& kv = p.cache;
  int64_t n, j, a, L, held;
  if (!p.cu_seqlens) {
    const uint32_t per = ((uint32_t)p.Tseq + P - 2) / P + 1;
    const uint32_t n32 = blockIdx.x / per;
    n = n32;
    j = blockIdx.x - n32 * per;
    a = n * p.Tseq;
    L = p.Tseq;
    held = kv.seq_lens[n];
  } else {
    const PackedItem it =
        find_packed(p.cu_seqlens, p.N, p.total_T, P, 2, blockIdx.x, kv.seq_lens, &held);
    n = it.n;
    j = it.item;
    a = it.start;
    L = it.end - it.start;
  }
  const AppendPage ap = append_page(held, kv.max_pages, P, j, a, L);
  if (ap.kept >= ap.stop) return;
  const int kept = ap.kept, stop = ap.stop;
  const int64_t page = kv.table[n * kv.max_pages + ap.pi];

  const T* __restrict__ in = static_cast<const T*>(is_k ? p.k_raw : p.v_raw) + head * D;
  const int64_t ld = is_k ? p.ld_k : p.ld_v;
  const int l = threadIdx.x % LPR;
  // the wave's rows
  const int wrow = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)) * append_rows_per_wave(P, D);
  const int row0 = wrow + (threadIdx.x & 63) / LPR;
  RopeArgs rope = p.rope;
  if (!is_k) rope.dim = 0;
  const LaneMap m = lane_map<D, INTER, false>(l, rope);
  if (kept == 0 && stop == P)                 // (the same for the workgroup: it has barriers)
    append_rows<T, D, INTER, P, true>(p, rope, m, in, ld, ap, page, head, is_k, wrow, row0, l);
  else
    append_rows<T, D, INTER, P, false>(p, rope, m, in, ld, ap, page, head, is_k, wrow, row0, l);
}

template <typename T, int D>
hipError_t launch_qk_t(const QkNormRopeArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)qk_norm_rope_blocks(a.rows, a.Hq, a.Hk, D));
  if (a.rope.inter) qk_norm_rope_kernel<T, D, true><<<grid, kThreads, 0, stream>>>(a);
  else qk_norm_rope_kernel<T, D, false><<<grid, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

template <typename T, int D, bool INTER>
hipError_t launch_append_t(const KvAppendArgs& a, hipStream_t stream) {
  const int P = a.cache.page_size;
  const dim3 grid((unsigned)kv_append_slots(a.N, a.total_T, a.Tseq, a.cu_seqlens != nullptr, P),
                  (unsigned)a.Hk, 2);
  auto threads = [](int page) { return 64 * page / append_rows_per_wave(page, D); };
  if (P == 16) kv_append_kernel<T, D, INTER, 16><<<grid, threads(16), 0, stream>>>(a);
  else if (P == 32) kv_append_kernel<T, D, INTER, 32><<<grid, threads(32), 0, stream>>>(a);
  else if (P == 64) kv_append_kernel<T, D, INTER, 64><<<grid, threads(64), 0, stream>>>(a);
  else kv_append_kernel<T, D, INTER, 128><<<grid, threads(128), 0, stream>>>(a);
  return hipGetLastError();
}

template <typename T>
hipError_t pick_append(const KvAppendArgs& a, hipStream_t s) {
  if (a.d == 128)
    return a.rope.inter ? launch_append_t<T, 128, true>(a, s) : launch_append_t<T, 128, false>(a, s);
  return a.rope.inter ? launch_append_t<T, 64, true>(a, s) : launch_append_t<T, 64, false>(a, s);
}

}  // namespace

int64_t qk_norm_rope_blocks(int64_t rows, int Hq, int Hk, int d) {
  const int64_t tb = kThreads / (d / 16);
  return (rows + tb - 1) / tb * ((Hq + kHeads - 1) / kHeads + (Hk + kHeads - 1) / kHeads);
}

int64_t kv_append_slots(int64_t N, int64_t total_T, int64_t Tseq, bool packed, int P) {
  return packed ? total_T / P + 2 * N : N * ((Tseq + P - 2) / P + 1);
}

hipError_t launch_qk_norm_rope(const QkNormRopeArgs& a, hipStream_t stream) {
  if (a.io == DType::F32)
    return a.d == 128 ? launch_qk_t<float, 128>(a, stream) : launch_qk_t<float, 64>(a, stream);
  return a.d == 128 ? launch_qk_t<bf16, 128>(a, stream) : launch_qk_t<bf16, 64>(a, stream);
}

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t stream) {
  return a.io == DType::F32 ? pick_append<float>(a, stream) : pick_append<bf16>(a, stream);
}

#ifdef GDN_CHECK
unsigned check_violations_attn_rope() { return take_check_violations(); }
#endif

}  // namespace gdn
