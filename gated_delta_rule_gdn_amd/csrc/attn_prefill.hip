// attn_prefill.hip -- causal softmax attention over packed prompts with
// grouped heads on gfx950, full or in a sliding window:
//
//   o_t = sum_s p_ts v_s / sum_s p_ts,   p_ts = exp(scale * q_t . k_s - m_t)
//
// in one pass over the keys with a running maximum m and sum for each query.
//
// Both kernels put the queries on the columns of the products,
//   S^T [tokens x queries] = K Q^T,    O^T [d x queries] += V^T P^T,
// so that a lane holds scores of one query only: the maximum and the sum are
// reduced in registers and across 2 (or 4) lanes, and the weights are, as they
// lie in the score accumulators, the k-values this lane supplies to the second
// product.  No weight crosses lanes or LDS.  The bf16 kernel rounds the weights to
// bf16 for it, half a step of 2^-8 of each like the output's own rounding (error
// against 64 bits 2.1e-3 for 8 prompts of 4096 tokens, 1.6e-3 with fp32 weights):
// in two terms they would take half as many products again.
//
// 4 d flops to a key that a query sees, against a few bytes: bound by the matrix
// cores, and with them by power (the clock falls to about 1.8 GHz).  bf16, 16
// heads of 128: one prompt of 32768 tokens over 2 key heads 3.66 to 3.89 ms on
// different cards, 1130 to 1200 TFLOP/s (a plain product of 8192 x 8192 x 8192
// reaches 1212); 8 prompts of 4096 over 16 key heads 527 to 549 us, 1000 to 1043
// TFLOP/s; 16 prompts, 32768 tokens in all, a window of 2048, 337 to 361 us, 954 to
// 1022 TFLOP/s.  Short prompts wait for memory at both ends of a tile (about 6 us
// of each workgroup).
#include "attn_device.hpp"

namespace gdn {
namespace {

constexpr int kThreads = 256;

// One workgroup's query tile: queries [q0, q0 + BM) of the sequence that is
// rows [a, a + L) of the packed tensors, and a query head.
struct Tile {
  int64_t a, L, q0;
  int hq;
  bool valid;
};

// Workgroup blk runs on XCD blk % 8, and each XCD has an L2 of its own, so the
// workgroups that follow each other on an XCD should read the same keys and
// values; and a query tile costs as many key tiles as lie before it, so the
// late tiles should start first.  The query heads of a key head always follow
// each other.  (All counts fit in 32 bits: the host bounds the grid.)
//
// Equal lengths, key heads of all sequences a multiple of 8: an XCD keeps its
// share of them, in groups of 4 query heads or more, and goes through each
// group's tiles from the last to the first.  64 workgroups
// of an XCD then walk the keys of 4 heads together (B 8, T 4096, 16 heads:
// 78 % of the L2 reads hit against 48 % with heads dealt round the XCDs).
// Otherwise tiles are dealt round the XCDs, the last tiles of all sequences
// first.
//
// Packed lengths: the tiles are dealt round the XCDs, the dear ones first
// (rank_tile_by): found by counting, so nothing is sorted.  (16 prompts, 32768
// tokens, a window of 2048: 367 us; in the order of the tokens 383 us.)
constexpr uint32_t kXcds = 8;
constexpr int64_t kMaxRanked = 1024;      // sequences that are ranked; more keep their order

template <int BM>
__device__ __forceinline__ Tile find_tile(const PrefillArgs& p, uint32_t blocks) {
  Tile t;
  const uint32_t blk = blockIdx.x;
  const uint32_t G = (uint32_t)(p.Hq / p.Hk), Hk = (uint32_t)p.Hk, N = (uint32_t)p.N;
  const uint32_t per = blocks / kXcds;                    // full rounds over the XCDs
  const uint32_t xcd = blk % kXcds, i = blk / kXcds;
  t.valid = true;
  if (!p.cu_seqlens) {
    const uint32_t tiles = ((uint32_t)p.Tseq + BM - 1) / BM, pairs = N * Hk;
    const uint32_t mine = pairs / kXcds;                  // pairs of an XCD
    uint32_t pair, tile, head;
    if (pairs % kXcds == 0) {
      const uint32_t gp = G >= 4 ? 1 : 4 / G;             // pairs of a group
      const uint32_t grp = i / (gp * tiles * G), w = i - grp * (gp * tiles * G);
      const uint32_t here = mine - grp * gp < gp ? mine - grp * gp : gp;
      const uint32_t level = w / (here * G), x = w - level * (here * G);
      tile = tiles - 1 - level;
      pair = xcd + kXcds * (grp * gp + x / G);
      head = x % G;
    } else {
      // unit = (tile from the last, pair); the last partial round is dealt plainly
      uint32_t unit;
      const uint32_t rounds = per / G;
      if (i < rounds * G) { unit = i / G * kXcds + xcd; head = i % G; }
      else { const uint32_t r = blk - rounds * G * kXcds; unit = rounds * kXcds + r / G; head = r % G; }
      tile = tiles - 1 - unit / pairs;
      pair = unit % pairs;
    }
    const uint32_t n = pair / Hk, hk = pair - n * Hk;
    t.a = n * p.Tseq;
    t.L = p.Tseq;
    t.q0 = (int64_t)tile * BM;
    t.hq = (int)(hk * G + head);
    return t;
  }
  uint32_t unit, head;
  const uint32_t rounds = per / G;
  if (i < rounds * G) {
    unit = i / G * kXcds + xcd;
    head = i % G;
  } else {
    const uint32_t r = blk - rounds * G * kXcds;
    unit = rounds * kXcds + r / G;
    head = r % G;
  }
  const uint32_t rank = unit / Hk;
  t.hq = (int)((unit - rank * Hk) * G + head);
  PackedItem it;
  // tiles from this number on see a whole window
  const int level = (int)((p.window > 0 && p.window < p.total_T ? p.window : p.total_T) + BM - 1) / BM;
  if (p.N <= 64)
    it = rank_tile<1>(p.cu_seqlens, (int)p.N, p.total_T, BM, level, (int)rank);
  else if (p.N <= kMaxRanked)
    it = rank_tile<kMaxRanked / 64>(p.cu_seqlens, (int)p.N, p.total_T, BM, level, (int)rank);
  else
    it = find_packed(p.cu_seqlens, p.N, p.total_T, BM, 1, (int64_t)rank);
  t.a = it.start;
  t.L = it.end - it.start;
  t.q0 = it.item * BM;
  t.valid = t.q0 >= 0 && t.q0 < t.L;
  return t;
}

// The products give unseen tokens a weight of zero, and zero times an infinite or
// NaN value is NaN: such a value would reach queries that do not see it.  A wave
// whose sums are not all finite looks at the values that its tiles hold and some
// of its queries [q0, q0 + rows) do not see (tiles end less than 160 tokens from
// q0 on either side of what is seen), and if any is not finite it computes its
// rows again by exact_rows, which touches seen tokens only.
// So does a wave of the bf16 kernel whose running maximum was huge: its weights
// are 2^(s c - m) with an unrounded product and m off by half a step, the same
// factor on all of a query's weights and so none on its output, until it leaves
// the range of fp32.  Below 2^24 it is 2 at most.  (The product rounded first
// takes another instruction for each of 32 weights.)
template <typename T, int D>
__device__ __forceinline__ bool unseen_not_finite(const T* __restrict__ v, int64_t ld, int L,
                                                  int window, int q0, int rows) {
  const int lane = threadIdx.x & 63;
  float z = 0.f;                            // times 0: NaN where a value is not finite
  auto scan = [&](int from, int to) {
#pragma unroll 1
    for (int s = from < 0 ? 0 : from; s < to && s < L; ++s)
#pragma unroll
      for (int c = 0; c < D; c += 64) z = __builtin_fmaf((float)v[s * ld + c + lane], 0.f, z);
  };
  scan(q0 + 1, q0 + 160);
  if (window) scan(q0 - window - 160, q0 + rows - window);
  return __any(z != z);
}

// Says that x points to global memory, as a kernel's own arguments do.
template <typename T>
__device__ __forceinline__ const T* in_global(const void* x) {
  return (const T*)(const __attribute__((address_space(1))) T*)x;
}

// Rows [q0, q0 + rows) of a sequence and head by a wave, one after another: 64
// keys at a time, a score to a lane, then D / 64 columns to a lane.  Bound by the
// latency of its loads (a prompt of 4096 tokens, 16 heads, with one NaN value: up
// to 13 ms for the wave that it sends here, 0.11 ms without; 32768 tokens 114).  A
// row all of whose columns are NaN is settled: where every value is NaN all waves
// come here (16384 tokens 138 ms walking on, 2 ms so).
template <typename T, int D>
__device__ __forceinline__ void exact_rows(const PrefillArgs& p, const Tile& tl, int hk, int window,
                                           int q0, int rows) {
  const int lane = threadIdx.x & 63, L = (int)tl.L;
  const float c_scale = p.scale * kLog2e;
  const T* kp = in_global<T>(p.k) + tl.a * p.ld_k + hk * D;
  const T* vp = in_global<T>(p.v) + tl.a * p.ld_v + hk * D;
  for (int t = q0; t < q0 + rows && t < L; ++t) {
    const T* qp = in_global<T>(p.q) + (tl.a + t) * p.ld_q + tl.hq * D;
    float m = kNone, l = 0.f, o[D / 64] = {};
    for (int s0 = window && t >= window ? t - window + 1 : 0; s0 <= t; s0 += 64) {
      const int s = s0 + lane <= t ? s0 + lane : t;
      float x = 0.f;
#pragma unroll 4
      for (int c = 0; c < D; c += 8) {
        float a[8], b[8];
        load_f32<8, T>(qp + c, a);
        load_f32<8, T>(kp + s * p.ld_k + c, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) x = __builtin_fmaf(a[i], b[i], x);
      }
      x = s0 + lane <= t ? x * c_scale : -__builtin_huge_valf();
      const float m_new = fmaxf(m, wave_max(x));
      const float alpha = exp2_fast(m - m_new), w = weight_of(x, m_new);
      m = m_new;
      float sum = w;
#pragma unroll
      for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off);
      l = l * alpha + sum;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) o[c] *= alpha;
#pragma unroll 1
      for (int i0 = 0; i0 < 64 && s0 + i0 <= t; i0 += 16) {
        float y[16][D / 64];                // values of 16 keys (t's again behind t)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int u = s0 + i0 + i;
          const T* row = vp + (u < t ? u : t) * p.ld_v + lane;
#pragma unroll
          for (int c = 0; c < D / 64; ++c) y[i][c] = (float)row[64 * c];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float wi = (float)(T)__shfl(w, i0 + i);
          const bool seen = s0 + i0 + i <= t;
#pragma unroll
          for (int c = 0; c < D / 64; ++c) o[c] = seen ? __builtin_fmaf(wi, y[i][c], o[c]) : o[c];
        }
      }
      bool nan = true;                      // every column: no later key changes that
#pragma unroll
      for (int c = 0; c < D / 64; ++c) nan = nan && o[c] != o[c];
      if (__all(nan)) break;
    }
    T* op = static_cast<T*>(p.o) + ((tl.a + t) * p.Hq + tl.hq) * (int64_t)D + lane;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) op[64 * c] = (T)(o[c] / l);
  }
}

// Both, for the end of a kernel: true if the rows are written (always if `huge`, the
// wave's maximum was).  The arguments are
// read from the kernel's argument segment again, where `p` is its first: kept in
// registers for this rare end they would spill others (2 % of a prompt).
template <typename T, int D>
__device__ __forceinline__ bool rows_again(const Tile& tl, int hk, int window, int q0, int rows,
                                           bool huge) {
#if __HIP_DEVICE_COMPILE__
  uint64_t at = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(at));
  const PrefillArgs p = *reinterpret_cast<const PrefillArgs*>(at);
  const T* v = in_global<T>(p.v) + tl.a * p.ld_v + hk * D;
  if (!huge && !unseen_not_finite<T, D>(v, p.ld_v, (int)tl.L, window, q0, rows)) return false;
  exact_rows<T, D>(p, tl, hk, window, q0, rows);
#endif
  return true;
}

// ---------------------------------------------------------------------------
// fp32: v_mfma_f32_16x16x4_f32.  A workgroup has 32 queries; waves 0 and 1 take
// 16 each over the first 16 tokens of every key tile of 16 KW, waves 2 and 3 the
// same queries over the next 16, and so on, with a running maximum and sum of
// their own, and they join through LDS at the end.  Short prompts have few query
// tiles, and this divides the time that one takes (KW 4 where there are few, see
// split_f32, else 2).  The next key tile is loaded
// into registers while this one is computed.  Bound by fp32 products and the
// vector work between them: 4096 tokens, 16 heads of 128: 675 us, 102 TFLOP/s (a
// plain fp32 product reaches 154).  (Without the bound on registers the compiler
// moves the sums to the accumulation registers and back in every tile: 790 us;
// key tiles double-buffered in LDS, which leaves room for two workgroups instead
// of three: 750 us.)
// ---------------------------------------------------------------------------
template <int D, int KW>
__global__ __launch_bounds__(128 * KW, KW == 4 ? 2 : D == 64 ? 4 : 3) void prefill_f32_kernel(PrefillArgs p, uint32_t blocks) {
  constexpr int BM = 32, BN = 16 * KW, LD = D + 4, KB = D / 32, MT = D / 16;
  constexpr int NT = 128 * KW;                        // threads
  constexpr int NL = BN * D / 4 / NT;                 // 16-byte loads of a thread and tile
  __shared__ __align__(16) float s_kv[2 * BN * LD];
  __shared__ float s_m[KW - 1][32], s_l[KW - 1][32];
  lds_nan_fill(s_kv, sizeof s_kv);
  float *s_k = s_kv, *s_v = s_kv + BN * LD;
  const Tile tl = find_tile<BM>(p, blocks);
  if (!tl.valid) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wq = wave & 1, wk = wave >> 1;
  const int g = lane >> 4, j = lane & 15;
  const int hk = tl.hq / (p.Hq / p.Hk);
  const int L = (int)tl.L;
  const int q0 = (int)tl.q0 + 16 * wq;      // the wave's first query
  const int tq = q0 + j;                    // this lane's query
  const float* kb_ = static_cast<const float*>(p.k) + tl.a * p.ld_k + hk * D;
  const float* vb_ = static_cast<const float*>(p.v) + tl.a * p.ld_v + hk * D;

  const int window = p.window > 0 && p.window < L ? (int)p.window : 0;
  int lo = window ? (int)tl.q0 - window + 1 : 0;      // first key that the tile sees
  lo = lo < 0 ? 0 : lo / BN * BN;
  const int stop = (int)tl.q0 + BM < L ? (int)tl.q0 + BM : L;
  float4 kr[NL], vr[NL];
  auto load_tile = [&](int k0) {            // rows past the sequence are zero: they may
#pragma unroll                              // belong to another one
    for (int e = 0; e < NL; ++e) {
      const int row = (e * NT + tid) / (D / 4), c = 4 * ((e * NT + tid) % (D / 4));
      kr[e] = vr[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 + row < L) {
        kr[e] = *reinterpret_cast<const float4*>(kb_ + (int64_t)(k0 + row) * p.ld_k + c);
        vr[e] = *reinterpret_cast<const float4*>(vb_ + (int64_t)(k0 + row) * p.ld_v + c);
      }
    }
  };
  load_tile(lo);
  Frag8<float> q[KB];
  {
    const float flip = p.scale < 0.f ? -1.f : 1.f;    // the scale below is positive
    const int row = tq < L ? tq : L - 1;
    const float* qp = static_cast<const float*>(p.q) + (tl.a + row) * p.ld_q + tl.hq * D + 8 * g;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      load_f32<8, float>(qp + 32 * kb, q[kb].v);
#pragma unroll
      for (int i = 0; i < 8; ++i) q[kb].v[i] *= flip;
    }
  }
  const float c_scale = fabsf(p.scale) * kLog2e;
  f32x4 o[MT];
#pragma unroll
  for (int c = 0; c < MT; ++c) o[c] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = kNone, l = 0.f;

  for (int k0 = lo; k0 < stop; k0 += BN) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < NL; ++e) {
      const int row = (e * NT + tid) / (D / 4), c = 4 * ((e * NT + tid) % (D / 4));
      lds_check(s_k + row * LD + c, 16);
      *reinterpret_cast<float4*>(s_k + row * LD + c) = kr[e];
      *reinterpret_cast<float4*>(s_v + row * LD + c) = vr[e];
    }
    __syncthreads();
    if (k0 + BN < stop) load_tile(k0 + BN);
    const int kw = k0 + 16 * wk;            // this wave's tokens
    if (kw > q0 + 15 || (window && kw + 15 <= q0 - window)) continue;   // nothing seen
    f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {       // two chains, so that products need not wait
      Frag8<float> a;
      load_f32<8, float>(s_k + (16 * wk + j) * LD + 32 * kb + 8 * g, a.v);
      mma32(acc[kb & 1], a, q[kb]);
    }
    float x[4], mx = -__builtin_huge_valf();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int u = kw + 4 * g + r;
      const bool seen = u <= tq && (!window || u > tq - window);
      x[r] = seen ? (acc[0][r] + acc[1][r]) * c_scale : -__builtin_huge_valf();
      mx = fmaxf(mx, x[r]);
    }
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
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float e = weight_of(x[r], m);
      l += e;
      const float* vl = s_v + (16 * wk + 4 * g + r) * LD + j;
#pragma unroll
      for (int c = 0; c < MT; ++c)
        o[c] = __builtin_amdgcn_mfma_f32_16x16x4f32(vl[16 * c], e, o[c], 0, 0, 0);
    }
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);

  // the other waves of the same queries hand over through the tiles
  static_assert((KW - 1) * 32 <= 2 * BN, "32 queries of sums for each");
  __syncthreads();
  if (wk > 0) {
#pragma unroll
    for (int c = 0; c < MT; ++c) {
      float* dst = s_kv + ((wk - 1) * 32 + 16 * wq + j) * LD + 16 * c + 4 * g;
      lds_check(dst, 16);
      *reinterpret_cast<float4*>(dst) = make_float4(o[c][0], o[c][1], o[c][2], o[c][3]);
    }
    if (g == 0) { s_m[wk - 1][16 * wq + j] = m; s_l[wk - 1][16 * wq + j] = l; }
  }
  __syncthreads();
  if (wk > 0) return;
#pragma unroll
  for (int w = 0; w < KW - 1; ++w) {
    const float m1 = s_m[w][16 * wq + j], mm = fmaxf(m, m1);
    const float f0 = exp2_fast(m - mm), f1 = exp2_fast(m1 - mm);
    m = mm;
    l = l * f0 + s_l[w][16 * wq + j] * f1;
#pragma unroll
    for (int c = 0; c < MT; ++c) {
      const float4 u = *reinterpret_cast<const float4*>(s_kv + (w * 32 + 16 * wq + j) * LD + 16 * c + 4 * g);
      o[c][0] = o[c][0] * f0 + u.x * f1;
      o[c][1] = o[c][1] * f0 + u.y * f1;
      o[c][2] = o[c][2] * f0 + u.z * f1;
      o[c][3] = o[c][3] * f0 + u.w * f1;
    }
  }
  const float inv = 1.f / l;                // a query sees itself, with a score above kNone: > 0
  float z = 0.f;                            // NaN where a sum is not finite
#pragma unroll
  for (int c = 0; c < MT; ++c)
#pragma unroll
    for (int r = 0; r < 4; ++r) z = __builtin_fmaf(o[c][r], 0.f, z);
  if (__any(z != z) && rows_again<float, D>(tl, hk, window, q0, 16, false)) return;
  float* op = static_cast<float*>(p.o) + ((tl.a + tq) * p.Hq + tl.hq) * (int64_t)D + 4 * g;
#pragma unroll
  for (int c = 0; c < MT; ++c)
    if (tq < L) store4<float>(op + 16 * c, o[c][0] * inv, o[c][1] * inv, o[c][2] * inv, o[c][3] * inv);
}

// ---------------------------------------------------------------------------
// bf16: v_mfma_f32_32x32x16_bf16, 32 queries to a wave, 128 to a workgroup (64
// where there are few, see split_bf16), key tiles of 64 tokens in LDS.
//
// Lane 32 h + i holds, of a 32 x 32 product, column i and rows
// 8 a + 4 h + b (a, b = 0..3), and supplies 8 k-values.  The score tile's rows
// of a 16-token block in a lane are tokens 4 h + b and 8 + 4 h + b, so V^T is
// read with the same 8 tokens: two transposing LDS reads of 4 tokens each.
//
// LDS rows are D elements; the 16-byte chunks of a row are permuted so that
// the lanes that read together fall on different banks (k_chunk: 16 rows at
// one chunk; v_chunk: 4 rows at 4 neighbouring chunks).
// ---------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ int k_chunk(int row, int c) {
  return D == 128 ? c ^ (row & 15) : c ^ ((row >> 1) & 7);
}
template <int D>
__device__ __forceinline__ int v_chunk(int row, int c) {
  return D == 128 ? c ^ ((row & 3) << 2) : c ^ (((row >> 1) & 1) << 2);
}

__device__ __forceinline__ bf16x4 read_tr16(const bf16* p) {
  lds_check(p, 8);
  typedef short v4s __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) v4s*)(p)));
}

// 16 bytes for each lane from base + voff + soff straight into LDS at
// lds + 16 * lane (lds is the same for the wave).  The load is counted by
// vmcnt like any other; the compiler does not know of it, so wait_tiles()
// stands before the barrier behind which the bytes are read.  m0 is set in the same
// block and named as clobbered; the compiler warns that it is a reserved register,
// which it sets before each use of its own.  (As an operand "{m0}" its writes are
// merged across the blocks, and tiles land in the wrong place.)
typedef int i32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void load_lds16(uint32_t lds, i32x4 base, uint32_t voff, uint32_t soff) {
#if __HIP_DEVICE_COMPILE__
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      ::"s"(lds), "v"(voff), "s"(base), "s"(soff) : "memory", "m0");
#pragma clang diagnostic pop
#endif
}
// This wave's loads have landed and its LDS reads are done; then all waves'.
__device__ __forceinline__ void wait_tiles() {
#if __HIP_DEVICE_COMPILE__
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
#endif
}
__device__ __forceinline__ i32x4 buffer_at(const void* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  i32x4 r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)u);
  r[1] = __builtin_amdgcn_readfirstlane((int)((u >> 32) & 0xffff));
  r[2] = -1;                              // offsets are kept in range by the caller
  r[3] = 0x00027000;
  return r;
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

// WIN: with the code of a window's mask (calls without a window are 1 to 2 % faster
// without it: 8 prompts of 4096 tokens 546 / 540 us, 4 short ones 11.0 / 10.7).
// SPLIT 2: 64 queries to a workgroup; waves 0 and 1 take the even key tiles, 2
// and 3 the odd ones, with a maximum and sum of their own, and join at the end.
//
// The loop over key tiles is pipelined by hand: while the weights of tile i
// are formed (VALU), the scores of tile i + 1 are on the matrix cores, and
// while the maximum of tile i + 1 is formed, tile i's product with V is.  K
// runs one tile ahead of V; both are double-buffered in LDS and loaded one
// iteration before they are read, with one barrier to an iteration.
template <int D, int SPLIT, bool WIN>
__global__ __launch_bounds__(kThreads, SPLIT == 2 ? 1 : D == 64 ? 3 : 2) void prefill_bf16_kernel(PrefillArgs p, uint32_t blocks) {
  constexpr int WQ = 4 / SPLIT;                       // waves with queries of their own
  constexpr int BM = 32 * WQ, BN = 64, KB = D / 16, MT = D / 32;
  constexpr int STEP = BN * SPLIT;                    // keys of an iteration
  constexpr int CH = D / 8;                           // 16-byte chunks of a row
  constexpr int NL = BN * CH / (64 * WQ);             // chunks a thread loads of a tile
  constexpr int RL = 64 * WQ / CH;                    // rows of one such load
  __shared__ __align__(16) bf16 s_k[2][STEP * D], s_v[2][STEP * D];
  lds_nan_fill(s_k, sizeof s_k);
  lds_nan_fill(s_v, sizeof s_v);
  const Tile tl = find_tile<BM>(p, blocks);
  if (!tl.valid) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wq = SPLIT == 1 ? wave : wave % WQ, wk = SPLIT == 1 ? 0 : wave / WQ;
  const int h = lane >> 5, i32 = lane & 31;
  const int hk = tl.hq / (p.Hq / p.Hk);
  const int L = __builtin_amdgcn_readfirstlane((int)tl.L);
  const int qt0 = __builtin_amdgcn_readfirstlane((int)tl.q0);
  const int q0 = qt0 + 32 * wq;             // the wave's first query
  const int tq = q0 + i32;                  // this lane's query
  const bf16* kb_ = static_cast<const bf16*>(p.k) + tl.a * p.ld_k + hk * D;
  const bf16* vb_ = static_cast<const bf16*>(p.v) + tl.a * p.ld_v + hk * D;

  const int window = WIN && p.window > 0 && p.window < L ? (int)p.window : 0;
  int lo = window ? qt0 - window + 1 : 0;             // first key that the tile sees
  lo = lo < 0 ? 0 : lo / BN * BN;
  const int stop = qt0 + BM < L ? qt0 + BM : L;
  // this wave needs keys before it; behind the prompt's end it has no queries: it
  // loads its share of the tiles and computes nothing
  const int mine = q0 >= L ? 0 : q0 + 32 < stop ? q0 + 32 : stop;

  // loads of one tile: row r0 + e RL, permuted so that LDS position pc of row r
  // gets chunk k_chunk(r, pc); rows past the sequence repeat its last one
  // (their scores are masked), so nothing of another sequence is read
  const int r0 = (SPLIT == 1 ? tid : tid % (64 * WQ)) / CH, pc = tid % CH;
  const uint32_t ck = 16 * k_chunk<D>(r0, pc), cv = 16 * v_chunk<D>(r0, pc);
  const uint32_t lk2 = (uint32_t)p.ld_k * 2, lv2 = (uint32_t)p.ld_v * 2;
  const uint32_t wave_lds = (uint32_t)wq * 1024;
  const uint32_t k_off = (uint32_t)r0 * lk2 + ck, v_off = (uint32_t)r0 * lv2 + cv;   // of a whole tile
  // K's chunks repeat after 16 rows: with 8 rows to a load, the odd loads' differ
  constexpr uint32_t ODD = D == 128 && RL == 8 ? 128 : 0;
  static_assert(RL % 16 == 0 || ODD, "the chunks of a thread's rows");
  const uint32_t k_odd = (uint32_t)r0 * lk2 + (ck ^ ODD);
  auto load_tile = [&](const bf16* base, int64_t ld, uint32_t ld2, uint32_t chunk, uint32_t odd,
                       const bf16* dst, int k0) {
    const i32x4 rs = buffer_at(base + k0 * ld);
    const uint32_t at = __builtin_amdgcn_readfirstlane(lds_address(dst)) + wave_lds;
    if (k0 + BN <= L) {
      const uint32_t voff[2] = {(uint32_t)r0 * ld2 + chunk, (uint32_t)r0 * ld2 + (chunk ^ odd)};
#pragma unroll
      for (int e = 0; e < NL; ++e)
        load_lds16(at + e * (1024 * WQ), rs, voff[e % 2], (uint32_t)(e * RL) * ld2);
    } else {
#pragma unroll
      for (int e = 0; e < NL; ++e) {
        const int row = r0 + e * RL < L - k0 ? r0 + e * RL : L - 1 - k0;
        load_lds16(at + e * (1024 * WQ), rs, (uint32_t)row * ld2 + (e % 2 ? chunk ^ odd : chunk), 0);
      }
    }
  };

  // The queries come in whole rows too, by way of the second key buffer (waves
  // 0 and 1) and the second value buffer: loads of a fragment's rows straight
  // into registers touch 64 rows each.
  const int lo_w = lo + BN * wk;            // this wave's first tile
  if (lo_w < stop) load_tile(kb_, p.ld_k, lk2, ck, ODD, s_k[0] + wk * BN * D, lo_w);
  constexpr int HALF = STEP / 32;           // waves whose queries fit into a key buffer
  bf16* sq = wave < HALF ? s_k[1] + wave * (32 * D) : s_v[1] + (wave - HALF) * (32 * D);
  {
    constexpr int RQ = 64 / CH;             // rows of a wave's load
    const i32x4 rs = buffer_at(static_cast<const bf16*>(p.q) + (tl.a + q0) * p.ld_q + tl.hq * D);
    const uint32_t at = __builtin_amdgcn_readfirstlane(lds_address(sq));
#pragma unroll
    for (int e = 0; e < 32 / RQ; ++e) {
      const int row = e * RQ + lane / CH;
      const int from = q0 + row < L ? row : L - 1 - q0;   // past the sequence: its last row
      if (q0 < L)                           // (a wave without a query loads none)
        load_lds16(at + e * 1024, rs, (uint32_t)from * (uint32_t)(p.ld_q * 2) +
                                                    16 * k_chunk<D>(row, lane % CH), 0);
    }
  }
  if (lo_w < stop) load_tile(vb_, p.ld_v, lv2, cv, 0u, s_v[0] + wk * BN * D, lo_w);
  wait_tiles();
  bf16x8 q[KB];
  {
    const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;   // the scale below is positive
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      const bf16* src = sq + i32 * D + 8 * k_chunk<D>(i32, 2 * kb + h);
      lds_check(src, 16);
      uint4 u = *reinterpret_cast<const uint4*>(src);
      u.x ^= flip; u.y ^= flip; u.z ^= flip; u.w ^= flip;
      q[kb] = __builtin_bit_cast(bf16x8, u);
    }
  }
  wait_tiles();                             // every wave has its queries
  if (lo_w + STEP < stop) load_tile(kb_, p.ld_k, lk2, ck, ODD, s_k[1] + wk * BN * D, lo_w + STEP);

  const float c_scale = fabsf(p.scale) * kLog2e;
  f32x16 o[MT];
#pragma unroll
  for (int c = 0; c < MT; ++c)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[c][r] = 0.f;
  float m = kNone, l = 0.f;
  bool huge = false;                        // some query's m was 2^24 or more (see above)

  auto scores = [&](const bf16* kt, f32x16* s) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) s[t][r] = 0.f;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int row = 32 * t + i32;
        const bf16* src = kt + row * D + 8 * k_chunk<D>(row, 2 * kb + h);
        lds_check(src, 16);
        s[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*reinterpret_cast<const bf16x8*>(src), q[kb],
                                                       s[t], 0, 0, 0);
      }
  };
  auto top = [&](const f32x16* s) {
    float mx = s[0][0];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[t][r]);
    return over_halves(mx) * c_scale;
  };

  f32x16 s[2];
  float mx = kNone;
  if (lo_w < mine) {
    check_true(q0 < L && lo_w < stop);      // the queries and the tile were loaded
    scores(s_k[0] + wk * BN * D, s);
    mx = top(s);
  }
  // One iteration: tile k0's scores are in s, V's buffer is `buf`; leaves the
  // next tile's scores in sn and their maximum in mx (behind the last tile: of what
  // the buffer holds, and nothing reads them).
  // INNER: the tiles to load exist and are whole; their loads are then spread
  // over the score products (all at once they keep a wave from its products for
  // as long as the address unit takes over four waves' 32 KB: 1.4 % of a 32K
  // prompt).
  auto step = [&](auto inner, int k0, int buf, f32x16* s, f32x16* sn) {
    constexpr bool INNER = decltype(inner)::value;
    wait_tiles();
    i32x4 rk, rv;
    uint32_t ak = 0, av = 0;
    if constexpr (INNER) {
      rk = buffer_at(kb_ + (k0 + 2 * STEP) * p.ld_k);
      rv = buffer_at(vb_ + (k0 + STEP) * p.ld_v);
      ak = __builtin_amdgcn_readfirstlane(lds_address(s_k[buf] + wk * BN * D)) + wave_lds;
      av = __builtin_amdgcn_readfirstlane(lds_address(s_v[buf ^ 1] + wk * BN * D)) + wave_lds;
    } else {
      if (k0 + 2 * STEP < stop)
        load_tile(kb_, p.ld_k, lk2, ck, ODD, s_k[buf] + wk * BN * D, k0 + 2 * STEP);
      if (k0 + STEP < stop)
        load_tile(vb_, p.ld_v, lv2, cv, 0u, s_v[buf ^ 1] + wk * BN * D, k0 + STEP);
      if (k0 >= mine) return;               // nothing left for this wave to see
    }
    check_true(q0 < L);
    constexpr int LP = 2 * KB / (2 * NL);   // score products to a load
    static_assert(!INNER || LP >= 1, "a place for every load");
    auto load_part = [&](int e) {           // K's loads, then V's
      if constexpr (INNER) {
        if (e < NL) load_lds16(ak + e * (1024 * WQ), rk, e % 2 ? k_odd : k_off, (uint32_t)(e * RL) * lk2);
        else if (e < 2 * NL) load_lds16(av + (e - NL) * (1024 * WQ), rv, v_off, (uint32_t)((e - NL) * RL) * lv2);
      }
    };
    // element (t, r) is token k0 + 4 h + at: not seen where at > tq - k0 - 4 h,
    // or at <= that less the window
    // (k0, the tiles and the queries' first are multiples of 64, so an inner tile ends
    // before the workgroup's queries; without the code of its mask a 32K prompt is 2 %
    // faster)
    const bool front = !INNER && k0 + BN - 1 > q0, back = window && k0 <= q0 + 31 - window;
    if (front) {
      const int last = tq - k0 - 4 * h;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (32 * t + 8 * (r / 4) + r % 4 > last) s[t][r] = -__builtin_huge_valf();
    }
    if (back) {
      const int before = tq - window - k0 - 4 * h;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (32 * t + 8 * (r / 4) + r % 4 <= before) s[t][r] = -__builtin_huge_valf();
    }
    if (front || back) mx = top(s);
    // The sums are kept relative to m, which need not be the maximum: it is
    // moved only when a score passes it by 2^8, so weights stay below 2^8 and
    // the output is rarely rescaled.
    if (__any(mx > m + 8.f)) {
      const float m_new = fmaxf(m, mx);
      const float alpha = exp2_fast(m - m_new);
      huge |= __any(fabsf(m_new) >= 0x1p24f && fabsf(m_new) < -kNone) != 0;
      m = m_new;
      l *= alpha;
#pragma unroll
      for (int c = 0; c < MT; ++c)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[c][r] *= alpha;
    }
    // One product to a line of this schedule, with LDS reads some products
    // ahead of their use and a share of the vector work behind each; the
    // compiler keeps the lines in order.
    constexpr int NQ = 2 * KB, NP = 4 * MT;   // products of scores and of the output
    constexpr int AK = 2, AV = 2;             // reads ahead (2 to 6 measure alike; 3 spill at D 64)
    constexpr int EW = 32 / NQ;               // weights to a score product
    bf16x8 kf[NQ], vf[NP], w[4];
    auto read_k = [&](int i) {
      const int row = 32 * (i % 2) + i32;
      const bf16* src = s_k[buf ^ 1] + wk * BN * D + row * D + 8 * k_chunk<D>(row, 2 * (i / 2) + h);
      lds_check(src, 16);
      kf[i] = *reinterpret_cast<const bf16x8*>(src);
    };
    auto read_v = [&](int j) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int li = lane & 15;
        const int row = 16 * (j / MT) + 8 * half + 4 * h + (li >> 2);
        const int col = 32 * (j % MT) + 16 * ((lane >> 4) & 1) + 4 * (li & 3);
        const bf16x4 u = read_tr16(s_v[buf] + wk * BN * D + row * D + 8 * v_chunk<D>(row, col / 8) + col % 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) vf[j][4 * half + i] = u[i];
      }
    };
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 16; ++r) sn[t][r] = 0.f;
#pragma unroll
    for (int i = 0; i < AK; ++i) read_k(i);
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      if (i + AK < NQ) read_k(i + AK);
      if (i >= NQ - AV) read_v(i - (NQ - AV));
      sn[i % 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[i], q[i / 2], sn[i % 2], 0, 0, 0);
      if constexpr (INNER) {
        if (i % LP == LP - 1) load_part(i / LP);
      }
#pragma unroll
      for (int e = EW * i; e < EW * i + EW; ++e) {
        const float x = exp2_fast(__builtin_fmaf(s[e / 16][e % 16], c_scale, -m));
        l += x;
        w[e / 8][e % 8] = (bf16)x;
      }
    }
    float top_n = -__builtin_huge_valf();
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      __builtin_amdgcn_sched_barrier(0);
      if (j + AV < NP) read_v(j + AV);
      o[j % MT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[j], w[j / MT], o[j % MT], 0, 0, 0);
      constexpr int EM = 32 / NP;
#pragma unroll
      for (int e = EM * j; e < EM * j + EM; ++e) top_n = fmaxf(top_n, sn[e / 16][e % 16]);
    }
    __builtin_amdgcn_sched_barrier(0);
    mx = over_halves(top_n) * c_scale;
  };
  f32x16 s1[2];
  int k0 = lo;
  const int dk = BN * wk;
  // (D 64 has no registers left for the two forms)
  for (; D == 128 && q0 < L && k0 + 3 * STEP < stop && k0 + 4 * STEP <= L; k0 += 2 * STEP) {
    step(std::bool_constant<D == 128>{}, k0 + dk, 0, s, s1);
    step(std::bool_constant<D == 128>{}, k0 + dk + STEP, 1, s1, s);
  }
  for (; k0 < stop; k0 += 2 * STEP) {
    step(std::false_type{}, k0 + dk, 0, s, s1);
    if (k0 + STEP < stop) step(std::false_type{}, k0 + dk + STEP, 1, s1, s);
  }
  l += __shfl_xor(l, 32);
  if constexpr (SPLIT == 2) {               // the second half hands over through V's tiles
    wait_tiles();
    float* so = reinterpret_cast<float*>(&s_v[0][0]) + wq * (16 * MT * 64) + lane;
    float* sm = reinterpret_cast<float*>(&s_k[1][0]) + wq * 128 + lane;
    uint32_t* s_huge = reinterpret_cast<uint32_t*>(&s_k[1][0]) + WQ * 128;
    static_assert(WQ * 16 * MT * 64 * sizeof(float) <= sizeof s_v && BM <= STEP, "the sums fit");
    if (wk == 1) {
#pragma unroll
      for (int c = 0; c < MT; ++c)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          lds_check(so + (16 * c + r) * 64, 4);
          so[(16 * c + r) * 64] = o[c][r];
        }
      sm[0] = m;
      sm[64] = l;
      if (lane == 0) s_huge[wq] = huge;
    }
    wait_tiles();
    if (wk == 1) return;
    huge |= s_huge[wq] != 0;
    const float m1 = sm[0], mm = fmaxf(m, m1);
    const float f0 = exp2_fast(m - mm), f1 = exp2_fast(m1 - mm);
    l = l * f0 + sm[64] * f1;
#pragma unroll
    for (int c = 0; c < MT; ++c)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[c][r] = o[c][r] * f0 + so[(16 * c + r) * 64] * f1;
  }
  const float inv = 1.f / l;                // a query sees itself, with a score above kNone: > 0
  // rows leave through LDS (this wave's part of the key tiles, which no wave
  // reads any more), so that a store covers whole rows
  if constexpr (SPLIT == 1) wait_tiles();
  if (q0 >= L) return;
  static_assert(BM <= 2 * STEP, "the waves' rows fit into the key tiles");
  float z[4] = {0.f, 0.f, 0.f, 0.f};        // NaN where a sum is not finite
#pragma unroll
  for (int c = 0; c < MT; ++c)
#pragma unroll
    for (int r = 0; r < 16; ++r) z[r % 4] = __builtin_fmaf(o[c][r], 0.f, z[r % 4]);
  z[0] += z[1] + (z[2] + z[3]);
  if ((huge || __any(z[0] != z[0])) && rows_again<bf16, D>(tl, hk, window, q0, 32, huge)) return;
  bf16* so = &s_k[0][0] + wq * 32 * D;
#pragma unroll
  for (int c = 0; c < MT; ++c)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      bf16* dst = so + i32 * D + 8 * ((4 * c + r / 4) ^ (i32 & (CH - 1))) + 4 * h;
      lds_check(dst, 8);
      store4<bf16>(dst, o[c][r] * inv, o[c][r + 1] * inv, o[c][r + 2] * inv, o[c][r + 3] * inv);
    }
  bf16* op = static_cast<bf16*>(p.o) + ((tl.a + q0) * p.Hq + tl.hq) * (int64_t)D;
#pragma unroll
  for (int e = 0; e < 32 * CH / 64; ++e) {
    const int row = (e * 64 + lane) / CH, c = (e * 64 + lane) % CH;
    if (q0 + row < L)
      *reinterpret_cast<uint4*>(op + row * (int64_t)p.Hq * D + 8 * c) =
          *reinterpret_cast<const uint4*>(so + row * D + 8 * (c ^ (row & (CH - 1))));
  }
}

int64_t blocks_of(int64_t N, int64_t total_T, int64_t Tseq, bool packed, int Hq, int64_t bm) {
  return (packed ? total_T / bm + N : N * ((Tseq + bm - 1) / bm)) * Hq;
}

// With few query tiles a CU has one workgroup or none, and the last tile's walk
// over its keys is the call's time: then more waves share a tile's keys.  It costs
// a tile twice the LDS and a hand-over, so not where a walk is short, nor where
// the tiles fill the CUs anyway.  The mean keys of a prompt's last query:
int64_t mean_keys(const PrefillArgs& a) {
  const int64_t len = a.cu_seqlens ? a.total_T / a.N : a.Tseq;
  return a.window > 0 && a.window < len ? a.window : len;
}
// bf16, us with 128 queries to a workgroup / 64 and the keys shared, d 128: 2048
// tokens, 8 heads 32.9 / 22.2; 512 tokens, 16 heads 13.0 / 10.9; 2 prompts of 704
// tokens in all, 12 heads 13.6 / 12.2; 4 of 128, 16 heads 8.1 / 7.7; with 256
// workgroups of the first kind: 4096 tokens, 8 heads 62 / 50, 1024 tokens, 32
// heads 21.6 / 22.8; with 512: 2048 tokens, 32 heads 46 / 67.  At d 64 two
// workgroups of the second kind fit a CU: 288, 2048 tokens, 18 heads 28.1 / 20.0;
// 384, 24 heads 28.8 / 25.9; 448, 28 heads 29.8 / 29.9; 315, 9 prompts of 640, 7
// heads 12.8 / 14.2.
bool split_bf16(int64_t blocks, int64_t keys, int d) {
  return blocks <= 256 ? keys >= 256 : d == 64 && blocks <= 384 && keys >= 768;
}
// fp32, us with 4 / 8 waves to 32 queries, d 128: 2352 tokens, 2 heads 138 / 121;
// 3 prompts of 257 tokens in all, 4 heads of 64 8.9 / 8.5; 24 prompts of 304 in all,
// 8 heads 8.4 / 9.4; with 512 workgroups: 2048 tokens, 8 heads 147 / 123; with 2048:
// 4096 tokens, 16 heads 677 / 853.
bool split_f32(int64_t blocks, int64_t keys) { return blocks <= 512 && keys >= 64; }

// rows_again reads PrefillArgs where a kernel's arguments begin.
using PrefillKernel = void (*)(PrefillArgs, uint32_t);
static_assert(std::is_same<decltype(&prefill_bf16_kernel<128, 1, true>), PrefillKernel>::value &&
                  std::is_same<decltype(&prefill_f32_kernel<128, 2>), PrefillKernel>::value,
              "PrefillArgs is the first argument");

template <int SPLIT>
void launch_bf16(const PrefillArgs& a, int64_t blocks, hipStream_t stream) {
  const dim3 grid((unsigned)blocks);
  const uint32_t n = (uint32_t)blocks;
  if (a.d == 128) {
    if (a.window) prefill_bf16_kernel<128, SPLIT, true><<<grid, kThreads, 0, stream>>>(a, n);
    else prefill_bf16_kernel<128, SPLIT, false><<<grid, kThreads, 0, stream>>>(a, n);
  } else {
    if (a.window) prefill_bf16_kernel<64, SPLIT, true><<<grid, kThreads, 0, stream>>>(a, n);
    else prefill_bf16_kernel<64, SPLIT, false><<<grid, kThreads, 0, stream>>>(a, n);
  }
}

}  // namespace

int64_t prefill_blocks(int64_t N, int64_t total_T, int64_t Tseq, bool packed, int Hq, DType io) {
  return blocks_of(N, total_T, Tseq, packed, Hq, io == DType::F32 ? 32 : 128);
}

hipError_t launch_attn_prefill(const PrefillArgs& a, hipStream_t stream) {
  const bool packed = a.cu_seqlens != nullptr;
  const int64_t blocks = prefill_blocks(a.N, a.total_T, a.Tseq, packed, a.Hq, a.io);
  const int64_t keys = mean_keys(a);
  const dim3 grid((unsigned)blocks);
  if (a.io == DType::F32) {
    if (split_f32(blocks, keys)) {
      if (a.d == 128) prefill_f32_kernel<128, 4><<<grid, 512, 0, stream>>>(a, (uint32_t)blocks);
      else prefill_f32_kernel<64, 4><<<grid, 512, 0, stream>>>(a, (uint32_t)blocks);
    } else {
      if (a.d == 128) prefill_f32_kernel<128, 2><<<grid, 256, 0, stream>>>(a, (uint32_t)blocks);
      else prefill_f32_kernel<64, 2><<<grid, 256, 0, stream>>>(a, (uint32_t)blocks);
    }
  } else if (split_bf16(blocks, keys, a.d)) {
    const int64_t twice = blocks_of(a.N, a.total_T, a.Tseq, packed, a.Hq, 64);
    launch_bf16<2>(a, twice, stream);
  } else {
    launch_bf16<1>(a, blocks, stream);
  }
  return hipGetLastError();
}

#ifdef GDN_CHECK
unsigned check_violations_attn_prefill() { return take_check_violations(); }
#endif

}  // namespace gdn
