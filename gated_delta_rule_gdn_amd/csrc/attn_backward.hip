// attn_backward.hip -- gradients of the causal softmax attention of
// attn_prefill.hip on gfx950.  With c = scale, p_ts = exp(c q_t . k_s - m_t) / l_t
// from the statistics that the forward left,
//
//   D_t = sum_s p_ts (d_o_t . v_s) = d_o_t . o_t
//   ds_ts = p_ts (d_o_t . v_s - D_t)
//   dq_t = c sum_s ds_ts k_s,   dk_s = c sum_t ds_ts q_t,   dv_s = sum_t p_ts d_o_t
//
// the last two over the query heads of the key head too.
//
// Two kernels form the probabilities again, each with the sums that it is after in
// registers: one walks the keys of a query tile (dq, and D and the statistics packed
// for the other), one the queries of a key tile (dk, dv).  That is 7 products of
// d x keys x queries where one kernel with both sums would do 5; but its dq (or dk and
// dv) would go through memory for every pair of tiles, as atomics, whose order changes
// the result, or as partial sums of four times the products' operands.  Here every sum
// has a fixed order.
//
// In both, what is summed over lies on the rows of the first products (S^T = K Q^T and
// dP^T = V dO^T for dq; S = Q K^T and dP = dO V^T for dk and dv), so p and ds are, as
// they lie in the accumulators, the k-values of the second products.
//
// 14 d flops to a key that a query sees, against a few bytes: bound by the matrix cores, at
// the clock that power leaves them (1.7 to 1.9 GHz), and by the waits between products, in
// which they are idle 41 to 51 % of the time.  Calls in a row, bf16, 16 heads of 128: a
// document of 16384 tokens over 2 key heads 3570 to 3660 us, 1050 to 1080 TFLOP/s (a plain
// product of 8192 x 8192 x 8192 reaches 1212); 8 prompts of 4096 tokens over 16 key heads
// 1970 to 1990 us, 970; 16 documents, 32768 tokens in all, a window of 2048 over 2 key heads
// 1210 to 1360 us by their lengths, 870 to 890.  Gradients in fp32 from bf16 rows: 2030 us
// for the 8 prompts, the document as before.  fp32, 4096 tokens, 16 heads of 128: 2200 us,
// 109 TFLOP/s (a product: 154).  Short documents are three launches and the walks of the
// longest one's tiles (29 of 282 tokens on average, 6 heads of 64 over 3: 52 to 55 us, traced
// 22 + 26 + 8).
#include <cmath>

#include "attn_shares.hpp"
#include "attn_tiles.hpp"

#include "hybrid_kernels.hpp"

namespace gdn {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ TileArgs tile_args(const AttnBwdArgs& p, int G) {
  return TileArgs{p.cu_seqlens, p.N, p.Tseq, p.total_T, p.window, p.Hk, G};
}

// One walk of a key tile: [k0, k0 + BK) of the sequence [a, a + L), steps [at, stop) of the
// `each` steps of each query head of the key head hk; its sums go to the outputs (slot -1)
// or to a slot of the workspace.
struct Walk {
  int64_t a;
  int L, k0, hk, each, at, stop, slot, pad;
};
// A worker's walks, and the tile that it begins and `behind` workers behind it go on with.
struct Worker {
  int first, count;
  int64_t row0;
  int rows, hk, behind, pad;
};
static_assert(sizeof(Walk) == 40 && sizeof(Worker) == 32, "10 and 8 floats");

// The workspace: 16 bytes for each query and head, the workers, their walks, and two
// partial tiles of dk and dv for each worker.
__host__ __device__ inline int64_t tiles_of(int64_t N, int64_t total_T, int64_t Tseq, bool packed, int64_t rows) {
  return packed ? total_T / rows + N : N * ((Tseq + rows - 1) / rows);
}
__device__ __forceinline__ uint4* aux_of(const AttnBwdArgs& p, int hq) {
  return reinterpret_cast<uint4*>(p.ws) + hq * p.total_T;
}
__device__ __forceinline__ Worker* workers_of(const AttnBwdArgs& p) {
  return reinterpret_cast<Worker*>(p.ws + 4 * p.total_T * p.Hq);
}
__device__ __forceinline__ Walk* walks_of(const AttnBwdArgs& p, int workers) {
  return reinterpret_cast<Walk*>(p.ws + 4 * p.total_T * p.Hq + 8 * workers);
}
__host__ __device__ inline int64_t walk_floats(int64_t tiles, int Hk, int workers) {
  return (10 * (tiles * Hk + workers) + 3) / 4 * 4;   // slots begin at 16 bytes
}
template <int D, int BK>
__device__ __forceinline__ float* slot_of(const AttnBwdArgs& p, int workers, int slot) {
  const int64_t tiles = tiles_of(p.N, p.total_T, p.Tseq, p.cu_seqlens != nullptr, BK);
  return p.ws + 4 * p.total_T * p.Hq + 8 * workers + walk_floats(tiles, p.Hk, workers) +
         (int64_t)slot * (BK * 2 * D);
}

// ---------------------------------------------------------------------------
// Who walks what.  A workgroup of the dk and dv kernel has either one key tile (`workers`
// 0, the dear ones first; see whole_tiles) or an equal share of all tiles' walks, in the order
// of sequence, key head and tile: then the first and the last walk of a share may be parts
// of one, whose sums go to the workspace and are joined in order by another kernel.  Shares
// that follow each other are on one XCD.  The shares are counted out by the first
// workgroups of the dq kernel, a wave to a worker.
// ---------------------------------------------------------------------------
constexpr int kLead = 4;                    // steps that a walk's beginning and end are worth
constexpr int64_t kLeast = 3;               // units of a share
constexpr int plan_blocks(int workers) { return (workers + 8 * 4 - 1) / (8 * 4) * 8; }   // whole rounds of the XCDs

__device__ __forceinline__ int64_t length_of(const AttnBwdArgs& p, int64_t i) {
  const int64_t l = clamp_i64(p.cu_seqlens[i + 1], 0, p.total_T) - clamp_i64(p.cu_seqlens[i], 0, p.total_T);
  return l > 0 ? l : 0;
}

template <int BK, int BQ>
__device__ __forceinline__ void plan_worker(const AttnBwdArgs& p, int workers, int worker) {
  if (worker >= workers) return;
  const int lane = threadIdx.x & 63;
  const WalkUnits u{p.window, BK, BQ, p.Hq / p.Hk, kLead};
  int64_t total;
  if (!p.cu_seqlens) {
    total = p.N * p.Hk * u.units(p.Tseq);
  } else {
    int64_t sum = 0;
    for (int64_t i = lane; i < p.N; i += 64) sum += u.units(length_of(p, i));
#pragma unroll
    for (int off = 32; off; off >>= 1) sum += __shfl_xor((long long)sum, off);
    total = sum * p.Hk;
  }
  const Shares s = shares_of(total, workers, kLeast);
  Worker me{0, 0, 0, 0, 0, 0, 0};
  int64_t x = 0, end = 0;
  if (worker < s.workers) {
    x = s.begin(worker);
    end = s.begin(worker + 1);
  }
  if (x < end) {
    // sequence n with its units [base, base + Hk per), its tile j of head hk from unit `from`
    // on; `tiles` before the sequence
    int64_t n = 0, base = 0, per = 1, a = 0, L = 0, tiles = 0;
    if (!p.cu_seqlens) {
      per = u.units(p.Tseq);
      n = x / (per * p.Hk);
      base = n * per * p.Hk;
      a = n * p.Tseq;
      L = p.Tseq;
      tiles = n * u.tiles(L);
    } else {
      for (int64_t i0 = 0; i0 < p.N; i0 += 64) {
        const int64_t l = i0 + lane < p.N ? length_of(p, i0 + lane) : 0;
        const int64_t mine = u.units(l) * p.Hk;
        int64_t upto = mine, tiles_to = u.tiles(l);
#pragma unroll
        for (int off = 1; off < 64; off *= 2) {
          const int64_t v = __shfl_up((long long)upto, off), t = __shfl_up((long long)tiles_to, off);
          if (lane >= off) { upto += v; tiles_to += t; }
        }
        const uint64_t m = __ballot(base + upto > x);
        if (m) {
          const int k = __ffsll((unsigned long long)m) - 1;
          n = i0 + k;
          L = read_lane(l, k);
          per = read_lane(mine, k) / p.Hk;
          base += read_lane(upto, k) - per * p.Hk;
          tiles += read_lane(tiles_to, k) - u.tiles(L);
          break;
        }
        base += read_lane(upto, 63);
        tiles += read_lane(tiles_to, 63);
      }
      a = clamp_i64(p.cu_seqlens[n], 0, p.total_T);
    }
    const int64_t r = x - base;
    int hk = (int)(r / per);
    int64_t j = u.tile_at(L, r - hk * per);
    int64_t from = base + hk * per + u.before(L, j);
    // each tile has a place of its own in the list, and each worker one more (ranges that
    // overlap can have more tiles than there is room for: those are not walked)
    const int64_t place = tiles * p.Hk + hk * u.tiles(L) + j + worker;
    const int64_t room = tiles_of(p.N, p.total_T, p.Tseq, p.cu_seqlens != nullptr, BK) * p.Hk + workers - place;
    me.first = room > 0 ? (int)place : 0;
    Walk* to = walks_of(p, workers) + me.first;
    while (x < end && me.count < room) {
      const WalkPart w = part_of(u, L, j, from, x, end);
      if (w.s1 > w.s0) {
        const Walk t{a, (int)L, (int)(j * BK), hk, (int)(w.all / u.G), (int)w.s0, (int)w.s1,
                     w.whole() ? -1 : 2 * worker + (w.s0 == 0), 0};
        if (lane == 0) to[me.count] = t;
        ++me.count;
        if (w.s0 == 0 && !w.whole()) {
          me.behind = s.owner(from + u.lead + w.all - 1) - worker;
          me.row0 = a + j * BK;
          me.rows = (int)(L - j * BK < BK ? L - j * BK : BK);
          me.hk = hk;
        }
      }
      x = w.next;
      from += u.lead + w.all;
      if (x < end && ++j == u.tiles(L)) {
        j = 0;
        if (++hk == p.Hk) {
          hk = 0;
          ++n;
          if (p.cu_seqlens) {
            while (n < p.N && length_of(p, n) == 0) ++n;
            if (n >= p.N) break;            // (offsets that changed under the call)
            a = clamp_i64(p.cu_seqlens[n], 0, p.total_T);
            L = length_of(p, n);
          } else {
            a += p.Tseq;
          }
        }
      }
    }
  }
  if (lane == 0) workers_of(p)[worker] = me;
}

// x, but what is computed from it is not taken out of a loop over walks: addresses kept
// through a walk would spill its sums.
__device__ __forceinline__ int each_walk(int x) {
#if __HIP_DEVICE_COMPILE__
  asm volatile("" : "+v"(x));
#endif
  return x;
}

// The walks of a workgroup: those of its worker, or its tile's.
template <int BK, int BQ>
struct Walks {
  int first, count;
  __device__ __forceinline__ Walks(const AttnBwdArgs& p, int workers) : first(0), count(1) {
    if (workers) {
      const int worker = blockIdx.x % kXcds * (workers / kXcds) + blockIdx.x / kXcds;   // (a multiple of kXcds)
      first = __builtin_amdgcn_readfirstlane(workers_of(p)[worker].first);
      count = __builtin_amdgcn_readfirstlane(workers_of(p)[worker].count);
    }
  }
  __device__ __forceinline__ Walk walk(const AttnBwdArgs& p, uint32_t blocks, int workers, int i) const {
    Walk w;
    if (workers) {
      w = walks_of(p, workers)[first + i];
      w.a = (int64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)w.a) |
            (int64_t)__builtin_amdgcn_readfirstlane((int)(w.a >> 32)) << 32;
    } else {
      const Tile t = find_tile<BK>(tile_args(p, 1), blockIdx.x, blocks);
      const WalkUnits u{p.window, BK, BQ, p.Hq / p.Hk, 0};
      // the first keys are seen by the most queries
      const int64_t j = t.valid ? (t.L + BK - 1) / BK - 1 - t.q0 / BK : 0;
      w.a = t.a; w.L = (int)t.L; w.k0 = (int)(j * BK); w.hk = t.hq;
      w.each = t.valid ? (int)u.steps(t.L, j) : 0;
      w.at = 0; w.stop = w.each * u.G; w.slot = -1;
    }
    w.L = __builtin_amdgcn_readfirstlane(w.L);
    w.k0 = __builtin_amdgcn_readfirstlane(w.k0);
    w.hk = __builtin_amdgcn_readfirstlane(w.hk);
    w.each = __builtin_amdgcn_readfirstlane(w.each);
    w.at = __builtin_amdgcn_readfirstlane(w.at);
    w.stop = __builtin_amdgcn_readfirstlane(w.stop);
    w.slot = __builtin_amdgcn_readfirstlane(w.slot);
    return w;
  }
};

// ---------------------------------------------------------------------------
// fp32: v_mfma_f32_16x16x4_f32, 32 queries (dq) or 32 keys (dk, dv) to a workgroup,
// tiles of 32 rows of the other in LDS (dq of few tiles: 64).  Waves 0 and 1 take 16 rows
// of their own over the first 16 rows of each tile, waves 2 and 3 (4 to 7) the same over the
// others, and their sums are added at the end.  (Every fragment from LDS serves one product: 4096 tokens, 16
// heads of 128 run at 0.71 of a plain product's rate.)
// ---------------------------------------------------------------------------
// KW pairs of waves share a tile's keys (see split_dq_f32).
template <int D, int KW>
__global__ __launch_bounds__(128 * KW, 2) void attn_dq_f32_kernel(AttnBwdArgs p, uint32_t blocks, int workers) {
  constexpr int kT = 128 * KW, BM = 32, BN = 16 * KW, LD = D + 4, KB = D / 32, MT = D / 16;
  constexpr int KEYS = 32, STEP = 32;       // of the dk and dv kernel
  constexpr int NL = BN * D / 4 / kT;
  __shared__ __align__(16) float s_kv[2 * BN * LD];
  lds_nan_fill(s_kv, sizeof s_kv);
  float *s_k = s_kv, *s_v = s_kv + BN * LD;
  const int G = p.Hq / p.Hk, plan = plan_blocks(workers);
  if ((int)blockIdx.x < plan) {
    if (threadIdx.x < 256) plan_worker<KEYS, STEP>(p, workers, 4 * blockIdx.x + (threadIdx.x >> 6));
    return;
  }
  const Tile tl = find_tile<BM>(tile_args(p, G), blockIdx.x - plan, blocks);
  if (!tl.valid) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wq = wave & 1, wk = wave >> 1;
  const int g = lane >> 4, j = lane & 15;
  const int hk = tl.hq / G, L = (int)tl.L;
  const int q0 = (int)tl.q0 + 16 * wq, tq = q0 + j;
  const float* kb_ = static_cast<const float*>(p.k) + tl.a * p.ld_k + hk * D;
  const float* vb_ = static_cast<const float*>(p.v) + tl.a * p.ld_v + hk * D;
  const int window = p.window > 0 && p.window < L ? (int)p.window : 0;
  int lo = window ? (int)tl.q0 - window + 1 : 0;
  lo = lo < 0 ? 0 : lo / BN * BN;
  const int stop = (int)tl.q0 + BM < L ? (int)tl.q0 + BM : L;
  float4 kr[NL], vr[NL];
  auto load_tile = [&](int k0) {            // rows past the sequence are zero
#pragma unroll
    for (int e = 0; e < NL; ++e) {
      const int row = (e * kT + tid) / (D / 4), c = 4 * ((e * kT + tid) % (D / 4));
      kr[e] = vr[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k0 + row < L) {
        kr[e] = *reinterpret_cast<const float4*>(kb_ + (int64_t)(k0 + row) * p.ld_k + c);
        vr[e] = *reinterpret_cast<const float4*>(vb_ + (int64_t)(k0 + row) * p.ld_v + c);
      }
    }
  };
  load_tile(lo);
  Frag8<float> q[KB], go[KB];
  float m, rl, dl = 0.f;
  {
    const int64_t row = tl.a + (tq < L ? tq : L - 1);
    const float* qp = static_cast<const float*>(p.q) + row * p.ld_q + tl.hq * D + 8 * g;
    const float* gp = static_cast<const float*>(p.d_o) + (row * p.Hq + tl.hq) * D + 8 * g;
    const float* op = static_cast<const float*>(p.o) + (row * p.Hq + tl.hq) * D + 8 * g;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      float o[8];
      load_f32<8, float>(qp + 32 * kb, q[kb].v);
      load_f32<8, float>(gp + 32 * kb, go[kb].v);
      load_f32<8, float>(op + 32 * kb, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) dl = __builtin_fmaf(go[kb].v[i], o[i], dl);
    }
    dl += __shfl_xor(dl, 16);
    dl += __shfl_xor(dl, 32);
    const float2 st = reinterpret_cast<const float2*>(p.stats)[row * p.Hq + tl.hq];
    m = st.x;
    rl = 1.f / st.y;
    if (wk == 0 && g == 0 && tq < L)
      reinterpret_cast<float4*>(aux_of(p, tl.hq))[row] = make_float4(m, rl, dl, 0.f);
  }
  const float c_scale = p.scale * kLog2e;
  f32x4 dq[MT];
#pragma unroll
  for (int c = 0; c < MT; ++c) dq[c] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int k0 = lo; k0 < stop; k0 += BN) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < NL; ++e) {
      const int row = (e * kT + tid) / (D / 4), c = 4 * ((e * kT + tid) % (D / 4));
      lds_check(s_v + row * LD + c, 16);
      *reinterpret_cast<float4*>(s_k + row * LD + c) = kr[e];
      *reinterpret_cast<float4*>(s_v + row * LD + c) = vr[e];
    }
    __syncthreads();
    if (k0 + BN < stop) load_tile(k0 + BN);
    const int kw = k0 + 16 * wk;
    if (kw > q0 + 15 || (window && kw + 15 <= q0 - window)) continue;   // nothing seen
    f32x4 s = {0.f, 0.f, 0.f, 0.f}, dp = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      Frag8<float> a;
      load_f32<8, float>(s_k + (16 * wk + j) * LD + 32 * kb + 8 * g, a.v);
      mma32(s, a, q[kb]);
      load_f32<8, float>(s_v + (16 * wk + j) * LD + 32 * kb + 8 * g, a.v);
      mma32(dp, a, go[kb]);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int u = kw + 4 * g + r;
      const bool seen = u <= tq && (!window || u > tq - window);
      const float pr = seen ? weight_of(s[r] * c_scale, m) * rl : 0.f;
      const float ds = pr * (dp[r] - dl);
      const float* kl = s_k + (16 * wk + 4 * g + r) * LD + j;
#pragma unroll
      for (int c = 0; c < MT; ++c)
        dq[c] = __builtin_amdgcn_mfma_f32_16x16x4f32(kl[16 * c], ds, dq[c], 0, 0, 0);
    }
  }
  __syncthreads();
  static_assert((KW - 1) * BM <= 2 * BN, "the sums fit");
  if (wk > 0) {
#pragma unroll
    for (int c = 0; c < MT; ++c) {
      float* dst = s_kv + ((wk - 1) * BM + 16 * wq + j) * LD + 16 * c + 4 * g;
      lds_check(dst, 16);
      *reinterpret_cast<float4*>(dst) = make_float4(dq[c][0], dq[c][1], dq[c][2], dq[c][3]);
    }
  }
  __syncthreads();
  if (wk > 0 || tq >= L) return;
  float* to = static_cast<float*>(p.dq) + (tl.a + tq) * p.ld_dq + tl.hq * D + 4 * g;
#pragma unroll
  for (int c = 0; c < MT; ++c) {
#pragma unroll
    for (int i = 0; i < KW - 1; ++i) {
      const float4 u = *reinterpret_cast<const float4*>(s_kv + (i * BM + 16 * wq + j) * LD + 16 * c + 4 * g);
      dq[c][0] += u.x; dq[c][1] += u.y; dq[c][2] += u.z; dq[c][3] += u.w;
    }
    store4<float>(to + 16 * c, dq[c][0] * p.scale, dq[c][1] * p.scale, dq[c][2] * p.scale, dq[c][3] * p.scale);
  }
}

// D 64: three workgroups to a CU (168 registers; the 171 that the compiler takes of itself
// leave room for two: 4096 tokens, 8 heads 693 -> 641 us with dq).
template <int D>
__global__ __launch_bounds__(kThreads, D == 64 ? 3 : 2) void attn_dkv_f32_kernel(AttnBwdArgs p, uint32_t blocks, int workers) {
  constexpr int BK = 32, BQ = 32, LD = D + 4, KB = D / 32, MT = D / 16;
  constexpr int NL = BQ * D / 4 / kThreads;
  __shared__ __align__(16) float s_qg[2 * BQ * LD];
  __shared__ __align__(16) float4 s_aux[BQ];
  lds_nan_fill(s_qg, sizeof s_qg);
  lds_nan_fill(s_aux, sizeof s_aux);
  float *s_q = s_qg, *s_g = s_qg + BQ * LD;
  const int G = p.Hq / p.Hk;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = wave & 1, wq = wave >> 1;
  const float c_scale = p.scale * kLog2e;
  const Walks<BK, BQ> walks(p, workers);
  for (int nth = 0; nth < walks.count; ++nth) {
    const Walk w = walks.walk(p, blocks, workers, nth);
    if (w.at >= w.stop) continue;
    const int tid = each_walk(threadIdx.x), lane = tid & 63, g = lane >> 4, j = lane & 15;
    const int hk = w.hk, L = w.L, k0 = w.k0;
    const int u0 = k0 + 16 * wk, tk = u0 + j;         // this lane's key
    const int window = p.window > 0 && p.window < L ? (int)p.window : 0;
    Frag8<float> k[KB], v[KB];
    {
      const int64_t row = w.a + (tk < L ? tk : L - 1);
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        load_f32<8, float>(static_cast<const float*>(p.k) + row * p.ld_k + hk * D + 32 * kb + 8 * g, k[kb].v);
        load_f32<8, float>(static_cast<const float*>(p.v) + row * p.ld_v + hk * D + 32 * kb + 8 * g, v[kb].v);
      }
    }
    f32x4 dk[MT], dv[MT];
#pragma unroll
    for (int c = 0; c < MT; ++c) dk[c] = dv[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    float4 qr[NL], gr[NL], ar;
    int head = w.at / w.each, tile = w.at - head * w.each;  // of the step to load
    int now = tile;                                         // of the step at hand
    auto load_tile = [&]() {                // rows past the sequence are zero
      const int t0 = k0 + tile * BQ, hq = hk * G + head;
#pragma unroll
      for (int e = 0; e < NL; ++e) {
        const int row = (e * kThreads + tid) / (D / 4), c = 4 * ((e * kThreads + tid) % (D / 4));
        qr[e] = gr[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t0 + row < L) {
          qr[e] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + (w.a + t0 + row) * p.ld_q + hq * D + c);
          gr[e] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.d_o) + ((w.a + t0 + row) * p.Hq + hq) * (int64_t)D + c);
        }
      }
      ar = make_float4(0.f, 0.f, 0.f, 0.f);
      if (tid < BQ && t0 + tid < L)
        ar = reinterpret_cast<const float4*>(aux_of(p, hq))[w.a + t0 + tid];
      if (++tile == w.each) { tile = 0; ++head; }
    };
    load_tile();
    for (int step = w.at; step < w.stop; ++step) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < NL; ++e) {
        const int row = (e * kThreads + tid) / (D / 4), c = 4 * ((e * kThreads + tid) % (D / 4));
        lds_check(s_g + row * LD + c, 16);
        *reinterpret_cast<float4*>(s_q + row * LD + c) = qr[e];
        *reinterpret_cast<float4*>(s_g + row * LD + c) = gr[e];
      }
      if (tid < BQ) {
        lds_check(s_aux + tid, 16);
        s_aux[tid] = ar;
      }
      __syncthreads();
      if (step + 1 < w.stop) load_tile();
      const int t0 = k0 + now * BQ + 16 * wq;         // this wave's queries
      if (++now == w.each) now = 0;
      if (t0 + 15 < u0 || t0 >= L || (window && t0 - window >= u0 + 15)) continue;
      f32x4 s = {0.f, 0.f, 0.f, 0.f}, dp = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        Frag8<float> a;
        load_f32<8, float>(s_q + (16 * wq + j) * LD + 32 * kb + 8 * g, a.v);
        mma32(s, a, k[kb]);
        load_f32<8, float>(s_g + (16 * wq + j) * LD + 32 * kb + 8 * g, a.v);
        mma32(dp, a, v[kb]);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * wq + 4 * g + r, t = t0 + 4 * g + r;
        lds_check(s_aux + row, 16);
        const float4 st = s_aux[row];
        const bool seen = tk <= t && t < L && (!window || tk > t - window);
        const float pr = seen ? weight_of(s[r] * c_scale, st.x) * st.y : 0.f;
        const float ds = pr * (dp[r] - st.z);
        const float *ql = s_q + row * LD + j, *gl = s_g + row * LD + j;
#pragma unroll
        for (int c = 0; c < MT; ++c) {
          dv[c] = __builtin_amdgcn_mfma_f32_16x16x4f32(gl[16 * c], pr, dv[c], 0, 0, 0);
          dk[c] = __builtin_amdgcn_mfma_f32_16x16x4f32(ql[16 * c], ds, dk[c], 0, 0, 0);
        }
      }
    }
    __syncthreads();
    if (wq == 1) {
#pragma unroll
      for (int c = 0; c < MT; ++c) {
        float* dst = s_qg + (16 * wk + j) * LD + 16 * c + 4 * g;
        lds_check(dst + BQ * LD, 16);
        *reinterpret_cast<float4*>(dst) = make_float4(dk[c][0], dk[c][1], dk[c][2], dk[c][3]);
        *reinterpret_cast<float4*>(dst + BQ * LD) = make_float4(dv[c][0], dv[c][1], dv[c][2], dv[c][3]);
      }
    }
    __syncthreads();
    if (wq == 0 && tk < L) {
      float *tok, *tov;
      if (w.slot < 0) {
        tok = static_cast<float*>(p.dk) + (w.a + tk) * p.ld_dk + hk * D;
        tov = static_cast<float*>(p.dv) + (w.a + tk) * p.ld_dv + hk * D;
      } else {
        tok = slot_of<D, BK>(p, workers, w.slot) + (tk - k0) * (2 * D);
        tov = tok + D;
      }
#pragma unroll
      for (int c = 0; c < MT; ++c) {
        const float* src = s_qg + (16 * wk + j) * LD + 16 * c + 4 * g;
        const float4 a = *reinterpret_cast<const float4*>(src);
        const float4 b = *reinterpret_cast<const float4*>(src + BQ * LD);
        store4<float>(tok + 16 * c + 4 * g, (dk[c][0] + a.x) * p.scale, (dk[c][1] + a.y) * p.scale,
                      (dk[c][2] + a.z) * p.scale, (dk[c][3] + a.w) * p.scale);
        store4<float>(tov + 16 * c + 4 * g, dv[c][0] + b.x, dv[c][1] + b.y, dv[c][2] + b.z, dv[c][3] + b.w);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// bf16: v_mfma_f32_32x32x16_bf16, 32 queries (dq) or keys (dk, dv) to a wave, 128 to
// a workgroup, tiles of 64 rows of the other, double-buffered in LDS.  p and ds are
// rounded to bf16 for the second products, half a step of 2^-8 of each like the
// outputs' own rounding.
//
// Lane 32 h + i holds, of a 32 x 32 product, column i and rows 8 a + 4 h + b
// (a, b = 0..3), and supplies 8 k-values: rows 4 h + b and 8 + 4 h + b of a block of
// 16, so the other operand of the second products is read with the same 8 rows, by two
// transposing LDS reads of 4 rows each.
//
// Every tile is read by rows and transposed.  Its 16-byte chunks are permuted so
// that both kinds of reads fall on different banks: 16 rows at one chunk go to 16
// places, and 4 neighbouring rows at 4 neighbouring chunks too.
// ---------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ int chunk_at(int row, int c) {
  return D == 128 ? c ^ ((row & 3) << 2 | ((row >> 2) & 3)) : c ^ (((row >> 1) & 1) << 2 | ((row >> 2) & 3));
}

// A tile of 64 rows of D elements, `rows` of them there (the last one repeats: what
// it gives is masked), into LDS by a workgroup.
template <int D>
__device__ __forceinline__ void load_tile64(const bf16* base, uint32_t ld2, int rows, const bf16* dst, int tid) {
  constexpr int CH = D / 8, RL = kThreads / CH, NL = 64 / RL;
  const i32x4 rs = buffer_at(base);
  const uint32_t at = __builtin_amdgcn_readfirstlane(lds_address(dst)) +
                      1024 * __builtin_amdgcn_readfirstlane(tid >> 6);
#pragma unroll
  for (int e = 0; e < NL; ++e) {
    const int r = e * RL + tid / CH;
    load_lds16(at + e * 4096, rs, (uint32_t)(r < rows ? r : rows - 1) * ld2 + 16 * chunk_at<D>(r, tid % CH), 0);
  }
}

// The rows [r0, r0 + 32) of a tile as the first operand of a product over d, and the
// rows [r0, r0 + 16) transposed, columns [32 c, +32), as that of one over rows.
template <int D>
__device__ __forceinline__ bf16x8 read_rows(const bf16* tile, int r0, int kb, int lane) {
  const int row = r0 + (lane & 31);
  const bf16* src = tile + row * D + 8 * chunk_at<D>(row, 2 * kb + (lane >> 5));
  lds_check(src, 16);
  return *reinterpret_cast<const bf16x8*>(src);
}
template <int D>
__device__ __forceinline__ bf16x8 read_columns(const bf16* tile, int r0, int c, int lane) {
  bf16x8 f;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int li = lane & 15;
    const int row = r0 + 8 * half + 4 * (lane >> 5) + (li >> 2);
    const int col = 32 * c + 16 * ((lane >> 4) & 1) + 4 * (li & 3);
    const bf16x4 u = read_tr16(tile + row * D + 8 * chunk_at<D>(row, col / 8) + col % 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[4 * half + i] = u[i];
  }
  return f;
}

// x as three bf16 terms (24 bits).
__device__ __forceinline__ uint2 three_terms(float x) {
  const bf16 a = (bf16)x;
  const float r = x - (float)a;
  const bf16 b = (bf16)r;
  const bf16x4 t = {a, b, (bf16)(r - (float)b), (bf16)0.f};
  return __builtin_bit_cast(uint2, t);
}

// 32 rows of a wave, row i32 in the lanes i32 and 32 + i32 as the products leave it, times
// f to memory by way of 64 D bytes (fp32: 128 D) of LDS of its own.
template <int D, typename TG>
__device__ __forceinline__ void rows_out(bf16* lds, const f32x16* acc, float f, TG* to, int64_t ld, int rows, int lane) {
  constexpr int N = 16 / sizeof(TG), CH = D / N;      // elements of a chunk, chunks of a row
  TG* so = reinterpret_cast<TG*>(lds);
  const int h = lane >> 5, i32 = lane & 31;
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      const int at = 32 * c + 2 * r + 4 * h;
      TG* dst = so + i32 * D + N * ((at / N) ^ (i32 & 7)) + at % N;
      lds_check(dst, 4 * sizeof(TG));
      store4<TG>(dst, acc[c][r] * f, acc[c][r + 1] * f, acc[c][r + 2] * f, acc[c][r + 3] * f);
    }
#pragma unroll
  for (int e = 0; e < 32 * CH / 64; ++e) {
    const int row = (e * 64 + lane) / CH, c = (e * 64 + lane) % CH;
    const TG* src = so + row * D + N * (c ^ (row & 7));
    lds_check(src, 16);
    if (row < rows) *reinterpret_cast<uint4*>(to + row * ld + N * c) = *reinterpret_cast<const uint4*>(src);
  }
}

// Two workgroups to a CU hide each other's waits.  D is formed from outputs of 16 bits (see
// low_bytes): from bf16 alone a gradient's error was 3.1e-3 of its norm instead of 2.7e-3 for
// documents of 16 tokens.  3 products: 970 TFLOP/s for 8 prompts of 4096 tokens, 16 heads of
// 128, 1080 to 1100 for a document of 16384.
// SPLIT 2: 64 queries to a workgroup, each 32 of them to two waves that take 32 keys of a
// tile each and add their sums at the end (see split_dq).
template <int D, typename TG, int SPLIT>
__global__ __launch_bounds__(kThreads, 2) void attn_dq_bf16_kernel(AttnBwdArgs p, uint32_t blocks, int workers) {
  constexpr int BM = 128 / SPLIT, BN = 64, KB = D / 16, MT = D / 32;
  constexpr int KEYS = 128, STEP = 64;      // of the dk and dv kernel
  __shared__ __align__(16) bf16 s_k[2][BN * D], s_v[2][BN * D];
  lds_nan_fill(s_k, sizeof s_k);
  lds_nan_fill(s_v, sizeof s_v);
  const int G = p.Hq / p.Hk, plan = plan_blocks(workers);
  if ((int)blockIdx.x < plan) {
    plan_worker<KEYS, STEP>(p, workers, 4 * blockIdx.x + (threadIdx.x >> 6));
    return;
  }
  const Tile tl = find_tile<BM>(tile_args(p, G), blockIdx.x - plan, blocks);
  if (!tl.valid) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, i32 = lane & 31;
  const int hk = tl.hq / G;
  const int L = __builtin_amdgcn_readfirstlane((int)tl.L);
  const int qt0 = __builtin_amdgcn_readfirstlane((int)tl.q0);
  const int q0 = qt0 + 32 * (wave / SPLIT), tq = q0 + i32, part = wave % SPLIT;
  const bf16* kb_ = static_cast<const bf16*>(p.k) + tl.a * p.ld_k + hk * D;
  const bf16* vb_ = static_cast<const bf16*>(p.v) + tl.a * p.ld_v + hk * D;
  const uint32_t lk2 = (uint32_t)p.ld_k * 2, lv2 = (uint32_t)p.ld_v * 2;
  const int window = p.window > 0 && p.window < L ? (int)p.window : 0;
  int lo = window ? qt0 - window + 1 : 0;
  lo = lo < 0 ? 0 : lo / BN * BN;
  const int stop = qt0 + BM < L ? qt0 + BM : L;
  load_tile64<D>(kb_ + lo * p.ld_k, lk2, L - lo, s_k[0], tid);
  load_tile64<D>(vb_ + lo * p.ld_v, lv2, L - lo, s_v[0], tid);

  const float c_scale = p.scale * kLog2e;
  bf16x8 q[KB], go[KB];
  float lse, dl = 0.f;
  {
    uint4 o[KB];
    uint2 low[KB];
    const int64_t row = tl.a + (tq < L ? tq : L - 1);
    const bf16* qp = static_cast<const bf16*>(p.q) + row * p.ld_q + tl.hq * D + 8 * h;
    const bf16* gp = static_cast<const bf16*>(p.d_o) + (row * p.Hq + tl.hq) * D + 8 * h;
    const bf16* op = static_cast<const bf16*>(p.o) + (row * p.Hq + tl.hq) * D + 8 * h;
    const uint8_t* lp = reinterpret_cast<const uint8_t*>(p.stats + 2 * p.total_T * p.Hq) +
                        (row * p.Hq + tl.hq) * D + 8 * h;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      q[kb] = *reinterpret_cast<const bf16x8*>(qp + 16 * kb);
      go[kb] = *reinterpret_cast<const bf16x8*>(gp + 16 * kb);
      o[kb] = *reinterpret_cast<const uint4*>(op + 16 * kb);
      low[kb] = *reinterpret_cast<const uint2*>(lp + 16 * kb);
    }
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      const float2 x[4] = {with_low_bytes<0>(o[kb].x, low[kb].x), with_low_bytes<2>(o[kb].y, low[kb].x),
                           with_low_bytes<0>(o[kb].z, low[kb].y), with_low_bytes<2>(o[kb].w, low[kb].y)};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        dl = __builtin_fmaf((float)go[kb][2 * i + 1], x[i].y, __builtin_fmaf((float)go[kb][2 * i], x[i].x, dl));
    }
    dl += __shfl_xor(dl, 32);
    const float2 st = reinterpret_cast<const float2*>(p.stats)[row * p.Hq + tl.hq];
    lse = st.x + __builtin_amdgcn_logf(st.y);
    if (h == 0 && part == 0 && tq < L) {
      const uint2 a = three_terms(-lse / c_scale), b = three_terms(-dl);
      aux_of(p, tl.hq)[row] = make_uint4(a.x, a.y, b.x, b.y);
    }
  }
  f32x16 dq[MT];
#pragma unroll
  for (int c = 0; c < MT; ++c)
#pragma unroll
    for (int r = 0; r < 16; ++r) dq[c][r] = 0.f;

  int buf = 0;
  for (int k0 = lo; k0 < stop; k0 += BN, buf ^= 1) {
    wait_tiles();
    if (k0 + BN < stop) {
      load_tile64<D>(kb_ + (k0 + BN) * p.ld_k, lk2, L - k0 - BN, s_k[buf ^ 1], tid);
      load_tile64<D>(vb_ + (k0 + BN) * p.ld_v, lv2, L - k0 - BN, s_v[buf ^ 1], tid);
    }
    if (q0 >= L) continue;
#pragma unroll
    for (int at = 0; at < BN; at += 32 * SPLIT) {
      const int sub = at + 32 * part, kw = k0 + sub;
      if (kw > q0 + 31 || (window && kw + 31 <= q0 - window)) continue;   // nothing seen
      f32x16 s, dp;
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = dp[r] = 0.f;
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(read_rows<D>(s_k[buf], sub, kb, lane), q[kb], s, 0, 0, 0);
        dp = __builtin_amdgcn_mfma_f32_32x32x16_bf16(read_rows<D>(s_v[buf], sub, kb, lane), go[kb], dp, 0, 0, 0);
      }
      if (kw + 31 > q0 || (window && kw <= q0 + 31 - window)) {
        const int last = tq - kw - 4 * h, before = window ? last - window : -1;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int u = 8 * (r / 4) + r % 4;
          if (u > last || u <= before) s[r] = -__builtin_huge_valf() * c_scale;
        }
      }
      bf16x8 ds[2];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float pr = exp2_fast(__builtin_fmaf(s[r], c_scale, -lse));
        ds[r / 8][r % 8] = (bf16)(pr * (dp[r] - dl));
      }
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int c = 0; c < MT; ++c)
          dq[c] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(read_columns<D>(s_k[buf], sub + 16 * b, c, lane), ds[b], dq[c], 0, 0, 0);
    }
  }
  wait_tiles();                             // the key tiles are free
  static_assert(sizeof s_k + sizeof s_v >= BM * D * sizeof(TG), "the rows fit");
  bf16* mine = (wave < 2 ? s_k[0] : s_v[0]) + (wave & 1) * BN * D;
  if constexpr (SPLIT == 2) {               // both waves of 32 queries have tiles of their own
    static_assert(sizeof s_k >= 32 * D * sizeof(float) && sizeof s_v >= 32 * D * sizeof(float), "the sums fit");
    float4* sums = reinterpret_cast<float4*>(wave < 2 ? s_k[0] : s_v[0]) + lane;
#pragma unroll
    for (int i = 0; i < 4 * MT; ++i) {
      const f32x16& x = dq[i / 4];
      const int r = i % 4 * 4;
      lds_check(sums + 64 * i, 16);
      if (part == 1) sums[64 * i] = make_float4(x[r], x[r + 1], x[r + 2], x[r + 3]);
    }
    __syncthreads();
    if (part == 1) return;
#pragma unroll
    for (int i = 0; i < 4 * MT; ++i) {
      f32x16& x = dq[i / 4];
      const int r = i % 4 * 4;
      lds_check(sums + 64 * i, 16);
      const float4 y = sums[64 * i];
      x[r] += y.x; x[r + 1] += y.y; x[r + 2] += y.z; x[r + 3] += y.w;
    }
  }
  if (q0 >= L) return;
  rows_out<D>(mine, dq, p.scale, static_cast<TG*>(p.dq) + (tl.a + q0) * p.ld_dq + tl.hq * D, p.ld_dq, L - q0, lane);
}

// Where a lane reads from a tile in LDS.  Rows: row i32, its 16-byte chunk 2 kb + h, is
// at rows ^ 32 kb; a tile's rows are 2 D bytes and its base a multiple of that, so the
// permutation's exclusive or goes through the whole address.  Columns [32 c, +32) of the
// rows [16 b, +16), transposed: at (cols ^ 64 c ^ 32 half) + (16 b + 8 half) 2 D.
struct LaneReads {
  uint32_t rows, cols;
};
template <int D>
__device__ __forceinline__ LaneReads lane_reads(uint32_t base, int lane) {
  const int h = lane >> 5, i32 = lane & 31, li = lane & 15;
  const int row = 4 * h + (li >> 2), chunk = 2 * ((lane >> 4) & 1) + ((li & 3) >> 1);
  return LaneReads{base + i32 * 2 * D + 16 * chunk_at<D>(i32, h),
                   base + row * 2 * D + 16 * chunk_at<D>(row, chunk) + 8 * (li & 1)};
}
template <typename T>
__device__ __forceinline__ T lds_read(uint32_t at) {
  T x{};
#if __HIP_DEVICE_COMPILE__
#ifdef GDN_CHECK
  check_true(at + sizeof(T) <= __builtin_amdgcn_groupstaticsize());
#endif
  x = *(const __attribute__((address_space(3))) T*)at;
#endif
  return x;
}
template <int D>
__device__ __forceinline__ bf16x8 rows_at(uint32_t rows, int kb, int offset) {
  return lds_read<bf16x8>((rows ^ (32 * kb)) + offset);
}
template <int D>
__device__ __forceinline__ bf16x8 columns_at(uint32_t cols, int b, int c, int offset) {
  bf16x8 f{};
#if __HIP_DEVICE_COMPILE__
  typedef short v4s __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint32_t at = (cols ^ (64 * c + 32 * half)) + (16 * b + 8 * half) * 2 * D + offset;
#ifdef GDN_CHECK
    check_true(at + 8 <= __builtin_amdgcn_groupstaticsize());
#endif
    const bf16x4 u = __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) v4s*)at));
#pragma unroll
    for (int i = 0; i < 4; ++i) f[4 * half + i] = u[i];
  }
#endif
  return f;
}

// The statistics enter the first products: a 17th block of 16 k-values holds, of each
// query, -(m + log2 l) / (c log2 e) and -D in three bf16 terms each, and ones on the
// side of the keys.  So the products give c q . k - m - log2 l (over c) and
// d_o . v - D without a vector operation, and without the 8 LDS reads that would bring
// them to the lanes, whose 16 rows are all different queries.
//
// Products with their registers chosen: sums that stay, and keys and values, in accumulation
// registers, which the vector unit does not see (the compiler would move them there and
// back for every product), scores in vector registers.  The compiler knows nothing of what
// a product takes, so:
//  - operands that the vector unit wrote go through settle() first (2 wait states);
//  - results are read by it behind 8 further products or more, or behind products_done()
//    (11 wait states); all these are volatile, so they keep their order, and in between
//    results are operands of nothing else;
//  - a sum comes around again 2 products later at the earliest, which needs no wait.
__device__ __forceinline__ void product_v0(f32x16& acc, const bf16x8& a, const bf16x8& b) {
#if __HIP_DEVICE_COMPILE__
  asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, 0" : "=&v"(acc) : "v"(a), "a"(b));
#endif
}
__device__ __forceinline__ void product_v(f32x16& acc, const bf16x8& a, const bf16x8& b) {
#if __HIP_DEVICE_COMPILE__
  asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+v"(acc) : "v"(a), "a"(b));
#endif
}
__device__ __forceinline__ void product_a(f32x16& acc, const bf16x8& a, const bf16x8& b) {
#if __HIP_DEVICE_COMPILE__
  asm volatile("v_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
#endif
}
__device__ __forceinline__ void settle(bf16x8& a, bf16x8& b) {
#if __HIP_DEVICE_COMPILE__
  asm volatile("s_nop 1" : "+v"(a), "+v"(b));
#endif
}
// Behind it the sums can be read, or copied by the compiler: it stands at the end of each
// loop that adds to them, since copies may be made anywhere behind that.
template <int N>
__device__ __forceinline__ void products_done(f32x16* a, f32x16* b) {
#if __HIP_DEVICE_COMPILE__
  if constexpr (N == 4)
    asm volatile("s_nop 11" : "+a"(a[0]), "+a"(a[1]), "+a"(a[2]), "+a"(a[3]), "+a"(b[0]), "+a"(b[1]), "+a"(b[2]), "+a"(b[3]));
  else
    asm volatile("s_nop 11" : "+a"(a[0]), "+a"(a[1]), "+a"(b[0]), "+a"(b[1]));
#endif
}
__device__ __forceinline__ void products_done(f32x16& a, f32x16& b) {
#if __HIP_DEVICE_COMPILE__
  asm volatile("s_nop 11" : "+v"(a), "+v"(b));
#endif
}
// Both have been read from LDS: one wait instead of two.
__device__ __forceinline__ void both_there(const bf16x8& a, const bf16x8& b) {
#if __HIP_DEVICE_COMPILE__
  asm volatile("" ::"v"(a), "v"(b));
#endif
}
// What is behind reads x where it stands now.
__device__ __forceinline__ void behind_v(f32x16& x) {
#if __HIP_DEVICE_COMPILE__
  asm volatile("" : "+v"(x));
#endif
}
__device__ __forceinline__ void keep_a(bf16x8& x) {
#if __HIP_DEVICE_COMPILE__
  asm volatile("" : "+a"(x));
#endif
}

// One wave to a SIMD: two sums of 32 keys x D and the keys and values themselves take
// 192 registers.  What hides latencies instead is a pipeline by hand over blocks of 32
// queries: the first products of the next block, with the weights of this one formed
// between them, then this one's second products; every LDS read some products ahead of its
// use; tiles in four buffers in LDS: the one in use, the next, whose first rows are read ahead
// of it, and two on their way (the last of them into the buffer that the tile before this one
// has left).  4 products: 850 to 890 TFLOP/s for 8 prompts of 4096 tokens, 16 heads of 128,
// 1030 to 1060 for a document of 16384 tokens (two waves to a SIMD, as the compiler schedules
// them, 640 and 690).  Of the 2.0 us that a step of 64 queries takes the products alone are
// 1.3, at the 1.7 GHz that power leaves them.  With the LDS reads, seven eighths of the weights
// or the loads and barriers left out it takes 1.8, 1.8 and 1.7.
template <int D, typename TG>
__global__ __launch_bounds__(kThreads, D == 64 ? 2 : 1) void attn_dkv_bf16_kernel(AttnBwdArgs p, uint32_t blocks, int workers) {
  constexpr int BK = 128, BQ = 64, KB = D / 16, MT = D / 32;
  constexpr int GO = BQ * D * 2;            // d_o behind q in a buffer
  constexpr int BUF = 2 * GO;
  constexpr int NB = 4;                     // buffers
  constexpr int LOADS = 2 * BQ * D / 8 / kThreads + 1;   // of a wave and tile
  __shared__ __align__(1024) bf16 s_t[NB][2 * BQ * D];
  __shared__ __align__(1024) uint4 s_aux[NB][BQ];
  lds_nan_fill(s_t, sizeof s_t);
  lds_nan_fill(s_aux, sizeof s_aux);
  const int G = p.Hq / p.Hk;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float c_scale = p.scale * kLog2e;
  const uint32_t lq2 = (uint32_t)p.ld_q * 2, lg2 = (uint32_t)p.Hq * D * 2;
  // a thread's part of a tile: row r0 and every RL-th behind it, whose chunks are the same
  constexpr int CH = D / 8, RL = kThreads / CH, NL = BQ / RL;
  static_assert(RL % 16 == 0, "chunks repeat after 16 rows");
  const int r0 = threadIdx.x / CH;
  const uint32_t chunk = 16 * chunk_at<D>(r0, threadIdx.x % CH);
  const uint32_t off_q = r0 * lq2 + chunk, off_g = r0 * lg2 + chunk;
  const uint32_t lds_t = __builtin_amdgcn_readfirstlane(lds_address(s_t)) + 1024 * wave;
  const uint32_t lds_aux = __builtin_amdgcn_readfirstlane(lds_address(s_aux)) + BQ * 4 * wave;

  // lanes 0..31 supply the terms, those of m and l first; what 32..63 supply counts for nothing
  const uint32_t one = 0x3f80;              // 1 in bf16
  const bool low = (threadIdx.x & 32) == 0;
  bf16x8 ones_s = __builtin_bit_cast(bf16x8, make_uint4(low ? one << 16 | one : 0, low ? one : 0, 0, 0));
  bf16x8 ones_d = __builtin_bit_cast(bf16x8, make_uint4(0, 0, low ? one << 16 | one : 0, low ? one : 0));
  const LaneReads at = lane_reads<D>(lds_address(s_t), threadIdx.x & 63);
  const uint32_t at_aux = lds_address(s_aux) + 16 * (threadIdx.x & 31);

  auto statistics = [&](uint32_t block) { return lds_read<bf16x8>(at_aux + block); };   // of 32 queries
  keep_a(ones_s);
  keep_a(ones_d);
  constexpr int NF = 2 * KB, NS = 4 * MT;   // first and second products of a block
  constexpr int AF = 4, AS = 4;             // reads ahead
  constexpr int E1 = 12;                    // weights' slots between first products; the others behind them
  constexpr uint32_t HALF = 64 * D, HALF_AUX = 512;   // the second block of a buffer
  const Walks<BK, BQ> walks(p, workers);
  for (int nth = 0; nth < walks.count; ++nth) {
  const Walk w = walks.walk(p, blocks, workers, nth);
  if (w.at >= w.stop) continue;
  const int tid = each_walk(threadIdx.x), lane = tid & 63, h = lane >> 5, i32 = lane & 31;
  const int hk = w.hk, L = w.L, k0 = w.k0;
  const int u0 = k0 + 32 * wave, tk = u0 + i32;       // this lane's key
  const int window = p.window > 0 && p.window < L ? (int)p.window : 0;
  if (nth > 0) wait_tiles();                // no wave reads a buffer any more
  int head = w.at / w.each, tile = w.at - head * w.each;   // of the step to load
  int now = tile;                                          // of the step at hand
  const bf16 *q_at, *g_at;                  // that step's first rows
  const uint4* aux_at;
  auto head_at = [&]() {
    const int hq = hk * G + head;
    const int64_t row = w.a + k0 + tile * BQ;
    q_at = static_cast<const bf16*>(p.q) + row * p.ld_q + hq * D;
    g_at = static_cast<const bf16*>(p.d_o) + (row * p.Hq + hq) * (int64_t)D;
    aux_at = aux_of(p, hq) + row;
  };
  head_at();
  auto load_step = [&](int buf) {
    const i32x4 rq = buffer_at(q_at), rg = buffer_at(g_at), ra = buffer_at(aux_at);
    const uint32_t to = lds_t + buf * BUF, to_aux = lds_aux + buf * (BQ * 16);
    const int rows = L - k0 - tile * BQ;    // that there are; the last one repeats (what it gives is masked)
    if (rows >= BQ) {
#pragma unroll
      for (int e = 0; e < NL; ++e) {
        load_lds16(to + e * 4096, rq, off_q, e * RL * lq2);
        load_lds16(to + GO + e * 4096, rg, off_g, e * RL * lg2);
      }
    } else {
#pragma unroll
      for (int e = 0; e < NL; ++e) {
        const int r = r0 + e * RL < rows ? r0 + e * RL : rows - 1;
        load_lds16(to + e * 4096, rq, r * lq2 + chunk, 0);
        load_lds16(to + GO + e * 4096, rg, r * lg2 + chunk, 0);
      }
    }
    if (lane < BQ / 4) {                    // a quarter of the statistics to a wave
      const int r = BQ / 4 * wave + lane;
      load_lds16(to_aux, ra, 16u * (uint32_t)(r < rows ? r : rows - 1), 0);
    }
    if (++tile == w.each) {
      tile = 0;
      ++head;
      head_at();
    } else {
      q_at += BQ * p.ld_q;
      g_at += BQ * (int64_t)p.Hq * D;
      aux_at += BQ;
    }
  };
  load_step(0);
  bf16x8 k[KB], v[KB];
  {
    const int64_t row = w.a + (tk < L ? tk : L - 1);
    const bf16* kp = static_cast<const bf16*>(p.k) + row * p.ld_k + hk * D + 8 * h;
    const bf16* vp = static_cast<const bf16*>(p.v) + row * p.ld_v + hk * D + 8 * h;
#pragma unroll
    for (int kb = 0; kb < KB; ++kb) {
      k[kb] = *reinterpret_cast<const bf16x8*>(kp + 16 * kb);
      v[kb] = *reinterpret_cast<const bf16x8*>(vp + 16 * kb);
    }
  }
  f32x16 zero, dk[MT], dv[MT];
#pragma unroll
  for (int r = 0; r < 16; ++r) zero[r] = 0.f;
#pragma unroll
  for (int c = 0; c < MT; ++c) dk[c] = dv[c] = zero;

  // A block's statistics and the rows of its first AF products, read ahead of it.
  bf16x8 x, ahead[AF];
  auto read_first = [&](uint32_t block, int i) { return rows_at<D>(at.rows + block, i / 2, i % 2 ? GO : 0); };

  // One block: its scores are in s and dp; leaves those of the block at `next` in sn, dpn,
  // and reads ahead of the one at `after`.
  auto step = [&](uint32_t cur, int t0, uint32_t next, uint32_t after, uint32_t after_aux, f32x16& s, f32x16& dp,
                  f32x16& sn, f32x16& dpn) {
    if (t0 < u0 + 31 || t0 + 31 >= L || (window && t0 + 31 - window >= u0)) {
      // element r is query t0 + 4 h + at: seen where it is at the key or behind it,
      // before the end, and less than the window behind it
      const int first = tk - t0 - 4 * h;
      int end = L - t0 - 4 * h;
      if (window && first + window < end) end = first + window;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int e = 8 * (r / 4) + r % 4;
        if (e < first || e >= end) s[r] = -__builtin_huge_valf() * c_scale;
      }
    }
    const uint32_t cols = at.cols + cur;
    bf16x8 f[NF], g[NS], pw[2], dw[2];
    auto read_second = [&](int j) { g[j] = columns_at<D>(cols, j / (2 * MT), j / 2 % MT, j % 2 ? 0 : GO); };
    // The weights in three stages, so that none waits for the one before it: slot n begins
    // weight n, takes weight n - 1 to the power and finishes weight n - 2.
    float y[16], pr[16];
    auto weights = [&](int from, int to) {
#pragma unroll
      for (int n = from; n < to; ++n) {
        if (n >= 2) {
          const int e = n - 2;
          pw[e / 8][e % 8] = (bf16)pr[e];
          dw[e / 8][e % 8] = (bf16)(pr[e] * dp[e]);
        }
        if (n < 16) y[n] = s[n] * c_scale;
        if (n >= 1 && n < 17) pr[n - 1] = exp2_fast(y[n - 1]);
      }
    };
#pragma unroll
    for (int i = 0; i < AF; ++i) f[i] = ahead[i];
    __builtin_amdgcn_sched_barrier(0);
    product_v0(sn, x, ones_s);
    product_v0(dpn, x, ones_d);
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      __builtin_amdgcn_sched_barrier(0);
      if (i % 2 == 0) {
#pragma unroll
        for (int n = i; n < i + 2; ++n) {
          if (n + AF < NF) f[n + AF] = read_first(next, n + AF);
          if (n >= NF - AS) read_second(n - (NF - AS));
        }
        both_there(f[i], f[i + 1]);
      }
      if (i % 2 == 0) product_v(sn, f[i], k[i / 2]);
      else product_v(dpn, f[i], v[i / 2]);
      weights(E1 * i / NF, E1 * (i + 1) / NF);
    }
    settle(pw[0], dw[0]);
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      __builtin_amdgcn_sched_barrier(0);
      if (j % 2 == 0) {
#pragma unroll
        for (int n = j; n < j + 2; ++n) {
          if (n + AS < NS) read_second(n + AS);
          else if (n + AS - NS < AF) ahead[n + AS - NS] = read_first(after, n + AS - NS);
        }
        both_there(g[j], g[j + 1]);
      }
      if (j == NS / 2) settle(pw[1], dw[1]);
      if (j == NS - 1) x = statistics(after_aux);
      const int b = j / (2 * MT), c = j / 2 % MT;
      if (j % 2 == 0) product_a(dv[c], g[j], pw[b]);
      else product_a(dk[c], g[j], dw[b]);
      if (j < NS / 2) weights(E1 + (18 - E1) * j / (NS / 2), E1 + (18 - E1) * (j + 1) / (NS / 2));
    }
    static_assert(AS >= AF && NS >= 8 && E1 >= 10, "every read has its line; products behind the scores; 8 weights before them");
    __builtin_amdgcn_sched_barrier(0);
    behind_v(sn);
    behind_v(dpn);
  };

  f32x16 s, dp, s1, dp1;
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    keep_a(k[kb]);
    keep_a(v[kb]);
  }
  wait_tiles();
  // (the second tile is needed a step later: the first products wait for one only; prompts of
  // 128 tokens, 16 heads, 438 -> 428 us with dq)
#pragma unroll
  for (int i = 1; i < NB - 1; ++i)
    if (w.at + i < w.stop) load_step(i);
  int buf = 0;
  auto next_buf = [](int i) { return (i + 1) % NB; };
  // The next tile is there, with the one behind it perhaps still on its way, and the last one free.
  auto next_tile = [&](int i) {
    if (i + 2 < w.stop) wait_tiles_but<LOADS>();
    else wait_tiles();
    if (i + NB - 1 < w.stop) load_step((buf + NB - 1) % NB);
  };
  if (u0 >= L) {                            // no key: this wave's share of the loads is all it does
    for (int i = w.at; i < w.stop; ++i) {
      next_tile(i);
      buf = next_buf(buf);
    }
    continue;
  }
  {
    x = statistics(0);
    product_v0(s, x, ones_s);
    product_v0(dp, x, ones_d);
    bf16x8 f[NF];
#pragma unroll
    for (int i = 0; i < NF; ++i) f[i] = read_first(0, i);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < NF; i += 2) {
      both_there(f[i], f[i + 1]);
      product_v(s, f[i], k[i / 2]);
      product_v(dp, f[i + 1], v[i / 2]);
    }
    products_done(s, dp);
    x = statistics(HALF_AUX);
#pragma unroll
    for (int i = 0; i < AF; ++i) ahead[i] = read_first(HALF, i);
  }
  for (int i = w.at; i < w.stop; ++i) {
    next_tile(i);
    const int t0 = k0 + now * BQ, nb = next_buf(buf);
    if (++now == w.each) now = 0;
    const uint32_t cur = buf * BUF, then = nb * BUF, then_aux = nb * (BQ * 16);
    step(cur, t0, cur + HALF, then, then_aux, s, dp, s1, dp1);
    step(cur + HALF, t0 + 32, then, then + HALF, then_aux + HALF_AUX, s1, dp1, s, dp);
    products_done<MT>(dk, dv);
    buf = nb;
  }
  // Rows leave through LDS, so that a store covers whole rows.  Waves that are still at the last
  // tile read its buffer (buf - 1) and, ahead of a tile that is none, the next (buf); the other two
  // have been read before the last barrier: a quarter of them to a wave.
  bf16* mine = s_t[(buf + 1 + (wave >> 1)) % NB] + (wave & 1) * BQ * D;
  const int rows = L - u0 < 32 ? L - u0 : 32;
  if (w.slot < 0) {
    const int64_t row0 = w.a + u0;
    rows_out<D>(mine, dk, p.scale, static_cast<TG*>(p.dk) + row0 * p.ld_dk + hk * D, p.ld_dk, rows, lane);
    rows_out<D>(mine, dv, 1.f, static_cast<TG*>(p.dv) + row0 * p.ld_dv + hk * D, p.ld_dv, rows, lane);
  } else {
    float* to = slot_of<D, BK>(p, workers, w.slot) + (int64_t)(32 * wave) * (2 * D);
    rows_out<D>(mine, dk, p.scale, to, 2 * D, rows, lane);
    rows_out<D>(mine, dv, 1.f, to + D, 2 * D, rows, lane);
  }
  }
}

// The parts of the tiles that several workers share, added in order: 16 rows of the tile
// that a worker begins to a workgroup, several parts on their way at a time.
template <typename TG, int D, int BK>
__global__ __launch_bounds__(kThreads) void attn_dkv_join_kernel(AttnBwdArgs p, int workers) {
  constexpr int LR = 2 * D / 4;             // threads of a row of dk and dv
  const int worker = blockIdx.x;
  const Worker t = workers_of(p)[worker];
  if (t.behind <= 0) return;
  constexpr int RB = kThreads / LR, R = 16 / RB;      // rows at a time, and of a thread
  const int c = 4 * (threadIdx.x % LR), r0 = 16 * blockIdx.y + threadIdx.x / LR;
  if (16 * blockIdx.y >= t.rows) return;
  // (rows behind the tile's last read what the slots hold there, and are not written)
  float4 v[R];
  const float* first = slot_of<D, BK>(p, workers, 2 * worker + 1) + r0 * (2 * D) + c;
#pragma unroll
  for (int r = 0; r < R; ++r) v[r] = *reinterpret_cast<const float4*>(first + r * RB * (2 * D));
  const float* src = slot_of<D, BK>(p, workers, 2 * worker + 2) + r0 * (2 * D) + c;
#pragma unroll 4
  for (int i = 0; i < t.behind; ++i, src += 2 * (BK * 2 * D))
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float4 x = *reinterpret_cast<const float4*>(src + r * RB * (2 * D));
      v[r].x += x.x; v[r].y += x.y; v[r].z += x.z; v[r].w += x.w;
    }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r0 + r * RB >= t.rows) break;
    const int64_t row = t.row0 + r0 + r * RB;
    if (c < D) store4<TG>(static_cast<TG*>(p.dk) + row * p.ld_dk + t.hk * D + c, v[r].x, v[r].y, v[r].z, v[r].w);
    else store4<TG>(static_cast<TG*>(p.dv) + row * p.ld_dv + t.hk * D + c - D, v[r].x, v[r].y, v[r].z, v[r].w);
  }
}

// The dq kernel with 64 queries to a workgroup instead of 128, where a CU would otherwise
// have room left for workgroups (us of a whole backward call, 128 / 64).  d 128: 2048 tokens,
// 8 heads (128 workgroups of 128 queries) 106 / 80; 4096 tokens, 8 heads (256) 212 / 166;
// 8192 tokens, 8 heads (512) 537 / 494; 4 prompts of 512, 32 heads (512) 83 / 86; 12
// prompts, 8191 tokens, 8 heads (600) 124 / 113; 2048 tokens, 40 heads (640) 188 / 196;
// 8192 tokens, 12 heads (768) 705 / 717.  d 64: 29 prompts, 8191 tokens, 6 heads (552)
// 61 / 54; 4096 tokens, 20 heads (640) 203 / 193; 8192 tokens, 12 heads (768) 409 / 399,
// 16 heads (1024) 506 / 512; 2048 tokens, 64 heads (1024) 162 / 167.
bool split_dq(int64_t blocks, int d) { return blocks <= (d == 128 ? 512 : 768); }

template <typename TG, int D>
hipError_t launch_bf16(const AttnBwdArgs& a, int workers, hipStream_t stream) {
  const bool packed = a.cu_seqlens != nullptr;
  const int64_t tiles = tiles_of(a.N, a.total_T, a.Tseq, packed, 128);
  const uint32_t nq = (uint32_t)(tiles * a.Hq), nk = workers ? (uint32_t)workers : (uint32_t)(tiles * a.Hk);
  if (split_dq(nq, D)) {
    const uint32_t twice = (uint32_t)(tiles_of(a.N, a.total_T, a.Tseq, packed, 64) * a.Hq);
    attn_dq_bf16_kernel<D, TG, 2><<<dim3(twice + plan_blocks(workers)), kThreads, 0, stream>>>(a, twice, workers);
  } else {
    attn_dq_bf16_kernel<D, TG, 1><<<dim3(nq + plan_blocks(workers)), kThreads, 0, stream>>>(a, nq, workers);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  attn_dkv_bf16_kernel<D, TG><<<dim3(nk), kThreads, 0, stream>>>(a, nk, workers);
  e = hipGetLastError();
  if (e != hipSuccess || workers == 0) return e;
  attn_dkv_join_kernel<TG, D, 128><<<dim3(nk, 8), kThreads, 0, stream>>>(a, workers);
  return hipGetLastError();
}
// fp32 with 8 waves to a tile of 64 keys instead of 4 to 32, where few query tiles have many
// keys (us of a backward call, 4 / 8 waves).  d 128: 2048 tokens, 2 heads (128 workgroups)
// 222 / 203; 8 heads (512) 393 / 353; 4096 tokens, 8 heads (1024) 1223 / 1284.  d 64: 1024
// tokens, 4 heads 85 / 76; 12 prompts, 2048 tokens, 8 heads (608) 77.5 / 73.2; 8 of 256, 4
// heads 33.7 / 33.5; 3 of 86, 4 heads 22.1 / 22.6; 24 of 13, 8 heads 19.8 / 21.1.
bool split_dq_f32(int64_t blocks, int64_t keys) { return blocks <= 640 && keys >= 128; }

template <int D>
hipError_t launch_f32(const AttnBwdArgs& a, int workers, hipStream_t stream) {
  const int64_t tiles = tiles_of(a.N, a.total_T, a.Tseq, a.cu_seqlens != nullptr, 32);
  const uint32_t nq = (uint32_t)(tiles * a.Hq), nk = workers ? (uint32_t)workers : (uint32_t)(tiles * a.Hk);
  const dim3 grid(nq + plan_blocks(workers));
  const int64_t len = a.cu_seqlens ? a.total_T / a.N : a.Tseq;
  if (split_dq_f32(nq, a.window > 0 && a.window < len ? a.window : len)) attn_dq_f32_kernel<D, 4><<<grid, 512, 0, stream>>>(a, nq, workers);
  else attn_dq_f32_kernel<D, 2><<<grid, 256, 0, stream>>>(a, nq, workers);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  attn_dkv_f32_kernel<D><<<dim3(nk), kThreads, 0, stream>>>(a, nk, workers);
  e = hipGetLastError();
  if (e != hipSuccess || workers == 0) return e;
  attn_dkv_join_kernel<float, D, 32><<<dim3(nk, 2), kThreads, 0, stream>>>(a, workers);
  return hipGetLastError();
}

}  // namespace

// Workgroups of the second kind stay on their CU to the end: as many as there is room for.
struct KeyTiles {
  int64_t rows, step, room;
};
static KeyTiles key_tiles(int d, DType io) {
  return io == DType::F32 ? KeyTiles{32, 32, d == 128 ? 512 : 768} : KeyTiles{128, 64, d == 128 ? 256 : 512};
}

AttnBwdPlan attn_bwd_plan(int64_t N, int64_t total_T, int64_t window, int Hq, int Hk, int d, DType io) {
  const KeyTiles kt = key_tiles(d, io);
  const int64_t tiles = total_T / kt.rows + N;
  int64_t workers = 0;
  // (more sequences than kMaxRanked would take a workgroup long to count)
  if (N <= kMaxRanked && tiles * Hk < 8 * kt.room) {
    const WalkUnits u{window, (int)kt.rows, (int)kt.step, Hq / Hk, kLead};
    const int64_t most = Hk * (u.units(total_T) + N * (2 * u.G + u.lead)) / kLeast + 1;   // shares that there can be
    workers = most < kt.room ? (most + kXcds - 1) / kXcds * kXcds : kt.room;
  }
  AttnBwdPlan r;
  r.workers = (int)workers;
  r.ws_floats = 4 * total_T * Hq;
  if (workers) r.ws_floats += 8 * workers + walk_floats(tiles, Hk, (int)workers) + workers * (2 * kt.rows * 2 * d);
  return r;
}

// Whether each key tile gets a workgroup of its own, the dear ones first.  Equal shares of
// their walks are even, but cost partial sums and a join: 9 to 20 steps of a workgroup's
// walk and a fiftieth of it (us with whole tiles / shares: 8 prompts of 64 tokens, 8 heads of
// 2 24 / 29; 8 of 1024, 16 heads 178 / 198; 8192 tokens, 16 heads 900 / 942; 32768 tokens, 8
// heads of 4 7010 / 7097).
// With r tiles to each of the workgroups that there is room for, all sequences of a length,
// whole tiles are as uneven as the next round of them makes it: tiles that see a window cost
// alike and r is rounded up; without one costs fall evenly to 0, so two rounds, the second
// backwards, are even, and what d = r mod 2 rounds are left over make the longest walk
// 2 (d - d^2 / 2) / r^2 longer than the mean; up to r = 1 it is the first tile's.  (us
// whole / shares, r = 1: 16384 tokens, 16 heads of 2 5264 / 3609; r = 3: 32768 tokens, 6 heads of 3, 5765 / 5365; 4 prompts
// of 4096, 12 heads of 6, 742 / 763; 16 prompts of 512, 12 heads, 105 / 125.)
// Lengths that differ are not known here: from 3 tiles on (fp32, whose tiles are shorter
// than the longest sequence by more: 2) the longest one's walks rarely decide (us whole /
// shares; 12 prompts of 16384 tokens, r = 2.2 425 / 376, 3.3 542 / 547, 4.4 702 / 719; 16 of
// 32768 with a window of 2048, r = 2.1 1401 / 1386, 4.3 1360 / 1410; fp32, 12 of 4096, r =
// 2.2 221 / 237, heads of 64, r = 2.9 178 / 206), and never where all tokens in one
// sequence would be a short walk.
static bool whole_tiles(const AttnBwdArgs& a) {
  const KeyTiles kt = key_tiles(a.d, a.io);
  const int64_t tiles = tiles_of(a.N, a.total_T, a.Tseq, a.cu_seqlens != nullptr, kt.rows) * a.Hk;
  const double r = (double)tiles / (double)kt.room;
  const WalkUnits u{a.window, (int)kt.rows, (int)kt.step, a.Hq / a.Hk, kLead};
  if (a.cu_seqlens && a.N > 1)
    return r >= (a.io == DType::F32 ? 2.0 : 3.0) || u.before(a.total_T, 1) < 9;
  const int64_t L = a.total_T / a.N;
  const double walk = (double)(a.N * a.Hk) * (double)u.units(L) / (double)kt.room, d = std::fmod(r, 2.0);
  const double longer = r <= 1.0 ? (double)u.before(L, 1) - walk
                        : a.window > 0 && a.window < L / 2 ? (std::ceil(r) / r - 1.0) * walk
                                                           : 2.0 * (d - 0.5 * d * d) / (r * r) * walk;
  return longer < 9.0 + std::fmin(11.0, walk / 4.0) + walk / 50.0;
}

int64_t attn_bwd_blocks(int64_t N, int64_t total_T, int64_t Tseq, bool packed, int Hq, DType io) {
  return tiles_of(N, total_T, Tseq, packed, io == DType::F32 ? 32 : 128) * Hq + plan_blocks(1024);
}

hipError_t launch_attn_bwd(const AttnBwdArgs& a, const AttnBwdPlan& plan, hipStream_t stream) {
  const int workers = whole_tiles(a) ? 0 : plan.workers;
  if (a.io == DType::F32)
    return a.d == 128 ? launch_f32<128>(a, workers, stream) : launch_f32<64>(a, workers, stream);
  if (a.grad == DType::F32)
    return a.d == 128 ? launch_bf16<float, 128>(a, workers, stream) : launch_bf16<float, 64>(a, workers, stream);
  return a.d == 128 ? launch_bf16<bf16, 128>(a, workers, stream) : launch_bf16<bf16, 64>(a, workers, stream);
}

#ifdef GDN_CHECK
unsigned check_violations_attn_bwd() { return take_check_violations(); }
#endif

}  // namespace gdn
