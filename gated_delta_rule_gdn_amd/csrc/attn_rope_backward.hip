// attn_rope_backward.hip -- the gradient of qk_norm_rope (attn_rope.hip):
//
//   (ga, gb) = f (da cos t + db sin t,  db cos t - da sin t)      the turn taken back
//   n = x / rms(x),  d_weight += g n  over all rows and heads
//   dx = (g w - n mean(n g w)) / rms(x)
//
// with g = dy on channels that do not turn and, without a norm, dx = g.
//
// Lanes hold the channels that they hold in the forward, so again only sums over a
// row cross lanes.  The norm's root is formed again from the raw row, which has to be
// read in any case.  Reads two rows and writes one at some twenty flops an element:
// HBM-bound for many rows: 32768 rows of 16 + 2 heads of 128, bf16, 84 us, 5.4 TB/s, and 8 for
// the join of the weights' gradients.
#include "rope_device.hpp"

#include "hybrid_kernels.hpp"
#include "join_parts.hpp"

namespace gdn {
namespace {

constexpr int kThreads = 256;
// Heads of a thread, sharing the angles (1 or 4: within 1 %), and workgroups that loop over
// the tokens: each leaves one partial gradient of the weights, and they are joined in a
// fixed order (1024 or 16384: within 1 %, the join against the loads in flight).
constexpr int kHeads = 2;
constexpr int64_t kBlocks = 4096;

struct Split {
  int gq, gk;                                 // groups of kHeads heads of each operand
  int64_t tb;                                 // workgroups of a group
};
__host__ __device__ inline Split split_of(int64_t rows, int Hq, int Hk, int d) {
  const int tokens = kThreads / (d / 16);
  Split s;
  s.gq = (Hq + kHeads - 1) / kHeads;
  s.gk = (Hk + kHeads - 1) / kHeads;
  const int64_t need = (rows + tokens - 1) / tokens, most = kBlocks / (s.gq + s.gk);
  s.tb = need <= most ? need : (most > 1 ? most : 1);   // (no rows: none, at any number of heads)
  return s;
}

// Sum over a wave's lanes that are equal modulo LPR (4 or 8), in the vector unit.
template <int LPR>
__device__ __forceinline__ float over_tokens(float s) {
  auto dpp = [](float v, auto ctrl) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
        0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xf, 0xf, false));
  };
  s += dpp(s, std::integral_constant<int, 0x128>{});                         // row_ror:8
  if constexpr (LPR == 4) s += dpp(s, std::integral_constant<int, 0x124>{});  // row_ror:4
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(s), __float_as_uint(s), false, false);
  s = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(s), __float_as_uint(s), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

template <typename T, typename G, int D, bool INTER>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_bwd_kernel(QkNormRopeBwdArgs p) {
  constexpr int LPR = D / 16;
  constexpr int TB = kThreads / LPR;          // tokens of a workgroup's pass
  __shared__ __align__(16) float s_w[4][D];
  lds_nan_fill(s_w, sizeof s_w);
  const Split sp = split_of(p.rows, p.Hq, p.Hk, D);
  const int64_t tb = blockIdx.x / (sp.gq + sp.gk);
  const int grp = (int)(blockIdx.x - tb * (sp.gq + sp.gk));
  const bool is_q = grp < sp.gq;
  const int H = is_q ? p.Hq : p.Hk;
  const int h0 = (is_q ? grp : grp - sp.gq) * kHeads;
  const int64_t ld = is_q ? p.ld_q : p.ld_k, ldo = is_q ? p.ld_dq : p.ld_dk;
  const float* weight = is_q ? p.q_weight : p.k_weight;
  const bool normed = weight != nullptr;
  const int l = threadIdx.x % LPR;
  const LaneMap m = lane_map<D, INTER, true>(l, p.rope);
  const T* raw = static_cast<const T*>(is_q ? p.q_raw : p.k_raw);
  const G* up = static_cast<const G*>(is_q ? p.dq : p.dk);
  G* out = static_cast<G*>(is_q ? p.dq_raw : p.dk_raw);

  float w[16], acc[16];
  load_weights(weight, m, w);
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  Freqs f;
  if (p.rope.dim) load_freqs(p.rope, m, f);

  for (int64_t r = tb * TB + threadIdx.x / LPR; r < p.rows; r += sp.tb * TB) {   // whole rows of lanes leave together
    Chunk8<T> xa[kHeads], xb[kHeads];
    Chunk8<G> ga[kHeads], gb[kHeads];
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      const int h = h0 + i < H ? h0 + i : H - 1;
      ga[i].load(up + (r * H + h) * (int64_t)D + m.c0);
      gb[i].load(up + (r * H + h) * (int64_t)D + m.c1);
      if (normed) {
        xa[i].load(raw + r * ld + h * D + m.c0);
        xb[i].load(raw + r * ld + h * D + m.c1);
      }
    }
    float c[8], s[8];
    if (p.rope.dim) turn<std::is_same<G, float>::value, 8>(p.positions[r], f, p.rope, m, c, s);
#pragma unroll
    for (int i = 0; i < kHeads; ++i) {
      if (h0 + i >= H) break;
      float g[16];
      ga[i].unpack(g);
      gb[i].unpack(g + 8);
      if (m.turns) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int ia = INTER ? 2 * e : e, ib = INTER ? 2 * e + 1 : 8 + e;
          const float a = g[ia], b = g[ib];
          g[ia] = a * c[e] + b * s[e];
          g[ib] = b * c[e] - a * s[e];
        }
      }
      if (normed) {
        float x[16], ss = 0.f, sg = 0.f;
        xa[i].unpack(x);
        xb[i].unpack(x + 8);
#pragma unroll
        for (int e = 0; e < 16; ++e) ss += x[e] * x[e];
        const float inv = __builtin_amdgcn_rsqf(lanes_sum<LPR>(ss) * (1.f / D) + p.rope.eps);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          x[e] *= inv;
          acc[e] += g[e] * x[e];
          g[e] *= w[e];
          sg += g[e] * x[e];
        }
        sg = lanes_sum<LPR>(sg) * (1.f / D);
#pragma unroll
        for (int e = 0; e < 16; ++e) g[e] = inv * (g[e] - x[e] * sg);
      }
      G* to = out + r * ldo + (h0 + i) * D;
      store8(to + m.c0, g);
      store8(to + m.c1, g + 8);
    }
  }
  if (!(is_q ? p.dq_weight : p.dk_weight)) return;
  // over the wave's tokens, the workgroup's waves, then (below) the workgroups
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = over_tokens<LPR>(acc[e]);
  if (lane < LPR) {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float* dst = &s_w[wave][(e < 8 ? m.c0 : m.c1 - 8) + e];
      lds_check(dst, 4);
      *dst = acc[e];
    }
  }
  __syncthreads();
  // the parts of an operand follow each other: q's, then k's
  const int64_t part = is_q ? tb * sp.gq + grp : sp.tb * sp.gq + tb * sp.gk + (grp - sp.gq);
  if (threadIdx.x < D)
    p.ws[part * D + threadIdx.x] = (s_w[0][threadIdx.x] + s_w[1][threadIdx.x]) +
                                                  (s_w[2][threadIdx.x] + s_w[3][threadIdx.x]);
}

// Sum of the workgroups' partial weight gradients: one workgroup for 16 channels of an operand.
constexpr int kJoinThreads = 1024;
template <int D>
__global__ __launch_bounds__(kJoinThreads) void qk_weight_join_kernel(QkNormRopeBwdArgs p) {
  const bool is_q = blockIdx.y == 0;
  float* to = is_q ? p.dq_weight : p.dk_weight;
  if (!to) return;
  const Split sp = split_of(p.rows, p.Hq, p.Hk, D);
  join_parts<kJoinThreads>(p.ws + (is_q ? 0 : sp.tb * sp.gq * D), D, (int)sp.tb * (is_q ? sp.gq : sp.gk),
                           16 * blockIdx.x, D, to);
}

template <typename T, typename G, int D>
hipError_t launch_d(const QkNormRopeBwdArgs& a, hipStream_t stream) {
  const Split s = split_of(a.rows, a.Hq, a.Hk, D);
  const dim3 grid((unsigned)(s.tb * (s.gq + s.gk)));
  if (grid.x > 0) {                         // (no rows: the weights' gradients are 0)
    if (a.rope.inter) qk_norm_rope_bwd_kernel<T, G, D, true><<<grid, kThreads, 0, stream>>>(a);
    else qk_norm_rope_bwd_kernel<T, G, D, false><<<grid, kThreads, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.dq_weight && !a.dk_weight) return hipSuccess;
  qk_weight_join_kernel<D><<<dim3(D / 16, 2), kJoinThreads, 0, stream>>>(a);
  return hipGetLastError();
}
template <typename T, typename G>
hipError_t launch_t(const QkNormRopeBwdArgs& a, hipStream_t stream) {
  return a.d == 128 ? launch_d<T, G, 128>(a, stream) : launch_d<T, G, 64>(a, stream);
}

}  // namespace

int64_t qk_bwd_ws_floats(int64_t rows, int Hq, int Hk, int d) {
  const Split s = split_of(rows, Hq, Hk, d);
  return s.tb * (s.gq + s.gk) * d;
}

hipError_t launch_qk_norm_rope_bwd(const QkNormRopeBwdArgs& a, hipStream_t stream) {
  if (a.io == DType::F32) return launch_t<float, float>(a, stream);
  return a.grad == DType::F32 ? launch_t<bf16, float>(a, stream) : launch_t<bf16, bf16>(a, stream);
}

#ifdef GDN_CHECK
unsigned check_violations_rope_bwd() { return take_check_violations(); }
#endif

}  // namespace gdn
