// attn_device.hpp -- device helpers of the attention kernels: packed-sequence
// lookup, 8-element chunks kept as loaded, reductions over lanes.
#pragma once

#include "attn_index.hpp"
#include "attn_kernels.hpp"
#include "gdn_device.hpp"

#include <type_traits>

namespace gdn {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// Running maximum (log2 units) before any token: at or below every finite score, and
// a masked one (-inf) less it is -inf.
constexpr float kNone = -3.402823466e+38f;

// The weight of a score x that is at most a little above the running maximum m.  Both
// are rounded, so their difference is small for the largest however large they are;
// fused with the product that gives x it would be off by half a step of m.
__device__ __forceinline__ float weight_of(float x, float m) {
#pragma clang fp contract(off)
  return exp2_fast(x - m);
}

__device__ __forceinline__ int64_t read_lane(int64_t x, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)x, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)((uint64_t)x >> 32), lane);
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// Item idx of packed offsets (find_packed_by), and lens[n] where lens is given.
// Up to 63 sequences are read by the lanes of a wave at once, lengths with
// them, and the answer comes from the lanes: one memory latency.  More are
// probed 64 at a time; every lane gets the answer.
__device__ __forceinline__ PackedItem find_packed(const int64_t* __restrict__ cu, int64_t N,
                                                  int64_t total, int unit, int extra, int64_t idx,
                                                  const int64_t* __restrict__ lens = nullptr,
                                                  int64_t* len = nullptr) {
  const int lane = threadIdx.x & 63;
  if (N < 64) {
    const int64_t c = clamp_i64(cu[lane < N ? lane : N], 0, total);
    const int64_t s = lens ? lens[lane < N ? lane : N - 1] : 0;
    const uint64_t m = __ballot(lane < N && c / unit + extra * lane <= idx);
    PackedItem r;
    r.n = m ? 63 - __builtin_clzll(m) : 0;
    r.start = read_lane(c, (int)r.n);
    r.end = read_lane(c, (int)r.n + 1);
    r.item = idx - (r.start / unit + extra * r.n);
    if (lens) *len = read_lane(s, (int)r.n);
    return r;
  }
  const PackedItem r =
      find_packed_by(cu, N, total, unit, extra, idx, [&](int64_t lo, int64_t step, int64_t hi) {
        const int64_t i = lo + lane * step;
        return (uint64_t)__ballot(i < hi && packed_at_or_before(cu, i, total, unit, extra, idx));
      });
  if (lens) *len = lens[r.n];
  return r;
}

// Sum over the wave: within the rows of 16 lanes by DPP moves, then four lanes.
__device__ __forceinline__ int wave_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xf, 0xf, false);   // quad_perm [1,0,3,2]
  v += __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xf, 0xf, false);   // quad_perm [2,3,0,1]
  v += __builtin_amdgcn_update_dpp(0, v, 0x141, 0xf, 0xf, false);  // row_half_mirror
  v += __builtin_amdgcn_update_dpp(0, v, 0x140, 0xf, 0xf, false);  // row_mirror
  return __builtin_amdgcn_readlane(v, 0) + __builtin_amdgcn_readlane(v, 16) +
         __builtin_amdgcn_readlane(v, 32) + __builtin_amdgcn_readlane(v, 48);
}

// rank_tile_by over at most 64 M sequences: each lane keeps the tiles of M of
// them, sequence 64 i + lane in c[i].  Everything fits in 32 bits: the host
// bounds the tiles.
template <int M>
__device__ __forceinline__ PackedItem rank_tile(const int64_t* __restrict__ cu, int N,
                                                int64_t total, int unit, int level, int rank) {
  const int lane = threadIdx.x & 63;
  int c[M];
#pragma unroll
  for (int i = 0; i < M; ++i) {
    const int n = 64 * i + lane;
    c[i] = n < N ? (int)packed_tiles(cu, n, total, unit) : 0;
  }
  auto count = [&](auto f) {
    int v = 0;
#pragma unroll
    for (int i = 0; i < M; ++i) v += f(64 * i + lane, c[i]);
    return wave_sum(v);
  };
  auto pick = [&](auto f, int k) {
    int found = 0;
#pragma unroll
    for (int i = 0; i < M; ++i) {
      uint64_t m = __ballot(f(c[i]));
      const int here = __popcll(m);
      if (k >= 0 && k < here) {
        for (int j = k; j > 0; --j) m &= m - 1;
        found = 64 * i + __ffsll((unsigned long long)m) - 1;
      }
      k -= here;
    }
    return found;
  };
  const RankedTile t = rank_tile_by(N, (int)((total + unit - 1) / unit), level, rank, count, pick);
  PackedItem r{0, 0, 0, 0};
  if (t.n < 0) return r;
  r.n = t.n;
  r.item = t.item;
  r.start = clamp_i64(cu[t.n], 0, total);
  r.end = clamp_i64(cu[t.n + 1], 0, total);
  return r;
}

// 8 consecutive elements kept as loaded, so that many rows are in flight at
// the cost of 4 (bf16) or 8 (fp32) registers each.
template <typename T> struct Chunk8;
template <> struct Chunk8<bf16> {
  uint4 u;
  __device__ __forceinline__ void load(const bf16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void unpack(float* out) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      out[2 * i] = __uint_as_float(w[i] << 16);
      out[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <> struct Chunk8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void unpack(float* out) const {
    out[0] = a.x; out[1] = a.y; out[2] = a.z; out[3] = a.w;
    out[4] = b.x; out[5] = b.y; out[6] = b.z; out[7] = b.w;
  }
};

__device__ __forceinline__ void store8(bf16* p, const float* v) {
  typedef __bf16 bf16x8s __attribute__((ext_vector_type(8)));
  bf16x8s h;
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = (bf16)v[i];
  *reinterpret_cast<bf16x8s*>(p) = h;
}
__device__ __forceinline__ void store8(float* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Sum over the L consecutive lanes (4 or 8, aligned) that hold one row.
template <int L>
__device__ __forceinline__ float lanes_sum(float s) {
  static_assert(L == 4 || L == 8, "lanes of a row");
  auto dpp = [](float v, auto ctrl) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
        0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xf, 0xf, false));
  };
  s += dpp(s, std::integral_constant<int, 0xB1>{});   // quad_perm [1,0,3,2]
  s += dpp(s, std::integral_constant<int, 0x4E>{});   // quad_perm [2,3,0,1]
  if constexpr (L == 8) s += dpp(s, std::integral_constant<int, 0x141>{});  // row_half_mirror
  return s;
}

// Maximum over the two lanes 32 apart.
__device__ __forceinline__ float over_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Maximum over the two lanes 16 apart in each half.
__device__ __forceinline__ float over_rows(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

__device__ __forceinline__ float wave_max(float x) {
  auto dpp = [](float v, auto ctrl) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
        0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xf, 0xf, false));
  };
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0xB1>{}));   // quad_perm [1,0,3,2]
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0x4E>{}));   // quad_perm [2,3,0,1]
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0x141>{}));  // row_half_mirror
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0x140>{}));  // row_mirror
  return over_halves(over_rows(x));
}

}  // namespace gdn
