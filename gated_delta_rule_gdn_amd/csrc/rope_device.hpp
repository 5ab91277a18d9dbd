// rope_device.hpp -- which channels and frequencies a lane holds, and the rotary
// position's angles, for the kernels that turn query and key rows (attn_rope.hip)
// and the gradients of those rows (attn_rope_backward.hip).
#pragma once

#include "attn_device.hpp"

namespace gdn {

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

__device__ __forceinline__ void load_weights(const float* weight, const LaneMap& m, float* w) {
  if (!weight) return;
  load_f32<8, float>(weight + m.c0, w);
  load_f32<8, float>(weight + m.c1, w + 8);
}

}  // namespace gdn
