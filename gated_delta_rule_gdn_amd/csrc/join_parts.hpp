// join_parts.hpp -- sums of the partial weight gradients that workgroups leave in a
// workspace, in a fixed order.
#pragma once

#include "gdn_device.hpp"

namespace gdn {

// out[c] = sum of src[i ld + c] over i < n, for the 16 columns of a workgroup from `col` on
// (as far as they are below `cols`, a multiple of 4).  4 columns to a thread and THREADS / 4
// parts at a time, several of them on their way: a call is a few latencies long (512 parts of
// 2048 columns 4.6 us, a column to a thread 36; 3640 parts of 128 columns 8.0, 8.7).
template <int THREADS>
__device__ __forceinline__ void join_parts(const float* __restrict__ src, int64_t ld, int n, int col, int cols,
                                           float* __restrict__ out) {
  constexpr int P = THREADS / 4;
  static_assert(THREADS >= 256 && P % 16 == 0, "256 threads for the second sum");
  __shared__ __align__(16) float s[P][20], s2[16][17];
  lds_nan_fill(s, sizeof s);
  lds_nan_fill(s2, sizeof s2);
  const int c = col + 4 * (threadIdx.x & 3), part = threadIdx.x >> 2;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < cols) {
#pragma unroll 8
    for (int i = part; i < n; i += P) {
      const float4 u = *reinterpret_cast<const float4*>(src + i * ld + c);
      v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
    }
  }
  lds_check(&s[part][4 * (threadIdx.x & 3)], 16);
  *reinterpret_cast<float4*>(&s[part][4 * (threadIdx.x & 3)]) = v;
  __syncthreads();
  const int k = threadIdx.x & 15, g = threadIdx.x >> 4;
  if (g < 16) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < P / 16; ++i) {
      lds_check(&s[16 * i + g][k], 4);
      t += s[16 * i + g][k];
    }
    lds_check(&s2[g][k], 4);
    s2[g][k] = t;
  }
  __syncthreads();
  if (threadIdx.x < 16 && col + threadIdx.x < cols) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += s2[i][threadIdx.x];
    out[col + threadIdx.x] = t;
  }
}

}  // namespace gdn
