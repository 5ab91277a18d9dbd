// norm_ops.hip -- the residual stream between a hybrid's layers, on gfx950:
//
//   add_norm     : r = x + res, y = r / sqrt(mean(r^2) + eps) * weight, y in the
//                  type of x or as e4m3 codes with a scale for each group of
//                  channels or each row.
//   add_norm_bwd : d_r = d_res_out + inv (w dy - n mean(n w dy)), n = r inv, and
//                  d_weight = sum over rows of dy n.
//
// Both read their rows once, hold them in registers through the sums over a row and
// write once, at a few flops per element: HBM-bound for many rows, launch latency
// for few.  32768 rows of 2048 channels, bf16 with the residual in fp32: 142.9 us, 5.64 TB/s
// (a copy of 1 GiB: 5.09), backward 193.1, 5.56; 8192 rows of 4096 to e4m3 44.7 us, 5.3.  One
// row 1.8 us, 5.1 to 5.9 with its call.  Backward of 4096 rows of 16384 channels: bf16 115 us,
// 4.7 TB/s, with the residual in fp32 189, 5.7, all in fp32 277, 3.9: a thread's 64 channels take
// all 512 registers there, and in fp32 82 more.
//
// A row is held by W waves (1 or 4) in CH chunks of 8 channels to a lane, chunk
// i of thread t being number t + 64 W i of the row, so that every access is
// 16 (or 2 x 16) bytes to a lane, neighbours next to each other.
#include "attn_device.hpp"

#include "hybrid_kernels.hpp"
#include "join_parts.hpp"

namespace gdn {
namespace {

constexpr int kThreads = 256;
// Waves of a row (us, 1 / 4, 16384 rows, bf16 with the residual in fp32: 1024 channels 33.6 /
// 34.9 and backward 37.2 / 49.2; 1536 50.7 / 51.4, 55.4 / 58.0; 2048 75.6 / 72.9, 79.9 / 76.1;
// 2560 94.4 / 92.0, 103 / 97; 4096 149 / 146, 189 / 156.  With the residual in bf16: 32768 rows of
// 2048 93.0 / 92.9, 77 / 94; 16384 of 4096 100 / 94, 98 / 76).
int waves_of(int C) { return C <= 1536 ? 1 : 4; }

__device__ __forceinline__ float wave_sum_f(float s) {
  auto dpp = [](float v, auto ctrl) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
        0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xf, 0xf, false));
  };
  s += dpp(s, std::integral_constant<int, 0xB1>{});   // quad_perm [1,0,3,2]
  s += dpp(s, std::integral_constant<int, 0x4E>{});   // quad_perm [2,3,0,1]
  s += dpp(s, std::integral_constant<int, 0x141>{});  // row_half_mirror
  s += dpp(s, std::integral_constant<int, 0x140>{});  // row_mirror
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(s), __float_as_uint(s), false, false);
  s = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(s), __float_as_uint(s), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Maximum over n = 4, 8 or 16 aligned lanes.
__device__ __forceinline__ float lanes_max(float x, int n) {
  auto dpp = [](float v, auto ctrl) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
        0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xf, 0xf, false));
  };
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0xB1>{}));
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0x4E>{}));
  if (n >= 8) x = fmaxf(x, dpp(x, std::integral_constant<int, 0x141>{}));
  if (n >= 16) x = fmaxf(x, dpp(x, std::integral_constant<int, 0x140>{}));
  return x;
}

// Magnitude as far as it counts for a scale: infinities and NaN do not.
__device__ __forceinline__ float counted(float x) {
  x = fabsf(x);
  return x < __builtin_huge_valf() ? x : 0.f;
}

// Eight e4m3 codes of y * inv, rounded to nearest even; what passes the largest code
// (infinities) becomes it, NaN stays NaN.
__device__ __forceinline__ uint2 codes8(const float* y, float inv) {
  float z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    z[i] = y[i] * inv;
    z[i] = z[i] == z[i] ? __builtin_amdgcn_fmed3f(z[i], -448.f, 448.f) : z[i];
  }
  int a = __builtin_amdgcn_cvt_pk_fp8_f32(z[0], z[1], 0, false);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(z[2], z[3], a, true);
  int b = __builtin_amdgcn_cvt_pk_fp8_f32(z[4], z[5], 0, false);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(z[6], z[7], b, true);
  return make_uint2((uint32_t)a, (uint32_t)b);
}

// Rows are held times a power of two, which changes no rounding: so squares below 2^120 add
// up to less than 2^128 over 16384 channels, and products with gradients below 2^60 too.  At
// the other end eps covers what that costs, but for one next to nothing: there a small row
// is summed again times kSmall as well.
constexpr float kFactor = 0x1p-8f, kSmall = 0x1p80f;
__device__ __forceinline__ bool sum_again(float eps, float mean) {      // (mean is the same in all lanes)
  return eps < 0x1p-100f && __builtin_amdgcn_readfirstlane(mean < 0x1p-80f);
}

// W 1: a workgroup has 4 rows; W 4: one.
template <typename TX, typename TR, int W, int CH, bool CODES>
__global__ __launch_bounds__(kThreads) void add_norm_kernel(AddNormArgs p) {
  __shared__ float s_sum[2][4], s_max[4];
  lds_nan_fill(s_sum, sizeof s_sum);
  lds_nan_fill(s_max, sizeof s_max);
  const int t = W == 1 ? threadIdx.x & 63 : threadIdx.x, wave = threadIdx.x >> 6;
  const int64_t row = W == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x;
  if (W == 1 && row >= p.rows) return;
  const int chunks = p.C / 8;
  const TX* x = static_cast<const TX*>(p.x) + row * p.ld_x;
  const TR* res = static_cast<const TR*>(p.res) + (p.res ? row * p.C : 0);
  Chunk8<TX> cx[CH];
  Chunk8<TR> cr[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + 64 * W * i;
    if (c < chunks) {
      cx[i].load(x + 8 * c);
      if (p.res) cr[i].load(res + 8 * c);
    }
  }
  float w[CH][8], r[CH][8], ss = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + 64 * W * i;
    if (p.weight && c < chunks) {
      load_f32<8, float>(p.weight + 8 * c, w[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[i][e] = 1.f;
    }
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + 64 * W * i;
#pragma unroll
    for (int e = 0; e < 8; ++e) r[i][e] = 0.f;
    if (c < chunks) {
      cx[i].unpack(r[i]);
      if (p.res) {
        float u[8];
        cr[i].unpack(u);
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i][e] += u[e];
      }
      if (p.res_out) store8(static_cast<TR*>(p.res_out) + row * p.C + 8 * c, r[i]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = r[i][e] * kFactor;
      ss += x * x;
    }
  }
  auto over_row = [&](float (&s)[4]) {
    ss = wave_sum_f(ss);
    if constexpr (W == 4) {
      lds_check(s + wave, 4);
      if ((threadIdx.x & 63) == 0) s[wave] = ss;
      __syncthreads();
      ss = (s[0] + s[1]) + (s[2] + s[3]);
    }
    return ss / (float)p.C;
  };
  float mean = over_row(s_sum[0]) + p.eps * (kFactor * kFactor), f = kFactor;
  if (sum_again(p.eps, mean)) {
    f = kFactor * kSmall;
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = r[i][e] * f;
        ss += x * x;
      }
    mean = over_row(s_sum[1]) + (p.eps * f) * f;
  }
  const float inv = __builtin_amdgcn_rsqf(mean) * f;
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) r[i][e] *= inv * w[i][e];
  if constexpr (!CODES) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + 64 * W * i;
      if (c < chunks) store8(static_cast<TX*>(p.y) + row * p.C + 8 * c, r[i]);
    }
  } else {
    const int per = p.group ? p.group / 8 : chunks;     // chunks of a scale
    const int groups = p.group ? p.C / p.group : 1;
    float a[CH], top = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      a[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) a[i] = fmaxf(a[i], counted(r[i][e]));
      top = fmaxf(top, a[i]);
    }
    if (!p.group) {
      top = wave_max(top);
      if constexpr (W == 4) {
        lds_check(s_max + wave, 4);
        if ((threadIdx.x & 63) == 0) s_max[wave] = top;
        __syncthreads();
        top = fmaxf(fmaxf(s_max[0], s_max[1]), fmaxf(s_max[2], s_max[3]));
      }
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + 64 * W * i;
      const float m = p.group ? lanes_max(a[i], per) : top;
      const float scale = fmaxf(m, 0x1p-100f) / 448.f;
      if (c < chunks) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + row * p.C + 8 * c) =
            codes8(r[i], 1.f / scale);
        if (c % per == 0) p.y_scale[row * groups + c / per] = scale;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward.  Workgroups loop over rows and keep their rows' part of d_weight in
// registers; it goes to the workspace once for each workgroup, and a second kernel
// adds the parts in a fixed order.  With two workgroups to a CU loads and stores of different
// rows overlap; more leave more parts (us, 256 / 512 / 768 workgroups, bf16 with the residual in
// fp32: 16384 rows of 1536 channels 55.1 / 55.5 / 63.5, of 2048 103 / 76 / 83, of 2560 118 / 97 /
// 103, of 4096 150 / 156 / 157).  From 4097 channels on with the residual in fp32, and from 8193 on
// in any type, registers leave room for one to a CU (8192 rows of 8192 149 / 152 / 158, 4096 of
// 16384 180 / 189 / 200, all in fp32 253 / 278 / 280).
// ---------------------------------------------------------------------------
constexpr int64_t kBwdBlocks = 512;
int64_t bwd_blocks(int64_t rows, int C) {
  const int64_t need = waves_of(C) == 1 ? (rows + 3) / 4 : rows;
  return need < kBwdBlocks ? need : kBwdBlocks;
}

template <typename TX, typename TR, int W, int CH>
__global__ __launch_bounds__(kThreads) void add_norm_bwd_kernel(AddNormBwdArgs p, int blocks) {
  __shared__ float s_sum[2][4][2];
  __shared__ __align__(16) float s_w[W == 1 ? 4 * CH * 512 : 4];
  lds_nan_fill(s_sum, sizeof s_sum);
  lds_nan_fill(s_w, sizeof s_w);
  const int t = W == 1 ? threadIdx.x & 63 : threadIdx.x, wave = threadIdx.x >> 6;
  const int chunks = p.C / 8;
  float acc[CH][8], w[CH][8];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = t + 64 * W * i;
#pragma unroll
    for (int e = 0; e < 8; ++e) { acc[i][e] = 0.f; w[i][e] = 1.f; }
    if (p.weight && c < chunks) load_f32<8, float>(p.weight + 8 * c, w[i]);
  }
  const int64_t step = W == 1 ? 4 * (int64_t)blocks : blocks;
  int turn = 0;
  for (int64_t row = W == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x; row < p.rows; row += step) {
    Chunk8<TR> cr[CH], cd[CH];
    Chunk8<TX> cy[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + 64 * W * i;
      if (c < chunks) {
        cr[i].load(static_cast<const TR*>(p.r) + row * p.C + 8 * c);
        cy[i].load(static_cast<const TX*>(p.dy) + row * p.C + 8 * c);
        if (p.d_res_out) cd[i].load(static_cast<const TR*>(p.d_res_out) + row * p.C + 8 * c);
      }
    }
    float r[CH][8], g[CH][8], ss = 0.f, sg = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + 64 * W * i;
#pragma unroll
      for (int e = 0; e < 8; ++e) r[i][e] = g[i][e] = 0.f;
      if (c < chunks) {
        cr[i].unpack(r[i]);
        cy[i].unpack(g[i]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        r[i][e] *= kFactor;
        ss += r[i][e] * r[i][e];
        sg += r[i][e] * (g[i][e] * w[i][e]);
      }
    }
    auto over_row = [&] {
      ss = wave_sum_f(ss);
      sg = wave_sum_f(sg);
      if constexpr (W == 4) {               // two sets in turn: one barrier to a sum
        float (*s)[2] = s_sum[turn];
        turn ^= 1;
        lds_check(s + wave, 8);
        if ((threadIdx.x & 63) == 0) { s[wave][0] = ss; s[wave][1] = sg; }
        __syncthreads();
        ss = (s[0][0] + s[1][0]) + (s[2][0] + s[3][0]);
        sg = (s[0][1] + s[1][1]) + (s[2][1] + s[3][1]);
      }
    };
    over_row();
    float f = kFactor, squares = ss / (float)p.C + p.eps * (kFactor * kFactor);
    if (sum_again(p.eps, squares)) {
      f = kFactor * kSmall;
      ss = sg = 0.f;
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          r[i][e] *= kSmall;
          ss += r[i][e] * r[i][e];
          sg += r[i][e] * (g[i][e] * w[i][e]);
        }
      over_row();
      squares = ss / (float)p.C + (p.eps * f) * f;
    }
    const float root = __builtin_amdgcn_rsqf(squares), inv = root * f;
    const float mean = sg / (float)p.C * root;         // of n w dy
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + 64 * W * i;
      float u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) u[e] = 0.f;
      if (p.d_res_out && c < chunks) cd[i].unpack(u);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = r[i][e] * root;
        acc[i][e] += g[i][e] * n;
        u[e] += inv * (g[i][e] * w[i][e] - n * mean);
      }
      if (c < chunks) {
        if (p.d_res) store8(static_cast<TR*>(p.d_res) + row * p.C + 8 * c, u);
        if (p.dx) store8(static_cast<TX*>(p.dx) + row * p.ld_dx + 8 * c, u);
      }
    }
  }
  if (!p.d_weight) return;
  float* to = p.ws + blockIdx.x * (int64_t)p.C;
  if constexpr (W == 1) {
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        float* dst = s_w + (wave * CH + i) * 512 + 8 * t + e;
        lds_check(dst, 16);
        *reinterpret_cast<float4*>(dst) = make_float4(acc[i][e], acc[i][e + 1], acc[i][e + 2], acc[i][e + 3]);
      }
    __syncthreads();
    for (int c = threadIdx.x; c < p.C; c += kThreads) {
      lds_check(s_w + 3 * CH * 512 + c, 4);
      to[c] = (s_w[c] + s_w[CH * 512 + c]) + (s_w[2 * CH * 512 + c] + s_w[3 * CH * 512 + c]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = t + 64 * W * i;
      if (c < chunks) store8(to + 8 * c, acc[i]);
    }
  }
}

// 16 channels to a workgroup.
__global__ __launch_bounds__(kThreads) void weight_join_kernel(const float* ws, float* out, int C, int parts) {
  join_parts<kThreads>(ws, C, parts, 16 * blockIdx.x, C, out);
}

template <typename TX, typename TR, bool CODES>
hipError_t add_norm_t(const AddNormArgs& a, hipStream_t stream) {
  const dim3 four((unsigned)((a.rows + 3) / 4)), one((unsigned)a.rows);
  if (a.C <= 512) add_norm_kernel<TX, TR, 1, 1, CODES><<<four, kThreads, 0, stream>>>(a);
  else if (a.C <= 1024) add_norm_kernel<TX, TR, 1, 2, CODES><<<four, kThreads, 0, stream>>>(a);
  else if (waves_of(a.C) == 1) add_norm_kernel<TX, TR, 1, 3, CODES><<<four, kThreads, 0, stream>>>(a);
  else if (a.C <= 2048) add_norm_kernel<TX, TR, 4, 1, CODES><<<one, kThreads, 0, stream>>>(a);
  else if (a.C <= 4096) add_norm_kernel<TX, TR, 4, 2, CODES><<<one, kThreads, 0, stream>>>(a);
  else if (a.C <= 8192) add_norm_kernel<TX, TR, 4, 4, CODES><<<one, kThreads, 0, stream>>>(a);
  else add_norm_kernel<TX, TR, 4, 8, CODES><<<one, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}
template <typename TX, typename TR>
hipError_t add_norm_o(const AddNormArgs& a, hipStream_t stream) {
  return a.group < 0 ? add_norm_t<TX, TR, false>(a, stream) : add_norm_t<TX, TR, true>(a, stream);
}

template <typename TX, typename TR>
hipError_t add_norm_bwd_t(const AddNormBwdArgs& a, hipStream_t stream) {
  const int n = (int)bwd_blocks(a.rows, a.C);
  if (n > 0) {
    const dim3 grid((unsigned)n);
    if (a.C <= 512) add_norm_bwd_kernel<TX, TR, 1, 1><<<grid, kThreads, 0, stream>>>(a, n);
    else if (a.C <= 1024) add_norm_bwd_kernel<TX, TR, 1, 2><<<grid, kThreads, 0, stream>>>(a, n);
    else if (waves_of(a.C) == 1) add_norm_bwd_kernel<TX, TR, 1, 3><<<grid, kThreads, 0, stream>>>(a, n);
    else if (a.C <= 2048) add_norm_bwd_kernel<TX, TR, 4, 1><<<grid, kThreads, 0, stream>>>(a, n);
    else if (a.C <= 4096) add_norm_bwd_kernel<TX, TR, 4, 2><<<grid, kThreads, 0, stream>>>(a, n);
    else if (a.C <= 8192) add_norm_bwd_kernel<TX, TR, 4, 4><<<grid, kThreads, 0, stream>>>(a, n);
    else add_norm_bwd_kernel<TX, TR, 4, 8><<<grid, kThreads, 0, stream>>>(a, n);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.d_weight) return hipSuccess;
  weight_join_kernel<<<dim3((unsigned)((a.C + 15) / 16)), kThreads, 0, stream>>>(a.ws, a.d_weight, a.C, n);
  return hipGetLastError();
}

}  // namespace

int64_t add_norm_bwd_ws_floats(int64_t rows, int C) { return bwd_blocks(rows, C) * C; }

hipError_t launch_add_norm(const AddNormArgs& a, hipStream_t stream) {
  if (a.io == DType::F32) return add_norm_o<float, float>(a, stream);
  return a.res_type == DType::F32 ? add_norm_o<bf16, float>(a, stream) : add_norm_o<bf16, bf16>(a, stream);
}

hipError_t launch_add_norm_bwd(const AddNormBwdArgs& a, hipStream_t stream) {
  if (a.io == DType::F32) return add_norm_bwd_t<float, float>(a, stream);
  return a.res_type == DType::F32 ? add_norm_bwd_t<bf16, float>(a, stream) : add_norm_bwd_t<bf16, bf16>(a, stream);
}

#ifdef GDN_CHECK
unsigned check_violations_norm_ops() { return take_check_violations(); }
#endif

}  // namespace gdn
