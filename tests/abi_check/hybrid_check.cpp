// Drives every entry point of hybrid_api.cpp over a grid of descriptors from valid to
// absurd, with fake device addresses and launchers that only count.  Under
// -fsanitize=address,undefined any signed overflow or out-of-bounds access in the
// validation aborts the run; a call that returns an error must have launched nothing,
// and small valid calls must launch.  Prints "ok <calls>".
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "gdn_hybrid.h"
#include "hybrid_kernels.hpp"

static long g_launches = 0;

// Stand-ins for the kernels' host code.
namespace gdn {
int64_t prefill_blocks(int64_t N, int64_t total_T, int64_t Tseq, bool packed, int Hq, DType) {
  return (packed ? total_T / 32 + N : N * ((Tseq + 31) / 32)) * Hq;
}
AttnBwdPlan attn_bwd_plan(int64_t, int64_t total_T, int64_t, int Hq, int Hk, int d, DType) {
  return AttnBwdPlan{8, 4 * total_T * Hq + 8 * total_T * Hk * 2 * d};
}
int64_t attn_bwd_blocks(int64_t N, int64_t total_T, int64_t Tseq, bool packed, int Hq, DType) {
  return (packed ? total_T / 32 + N : N * ((Tseq + 31) / 32)) * Hq;
}
int64_t qk_bwd_ws_floats(int64_t rows, int Hq, int Hk, int d) { return rows > 0 ? ((int64_t)Hq + Hk) * 8 * d : 0; }
int64_t add_norm_bwd_ws_floats(int64_t rows, int C) { return (rows < 512 ? rows : 512) * C; }
hipError_t launch_attn_prefill(const PrefillArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_attn_bwd(const AttnBwdArgs&, const AttnBwdPlan&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_qk_norm_rope_bwd(const QkNormRopeBwdArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_add_norm(const AddNormArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_add_norm_bwd(const AddNormBwdArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
}  // namespace gdn

namespace {

long calls = 0, failures = 0;

void* P(int i) { return reinterpret_cast<void*>((uintptr_t)(i + 1) << 44); }
float* F(int i) { return static_cast<float*>(P(i)); }
const int64_t* I(int i) { return static_cast<const int64_t*>(P(i)); }

void check(gdn_status st, long before, const char* what) {
  ++calls;
  if (st < GDN_OK || st > GDN_ERR_HIP || (st != GDN_OK && g_launches != before)) {
    std::printf("%s: status %d, %ld launches\n", what, (int)st, g_launches - before);
    ++failures;
  }
}
void must(bool ok, const char* what) {
  ++calls;
  if (!ok) { std::printf("%s\n", what); ++failures; }
}

const int64_t kSizes[] = {-1, 0, 1, 17, 4096, (int64_t)1 << 31, INT64_MAX};
const int64_t kLds[] = {-8, 0, 128, 512, 1 << 20, ((int64_t)1 << 31) - 8, INT64_MAX};
const int32_t kHeads[] = {-1, 0, 1, 4, 65536, INT32_MAX};
const int32_t kDims[] = {-1, 0, 64, 128, 256, 16384, INT32_MAX};
const int32_t kTypes[] = {-1, GDN_F32, GDN_BF16, 5};
const int32_t kGroups[] = {-2, -1, 0, 32, 48, 128, INT32_MAX};
const float kFloats[] = {1.f, 0.f, -1.f, NAN, INFINITY, 1e-38f};

void fuzz() {
  for (int64_t n : kSizes)
    for (int64_t t : kSizes)
      for (int32_t h : kHeads)
        for (int32_t d : kDims)
          for (int32_t io : kTypes)
            for (int64_t ld : kLds)
              for (float f : kFloats) {
                long b = g_launches;
                gdn_attn_prefill_desc p{n, t, ld, ld, ld, n, h, h, d, io, f};
                check(gdn_attn_prefill_save(&p, nullptr, P(0), P(1), P(2), P(3), F(4), nullptr), b, "save");
                for (int32_t g : kTypes) {
                  gdn_attn_bwd_desc w{n, t, ld, ld, ld, ld, ld, ld, n, h, h, d, io, g, f};
                  (void)gdn_attn_backward_workspace_size(&w);
                  b = g_launches;
                  check(gdn_attn_backward(&w, I(11), P(0), P(1), P(2), P(3), P(4), F(5), P(6), SIZE_MAX, P(7), P(8),
                                          P(9), nullptr), b, "backward");
                  gdn_qk_bwd_desc q{t, ld, ld, ld, ld, h, 1, d, 64, GDN_ROPE_HALF, io, g, f, 1e-6f};
                  (void)gdn_qk_norm_rope_backward_workspace_size(&q);
                  b = g_launches;
                  check(gdn_qk_norm_rope_backward(&q, h > 0 ? P(0) : nullptr, P(1), h > 0 ? P(2) : nullptr, P(3),
                                                  nullptr, F(4), I(5), F(6), P(7), SIZE_MAX, h > 0 ? P(8) : nullptr,
                                                  P(9), nullptr, F(10), nullptr), b, "rope");
                }
              }
  for (int64_t r : kSizes)
    for (int64_t ld : kLds)
      for (int32_t C : kDims)
        for (int32_t io : kTypes)
          for (int32_t rt : kTypes)
            for (float eps : kFloats) {
              for (int32_t g : kGroups) {
                const long b = g_launches;
                gdn_add_norm_desc a{r, ld, C, io, rt, g, eps};
                check(gdn_add_norm(&a, P(0), P(1), F(2), P(3), P(4), g < 0 ? nullptr : F(5), nullptr), b, "norm");
              }
              const long b = g_launches;
              gdn_add_norm_bwd_desc w{r, ld, C, io, rt, eps};
              (void)gdn_add_norm_backward_workspace_size(&w);
              check(gdn_add_norm_backward(&w, P(0), P(1), F(2), P(3), P(4), SIZE_MAX, P(5), P(6), F(7), nullptr), b,
                    "norm backward");
            }
}

void small_calls_launch() {
  long b = g_launches;
  gdn_attn_bwd_desc w{2, 8, 1024, 1024, 1024, 1024, 1024, 1024, 0, 4, 2, 128, GDN_BF16, GDN_BF16, 0.1f};
  char* x = static_cast<char*>(P(7));
  const size_t need = gdn_attn_backward_workspace_size(&w);
  must(gdn_attn_backward(&w, nullptr, P(0), P(1), P(2), P(3), P(4), F(5), P(6), need, x, x + 1024, x + 1536, nullptr) ==
           GDN_OK && g_launches == b + 1, "column blocks of one buffer");
  b = g_launches;
  gdn_qk_bwd_desc q{8, 512, 256, 512, 256, 4, 2, 128, 0, GDN_ROPE_HALF, GDN_BF16, GDN_F32, 1.f, 0.f};
  must(gdn_qk_norm_rope_backward(&q, P(0), P(1), nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, P(0),
                                 P(1), nullptr, nullptr, nullptr) == GDN_OK && g_launches == b + 1, "in place");
  b = g_launches;
  gdn_add_norm_desc a{8, 256, 256, GDN_BF16, GDN_BF16, -1, 0.f};
  must(gdn_add_norm(&a, P(0), P(1), nullptr, P(1), P(0), nullptr, nullptr) == GDN_OK && g_launches == b + 1,
       "norm in place");
  b = g_launches;
  gdn_add_norm_bwd_desc v{8, 256, 256, GDN_BF16, GDN_F32, 0.f};
  must(gdn_add_norm_backward(&v, P(0), P(1), nullptr, P(3), nullptr, 0, P(0), P(3), nullptr, nullptr) == GDN_OK &&
           g_launches == b + 1, "norm backward in place");
}

}  // namespace

int main() {
  fuzz();
  small_calls_launch();
  must(g_launches > 100, "the grid holds valid calls");
  if (failures) return 1;
  std::printf("ok %ld\n", calls);
  return 0;
}
