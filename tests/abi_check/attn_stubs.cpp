// Host-only stand-ins for the attention kernels' launchers, so that
// attn_api.cpp can be built with g++ under the sanitizers and driven without a
// GPU.  The functions of sizes are the formulas of the kernels' host code.
#include <hip/hip_runtime.h>

#include "attn_kernels.hpp"

long g_launches = 0;

namespace gdn {
int64_t qk_norm_rope_blocks(int64_t rows, int Hq, int Hk, int) {
  return (rows + 31) / 32 * ((Hq + 3) / 4 + (Hk + 3) / 4);
}
int64_t kv_append_slots(int64_t N, int64_t total_T, int64_t Tseq, bool packed, int P) {
  return packed ? total_T / P + 2 * N : N * ((Tseq + P - 2) / P + 1);
}
int64_t prefill_blocks(int64_t N, int64_t total_T, int64_t Tseq, bool packed, int Hq, DType) {
  return (packed ? total_T / 32 + N : N * ((Tseq + 31) / 32)) * Hq;
}
AttnDecodePlan attn_decode_plan(int64_t N, int64_t max_tokens, int64_t, int Hq, int Hk, int d) {
  const int64_t rounds = N * Hk * ((Hq / Hk + 15) / 16) * ((max_tokens + 127) / 128);
  const int64_t b = rounds < 512 ? rounds : 512;
  return AttnDecodePlan{b, rounds, max_tokens > 512 ? b * (2 * 16 * (d + 4) + 2) : 0};
}
hipError_t launch_qk_norm_rope(const QkNormRopeArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_kv_append(const KvAppendArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_attn_prefill(const PrefillArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_attn_decode(const AttnDecodeArgs&, hipStream_t) { ++g_launches; return hipSuccess; }
}  // namespace gdn
