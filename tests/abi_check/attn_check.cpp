// Drives every entry point of attn_api.cpp (built with attn_stubs.cpp) over a
// grid of descriptors from valid to absurd, with fake device addresses.  Under
// -fsanitize=address,undefined any signed overflow or out-of-bounds access in
// the validation aborts the run; a call that returns an error must have
// launched nothing, and small valid calls must launch.  Prints "ok <calls>".
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "gdn_attn.h"

extern long g_launches;

namespace {

long calls = 0, failures = 0;

void* P(int i) { return reinterpret_cast<void*>((uintptr_t)(i + 1) << 44); }
float* F(int i) { return static_cast<float*>(P(i)); }
const int64_t* I(int i) { return static_cast<const int64_t*>(P(i)); }
const int32_t* T(int i) { return static_cast<const int32_t*>(P(i)); }

void check(gdn_status st, long before, const char* what) {
  ++calls;
  if (st < GDN_OK || st > GDN_ERR_HIP || (st != GDN_OK && g_launches != before)) {
    std::printf("%s: status %d, %ld launches\n", what, (int)st, g_launches - before);
    ++failures;
  }
}

const int64_t kSizes[] = {-1, 0, 1, 17, 4096, (int64_t)1 << 31, INT64_MAX};
const int64_t kLds[] = {-8, 0, 128, 512, 1 << 20, ((int64_t)1 << 31) - 8, INT64_MAX};
const int32_t kHeads[] = {-1, 0, 1, 4, 65536, INT32_MAX};
const int32_t kDims[] = {-1, 0, 64, 128, 256};
const int32_t kTypes[] = {-1, GDN_F32, GDN_BF16, 5};
const int32_t kPages[] = {-1, 0, 16, 24, 128, INT32_MAX};
const int32_t kRope[] = {-16, 0, 8, 64, 128, INT32_MAX};
const float kFloats[] = {1.f, 0.f, -1.f, NAN, INFINITY};

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
                check(gdn_attn_prefill(&p, nullptr, P(0), P(1), P(2), P(3), nullptr), b, "prefill");
                b = g_launches;
                check(gdn_attn_prefill(&p, I(4), P(0), P(1), P(2), P(3), nullptr), b, "prefill cu");
                for (int32_t rd : kRope) {
                  gdn_qk_desc q{t, ld, ld, h, 1, d, rd, GDN_ROPE_HALF, io, f, 1e-6f};
                  b = g_launches;
                  check(gdn_qk_norm_rope(&q, h > 0 ? P(0) : nullptr, P(1), F(2), F(3),
                                         rd ? I(4) : nullptr, rd ? F(5) : nullptr,
                                         h > 0 ? P(6) : nullptr, P(7), nullptr), b, "norm_rope");
                }
              }
  for (int64_t n : kSizes)
    for (int64_t t : kSizes)
      for (int64_t pages : kSizes)
        for (int64_t width : kSizes)
          for (int32_t h : kHeads)
            for (int32_t ps : kPages)
              for (int32_t d : {64, 128})
                for (float f : kFloats) {
                  long b = g_launches;
                  gdn_attn_decode_desc a{n, pages, width, t, h, h, d, ps, GDN_BF16, f};
                  (void)gdn_attn_decode_workspace_size(&a);
                  check(gdn_attn_decode(&a, P(0), P(1), P(2), F(3), F(4), T(5), I(6), P(7), P(8),
                                        (size_t)1 << 43, nullptr), b, "decode");
                  gdn_kv_append_desc k{n, t, 512, 512, pages, width, h, d, ps, 64,
                                       GDN_ROPE_INTERLEAVED, GDN_BF16, f, 1e-6f};
                  for (const int64_t* cu : {(const int64_t*)nullptr, I(11)}) {
                    b = g_launches;
                    check(gdn_kv_append(&k, cu, I(0), T(1), P(2), P(3), F(4), F(5), P(6), P(7),
                                        F(8), F(9), nullptr), b, "append");
                  }
                }
}

void must_launch(gdn_status st, long before, const char* what) {
  check(st, before, what);
  if (st != GDN_OK || g_launches != before + 1) {
    std::printf("%s: a valid call did not launch (status %d)\n", what, (int)st);
    ++failures;
  }
}

}  // namespace

int main() {
  fuzz();
  long b = g_launches;
  gdn_qk_desc q{5, 768, 768, 4, 1, 128, 64, GDN_ROPE_HALF, GDN_BF16, 1.f, 1e-6f};
  must_launch(gdn_qk_norm_rope(&q, P(0), P(1), F(2), F(3), I(4), F(5), P(6), P(7), nullptr), b, "norm_rope");
  b = g_launches;
  gdn_kv_append_desc k{3, 9, 512, 512, 10, 4, 2, 128, 16, 0, GDN_ROPE_HALF, GDN_F32, 1.f, 1e-6f};
  must_launch(gdn_kv_append(&k, nullptr, I(0), T(1), P(2), P(3), nullptr, nullptr, P(6), P(7), F(8), F(9),
                            nullptr), b, "append");
  b = g_launches;
  gdn_attn_prefill_desc p{3, 9, 512, 512, 512, 0, 4, 2, 128, GDN_BF16, -0.1f};
  must_launch(gdn_attn_prefill(&p, nullptr, P(0), P(1), P(2), P(3), nullptr), b, "prefill");
  b = g_launches;
  gdn_attn_decode_desc a{3, 10, 4, 0, 4, 2, 128, 16, GDN_BF16, 0.1f};
  must_launch(gdn_attn_decode(&a, P(0), P(1), P(2), F(3), F(4), T(5), I(6), P(7), nullptr, 0, nullptr), b, "decode");
  for (gdn_status st : {gdn_qk_norm_rope(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr),
                        gdn_kv_append(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                      nullptr, nullptr, nullptr, nullptr),
                        gdn_attn_prefill(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr),
                        gdn_attn_decode(nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr,
                                        nullptr, 0, nullptr)})
    if (st != GDN_ERR_INVALID_ARG) ++failures;
  if (gdn_attn_decode_workspace_size(nullptr) != 0 || gdn_attn_abi_version() != GDN_ATTN_ABI_VERSION) ++failures;
  if (failures) return 1;
  std::printf("ok %ld\n", calls);
  return 0;
}
