// How a decode call divides the caches (attn_index.hpp), on the host under the
// sanitizers: windows up to the largest of their type add up without overflow,
// a window that hides nothing gives the plan of none, and no cache has more
// rounds than the plan says.  Prints "ok <plans>".
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "attn_index.hpp"

using namespace gdn;

int main() {
  long n = 0;
  const int64_t most = INT64_MAX;
  for (int64_t width : {1, 2, 7, 12, 48, 2048, 1 << 20})
    for (int P : {16, 32, 64, 128})
      for (int Hk : {1, 4})
        for (int G : {1, 8, 16, 21}) {
          const int64_t cap = width * P;
          const DecodePlan all = decode_plan(3, cap, 0, G * Hk, Hk);
          for (int64_t w : {most, most - 1, most - 31, most - 32, most / 2, cap, cap - 1, cap - 31, cap - 32, cap - 33,
                            (int64_t)1, (int64_t)700, (int64_t)737}) {
            if (w < 1) continue;
            ++n;
            const DecodePlan p = decode_plan(3, cap, w, G * Hk, Hk);
            bool ok = p.blocks >= 1 && p.blocks <= all.rounds && p.rounds <= all.rounds;
            if (w >= cap) ok = ok && p.blocks == all.blocks && p.rounds == all.rounds && p.part_rows == all.part_rows;
            const int64_t per = p.rounds / (3 * Hk * ((G + 15) / 16));     // of one segment
            for (int64_t len : {(int64_t)0, w < cap ? w : cap, cap - 1, cap, most})
              ok = ok && decode_rounds(len, width, P, w, kDecodeRound, kDecodeStep) <= per;
            if (p.part_rows == 0) ok = ok && per <= kDecodeDirect / kDecodeRound;
            if (!ok) {
              std::printf("width %ld P %d G %d window %ld: %ld workgroups, %ld rounds, rows %ld\n", (long)width, P, G,
                          (long)w, (long)p.blocks, (long)p.rounds, (long)p.part_rows);
              return 1;
            }
          }
        }
  std::printf("ok %ld plans\n", n);
  return 0;
}
