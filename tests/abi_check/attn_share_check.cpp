// The shares that a decode step's rounds are dealt in: consecutive, complete,
// equal to within one, and every round's owner the block that has it.
#include <cstdio>
#include <initializer_list>

#include "attn_index.hpp"

int main() {
  long n = 0;
  for (int blocks : {1, 2, 3, 7, 64, 200, 511, 512})
    for (int total = 0; total < 1700; total += total < 40 ? 1 : 37) {
      int at = 0;
      for (int b = 0; b < blocks; ++b, ++n) {
        const gdn::DecodeShare s = gdn::decode_share(total, blocks, b);
        const int least = total / blocks;
        bool ok = s.at == at && (s.count == least || s.count == least + 1);
        for (int r = s.at; r < s.at + s.count; ++r) ok = ok && gdn::decode_owner(total, blocks, r) == b;
        if (!ok) { printf("blocks %d total %d block %d\n", blocks, total, b); return 1; }
        at += s.count;
      }
      if (at != total) { printf("blocks %d total %d: %d dealt\n", blocks, total, at); return 1; }
    }
  const int big = 0x7fffff00;              // as many rounds as the host lets pass
  for (int b : {0, 1, 255, 511}) {
    const gdn::DecodeShare s = gdn::decode_share(big, 512, b);
    if (gdn::decode_owner(big, 512, s.at) != b || gdn::decode_owner(big, 512, s.at + s.count - 1) != b) return 1;
  }
  printf("ok %ld shares\n", n);
}
