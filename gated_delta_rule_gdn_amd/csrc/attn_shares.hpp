// attn_shares.hpp -- how the walks of the key tiles of a backward call are dealt to
// workgroups in equal shares.  Plain C++, so that it can be checked on the host too.
#pragma once

#include "attn_index.hpp"

namespace gdn {

// A key tile of `rows` keys is walked in steps of `step` queries (rows % step == 0), all
// that see it of each of the G query heads of its key head.  Its cost is that many units
// and `lead` more for what stands before and behind a walk.
struct WalkUnits {
  int64_t window;                     // 0: none
  int rows, step, G, lead;

  GDN_HD int64_t tiles(int64_t L) const { return (L + rows - 1) / rows; }
  // steps of the tile j of a sequence of L tokens, for one query head
  GDN_HD int64_t steps(int64_t L, int64_t j) const {
    const int64_t all = (L + step - 1) / step - rows / step * j, cap = most(L);
    return all < cap ? all : cap;
  }
  // units of its tiles before tile j
  GDN_HD int64_t before(int64_t L, int64_t j) const {
    const int64_t a = (L + step - 1) / step, m = rows / step, cap = most(L);
    int64_t capped = a > cap ? (a - cap + m - 1) / m : 0;   // tiles that see a whole window
    if (capped > j) capped = j;
    const int64_t s = capped * (capped > 0 ? cap : 0) + (j - capped) * a -
                      m * (j * (j - 1) / 2 - capped * (capped - 1) / 2);
    return G * s + lead * j;
  }
  GDN_HD int64_t units(int64_t L) const { return before(L, tiles(L)); }
  // the tile that has unit r < units(L)
  GDN_HD int64_t tile_at(int64_t L, int64_t r) const {
    int64_t lo = 0, hi = tiles(L);
    while (hi - lo > 1) {
      const int64_t mid = lo + (hi - lo) / 2;
      if (before(L, mid) <= r) lo = mid; else hi = mid;
    }
    return lo;
  }

 private:
  GDN_HD int64_t most(int64_t L) const {
    return window > 0 && window < L ? (rows - 1 + window + step - 1) / step : INT64_MAX / 4;
  }
};

// `total` units in shares that differ by one at most, to as many of the workers as get
// `least` of them.
struct Shares {
  int64_t each, more;
  int workers;
  GDN_HD int64_t begin(int64_t w) const { return w * each + (w < more ? w : more); }
  GDN_HD int owner(int64_t x) const {     // the worker of unit x
    const int64_t in_more = more * (each + 1);
    return (int)(x < in_more ? x / (each + 1) : more + (x - in_more) / (each > 0 ? each : 1));
  }
};
GDN_HD Shares shares_of(int64_t total, int workers, int64_t least) {
  int64_t n = total / least;
  n = n < 1 ? 1 : (n > workers ? workers : n);
  return Shares{total / n, total % n, (int)n};
}

// The part [s0, s1) of a tile's steps (over all G heads) that the units [x, end) of a
// share hold, the tile beginning at unit `from`: none where s1 <= s0.  Steps behind the
// first are another worker's part of the same tile.
struct WalkPart {
  int64_t s0, s1, all, next;              // next: the unit behind the part
  GDN_HD bool whole() const { return s0 == 0 && s1 == all; }
};
GDN_HD WalkPart part_of(const WalkUnits& u, int64_t L, int64_t j, int64_t from, int64_t x, int64_t end) {
  WalkPart p;
  p.all = u.G * u.steps(L, j);
  const int64_t stop = from + u.lead + p.all;
  p.next = end < stop ? end : stop;
  p.s0 = x - from > u.lead ? x - from - u.lead : 0;
  p.s1 = p.next - from - u.lead;
  return p;
}

}  // namespace gdn
