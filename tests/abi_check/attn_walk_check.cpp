// The shares of a backward call's walks (attn_shares.hpp) against counting one by one:
// steps and units of tiles, the tile of a unit, shares that are equal to within one and
// cover every step of every tile once and in order, and the owners of the parts.
// Prints "ok <checks>".
#include <cstdint>
#include <cstdio>
#include <vector>

#include "attn_shares.hpp"

using namespace gdn;

namespace {

long checks = 0, failures = 0;
void must(bool ok, const char* what, long a = 0, long b = 0, long c = 0) {
  ++checks;
  if (!ok && ++failures < 20) std::printf("%s: %ld %ld %ld\n", what, a, b, c);
}

// steps of `step` queries from the tile's first key on that see one of its keys
int64_t count_steps(int64_t L, int64_t k0, int rows, int step, int64_t window) {
  int64_t last = -1;
  for (int64_t t = k0; t < L; ++t) {
    const int64_t lo = window && t - window + 1 > 0 ? t - window + 1 : 0;
    const int64_t hi = t;                  // sees keys lo .. hi
    if (hi >= k0 && lo < k0 + rows) last = t;
  }
  return last < 0 ? 0 : (last - k0) / step + 1;
}

void tiles_of_a_sequence(const WalkUnits& u, int64_t L) {
  int64_t sum = 0;
  for (int64_t j = 0; j < u.tiles(L); ++j) {
    must(u.before(L, j) == sum, "units before a tile", L, j, u.window);
    const int64_t n = u.steps(L, j);
    must(n == count_steps(L, j * u.rows, u.rows, u.step, u.window < L ? u.window : 0), "steps of a tile", L, j, u.window);
    must(n > 0, "a tile without steps", L, j);
    for (int64_t r : {sum, sum + (u.G * n + u.lead) / 2, sum + u.G * n + u.lead - 1})
      must(u.tile_at(L, r) == j, "tile of a unit", L, j, r);
    sum += u.G * n + u.lead;
  }
  must(u.units(L) == sum, "units of a sequence", L);
}

struct TileAt { int64_t L, j, from, all; };

void shares_of_all(const WalkUnits& u, const std::vector<int64_t>& lens, int Hk, int workers, int64_t least) {
  std::vector<TileAt> tiles;
  int64_t total = 0;
  for (int64_t L : lens)
    for (int h = 0; h < Hk; ++h)
      for (int64_t j = 0; j < u.tiles(L); ++j) {
        const int64_t all = u.G * u.steps(L, j);
        tiles.push_back(TileAt{L, j, total, all});
        total += u.lead + all;
      }
  if (total == 0) return;
  const Shares s = shares_of(total, workers, least);
  must(s.workers >= 1 && s.workers <= workers && s.begin(0) == 0 && s.begin(s.workers) == total, "shares", total);
  std::vector<int64_t> done(tiles.size(), 0);
  std::vector<int> opened(tiles.size(), -1);
  for (int w = 0; w < s.workers; ++w) {
    const int64_t x0 = s.begin(w), x1 = s.begin(w + 1);
    must(x1 - x0 == s.each || x1 - x0 == s.each + 1, "size of a share", w, x1 - x0, s.each);
    int64_t x = x0;
    int parts = 0;
    for (size_t i = 0; i < tiles.size() && x < x1; ++i) {
      const TileAt& t = tiles[i];
      const int64_t end = t.from + u.lead + t.all;
      if (x >= end || x1 <= t.from) continue;
      const WalkPart p = part_of(u, t.L, t.j, t.from, x, x1);
      must(p.all == t.all && p.next > x && p.next <= x1, "progress", w, (long)i);
      if (p.s1 > p.s0) {
        must(p.s0 == done[i] && p.s1 <= t.all, "order of a tile's parts", w, (long)i, p.s0);
        done[i] = p.s1;
        if (p.s0 == 0 && !p.whole()) { opened[i] = w; must(p.next == x1, "a tile left open ends the share", w); }
        if (p.s0 > 0) { must(x == x0, "a tile gone on with begins the share", w); }
        if (p.s0 > 0 && p.s1 == t.all) {
          must(opened[i] >= 0 && opened[i] + (s.owner(end - 1) - opened[i]) == w, "last owner", w, (long)i);
        }
        if (!p.whole()) ++parts;
      }
      for (int64_t y : {x, p.next - 1}) must(s.owner(y) == w, "owner", w, y);
      x = p.next;
    }
    must(x == x1 && parts <= 2, "the share's end", w, x, x1);
  }
  for (size_t i = 0; i < tiles.size(); ++i) must(done[i] == tiles[i].all, "every step once", (long)i, done[i], tiles[i].all);
}

}  // namespace

int main() {
  for (int rows : {32, 128})
    for (int64_t window : {(int64_t)0, (int64_t)1, (int64_t)20, (int64_t)64, (int64_t)129, (int64_t)1000, INT64_MAX})
      for (int G : {1, 3, 8})
        for (int lead : {0, 1, 4}) {
          const WalkUnits u{window, rows, rows == 32 ? 32 : 64, G, lead};
          for (int64_t L : {1, 2, 31, 32, 33, 64, 65, 127, 128, 129, 191, 192, 193, 500, 1025, 1500}) tiles_of_a_sequence(u, L);
          must(u.units(0) == 0 && u.tiles(0) == 0, "no tokens");
          for (int workers : {8, 64, 512})
            for (int64_t least : {1, 3, 8})
              for (const std::vector<int64_t>& lens : std::vector<std::vector<int64_t>>{
                       {1}, {300, 0, 5, 129}, {1500}, {64, 64, 64, 64, 64}, {0, 0, 700, 1, 1, 1}, {2000, 3}})
                shares_of_all(u, lens, G == 3 ? 2 : 1, workers, least);
        }
  // far from any overflow: 2^31 tokens, 128 heads of 16
  const WalkUnits big{0, 128, 64, 16, 4};
  must(big.units((int64_t)1 << 31) > 0 && big.before((int64_t)1 << 31, 1 << 20) > 0, "long sequences");
  if (failures) return 1;
  std::printf("ok %ld\n", checks);
  return 0;
}
