// The index arithmetic of the attention kernels (attn_index.hpp) on the host,
// over well-formed and malformed offsets, lengths and page tables: every row,
// page and token that a workgroup would touch lies within the tensors, and for
// well-formed input each is touched exactly once.  Prints "ok <items>".
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <vector>

#include "attn_index.hpp"

using namespace gdn;

namespace {
long items = 0;
void need(bool ok, const char* what) {
  if (!ok) { std::printf("violated: %s\n", what); std::exit(1); }
}

PackedItem find(const std::vector<int64_t>& cu, int64_t N, int64_t total, int unit, int extra, int64_t idx) {
  return find_packed_by(cu.data(), N, total, unit, extra, idx, [&](int64_t lo, int64_t step, int64_t hi) {
    uint64_t m = 0;
    for (int64_t lane = 0; lane < 64; ++lane) {
      const int64_t i = lo + lane * step;
      if (i < hi) {
        need(i >= 0 && i < N, "probe within the offsets");
        if (packed_at_or_before(cu.data(), i, total, unit, extra, idx)) m |= 1ull << lane;
      }
    }
    return m;
  });
}

std::vector<int64_t> offsets(std::mt19937& r, int64_t N, int64_t& total, bool good) {
  std::vector<int64_t> cu(N + 1, 0);
  for (int64_t n = 0; n < N; ++n) cu[n + 1] = cu[n] + (r() % 3 ? r() % 300 : r() % 2);
  total = cu[N];
  if (!good)
    for (auto& c : cu)
      if (r() % 3 == 0) c = (int64_t)(r() % 2000) - 500;
  if (!good && r() % 4 == 0) cu[r() % (N + 1)] = r() % 2 ? INT64_MIN : INT64_MAX;
  return cu;
}

void append(std::mt19937& r, bool good) {
  const int64_t N = 1 + r() % (r() % 4 ? 9 : 200);
  int64_t total;
  const auto cu = offsets(r, N, total, good);
  const int P = 16 << (r() % 4);
  const int64_t width = 1 + r() % 30;
  std::vector<int64_t> len(N);
  for (auto& s : len) s = good ? r() % 200 : (int64_t)(r() % 4000) - 1000;
  if (!good) len[r() % N] = r() % 2 ? INT64_MAX : INT64_MIN;
  std::map<std::pair<int64_t, int64_t>, int> written;      // (sequence, position)
  for (int64_t x = 0; x < total / P + 2 * N; ++x, ++items) {
    const PackedItem it = find(cu, N, total, P, 2, x);
    need(it.n >= 0 && it.n < N && it.start >= 0 && it.start <= total && it.end >= 0 && it.end <= total, "sequence");
    const AppendPage a = append_page(len[it.n], width, P, it.item, it.start, it.end - it.start);
    if (a.kept >= a.stop) continue;
    need(a.pi >= 0 && a.pi < width, "entry within the page table");
    need(a.kept >= 0 && a.stop <= P, "rows within the page");
    need(a.tok0 + a.kept >= it.start && a.tok0 + a.stop <= it.end, "input rows within the sequence");
    for (int row = a.kept; row < a.stop; ++row) {
      const int64_t pos = a.pi * P + row;
      if (good) need(a.tok0 + row - it.start == pos - clamp_i64(len[it.n], 0, width * P), "position of the row");
      ++written[{it.n, pos}];
    }
  }
  if (!good) return;
  for (int64_t n = 0; n < N; ++n) {
    const int64_t cap = width * P, s = len[n] < cap ? len[n] : cap;
    for (int64_t p = s; p < s + cu[n + 1] - cu[n] && p < cap; ++p) {
      need((written[{n, p}]) == 1, "each new token written once");
      written.erase({n, p});
    }
  }
  need(written.empty(), "nothing else written");
}

void append_equal(std::mt19937& r) {       // equal numbers of tokens: N ((T + P - 2) / P + 1) workgroups
  const int P = 16 << (r() % 4);
  const int64_t T = 1 + r() % 300, width = 1 + r() % 40, len = (int64_t)(r() % 700) - 20;
  const int64_t cap = width * P, s = clamp_i64(len, 0, cap);
  std::vector<int> seen(cap, 0);
  for (int64_t j = 0; j < (T + P - 2) / P + 1; ++j, ++items) {
    const AppendPage a = append_page(len, width, P, j, 1000, T);
    for (int row = a.kept; row < a.stop; ++row) {
      need(a.pi >= 0 && a.pi < width, "entry within the page table");
      need(a.tok0 + row == 1000 + a.pi * P + row - s, "input row");
      ++seen[a.pi * P + row];
    }
  }
  for (int64_t p = 0; p < cap; ++p) need(seen[p] == (p >= s && p < s + T), "each new token written once");
}

void tiles(std::mt19937& r, bool good) {   // a prefill's query tiles
  const int64_t N = 1 + r() % (r() % 4 ? 9 : 200);
  int64_t total;
  const auto cu = offsets(r, N, total, good);
  const int BM = r() % 2 ? 32 : 128;
  std::vector<int> seen(total, 0);
  for (int64_t x = 0; x < total / BM + N; ++x, ++items) {
    const PackedItem it = find(cu, N, total, BM, 1, x);
    const int64_t L = it.end - it.start, q0 = it.item * BM;
    if (q0 < 0 || q0 >= L) continue;
    for (int64_t q = q0; q < q0 + BM && q < L; ++q) {
      need(it.start + q >= 0 && it.start + q < total, "query row");
      ++seen[it.start + q];
    }
  }
  if (good)
    for (int64_t t = 0; t < total; ++t) need(seen[t] == 1, "each query computed once");
}

void ranked_tiles(std::mt19937& r, bool good) {   // the same tiles, the dear ones first
  const int64_t N = 1 + r() % (r() % 4 ? 9 : 200);
  int64_t total;
  const auto cu = offsets(r, N, total, good);
  const int BM = r() % 2 ? 32 : 128;
  const int level = r() % 2 ? (int)(total / BM) + 1 : 1 + (int)(r() % 6);
  std::vector<int> c(N);
  for (int64_t n = 0; n < N; ++n) c[n] = (int)packed_tiles(cu.data(), n, total, BM);
  auto count = [&](auto f) {
    int v = 0;
    for (int n = 0; n < (int)N; ++n) v += f(n, c[n]);
    return v;
  };
  auto pick = [&](auto f, int k) {
    int n = 0;
    for (; n < (int)N; ++n) if (f(c[n]) && k-- == 0) break;
    return n < (int)N ? n : 0;
  };
  std::vector<int> seen(total, 0);
  int64_t before = INT64_MAX;
  for (int64_t x = 0; x < total / BM + N; ++x, ++items) {
    const RankedTile it = rank_tile_by((int)N, (int)((total + BM - 1) / BM), level, (int)x, count, pick);
    if (it.n < 0) continue;
    need(it.n < N, "sequence");
    const int64_t start = clamp_i64(cu[it.n], 0, total), L = clamp_i64(cu[it.n + 1], 0, total) - start;
    const int64_t q0 = (int64_t)it.item * BM;
    if (q0 < 0 || q0 >= L) continue;
    const int64_t cost = it.item < level ? it.item : level;
    need(cost <= before, "falling order of the costs");
    before = cost;
    for (int64_t q = q0; q < q0 + BM && q < L; ++q) {
      need(start + q >= 0 && start + q < total, "query row");
      ++seen[start + q];
    }
  }
  if (good)
    for (int64_t t = 0; t < total; ++t) need(seen[t] == 1, "each query computed once");
}

void decode(std::mt19937& r) {
  const int P = 16 << (r() % 4), step = 32, round = 128;
  const int64_t width = 1 + r() % 50, cap = width * P;
  const int64_t window = r() % 2 ? 0 : 1 + r() % (2 * cap);
  int64_t len = (int64_t)(r() % (2 * cap + 40)) - 20;
  if (r() % 20 == 0) len = r() % 2 ? INT64_MAX : INT64_MIN;
  const int64_t L = clamp_i64(len, 0, cap), lo = window && L > window ? L - window : 0;
  const DecodeSpan d = decode_span(len, width, P, window, step);
  need(d.len == L && d.lo == lo && d.first <= lo && d.first % step == 0 && d.first > lo - step, "range");
  const int rounds = decode_rounds(len, width, P, window, round, step);
  const int64_t most = window > 0 && window + step < cap ? window + step : cap;
  need(rounds >= 1 && rounds <= (most + round - 1) / round, "rounds within what the host expects");
  std::vector<int> seen(cap, 0);
  for (int i = 0; i < rounds; ++i, ++items)
    for (int64_t t0 = d.first + (int64_t)i * round; t0 < d.first + (int64_t)(i + 1) * round; t0 += step)
      for (int64_t tile = t0; tile < t0 + step; tile += 16) {
        if (tile >= d.len) continue;
        need(tile >= 0 && tile / P < width && tile % P + 16 <= P, "tile within a page of the table");
        for (int64_t t = tile; t < tile + 16; ++t)
          if (t >= d.lo && t < d.len) ++seen[t];
      }
  for (int64_t t = 0; t < cap; ++t) need(seen[t] == (t >= lo && t < L), "each token seen once");
}
}  // namespace

int main() {
  std::mt19937 r(1);
  for (int i = 0; i < 1500; ++i) {
    append(r, true);
    append(r, false);
    append_equal(r);
    tiles(r, true);
    tiles(r, false);
    ranked_tiles(r, true);
    ranked_tiles(r, false);
    decode(r);
  }
  std::printf("ok %ld\n", items);
  return 0;
}
