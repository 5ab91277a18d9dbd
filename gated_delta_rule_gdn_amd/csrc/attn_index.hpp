// attn_index.hpp -- which rows, pages and tokens a workgroup of the attention
// kernels touches, from offsets, lengths and page tables that live on the
// device and may hold anything.  Plain C++, so that the bounds can be checked
// on the host too.
#pragma once

#include <stdint.h>

#ifdef __HIP__
#include <hip/hip_runtime.h>
#define GDN_HD __host__ __device__ __forceinline__
#else
#define GDN_HD inline
#endif

namespace gdn {

GDN_HD int64_t clamp_i64(int64_t x, int64_t lo, int64_t hi) {
  return x < lo ? lo : (x > hi ? hi : x);
}

// Packed offsets: sequence n owns the work items from floor(cu[n] / unit) +
// extra n onwards, so a sequence of L tokens has at least floor(L / unit) +
// extra of them, and all sequences together at most total / unit + extra N.
// The item `idx` is number `item` of sequence n, whose tokens are [start, end)
// (within [0, total]).  For malformed offsets n is some sequence, and item may
// be negative or end before start.
struct PackedItem {
  int64_t n, item, start, end;
};
// mask(lo, step, hi): bit i is set where lo + i step < hi and that sequence's
// first item is at or before idx (i < 64).
template <typename Mask>
GDN_HD PackedItem find_packed_by(const int64_t* cu, int64_t N, int64_t total, int unit, int extra,
                                 int64_t idx, Mask mask) {
  int64_t lo = 0, hi = N;
  while (hi - lo > 1) {
    const int64_t step = (hi - lo + 63) >> 6;
    const uint64_t m = mask(lo, step, hi);
    lo += m ? (63 - __builtin_clzll(m)) * step : 0;
    hi = lo + step < hi ? lo + step : hi;
  }
  PackedItem r;
  r.n = lo;
  r.start = clamp_i64(cu[lo], 0, total);
  r.end = clamp_i64(cu[lo + 1], 0, total);
  r.item = idx - (r.start / unit + extra * lo);
  return r;
}
GDN_HD bool packed_at_or_before(const int64_t* cu, int64_t n, int64_t total, int unit, int extra,
                                int64_t idx) {
  return clamp_i64(cu[n], 0, total) / unit + extra * n <= idx;
}

// Tiles of `unit` tokens of packed sequences, the dear ones first: which tile is
// `rank`-th.  A tile costs as much as its number within the sequence, but no
// more than number `level` (a window).  First come the tiles from `level` on,
// sequence by sequence, so that neighbours follow each other; then the others
// in falling order of their number (equal numbers by sequence).  No sequence has
// more than `most`.  count(f) is the sum of f(n, tiles of n) over the sequences,
// pick(f, k) the k-th sequence (from 0) with f(tiles) true.
GDN_HD int64_t packed_tiles(const int64_t* cu, int64_t n, int64_t total, int unit) {
  const int64_t L = clamp_i64(cu[n + 1], 0, total) - clamp_i64(cu[n], 0, total);
  return L > 0 ? (L + unit - 1) / unit : 0;
}
struct RankedTile {
  int n, item;    // sequence, number of the tile in it; n < 0: none
};
template <typename Count, typename Pick>
GDN_HD RankedTile rank_tile_by(int N, int most, int level, int rank, Count count, Pick pick) {
  const int dear = count([&](int, int c) { return c > level ? c - level : 0; });
  if (rank < dear) {
    // largest n with so many dear tiles before it at most
    int lo = 0, hi = N, before = 0;
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2;
      const int v = count([&](int n, int c) { return n < mid && c > level ? c - level : 0; });
      if (v <= rank) { lo = mid; before = v; } else { hi = mid; }
    }
    return RankedTile{lo, level + rank - before};
  }
  rank -= dear;
  if (count([&](int, int c) { return c < level ? c : level; }) <= rank) return RankedTile{-1, 0};
  // largest j with sum_n max(0, min(tiles_n, level) - j) > rank
  int lo = 0, hi = most < level ? most : level;
  auto from = [&](int j) {
    return count([&](int, int c) { return c > j ? (c < level ? c : level) - j : 0; });
  };
  int above = 0;                            // from(hi)
  while (hi - lo > 1) {
    const int j = lo + (hi - lo) / 2;
    const int v = from(j);
    if (v > rank) { lo = j; } else { hi = j; above = v; }
  }
  return RankedTile{pick([&](int c) { return c > lo; }, rank - above), lo};
}

// New rows [kept, stop) of the j-th page that L new tokens (rows a .. a + L of
// the input) touch behind seq_len held ones; none when kept >= stop.
struct AppendPage {
  int64_t pi;     // page of the sequence: index into its row of the table
  int64_t tok0;   // input row of the page's row 0 (meaningful from `kept` on)
  int kept, stop;
};
GDN_HD AppendPage append_page(int64_t seq_len, int64_t max_pages, int P, int64_t j, int64_t a,
                              int64_t L) {
  AppendPage r{0, 0, 0, 0};
  if (j < 0 || L <= 0) return r;
  const int64_t cap = max_pages * P;
  const int64_t s = clamp_i64(seq_len, 0, cap);
  r.pi = s / P + j;
  int64_t end = s + L < cap ? s + L : cap;
  if (end > (r.pi + 1) * P) end = (r.pi + 1) * P;
  const int64_t first = s > r.pi * P ? s : r.pi * P;
  if (first >= end) return r;
  r.tok0 = a + (r.pi * P - s);
  r.kept = (int)(first - r.pi * P);
  r.stop = (int)(end - r.pi * P);
  return r;
}

// How a decode call divides the caches.  The tokens that a sequence can hold are
// known on the host (the width of the page table), its length is not.
constexpr int kDecodeStep = 32;                     // tokens of a wave's step
constexpr int kDecodeRound = 4 * kDecodeStep;       // of a workgroup's: 4 waves
constexpr int64_t kDecodeBlocks = 512;              // workgroups that fill the chip: 2 to a CU
constexpr int64_t kDecodeDirect = 6 * kDecodeRound; // tokens of a cache that one workgroup takes whole
struct DecodePlan {
  int64_t blocks, rounds;  // workgroups; most rounds of work there can be
  int64_t part_rows;       // rows of a partial result; 0: every workgroup has a whole segment
};
GDN_HD DecodePlan decode_plan(int64_t N, int64_t max_tokens, int64_t window, int Hq, int Hk) {
  // (a window may be as large as its type: nothing is added to it before it is small)
  if (window > 0 && window < max_tokens - kDecodeStep) max_tokens = window + kDecodeStep;
  const int64_t G = Hq / Hk, segments = N * Hk * ((G + 15) / 16);
  const int64_t rounds = segments * ((max_tokens + kDecodeRound - 1) / kDecodeRound);
  if (max_tokens <= kDecodeDirect) return DecodePlan{segments, rounds, 0};
  return DecodePlan{rounds < kDecodeBlocks ? rounds : kDecodeBlocks, rounds, G < 16 ? G : 16};
}

// Tokens [lo, len) that a decode step sees.  They are taken in rounds of
// `round` tokens from `first` on, a multiple of `step`; a sequence without
// tokens has one (empty) round.
struct DecodeSpan {
  int64_t len, lo, first;
  GDN_HD int rounds(int round) const {
    const int64_t r = (len - first + round - 1) / round;
    return r > 0 ? (int)r : 1;
  }
};
GDN_HD DecodeSpan decode_span(int64_t seq_len, int64_t max_pages, int P, int64_t window,
                              int step) {
  DecodeSpan r;
  r.len = clamp_i64(seq_len, 0, max_pages * P);
  r.lo = window && r.len > window ? r.len - window : 0;
  r.first = r.lo / step * step;
  return r;
}
GDN_HD int decode_rounds(int64_t seq_len, int64_t max_pages, int P, int64_t window, int round,
                         int step) {
  return decode_span(seq_len, max_pages, P, window, step).rounds(round);
}

// The rounds of all segments dealt to `blocks` workgroups in order, in shares
// that differ by one at most: block b has rounds [at, at + count).
struct DecodeShare {
  int at, count;
};
GDN_HD DecodeShare decode_share(int total, int blocks, int b) {
  const int each = total / blocks, more = total - each * blocks;
  return DecodeShare{b * each + (b < more ? b : more), each + (b < more ? 1 : 0)};
}
// The block that has round r < total.
GDN_HD int decode_owner(int total, int blocks, int r) {
  const int each = total / blocks, more = total - each * blocks;
  const int in_more = more * (each + 1);
  return r < in_more ? r / (each + 1) : more + (r - in_more) / (each > 0 ? each : 1);
}

}  // namespace gdn
