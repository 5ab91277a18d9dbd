// attn_tiles.hpp -- which tile of which sequence and head a workgroup of the
// attention kernels has, and the loads that bring tiles straight into LDS.
#pragma once

#include "attn_device.hpp"

namespace gdn {

// Sequences, key heads and the G workgroups that each tile of a key head has.
struct TileArgs {
  const int64_t* cu_seqlens;          // device [N + 1] or NULL
  int64_t N, Tseq, total_T, window;
  int Hk, G;
};

// One workgroup's query tile: queries [q0, q0 + BM) of the sequence that is
// rows [a, a + L) of the packed tensors, and a query head.
struct Tile {
  int64_t a, L, q0;
  int hq;
  bool valid;
};

// Workgroup blk runs on XCD blk % 8, and each XCD has an L2 of its own, so the
// workgroups that follow each other on an XCD should read the same keys and
// values; and a query tile costs as many key tiles as lie before it, so the
// late tiles should start first.  The query heads of a key head always follow
// each other.  (All counts fit in 32 bits: the host bounds the grid.)
//
// Equal lengths, key heads of all sequences a multiple of 8: an XCD keeps its
// share of them, in groups of 4 query heads or more, and goes through each
// group's tiles from the last to the first.  64 workgroups
// of an XCD then walk the keys of 4 heads together (B 8, T 4096, 16 heads:
// 78 % of the L2 reads hit against 48 % with heads dealt round the XCDs).
// Otherwise tiles are dealt round the XCDs, the last tiles of all sequences
// first.
//
// Packed lengths: the tiles are dealt round the XCDs, the dear ones first
// (rank_tile_by): found by counting, so nothing is sorted.  (16 prompts, 32768
// tokens, a window of 2048: 367 us; in the order of the tokens 383 us.)
constexpr uint32_t kXcds = 8;
constexpr int64_t kMaxRanked = 1024;      // sequences that are ranked; more keep their order

template <int BM>
__device__ __forceinline__ Tile find_tile(const TileArgs& p, uint32_t blk, uint32_t blocks) {
  Tile t;
  const uint32_t G = (uint32_t)p.G, Hk = (uint32_t)p.Hk, N = (uint32_t)p.N;
  const uint32_t per = blocks / kXcds;                    // full rounds over the XCDs
  const uint32_t xcd = blk % kXcds, i = blk / kXcds;
  t.valid = true;
  if (!p.cu_seqlens) {
    const uint32_t tiles = ((uint32_t)p.Tseq + BM - 1) / BM, pairs = N * Hk;
    const uint32_t mine = pairs / kXcds;                  // pairs of an XCD
    uint32_t pair, tile, head;
    if (pairs % kXcds == 0) {
      const uint32_t gp = G >= 4 ? 1 : 4 / G;             // pairs of a group
      const uint32_t grp = i / (gp * tiles * G), w = i - grp * (gp * tiles * G);
      const uint32_t here = mine - grp * gp < gp ? mine - grp * gp : gp;
      const uint32_t level = w / (here * G), x = w - level * (here * G);
      tile = tiles - 1 - level;
      pair = xcd + kXcds * (grp * gp + x / G);
      head = x % G;
    } else {
      // unit = (tile from the last, pair); the last partial round is dealt plainly
      uint32_t unit;
      const uint32_t rounds = per / G;
      if (i < rounds * G) { unit = i / G * kXcds + xcd; head = i % G; }
      else { const uint32_t r = blk - rounds * G * kXcds; unit = rounds * kXcds + r / G; head = r % G; }
      tile = tiles - 1 - unit / pairs;
      pair = unit % pairs;
    }
    const uint32_t n = pair / Hk, hk = pair - n * Hk;
    t.a = n * p.Tseq;
    t.L = p.Tseq;
    t.q0 = (int64_t)tile * BM;
    t.hq = (int)(hk * G + head);
    return t;
  }
  uint32_t unit, head;
  const uint32_t rounds = per / G;
  if (i < rounds * G) {
    unit = i / G * kXcds + xcd;
    head = i % G;
  } else {
    const uint32_t r = blk - rounds * G * kXcds;
    unit = rounds * kXcds + r / G;
    head = r % G;
  }
  const uint32_t rank = unit / Hk;
  t.hq = (int)((unit - rank * Hk) * G + head);
  PackedItem it;
  // tiles from this number on see a whole window
  const int level = (int)((p.window > 0 && p.window < p.total_T ? p.window : p.total_T) + BM - 1) / BM;
  if (p.N <= 64)
    it = rank_tile<1>(p.cu_seqlens, (int)p.N, p.total_T, BM, level, (int)rank);
  else if (p.N <= kMaxRanked)
    it = rank_tile<kMaxRanked / 64>(p.cu_seqlens, (int)p.N, p.total_T, BM, level, (int)rank);
  else
    it = find_packed(p.cu_seqlens, p.N, p.total_T, BM, 1, (int64_t)rank);
  t.a = it.start;
  t.L = it.end - it.start;
  t.q0 = it.item * BM;
  t.valid = t.q0 >= 0 && t.q0 < t.L;
  return t;
}

__device__ __forceinline__ bf16x4 read_tr16(const bf16* p) {
  lds_check(p, 8);
  typedef short v4s __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) v4s*)(p)));
}

// 16 bytes for each lane from base + voff + soff straight into LDS at
// lds + 16 * lane (lds is the same for the wave).  The load is counted by
// vmcnt like any other; the compiler does not know of it, so wait_tiles()
// stands before the barrier behind which the bytes are read.  m0 is set in the same
// block and named as clobbered; the compiler warns that it is a reserved register,
// which it sets before each use of its own.  (As an operand "{m0}" its writes are
// merged across the blocks, and tiles land in the wrong place.)
typedef int i32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void load_lds16(uint32_t lds, i32x4 base, uint32_t voff, uint32_t soff) {
#if __HIP_DEVICE_COMPILE__
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %1, %2, %3 offen lds"
      ::"s"(lds), "v"(voff), "s"(base), "s"(soff) : "memory", "m0");
#pragma clang diagnostic pop
#endif
}
// This wave's loads have landed and its LDS reads are done; then all waves'.
__device__ __forceinline__ void wait_tiles() {
#if __HIP_DEVICE_COMPILE__
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
#endif
}
// The same, but for this wave's last N loads.
template <int N>
__device__ __forceinline__ void wait_tiles_but() {
#if __HIP_DEVICE_COMPILE__
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
#endif
}
__device__ __forceinline__ i32x4 buffer_at(const void* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  i32x4 r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)u);
  r[1] = __builtin_amdgcn_readfirstlane((int)((u >> 32) & 0xffff));
  r[2] = -1;                              // offsets are kept in range by the caller
  r[3] = 0x00027000;
  return r;
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

}  // namespace gdn
