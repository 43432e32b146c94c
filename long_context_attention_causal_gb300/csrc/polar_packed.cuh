// What the two packed prefill kernels share: how the query rows of packed
// sequences with grouped heads become tiles, and which tile a CTA takes.
//
// The rows of a tile are (token, query head of the group), token-major: G heads
// share a KV head, so a tile of R rows is R / G tokens, in memory as it is in
// the tile, and every key it reads serves G heads.  The tiles of all sequences
// are ranked by their keys, longest first, and CTA i takes tile i: the order in
// which CTAs start is then that of a longest-first schedule, without a list: a
// tile's rank is found from the lengths alone.  F(p) = sum_b max(0, n_b - p)
// tiles have an index of p or more in their sequence (n_b: tiles of sequence
// b), so rank e has the index p with F(p + 1) <= e < F(p), and is the (e - F(p +
// 1))-th of the sequences with n_b > p.  Measured against tiles in the order of
// the sequences: see the kernels.
#pragma once

#include "polar_device.cuh"
#include "polar_internal.h"

namespace polar {

struct PackedTile {
  int head;   // KV head; -1: no tile for this CTA
  int index;  // of the sequence's tiles
  int len;    // tokens of the sequence
  int start;  // its first token
};

// Tokens [start, start + len) of sequence b; offsets out of bounds are cut.
__device__ __forceinline__ int2 packed_seq(const int* cu, int b, int N, bool* bad) {
  const int lo = __ldg(cu + b), hi = __ldg(cu + b + 1);
  const int s = min(max(lo, 0), N), e = min(max(hi, s), N);
  if (s != lo || e != hi) *bad = true;
  return make_int2(s, e - s);
}

// The tile of CTA `cta`, by one converged warp.  tokens: of a tile;
// head_group: KV heads whose tiles are ranked together (their K and V stay in
// L2), group after group.
__device__ __forceinline__ PackedTile packed_tile(const int* cu, int B, int N, int Hkv,
                                                  int head_group, int tokens, long long cta,
                                                  int* status) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  auto tiles = [&](int b) {
    return b < B ? (packed_seq(cu, b, N, &bad).y + tokens - 1) / tokens : 0;
  };
  // up to 256 sequences stay in registers
  constexpr int kHeld = 8;
  int held[kHeld];
#pragma unroll
  for (int i = 0; i < kHeld; ++i) held[i] = tiles(lane + 32 * i);
  auto above = [&](int p) -> int {  // F(p)
    int f = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) f += max(0, held[i] - p);
    for (int b = lane + 32 * kHeld; b < B; b += 32) f += max(0, tiles(b) - p);
    return (int)__reduce_add_sync(0xffffffffu, (unsigned)f);
  };
  int most = 0;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) most = max(most, held[i]);
  for (int b = lane + 32 * kHeld; b < B; b += 32) most = max(most, tiles(b));
  most = __reduce_max_sync(0xffffffffu, most);
  const int total = above(0);
  if (__any_sync(0xffffffffu, bad) && cta == 0 && lane == 0) atomicExch(status, 3);
  PackedTile t{-1, 0, 0, 0};
  if (total == 0 || cta >= (long long)total * Hkv) return t;
  const long long per_group = (long long)total * head_group;
  const int g = (int)(cta / per_group);
  const int rem = (int)(cta - g * per_group);
  const int hg = min(head_group, Hkv - g * head_group);
  const int rank = rem / hg;
  t.head = g * head_group + rem % hg;
  int lo = 0, hi = most - 1;  // F(lo) > rank; F(hi + 1) <= rank
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (above(mid) > rank) lo = mid;
    else hi = mid - 1;
  }
  t.index = lo;
  int left = rank - above(lo + 1);  // sequences with more than lo tiles before it
  for (int b0 = 0; b0 < B; b0 += 32) {
    const unsigned here = __ballot_sync(0xffffffffu, tiles(b0 + lane) > lo);
    const int n = __popc(here);
    if (left < n) {
      const bool mine = ((here >> lane) & 1u) && __popc(here & ((1u << lane) - 1u)) == left;
      const int b = b0 + __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
      const int2 s = packed_seq(cu, b, N, &bad);
      t.start = s.x;
      t.len = s.y;
      return t;
    }
    left -= n;
  }
  t.head = -1;  // not reached
  return t;
}

}  // namespace polar
