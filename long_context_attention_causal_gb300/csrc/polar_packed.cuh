// What the two packed prefill kernels share: how the query rows of packed
// sequences with grouped heads become tiles, and which tile has which rank.
//
// The rows of a tile are (token, query head of the group), token-major: G heads
// share a KV head, so a tile of R rows is R / G tokens, in memory as it is in
// the tile, and every key it reads serves G heads.  The tiles of all sequences
// are ranked by their keys, longest first, so that CTAs which take them by rank
// follow a longest-first schedule without a list: the tile of a rank is found
// from the lengths alone.  F(p) = sum_b max(0, n_b - p) tiles have an index of p
// or more in their sequence (n_b: tiles of sequence b), so rank e has the index p
// with F(p + 1) <= e < F(p), and is the (e - F(p + 1))-th of the sequences with
// n_b > p.
#pragma once

#include "polar_device.cuh"
#include "polar_internal.h"

namespace polar {

struct PackedTile {
  int head;   // KV head; -1: no tile of this rank
  int index;  // of the sequence's tiles
  int len;    // tokens of the sequence
  int start;  // its first token
};

// The tiles of a call; all members are run by one converged warp, whose lanes hold
// equal values but for `held`.
struct PackedTiles {
  static constexpr int kHeld = 8;
  static constexpr int kFew = 32 * kHeld;  // sequences whose tiles stay in registers

  const int* cu;
  int N, B, Hkv, tokens;
  int head_group;  // KV heads whose tiles are ranked together (their K and V stay in L2)
  int most, total;       // tiles of the longest sequence, of all
  int at, first, behind;  // index p last found, and its ranks [F(p + 1), F(p))
  // B <= kFew: n_b of sequence lane + 32 i.  Else: of 256 runs of `run` sequences
  // each, how many with n_b > at are in run lane + 32 i.
  int held[kHeld];
  int run;

  // Tokens [start, start + len) of sequence b; offsets out of bounds are cut.
  __device__ __forceinline__ int2 seq(int b) const {
    const int s = min(max(__ldg(cu + b), 0), N), e = min(max(__ldg(cu + b + 1), 0), N);
    return make_int2(s, e - s);
  }
  __device__ __forceinline__ int tiles(int b) const {
    return b < B ? (seq(b).y + tokens - 1) / tokens : 0;
  }

  // Sequences from the first descending offset on have no tiles (they could overlap
  // others, and be many times the rows); that, and offsets out of bounds, are recorded.
  __device__ __forceinline__ PackedTiles(const int* cu_, int B_, int N_, int Hkv_, int head_group_,
                                         int tokens_, int* status)
      : cu(cu_), N(N_), B(B_), Hkv(Hkv_), tokens(tokens_), head_group(head_group_), at(-1), first(0),
        behind(0), run((B_ + 32 * kFew - 1) / (32 * kFew) * 32) {
    const int lane = threadIdx.x & 31;
    bool bad = false;
    int good = B;
    most = 0;
    for (int b = lane; b < B; b += 32) {
      const int lo = __ldg(cu + b), hi = __ldg(cu + b + 1);
      if (lo < 0 || hi > N || hi < lo) bad = true;
      if (hi < lo) good = min(good, b);
      most = max(most, (seq(b).y + tokens - 1) / tokens);
    }
    B = (int)__reduce_min_sync(0xffffffffu, (unsigned)good);
    most = __reduce_max_sync(0xffffffffu, most);
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicExch(status, 3);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) held[i] = B <= kFew ? tiles(lane + 32 * i) : 0;
    total = above(0);
  }

  __device__ __forceinline__ int above(int p) const {  // F(p)
    int f = 0;
    if (B <= kFew) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i) f += max(0, held[i] - p);
    } else {
      for (int b = threadIdx.x & 31; b < B; b += 32) f += max(0, tiles(b) - p);
    }
    return (int)__reduce_add_sync(0xffffffffu, (unsigned)f);
  }

  // Position in the warp's ballots of the `left`-th set bit of `mask`.
  __device__ __forceinline__ static int nth(unsigned mask, int left) {
    const int lane = threadIdx.x & 31;
    const bool mine = ((mask >> lane) & 1u) && __popc(mask & ((1u << lane) - 1u)) == left;
    return __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
  }

  __device__ __forceinline__ PackedTile find(long long place) {
    const int lane = threadIdx.x & 31;
    PackedTile t{-1, 0, 0, 0};
    if (total == 0 || place >= (long long)total * Hkv) return t;
    // head groups, one after another; in one, the heads of a rank side by side
    const long long per_group = (long long)total * head_group;
    const int g = (int)(place / per_group);
    const int hg = min(head_group, Hkv - g * head_group);
    const long long rem = place - g * per_group;
    const int rank = (int)(rem / hg);
    if (at < 0 || rank < first || rank >= behind) {
      int lo = 0, hi = most - 1;  // F(lo) > rank; F(hi + 1) <= rank
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (above(mid) > rank) lo = mid;
        else hi = mid - 1;
      }
      at = lo;
      first = above(lo + 1);
      behind = above(lo);
      if (B > kFew) {
        const int pieces = run / 32;  // of 32 sequences in a run
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
          held[i] = 0;
#pragma unroll 4
          for (int c = 0; c < 32 * pieces; ++c) {
            const int b0 = 32 * (i * 32 * pieces + c);
            if (b0 >= B) break;
            const int n = __popc(__ballot_sync(0xffffffffu, tiles(b0 + lane) > at));
            if (lane == c / pieces) held[i] += n;
          }
        }
      }
    }
    int left = rank - first;  // sequences with more than `at` tiles before it
    int b = -1;
    if (B <= kFew) {
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        const unsigned here = __ballot_sync(0xffffffffu, held[i] > at);
        if (b < 0 && left < __popc(here)) b = 32 * i + nth(here, left);
        left -= __popc(here);
      }
    } else {
      int b0 = -1, skip = 0;
#pragma unroll
      for (int i = 0; i < kHeld; ++i) {
        int upto = held[i];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int u = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += u;
        }
        const unsigned past = __ballot_sync(0xffffffffu, upto > left);
        if (b0 < 0 && past) {
          const int l = __ffs(past) - 1;
          b0 = (l + 32 * i) * run;
          skip = left - __shfl_sync(0xffffffffu, upto - held[i], l);
        }
        left -= __shfl_sync(0xffffffffu, upto, 31);
      }
#pragma unroll 1
      for (int o = 0; b0 >= 0 && b < 0 && o < run; o += 32) {
        const unsigned here = __ballot_sync(0xffffffffu, tiles(b0 + o + lane) > at);
        if (skip < __popc(here)) b = b0 + o + nth(here, skip);
        skip -= __popc(here);
      }
    }
    if (b < 0 || b >= B) return t;  // not reached
    const int2 s = seq(b);
    t.head = g * head_group + (int)(rem % hg);
    t.index = at;
    t.start = s.x;
    t.len = s.y;
    return t;
  }
};

}  // namespace polar
