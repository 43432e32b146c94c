// The paged cache in 4 bits: layout and rounding.
//
// 32 consecutive channels of a row share a bf16 scale s = max |x| / 7 (rounded
// to nearest), and a channel is kept as n = x / s, rounded to nearest, ties to
// even, -7 <= n <= 7.  (|x| <= 7 s (1 + 2^-8), so only scales below the normal
// range can push n past 7; it is cut there.)  A group with an infinity or a NaN
// gets the scale NaN, and reads as NaN.
// The block of one (page, head) holds the rows' codes, d / 2 bytes each, then
// the rows' scales, d / 16 bytes each.  Four channels 4 p + j make 16 bits,
// signs in bits 15, 11, 7, 3 and |n| from bits 4, 0, 12, 8 on: with the mask
// 0x8070 the 16 bits, shifted left by 4 for odd j and with their bytes swapped
// for j >= 2, are a bf16 number of n 2^-129 (a subnormal, exact, and a full
// operand of a matrix product), so a code costs an instruction or less to
// unpack.  Two pieces make a 32-bit word, and word w = 4 i + c of a row (i:
// the scale's group) stands in place c d / 32 + i: lane c of a quad then reads
// its words of all groups at once.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace polar {

constexpr int kQ4Group = 32;
__host__ __device__ constexpr int q4_row_bytes(int d) { return d / 2 + d / 16; }

// Byte offset of the block of (page, head).
__device__ __forceinline__ size_t q4_block(long long page, int head, int Hkv, int shift, int d) {
  return (size_t)((page * Hkv + head) << shift) * q4_row_bytes(d);
}
// Place of word w (channels 8 w .. 8 w + 7) in its row.
__device__ __forceinline__ int q4_place(int w, int d) { return (w & 3) * (d / 32) + (w >> 2); }

// Bit of |n| of channel j (0..3) in its 16 bits; its sign is bit 15 - 4 j.
__host__ __device__ constexpr int q4_at(int j) { return j == 0 ? 4 : j == 1 ? 0 : j == 2 ? 12 : 8; }

__device__ __forceinline__ int q4_value(uint32_t piece, int j) {
  const int size = (int)(piece >> q4_at(j)) & 7;
  return (piece & (0x8000u >> (4 * j))) ? -size : size;
}

}  // namespace polar
