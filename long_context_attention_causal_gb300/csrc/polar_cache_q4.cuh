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

// Sign and size of channel j (0..3) in its 16 bits.
__device__ __forceinline__ uint32_t q4_code(int n, int j) {
  const uint32_t size = (uint32_t)(n < 0 ? -n : n);
  const int at = j == 0 ? 4 : j == 1 ? 0 : j == 2 ? 12 : 8;
  return (size << at) | (n < 0 ? 0x8000u >> (4 * j) : 0u);
}
__device__ __forceinline__ int q4_value(uint32_t piece, int j) {
  const int at = j == 0 ? 4 : j == 1 ? 0 : j == 2 ? 12 : 8;
  const int size = (int)(piece >> at) & 7;
  return (piece & (0x8000u >> (4 * j))) ? -size : size;
}

// n of x for a scale s > 0 (exact: the nearest integer to x / s, ties to even).
// x * inv is within 2^-22 of x / s, so m is that integer or, near a border, its
// neighbour; the remainder x - m s is exact there and decides.
__device__ __forceinline__ int q4_round(float x, float s, float inv) {
  const float m = rintf(x * inv);
  const float r = fmaf(-m, s, x), h = 0.5f * s;
  int n = (int)m;
  if (fabsf(r) > h || (fabsf(r) == h && (n & 1))) n += r > 0.f ? 1 : -1;
  return n;
}

}  // namespace polar
