// Rows of k and v into a paged 4-bit cache, and back.  (No counterpart on the
// pages; layout and rounding: polar_cache_q4.cuh.)
//
// The rows are read once and 9 bits are written for each 32 (bf16: 16) of a value,
// so DRAM is the floor; the append's arithmetic, 22 instructions a channel with what
// a row costs, takes longer.  Measured: 32768 tokens of 4 heads, d = 128, bf16 in 29 us
// (eight channels a thread 37), fp32 out 34 us, 4.5 TB/s (rows in the order of the
// heads 37; 16 bytes a thread 35 to 39; CTAs that stay, with loads ahead, 35 to 43).
// A scale's maximum is that of the bits of |x|, whose order
// as integers is that of the numbers, with infinity and NaN above.
#include <algorithm>
#include <climits>
#include <cstdint>

#include "polar_cache_q4.cuh"
#include "polar_device.cuh"
#include "polar_internal.h"
#include "polar_span.h"

namespace polar {

namespace {

constexpr int kThreads = 256;

struct Q4Args {
  const void* rows[2];  // k, v
  void* out[2];         // cache_read: k, v
  uint8_t* pages[2];
  const int* slots;
  long long stride[2];  // elements between tokens
  int N, Hkv, shift, num_pages;
  int* status;
};

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 u = __ldg(reinterpret_cast<const float4*>(p));
  const float4 v = __ldg(reinterpret_cast<const float4*>(p) + 1);
  x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
  x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                            pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Page and row of a slot, or false (negative: none; past the pool: recorded).
__device__ __forceinline__ bool place(const Q4Args& a, int slot, int& page, int& row) {
  page = slot >> a.shift;
  row = slot & ((1 << a.shift) - 1);
  if (slot < 0) return false;
  if (page >= a.num_pages) {
    atomicExch(a.status, 3);
    return false;
  }
  return true;
}

// Nearest bf16 (ties to even) to top / 7, top in the normal range, as its bits: the
// upper half of the bits of top (1 / 7) is it or its neighbour below or above, and
// seven times the border between two neighbours is exact in fp32 (9 bits by 3).
__device__ __forceinline__ uint32_t q4_scale(float top) {
  const uint32_t low = __float_as_uint(top * (1.0f / 7.0f)) >> 16;
  const uint32_t border = __float_as_uint(__uint_as_float(low << 16 | 0x8000u) * 7.0f);
  return low + (__float_as_uint(top) + (low & 1u) > border ? 1u : 0u);
}

// The word of codes of x[0..7] for a scale s in the range where 1 / s and the
// borders below keep their bits.  |x| (1 / s) + 2^23, rounded down, holds m = floor
// (|x| / s), or a neighbour where |x| / s is near an integer; either way |n| is m
// or m + 1, and the border between them, (m + 1/2) s, is exact in fp32 (8 bits by
// 4).  A tie goes to the even one: as integers, the bits of |x| plus m's parity
// are compared with the border's.
__device__ __forceinline__ uint32_t q4_word(const float (&x)[8], float s) {
  constexpr float kTwo23 = 8388608.0f;
  constexpr uint32_t kBits = 0x4B000000u;  // of 2^23
  const float h = 0.5f * s;
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  uint32_t word = 0, excess = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int at = q4_at(i & 3) + 16 * (i >> 2);
    const uint32_t size = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    const float t = __fmaf_rz(__uint_as_float(size), inv, kTwo23);
    const uint32_t tb = __float_as_uint(t);
    const uint32_t border = __float_as_uint(fmaf(t - kTwo23, s, h));
    word += tb << at;
    excess += kBits << at;
    if (size + (tb & 1u) > border) word += 1u << at;
  }
  word -= excess;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int sign = 15 - 4 * (i & 3) + 16 * (i >> 2);
    word |= (__float_as_uint(x[i]) >> (31 - sign)) & (1u << sign);
  }
  return word;
}

// The same for any scale s > 0, in fp64 (near the subnormal range).
__device__ __noinline__ uint32_t q4_word_small(float x0, float x1, float x2, float x3, float x4,
                                               float x5, float x6, float x7, float s) {
  const float x[8] = {x0, x1, x2, x3, x4, x5, x6, x7};
  uint32_t word = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t n = (uint32_t)fmin(rint(fabs((double)x[i]) / (double)s), 7.0);
    word |= n << (q4_at(i & 3) + 16 * (i >> 2));
    word |= (__float_as_uint(x[i]) & 0x80000000u) >> (16 + 4 * (i & 3) - 16 * (i >> 2));
  }
  return word;
}

// Both kernels: rows of k (blockIdx.y 0) and v (1), (token, head) by (token, head),
// W threads a row; the read with two rows a thread, whose loads are in flight
// together.
constexpr int kReadBatch = 2;

// Two words a thread, so that what a row costs beside its codes (place, scale,
// addresses) is spread over 16 channels; two threads share a scale.
template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 5) q4_append_kernel(const Q4Args a) {
  constexpr int W = D / 16;  // threads of a row
  const bool is_v = blockIdx.y != 0;
  const int w = threadIdx.x % W;
  const uint32_t rows = (uint32_t)a.N * (uint32_t)a.Hkv;
  const uint32_t id = blockIdx.x * (kThreads / W) + threadIdx.x / W;
  const uint32_t token = id / (uint32_t)a.Hkv;
  const int head = (int)(id - token * (uint32_t)a.Hkv);
  float x[2][8];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 8; ++i) x[h][i] = 0.f;
  int slot = -1;
  if (id < rows) {  // the same for a group's threads
    const T* src = static_cast<const T*>(is_v ? a.rows[1] : a.rows[0]) +
                   (long long)token * (is_v ? a.stride[1] : a.stride[0]) + head * D + 16 * w;
    load8(src, x[0]);
    load8(src + 8, x[1]);
    slot = __ldg(a.slots + token);
  }
  uint32_t top = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(x[h][i]) & 0x7FFFFFFFu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  uint32_t scale = 0, code[2] = {0, 0};
  if (top >= 0x7F800000u) {
    scale = 0x7FFF;  // an infinity or NaN: the group reads as NaN
  } else if (top > 0x10000000u) {  // 2^-95
    scale = q4_scale(__uint_as_float(top));
#pragma unroll
    for (int h = 0; h < 2; ++h) code[h] = q4_word(x[h], __uint_as_float(scale << 16));
  } else if (top > 0) {
    const __nv_bfloat16 sb = __float2bfloat16_rn(__uint_as_float(top) / 7.0f);
    scale = __bfloat16_as_ushort(sb);
    if (scale > 0)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        code[h] = q4_word_small(x[h][0], x[h][1], x[h][2], x[h][3], x[h][4], x[h][5], x[h][6],
                                x[h][7], __bfloat162float(sb));
  }
  int page, row;
  if (!place(a, slot, page, row)) return;
  uint8_t* block = (is_v ? a.pages[1] : a.pages[0]) + q4_block(page, head, a.Hkv, a.shift, D);
  uint32_t* codes = reinterpret_cast<uint32_t*>(block + (size_t)row * (D / 2));
#pragma unroll
  for (int h = 0; h < 2; ++h) codes[q4_place(2 * w + h, D)] = code[h];
  if ((w & 1) == 0) {
    uint8_t* scales = block + ((size_t)(D / 2) << a.shift);
    reinterpret_cast<uint16_t*>(scales + (size_t)row * (D / 16))[w >> 1] = (uint16_t)scale;
  }
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) q4_read_kernel(const Q4Args a) {
  constexpr int kBatch = kReadBatch;
  constexpr int W = D / 8;
  constexpr int R = kThreads / W;
  const bool is_v = blockIdx.y != 0;
  const int w = threadIdx.x % W;
  const uint32_t rows = (uint32_t)a.N * (uint32_t)a.Hkv;
  const uint8_t* pages = is_v ? a.pages[1] : a.pages[0];
  uint32_t code[kBatch], scale[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const uint32_t id = (blockIdx.x * kBatch + u) * R + threadIdx.x / W;
    code[u] = scale[u] = 0;
    int page, row;
    if (id < rows && place(a, __ldg(a.slots + id / (uint32_t)a.Hkv), page, row)) {
      const uint8_t* block =
          pages + q4_block(page, (int)(id % (uint32_t)a.Hkv), a.Hkv, a.shift, D);
      code[u] = reinterpret_cast<const uint32_t*>(block + (size_t)row * (D / 2))[q4_place(w, D)];
      const uint8_t* scales = block + ((size_t)(D / 2) << a.shift);
      scale[u] = reinterpret_cast<const uint16_t*>(scales + (size_t)row * (D / 16))[w >> 2];
    }
  }
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const uint32_t id = (blockIdx.x * kBatch + u) * R + threadIdx.x / W;
    if (id >= rows) break;
    const float s = __uint_as_float(scale[u] << 16);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = s * (float)q4_value(code[u] >> (16 * (i >> 2)), i & 3);
    store8(static_cast<T*>(is_v ? a.out[1] : a.out[0]) + (size_t)id * D + 8 * w, x);
  }
}

template <bool kRead>
cudaError_t launch(const Q4Args& a, int d, int dtype, cudaStream_t s) {
  const long long rows = (long long)a.N * a.Hkv;
  const long long per = kRead ? (long long)kReadBatch * (kThreads / (d / 8)) : kThreads / (d / 16);
  const dim3 grid((unsigned)((rows + per - 1) / per), 2);
#define POLAR_Q4(D, T)                                       \
  if (kRead) q4_read_kernel<D, T><<<grid, kThreads, 0, s>>>(a); \
  else q4_append_kernel<D, T><<<grid, kThreads, 0, s>>>(a)
  if (dtype == POLAR_BF16) {
    if (d == 64) { POLAR_Q4(64, __nv_bfloat16); }
    else { POLAR_Q4(128, __nv_bfloat16); }
  } else {
    if (d == 64) { POLAR_Q4(64, float); }
    else { POLAR_Q4(128, float); }
  }
#undef POLAR_Q4
  return cudaGetLastError();
}

int check(const Q4Args& a, int d, int page_size, int dtype, int* shift) {
  if (a.N < 0 || a.Hkv < 1 || a.num_pages < 1) return POLAR_ERR_INVALID;
  if ((d != 64 && d != 128) || (dtype != POLAR_F32 && dtype != POLAR_BF16))
    return POLAR_ERR_UNSUPPORTED;
  if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) != 0)
    return POLAR_ERR_UNSUPPORTED;
  if ((long long)a.num_pages * page_size > INT_MAX || a.Hkv > 4096 ||
      (long long)a.N * a.Hkv > INT_MAX)
    return POLAR_ERR_UNSUPPORTED;
  *shift = 0;
  while ((1 << *shift) < page_size) ++*shift;
  if (a.N == 0) return POLAR_OK;
  if (!a.pages[0] || !a.pages[1] || !a.slots) return POLAR_ERR_INVALID;
  if (!aligned16(a.pages[0]) || !aligned16(a.pages[1]) ||
      (reinterpret_cast<uintptr_t>(a.slots) & 3u))
    return POLAR_ERR_MISALIGNED;
  return POLAR_OK;
}

}  // namespace

}  // namespace polar

using namespace polar;

extern "C" {

int polar_cache_append_q4(const void* k, const void* v, const int* slots, void* k_pages,
                          void* v_pages, long long k_stride, long long v_stride, int N, int Hkv,
                          int d, int page_size, int num_pages, int dtype, void* stream) {
  Q4Args a{{k, v}, {nullptr, nullptr}, {static_cast<uint8_t*>(k_pages), static_cast<uint8_t*>(v_pages)},
           slots, {k_stride, v_stride}, N, Hkv, 0, num_pages, nullptr};
  int st = check(a, d, page_size, dtype, &a.shift);
  if (st != POLAR_OK || N == 0) return st;
  if (!k || !v) return POLAR_ERR_INVALID;
  const long long width = (long long)Hkv * d;
  const size_t es = dtype == POLAR_BF16 ? 2 : 4;
  const int vec = (int)(16 / es);
  if (N > 1 && (k_stride < width || v_stride < width)) return POLAR_ERR_INVALID;
  if (!aligned16(k) || !aligned16(v) || (N > 1 && (k_stride % vec || v_stride % vec)))
    return POLAR_ERR_MISALIGNED;
  const size_t pool = (size_t)num_pages * Hkv * page_size * q4_row_bytes(d);
  const Strided ins[] = {{k, (size_t)N, (size_t)width * es, (size_t)k_stride * es},
                         {v, (size_t)N, (size_t)width * es, (size_t)v_stride * es},
                         span(slots, (size_t)N * 4)};
  for (const Strided& i : ins)
    if (meet(i, span(k_pages, pool)) || meet(i, span(v_pages, pool))) return POLAR_ERR_INVALID;
  if (meet(span(k_pages, pool), span(v_pages, pool))) return POLAR_ERR_INVALID;
  st = check_device(nullptr);
  if (st != POLAR_OK) return st;
  a.status = status_word();
  if (!a.status) return cuda_status("cudaGetSymbolAddress", cudaGetLastError());
  return cuda_status("4-bit append launch",
                     launch<false>(a, d, dtype, static_cast<cudaStream_t>(stream)));
}

int polar_cache_read_q4(const void* k_pages, const void* v_pages, const int* slots, void* k,
                        void* v, int N, int Hkv, int d, int page_size, int num_pages, int dtype,
                        void* stream) {
  Q4Args a{{nullptr, nullptr}, {k, v},
           {static_cast<uint8_t*>(const_cast<void*>(k_pages)),
            static_cast<uint8_t*>(const_cast<void*>(v_pages))},
           slots, {0, 0}, N, Hkv, 0, num_pages, nullptr};
  int st = check(a, d, page_size, dtype, &a.shift);
  if (st != POLAR_OK || N == 0) return st;
  if (!k || !v) return POLAR_ERR_INVALID;
  if (!aligned16(k) || !aligned16(v)) return POLAR_ERR_MISALIGNED;
  const size_t pool = (size_t)num_pages * Hkv * page_size * q4_row_bytes(d);
  const size_t rows = (size_t)N * Hkv * d * (dtype == POLAR_BF16 ? 2 : 4);
  const Strided ins[] = {span(k_pages, pool), span(v_pages, pool), span(slots, (size_t)N * 4)};
  for (const Strided& i : ins)
    if (meet(i, span(k, rows)) || meet(i, span(v, rows))) return POLAR_ERR_INVALID;
  if (meet(span(k, rows), span(v, rows))) return POLAR_ERR_INVALID;
  st = check_device(nullptr);
  if (st != POLAR_OK) return st;
  a.status = status_word();
  if (!a.status) return cuda_status("cudaGetSymbolAddress", cudaGetLastError());
  return cuda_status("4-bit read launch",
                     launch<true>(a, d, dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
