// Device helpers of the decayed linear attention kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "polar_device.cuh"
#include "polar_internal.h"

namespace polar {

// Tokens of sequence b: lengths[b] clamped to [0, T] (all T without lengths);
// a length outside records status 3.
__device__ __forceinline__ int linear_length(const int* lengths, int b, int T, int* status) {
  if (!lengths) return T;
  const int n = lengths[b];
  if ((n < 0 || n > T) && status && threadIdx.x == 0) atomicExch(status, 3);
  return min(max(n, 0), T);
}

// ln of a head's decay.  Below -200 the first power is 0 in fp32 already;
// the clamp keeps -inf * 0 = NaN out of the zeroth power.  NaN passes.
__device__ __forceinline__ float linear_log_decay(const float* log_decay, int h) {
  const float x = log_decay[h];
  return x < -200.f ? -200.f : x;
}
// and log2 of it
__device__ __forceinline__ float linear_log2_decay(const float* log_decay, int h) {
  return linear_log_decay(log_decay, h) * 1.4426950408889634f;
}

// g^n for n >= 0.  The product's rounding moves the result by 2^-24 |n l2|
// relative: a power that still weighs (above 2^-24) is right to 1e-6.
__device__ __forceinline__ float linear_power(float l2, int n) { return exp2f(l2 * (float)n); }

// g^n = hi + lo, for a state that is multiplied by the same power again and
// again: a power near 1 that is rounded to fp32 (up to 2^-25 off) puts every
// decay off by the same factor, as often as a state lives through it.  Of the
// state's 2-norm, rounded: 6e-6 over 16384 tokens by chunks of 64, 2e-6 by
// tiles of 128, 9e-5 over 4096 single tokens; in two parts 3e-7 for fp32
// prompts.  Costs a second fma.  Fast decays forget sooner than that shows, and
// lo is 0.  ln: linear_log_decay.
struct LinearDecay {
  float hi, lo;
  // g^n s + add, by pairs
  __device__ __forceinline__ float2 join(float2 s, float2 add) const {
    return ffma2(make_float2(hi, hi), s, ffma2(make_float2(lo, lo), s, add));
  }
  __device__ __forceinline__ float4 join(float4 s, float4 add) const {
    const float2 a = join(make_float2(s.x, s.y), make_float2(add.x, add.y));
    const float2 b = join(make_float2(s.z, s.w), make_float2(add.z, add.w));
    return make_float4(a.x, a.y, b.x, b.y);
  }
};
__device__ __forceinline__ LinearDecay linear_decay(float ln, int n) {
  const float x = ln * (float)n;
  if (fabsf(x) < 0.5f) {
    const float em = expm1f(x), hi = 1.f + em;
    return {hi, em - (hi - 1.f)};  // hi - 1 is exact
  }
  return {linear_power(ln * 1.4426950408889634f, n), 0.f};
}

// Programmatic launch: the kernels of one call follow each other without a
// drain between them.  A kernel lets its successor start (once all of its own
// CTAs have) and waits for its predecessor before it touches what that wrote
// or still reads; tensors of the call that no kernel of it writes need no wait.
__device__ __forceinline__ void linear_let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void linear_wait_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Launch of `kern`, chained to the kernel before it in the stream or not.
template <typename K, typename... A>
inline cudaError_t linear_launch(K kern, dim3 grid, int threads, int smem, cudaStream_t s,
                                 bool chained, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = chained ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// The tiles of one head that one run holds.
struct LinearPortion {
  int bh;
  int first, last;  // tiles [first, last) of the head
  int len;          // tokens of the sequence
  int live;         // tiles of the portion that hold tokens: [first, first + live)
  bool cut_left, cut_right;  // the run's boundary cuts the head there
  __device__ __forceinline__ int row(int tile) const { return tile * kLinearTile; }
  __device__ __forceinline__ int tokens(int tile) const {
    return min(kLinearTile, len - tile * kLinearTile);
  }
};

// Number of heads that run `part` touches, and the i-th of them in order.
__device__ __forceinline__ int linear_portions(const LinearSplit& s, int BH, int part) {
  const long long i0 = (long long)part * s.per;
  const long long i1 = min(i0 + s.per, (long long)BH * s.tiles);
  return (int)((i1 - 1) / s.tiles - i0 / s.tiles) + 1;
}
__device__ __forceinline__ LinearPortion linear_portion(const LinearSplit& s, int BH, int H, int T,
                                                        const int* lengths, int* status, int part,
                                                        int i) {
  const long long i0 = (long long)part * s.per;
  const long long i1 = min(i0 + s.per, (long long)BH * s.tiles);
  LinearPortion p;
  p.bh = (int)(i0 / s.tiles) + i;
  const long long h0 = (long long)p.bh * s.tiles;
  p.first = (int)(i0 > h0 ? i0 - h0 : 0);
  p.last = (int)(i1 < h0 + s.tiles ? i1 - h0 : s.tiles);
  p.cut_left = p.first > 0;
  p.cut_right = p.last < s.tiles;
  p.len = linear_length(lengths, p.bh / H, T, status);
  const int end = min(p.last, (p.len + kLinearTile - 1) / kLinearTile);
  p.live = max(end - p.first, 0);
  return p;
}

__device__ __forceinline__ float linear_load(const float* p) { return *p; }
__device__ __forceinline__ float linear_load(const __nv_bfloat16* p) {
  return __bfloat162float(*p);
}
__device__ __forceinline__ void linear_store(float* p, float x) { *p = x; }
__device__ __forceinline__ void linear_store(__nv_bfloat16* p, float x) {
  *p = __float2bfloat16_rn(x);
}

}  // namespace polar
