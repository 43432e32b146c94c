// Rotary positions of q and k.  (No counterpart on the pages.)
//
// Pair i < r/2 of a head's first r channels turns by the angle p f_i, p the
// token's position:
//   y_a = s (x_a cos - x_b sin),   y_b = s (x_b cos + x_a sin)
// with (a, b) = (i, i + r/2) (halves) or (2 i, 2 i + 1) (interleaved); the
// inverse, whose angle is negative, is the gradient, as s R^T is.
// A far position's angle in fp32 would be off by tenths of a radian, so the
// angle is kept in turns, as a 64-bit fraction: f_i / (2 pi) * 2^64 cut to an
// integer once a block, times the position, modulo 2^64 (whole turns drop out).
// Its upper 24 bits, h, are an fp32 number exactly, for one sincospi in [-1, 1); the
// next 16 are an angle e below 2^-21 beside it,
//   cos(h + e) = cos h - e sin h,   sin(h + e) = sin h + e cos h   (up to e^2 / 2).
// (Upper bits rounded to fp32 had left up to 2^-26 of a turn.)
// Bound by DRAM: q and k are read and written once.  A thread owns 16 bytes of
// the pairs of one token, whose sines it computes once, and walks over heads;
// with few tokens the heads are spread over threads instead.  Measured: 32768 tokens
// of 20 heads, d = 128 bf16, 58 us, 5.8 TB/s (2 heads a thread 81, 4 59, 8 57, 20 58).
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "polar_device.cuh"
#include "polar_internal.h"
#include "polar_span.h"

namespace polar {

namespace {

constexpr int kThreads = 256;

struct RopeArgs {
  const void *q, *k;
  void *q_out, *k_out;
  const int* positions;
  const double* inv_freq;  // [rot / 2] radians a token
  long long qs, ks, qos, kos;  // elements between tokens
  int N, Hq, Hkv, d, rot;
  int units, rot_units;  // threads of a token and of its turned part
  int heads;             // rows (of q, then of k) a thread walks over
  float scale;
};

__device__ __forceinline__ void unpack16(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack16(const uint4& u, float (&x)[4]) {
  x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y);
  x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void store16(void* p, const float (&x)[8]) {
  *static_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                       pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store16(void* p, const float (&x)[4]) {
  *static_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}

__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }

// One pair, in one order of roundings wherever it is computed.
__device__ __forceinline__ void turn(float xa, float xb, float c, float s, float& ya, float& yb) {
  ya = fmaf(xa, c, -__fmul_rn(xb, s));
  yb = fmaf(xb, c, __fmul_rn(xa, s));
}

// kVec: 16-byte accesses (8 bf16 or 4 fp32 channels a thread); without, one
// pair or one channel a thread, for parts of a head and strides that are not
// multiples of that.
template <typename T, bool kVec, bool kInterleaved, bool kInverse>
__global__ void __launch_bounds__(kThreads, 3) rope_kernel(const RopeArgs a) {
  constexpr int V = kVec ? 16 / (int)sizeof(T) : 1;
  __shared__ unsigned long long turns[64];
  if ((int)threadIdx.x < a.rot / 2) {
    double t = a.inv_freq[threadIdx.x] * 0.15915494309189533577;  // 1 / (2 pi)
    t -= floor(t);
    turns[threadIdx.x] = (unsigned long long)(t * 18446744073709551616.0);  // 2^64
  }
  __syncthreads();
  const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long token = id / a.units;
  if (token >= a.N) return;
  const int unit = (int)(id - token * a.units);
  const int rows = a.Hq + a.Hkv;
  const int row0 = (int)blockIdx.y * a.heads, row1 = min(rows, row0 + a.heads);
  const T* q = static_cast<const T*>(a.q) + token * a.qs;
  const T* k = static_cast<const T*>(a.k) + token * a.ks;
  T* qo = static_cast<T*>(a.q_out) + token * a.qos;
  T* ko = static_cast<T*>(a.k_out) + token * a.kos;
  auto src = [&](int r) { return r < a.Hq ? q + r * a.d : k + (r - a.Hq) * a.d; };
  auto dst = [&](int r) { return r < a.Hq ? qo + r * a.d : ko + (r - a.Hq) * a.d; };
  if (unit >= a.rot_units) {
    // the part of a head that keeps its values (not reached in place)
    const int off = a.rot + (unit - a.rot_units) * V;
    for (int r = row0; r < row1; ++r) {
      if (kVec) *reinterpret_cast<uint4*>(dst(r) + off) = *reinterpret_cast<const uint4*>(src(r) + off);
      else dst(r)[off] = src(r)[off];
    }
    return;
  }
  float cs[V], sn[V];
  const unsigned long long p = (unsigned long long)(long long)a.positions[token];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const unsigned long long t = p * turns[unit * V + i];
    const float x = (float)((int)(t >> 32) >> 8) * 1.1920928955078125e-7f;  // 2^-23: half turns
    const float e = (float)(int)((t >> 24) & 0xFFFFu) * 5.714523747137342e-12f;  // 2 pi 2^-40
    float s, c;
    sincospif(x, &s, &c);
    cs[i] = fmaf(-e, s, c) * a.scale;
    sn[i] = fmaf(e, c, s) * (kInverse ? -a.scale : a.scale);
  }
  const int off0 = kInterleaved ? 2 * unit * V : unit * V;
  const int off1 = kInterleaved ? off0 + V : off0 + a.rot / 2;
  if constexpr (kVec) {
    // four rows' loads in flight together, as they are: 118 registers of floats
    // had left half the warps and 86 us for 32768 tokens of 20 heads, d = 128 bf16
    constexpr int kBatch = 4;
    for (int r0 = row0; r0 < row1; r0 += kBatch) {
      uint4 u0[kBatch], u1[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (r0 + u < row1) {
          u0[u] = *reinterpret_cast<const uint4*>(src(r0 + u) + off0);
          u1[u] = *reinterpret_cast<const uint4*>(src(r0 + u) + off1);
        }
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (r0 + u < row1) {
          float x0[V], x1[V], y0[V], y1[V];
          unpack16(u0[u], x0);
          unpack16(u1[u], x1);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            if constexpr (kInterleaved) {
              // pair i: channels 2 i and 2 i + 1 of the two vectors in a row
              const float xa = i < V / 2 ? x0[2 * i % V] : x1[2 * i % V];
              const float xb = i < V / 2 ? x0[(2 * i + 1) % V] : x1[(2 * i + 1) % V];
              float(&y)[V] = i < V / 2 ? y0 : y1;
              turn(xa, xb, cs[i], sn[i], y[2 * i % V], y[(2 * i + 1) % V]);
            } else {
              turn(x0[i], x1[i], cs[i], sn[i], y0[i], y1[i]);
            }
          }
          store16(dst(r0 + u) + off0, y0);
          store16(dst(r0 + u) + off1, y1);
        }
    }
  } else {
    for (int r = row0; r < row1; ++r) {
      const float x0 = as_float(src(r)[off0]), x1 = as_float(src(r)[off1]);
      float y0, y1;
      turn(x0, x1, cs[0], sn[0], y0, y1);
      put(dst(r) + off0, y0);
      put(dst(r) + off1, y1);
    }
  }
}

template <typename T, bool kVec>
cudaError_t launch(const RopeArgs& a, dim3 grid, bool interleaved, bool inverse, cudaStream_t s) {
  if (interleaved) {
    if (inverse) rope_kernel<T, kVec, true, true><<<grid, kThreads, 0, s>>>(a);
    else rope_kernel<T, kVec, true, false><<<grid, kThreads, 0, s>>>(a);
  } else {
    if (inverse) rope_kernel<T, kVec, false, true><<<grid, kThreads, 0, s>>>(a);
    else rope_kernel<T, kVec, false, false><<<grid, kThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

bool in_place(const void* x, long long xs, const void* y, long long ys, int N) {
  return x == y && (xs == ys || N < 2);
}

}  // namespace

}  // namespace polar

using namespace polar;

extern "C" {

int polar_rope(const void* q, const void* k, const int* positions, const double* inv_freq,
               void* q_out, void* k_out, long long q_stride, long long k_stride,
               long long q_out_stride, long long k_out_stride, int N, int Hq, int Hkv, int d,
               int rot, int dtype, int interleaved, int inverse, float scale, void* stream) {
  if (N < 0 || Hq < 0 || Hkv < 0 || rot < 2 || rot > d || rot % 2 != 0 || !std::isfinite(scale))
    return POLAR_ERR_INVALID;
  if (dtype != POLAR_F32 && dtype != POLAR_BF16) return POLAR_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return POLAR_ERR_UNSUPPORTED;
  if (Hq > 4096 || Hkv > 4096) return POLAR_ERR_UNSUPPORTED;
  if (N == 0 || Hq + Hkv == 0) return POLAR_OK;
  if ((Hq && (!q || !q_out)) || (Hkv && (!k || !k_out)) || !positions || !inv_freq)
    return POLAR_ERR_INVALID;
  const long long qw = (long long)Hq * d, kw = (long long)Hkv * d;
  if (N > 1 && ((Hq && (q_stride < qw || q_out_stride < qw)) ||
                (Hkv && (k_stride < kw || k_out_stride < kw))))
    return POLAR_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) ||
      (reinterpret_cast<uintptr_t>(positions) & 3u) || (reinterpret_cast<uintptr_t>(inv_freq) & 7u))
    return POLAR_ERR_MISALIGNED;
  const size_t es = dtype == POLAR_BF16 ? 2 : 4;
  const int vec = (int)(16 / es);
  auto rows_of = [&](const void* p, long long w, long long stride) {
    return Strided{w ? p : nullptr, (size_t)N, (size_t)w * es, (size_t)stride * es};
  };
  const bool q_same = in_place(q, q_stride, q_out, q_out_stride, N);
  const bool k_same = in_place(k, k_stride, k_out, k_out_stride, N);
  {
    const Strided sq = rows_of(q, qw, q_stride), sk = rows_of(k, kw, k_stride);
    const Strided oq = rows_of(q_out, qw, q_out_stride), ok = rows_of(k_out, kw, k_out_stride);
    const Strided sp = span(positions, (size_t)N * 4), sf = span(inv_freq, (size_t)rot * 4);
    if (meet(oq, ok) || meet(oq, sk) || meet(ok, sq) || (!q_same && meet(oq, sq)) ||
        (!k_same && meet(ok, sk)) || meet(oq, sp) || meet(ok, sp) || meet(oq, sf) || meet(ok, sf))
      return POLAR_ERR_INVALID;
  }
  const long long strides[4] = {q_stride, q_out_stride, k_stride, k_out_stride};
  bool wide = rot % (2 * vec) == 0;
  for (int i = 0; i < 4; ++i)
    if (i < 2 ? Hq : Hkv) wide = wide && (strides[i] % vec == 0 || N < 2);
  int sms = 0;
  const int st = check_device(&sms);
  if (st != POLAR_OK) return st;
  RopeArgs a{q, k, q_out, k_out, positions, inv_freq, q_stride, k_stride, q_out_stride, k_out_stride,
             N, Hq, Hkv, d, rot, 0, 0, 0, scale};
  const int v = wide ? vec : 1;
  const bool copy = (Hq && !q_same) || (Hkv && !k_same);
  a.rot_units = rot / 2 / v;
  a.units = a.rot_units + (copy ? (d - rot) / v : 0);
  // Heads to a thread: as many as leave every SM its 2048 threads, at most 32.
  const long long threads = (long long)N * a.units, rows = Hq + Hkv;
  const long long groups =
      std::max(std::min(rows, (2048LL * sms + threads - 1) / threads), (rows + 31) / 32);
  a.heads = (int)((rows + groups - 1) / groups);
  const long long blocks = (threads + kThreads - 1) / kThreads;
  if (blocks > INT_MAX) return POLAR_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)blocks, (unsigned)((rows + a.heads - 1) / a.heads));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == POLAR_BF16)
    e = wide ? launch<__nv_bfloat16, true>(a, grid, interleaved != 0, inverse != 0, s)
             : launch<__nv_bfloat16, false>(a, grid, interleaved != 0, inverse != 0, s);
  else
    e = wide ? launch<float, true>(a, grid, interleaved != 0, inverse != 0, s)
             : launch<float, false>(a, grid, interleaved != 0, inverse != 0, s);
  return cuda_status("rotary positions launch", e);
}

}  // extern "C"
