// Causal Polar Attention over packed sequences with grouped heads, fp32, on the
// FP32 pipes, and the entry point of both types.
//
// "ATMA", §2.1 and §2.2 (online participation ratio, squared correction
// factors); tiles as in polar_packed.cuh.  One bf16 term of an fp32 input is not
// enough for the tensor cores (three of each are, as in the decode over the 4-bit
// cache, at six products for one; not built here): the two products run as
// register-tiled matrix products: a CTA of 256 threads owns 64 rows (64 / G tokens of a group's G heads) and walks over
// keys 64 at a time.  Thread (y, x) of a 16 x 16 grid scores rows 4 y .. 4 y + 3
// against keys x, x + 16, x + 32, x + 48 (64 products for 8 reads of 16 bytes),
// the 16 threads of a row share its maximum and sums by shuffles, P goes
// through shared memory, and the thread adds the tile's values to 4 rows x D / 16
// channels.  K of the next tile is copied (cp.async) while P V runs, V while the
// next scores do.  Bound by a tile's chain, its four block barriers with two CTAs a
// SM, not by a pipe: FMA 34 % (packed), LSU 28 %, 1.9 instructions a clock.  4
// prompts of up to 1500 tokens, 8 query on 2 KV heads, d = 128, 287 us (29 TFLOP/s;
// with single instead of packed multiply-adds 327).
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "polar_device.cuh"
#include "polar_internal.h"
#include "polar_packed.cuh"
#include "polar_span.h"

namespace polar {

namespace {

constexpr int kRows = 64;
constexpr int kKeys = 64;
constexpr int kThreads = 256;
constexpr int kTurns = 32;

template <int D>
struct Smem {
  // 16-byte pieces of a row are permuted (piece), so that the rows that a warp
  // reads at once lie in different banks
  float q[kRows][D], k[kKeys][D], v[kKeys][D];
  float p[kRows][kKeys];
  PackedTile tiles[kTurns];
};

// Place of piece ch of a row: neighbouring keys, and rows 4 apart, differ.
__device__ __forceinline__ int key_piece(int key, int ch) { return 4 * (ch ^ (key & 7)); }
__device__ __forceinline__ int row_piece(int row, int ch) { return 4 * (ch ^ ((row >> 2) & 7)); }

struct PackedF32Params {
  const float *q, *k, *v, *mem, *w_count;
  float *out, *n_eff, *conf;
  const int* cu;
  int* status;
  long long qs, ks, vs;
  int N, B, Hq, Hkv, head_group;
  int turns;  // tiles found at a time: 1 (and one a CTA) or kTurns
  polar_consts_t c;
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Sum and maximum over the 16 threads of a row.
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

template <int D, int G>
__global__ void __launch_bounds__(kThreads, 2) polar_packed_f32_kernel(const PackedF32Params p) {
  constexpr int TT = kRows / G;  // tokens of a tile
  constexpr int C = D / 4;       // 16-byte pieces of a row
  constexpr int CX = D / 64;     // float4s of channels a thread owns: x, x + 16
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem<D>& sm = *reinterpret_cast<Smem<D>*>(smem_raw);
  const int tid = threadIdx.x, x = tid & 15, y = tid >> 4;
  for (int k = 0;; ++k) {
    if (k % p.turns == 0) {
      __syncthreads();  // the last list is read
      if (tid < 32) {
        PackedTiles tiles(p.cu, p.B, p.N, p.Hkv, p.head_group, TT, p.status);
        for (int i = k; i < k + p.turns; ++i) {
          const PackedTile t = tiles.find((long long)i * gridDim.x +
                                          ((i & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x));
          if (tid == 0) sm.tiles[i - k] = t;
        }
      }
    }
    __syncthreads();
    const PackedTile tile = sm.tiles[k % p.turns];
    if (tile.head < 0) return;
    const int tok0 = tile.index * TT, cnt = min(tile.len - tok0, TT);
    const int keys = tok0 + cnt;  // keys of the tile's last row
    const size_t first = (size_t)tile.start;

    auto load_k = [&](int j0) {
      for (int i = tid; i < kKeys * C; i += kThreads) {
        const int key = i / C, ch = i % C;
        if (j0 + key < keys)
          cp_async16(&sm.k[key][key_piece(key, ch)],
                     p.k + (first + j0 + key) * (size_t)p.ks + (size_t)tile.head * D + 4 * ch);
      }
      cp_async_commit();
    };
    auto load_v = [&](int j0) {
      for (int i = tid; i < kKeys * C; i += kThreads) {
        const int key = i / C, ch = i % C;
        if (j0 + key < keys)
          cp_async16(&sm.v[key][4 * ch],
                     p.v + (first + j0 + key) * (size_t)p.vs + (size_t)tile.head * D + 4 * ch);
        else  // weighted by 0, and so a number
          *reinterpret_cast<float4*>(&sm.v[key][4 * ch]) = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      cp_async_commit();
    };
    for (int i = tid; i < kRows * C; i += kThreads) {
      const int row = i / C, ch = i % C;
      float4 u = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row / G < cnt)
        u = __ldg(reinterpret_cast<const float4*>(p.q + (first + tok0 + row / G) * (size_t)p.qs +
                                                  ((size_t)tile.head * G + row % G) * D) + ch);
      *reinterpret_cast<float4*>(&sm.q[row][row_piece(row, ch)]) = u;
    }
    load_k(0);
    load_v(0);

    float scale[4], m[4], l[4], q2[4];
    float2 acc[4][2 * CX];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int token = tok0 + (4 * y + i) / G;
      scale[i] = polar_tau((float)(token + 1), p.c.log_t0) * rsqrtf((float)D);
      m[i] = -INFINITY;
      l[i] = q2[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 2 * CX; ++e) acc[i][e] = make_float2(0.f, 0.f);
    }
    for (int j0 = 0; j0 < keys; j0 += kKeys) {
      cp_async_wait<1>();  // K (V may still be on its way)
      __syncthreads();
      // (packed pairs: the sums of even and odd channels)
      float2 s2[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) s2[i][u] = make_float2(0.f, 0.f);
#pragma unroll 2
      for (int ch = 0; ch < C; ++ch) {
        float4 qv[4], kv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          qv[i] = *reinterpret_cast<const float4*>(&sm.q[4 * y + i][row_piece(4 * y, ch)]);
          kv[i] = *reinterpret_cast<const float4*>(&sm.k[x + 16 * i][key_piece(x, ch)]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            float2& a = s2[i][u];
            a = ffma2(make_float2(qv[i].x, qv[i].y), make_float2(kv[u].x, kv[u].y), a);
            a = ffma2(make_float2(qv[i].z, qv[i].w), make_float2(kv[u].z, kv[u].w), a);
          }
      }
      float s[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) s[i][u] = s2[i][u].x + s2[i][u].y;
      __syncthreads();  // K is read
      if (j0 + kKeys < keys) load_k(j0 + kKeys);
      else cp_async_commit();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int token = tok0 + (4 * y + i) / G;
        float mt = -INFINITY;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          s[i][u] = j0 + x + 16 * u <= token && j0 + x + 16 * u < keys ? s[i][u] * scale[i]
                                                                         : -INFINITY;
          mt = fmaxf(mt, s[i][u]);
        }
        const float mn = fmaxf(m[i], row_max(mt));
        const float alpha = m[i] == mn ? 1.f : expf(m[i] - mn);  // 0 while m = -inf
        float ps = 0.f, pq = 0.f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float w = s[i][u] == -INFINITY ? 0.f : expf(s[i][u] - mn);
          ps += w;
          pq = fmaf(w, w, pq);
          sm.p[4 * y + i][row_piece(4 * y, (x >> 2) + 4 * u) + (x & 3)] = w;
        }
        l[i] = l[i] * alpha + ps;
        q2[i] = q2[i] * alpha * alpha + pq;  // squared correction factor
        m[i] = mn;
#pragma unroll
        for (int e = 0; e < 2 * CX; ++e) acc[i][e].x *= alpha, acc[i][e].y *= alpha;
      }
      cp_async_wait<1>();  // V (the next K may still be on its way)
      __syncthreads();
#pragma unroll 2
      for (int k4 = 0; k4 < kKeys / 4; ++k4) {
        float pv[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 u = *reinterpret_cast<const float4*>(&sm.p[4 * y + i][row_piece(4 * y, k4)]);
          pv[i][0] = u.x, pv[i][1] = u.y, pv[i][2] = u.z, pv[i][3] = u.w;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int cx = 0; cx < CX; ++cx) {
            const float4 vv = *reinterpret_cast<const float4*>(&sm.v[4 * k4 + u][4 * x + 64 * cx]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 pp = make_float2(pv[i][u], pv[i][u]);
              acc[i][2 * cx] = ffma2(pp, make_float2(vv.x, vv.y), acc[i][2 * cx]);
              acc[i][2 * cx + 1] = ffma2(pp, make_float2(vv.z, vv.w), acc[i][2 * cx + 1]);
            }
          }
      }
      __syncthreads();  // V and P are read
      if (j0 + kKeys < keys) load_v(j0 + kKeys);
      else cp_async_commit();
    }
    cp_async_wait<0>();
    // (the pieces' order does not matter to a sum over a row)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 4 * y + i, token = tok0 + row / G, head = tile.head * G + row % G;
      float a2 = 0.f, qq = 0.f;
#pragma unroll
      for (int e = 0; e < 2 * CX; ++e)
        a2 = fmaf(acc[i][e].x, acc[i][e].x, fmaf(acc[i][e].y, acc[i][e].y, a2));
#pragma unroll
      for (int e = 0; e < D / 16; ++e) qq = fmaf(sm.q[row][x + 16 * e], sm.q[row][x + 16 * e], qq);
      a2 = row_sum(a2);
      qq = row_sum(qq);
      const float ls = row_sum(l[i]), qs = row_sum(q2[i]);
      if (row / G >= cnt) continue;
      const RowResult res =
          polar_finish(m[i], ls, qs, a2, qq, (float)(token + 1), D, p.c);
      const size_t at = (first + token) * p.Hq + head;
#pragma unroll
      for (int cx = 0; cx < CX; ++cx) {
        const int ch = 4 * x + 64 * cx;
        const float4 mv = __ldg(reinterpret_cast<const float4*>(p.mem + at * D + ch));
        const float4 wv = __ldg(reinterpret_cast<const float4*>(p.w_count + (size_t)head * D + ch));
        *reinterpret_cast<float4*>(p.out + at * D + ch) =
            make_float4(fmaf(acc[i][2 * cx].x, res.scale_u, fmaf(res.count, wv.x, mv.x)),
                        fmaf(acc[i][2 * cx].y, res.scale_u, fmaf(res.count, wv.y, mv.y)),
                        fmaf(acc[i][2 * cx + 1].x, res.scale_u, fmaf(res.count, wv.z, mv.z)),
                        fmaf(acc[i][2 * cx + 1].y, res.scale_u, fmaf(res.count, wv.w, mv.w)));
      }
      if (x == 0) {
        p.n_eff[at] = res.n_eff;
        if (p.conf) p.conf[at] = res.conf;
      }
    }
    if (p.turns == 1) return;
  }
}

template <int D, int G>
cudaError_t launch_g(const PackedArgs& a, cudaStream_t s) {
  constexpr int kTokens = kRows / G;
  PackedF32Params p{static_cast<const float*>(a.q), static_cast<const float*>(a.k),
                    static_cast<const float*>(a.v), static_cast<const float*>(a.mem), a.w_count,
                    static_cast<float*>(a.out), a.n_eff, a.conf, a.cu, a.status, a.qs, a.ks, a.vs,
                    a.N, a.B, a.Hq, a.Hkv, l2_head_group(a.Hkv, 8.0 * (double)a.N * D), 1, a.c};
  auto kern = polar_packed_f32_kernel<D, G>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)sizeof(Smem<D>));
  static_assert(2 * (sizeof(Smem<D>) + 1024) <= 233472, "two CTAs a SM");
  if (e != cudaSuccess) return e;
  const long long tiles = std::min((long long)a.N / kTokens + a.B, (long long)a.N) * a.Hkv;
  long long ctas = tiles;
  // Finding a tile costs what the sequences are many: past those that a warp keeps in
  // registers CTAs stay and find many tiles at a time.  65536 sequences of 16
  // tokens, 8 query on 2 KV heads, d = 64: 520 ms with a CTA a tile, 26 so.
  if (a.B > PackedTiles::kFew) {
    p.turns = kTurns;
    ctas = std::min(tiles, 8LL * a.sms);
  }
  kern<<<(unsigned)ctas, kThreads, sizeof(Smem<D>), s>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const PackedArgs& a, cudaStream_t s) {
  switch (a.Hq / a.Hkv) {
    case 1: return launch_g<D, 1>(a, s);
    case 2: return launch_g<D, 2>(a, s);
    case 4: return launch_g<D, 4>(a, s);
    default: return launch_g<D, 8>(a, s);
  }
}

}  // namespace

cudaError_t launch_packed_f32(const PackedArgs& a, cudaStream_t s) {
  return a.d == 64 ? launch_d<64>(a, s) : launch_d<128>(a, s);
}

}  // namespace polar

using namespace polar;

extern "C" int polar_attn_fwd_packed(const void* q, const void* k, const void* v, const void* mem,
                                     const float* w_count, const int* cu_seqlens, void* out,
                                     float* n_eff, float* conf, long long q_stride,
                                     long long k_stride, long long v_stride, int N, int B, int Hq,
                                     int Hkv, int d, int dtype, const polar_consts_t* c,
                                     void* stream) {
  if (N < 0 || B < 0 || Hq < 1 || Hkv < 1) return POLAR_ERR_INVALID;
  if (dtype != POLAR_F32 && dtype != POLAR_BF16) return POLAR_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return POLAR_ERR_UNSUPPORTED;
  if (Hq % Hkv != 0) return POLAR_ERR_UNSUPPORTED;
  const int G = Hq / Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8) return POLAR_ERR_UNSUPPORTED;
  const polar_consts_t cc = c ? *c : defaults();
  if (!consts_ok(cc)) return POLAR_ERR_INVALID;
  if (N == 0 || B == 0) return POLAR_OK;
  if (!q || !k || !v || !mem || !w_count || !cu_seqlens || !out || !n_eff) return POLAR_ERR_INVALID;
  const long long qw = (long long)Hq * d, kw = (long long)Hkv * d;
  if (N > 1 && (q_stride < qw || k_stride < kw || v_stride < kw)) return POLAR_ERR_INVALID;
  const size_t es = dtype == POLAR_BF16 ? 2 : 4;
  if (N == 1) q_stride = qw, k_stride = v_stride = kw;
  const long long vec = (long long)(16 / es);
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(mem) || !aligned16(w_count) ||
      !aligned16(out) || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) ||
      (reinterpret_cast<uintptr_t>(n_eff) & 3u) || (reinterpret_cast<uintptr_t>(conf) & 3u) ||
      q_stride % vec || k_stride % vec || v_stride % vec)
    return POLAR_ERR_MISALIGNED;
  // a tensor map's strides stay below 2^40 bytes, a grid below 2^31 CTAs
  const long long most = 1LL << 37;
  if (q_stride > most || k_stride > most || v_stride > most || N > (1 << 30) || B > (1 << 18) ||
      (long long)N + B > INT_MAX / 2 || (((long long)N * G) / 64 + B + 1) * Hkv > INT_MAX)
    return POLAR_ERR_UNSUPPORTED;
  {
    const size_t rows = (size_t)N * Hq;
    const Strided outs[] = {span(out, rows * d * es), span(n_eff, rows * 4), span(conf, rows * 4)};
    const Strided ins[] = {{q, (size_t)N, (size_t)qw * es, (size_t)q_stride * es},
                           {k, (size_t)N, (size_t)kw * es, (size_t)k_stride * es},
                           {v, (size_t)N, (size_t)kw * es, (size_t)v_stride * es},
                           span(mem, rows * d * es), span(w_count, (size_t)qw * 4),
                           span(cu_seqlens, ((size_t)B + 1) * 4)};
    for (const Strided& o : outs) {
      for (const Strided& i : ins)
        if (meet(o, i)) return POLAR_ERR_INVALID;
      for (const Strided& other : outs)
        if (&other != &o && meet(o, other)) return POLAR_ERR_INVALID;
    }
  }
  int sms = 0;
  const int st = check_device(&sms);
  if (st != POLAR_OK) return st;
  PackedArgs a{q, k, v, mem, w_count, cu_seqlens, out, n_eff, conf, q_stride, k_stride, v_stride,
               N, B, Hq, Hkv, d, cc, status_word(), sms};
  if (!a.status) return cuda_status("cudaGetSymbolAddress", cudaGetLastError());
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == POLAR_F32)
    return cuda_status("packed prefill (fp32) launch", launch_packed_f32(a, s));
  CUtensorMap maps[3];
  if (!make_map_tokens(&maps[0], q, N, Hq, d, q_stride, G, 128 / G) ||
      !make_map_tokens(&maps[1], k, N, Hkv, d, k_stride, 1, 128) ||
      !make_map_tokens(&maps[2], v, N, Hkv, d, v_stride, 1, 128))
    return POLAR_ERR_CUDA;
  return cuda_status("packed prefill (tcgen05) launch", launch_packed_tc(a, maps, s));
}
