// Paged, grouped-query decode split kernel over a 4-bit cache.
//
// The mathematics is polar_decode_paged's (per query head: l = sum p, Q2 = sum
// p^2, acc = sum p v over the split's keys, merged by the same combine
// kernel); the rows are those of polar_cache_q4.cuh.  With the codes n and
// the scales s of a key's 32-channel groups g,
//   q . k_j = sum_g sk_jg (q_g . n_jg),     acc_g += sum_j (p_j sv_jg) n_jg
// so the scales never meet the codes: a key's score is a sum of d / 32 partial
// products, and V's scales go into the weights.
//
// A row of K or V is 9 d / 16 bytes, so at the rate of DRAM about 42 codes a
// clock pass through each SM, and the instructions that unpack them are the
// other bound (128 lanes a clock and SM).  Hence warp products (m16n8k16, bf16,
// fp32 sums) whose A operand is unpacked from the packed words in registers, in
// at most one instruction a code: a code masked out of its word is the bf16
// subnormal n 2^-129, exactly; the factor 2^64 that q and the weights carry
// keeps the sums in fp32's normal range.  A tensor-core instruction that
// reads its operand from shared memory would need the unpacked rows
// written there, 4 bytes for each byte that DRAM delivers.
//   S (16 keys x 8 heads) = K codes (A, 16 x 16 channels) . q^T (B)
//   O^T (16 channels x 8 heads) += V codes^T (A, 16 channels x 16 keys) . P'^T (B)
// P' comes from S's registers by movmatrix.  fp32 queries are split into three
// bf16 terms, whose sum is q, and so are the weights: three products each.
//
// 160 threads: warps 0-3 compute, 16 keys at a time, each with its own running
// maxima, sums and O; warp 4 copies (cp.async.bulk, a ring of stages of 128
// keys; a piece of min(page, 128) rows is one copy of codes and one of scales).
// The warps' states are joined in shared memory at the end.
#include <algorithm>
#include <climits>
#include <cmath>

#include "polar_cache_q4.cuh"
#include "polar_device.cuh"
#include "polar_internal.h"

namespace polar {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kSK = 128;  // keys a stage
constexpr int kStages = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;  // log2 units
constexpr float kTwo64 = 18446744073709551616.0f;
constexpr float kTwo65 = 36893488147419103232.0f;
constexpr uint32_t kCodeMask = 0x80708070u;

template <int D>
struct Q4Smem {
  uint8_t kc[kStages][kSK * D / 2], vc[kStages][kSK * D / 2];
  uint8_t ks[kStages][kSK * D / 16], vs[kStages][kSK * D / 16];
  uint32_t valid[kStages];  // a bit for each 8 keys of the stage
  uint64_t full[kStages], empty[kStages];
  float m[kWarps][8], l[kWarps][8], q2[kWarps][8];
  int abort_flag;
  static_assert(sizeof(float) * kWarps * 8 * D <= (size_t)kStages * kSK * D / 2, "warps' O over kc");
};

struct Q4DecodeParams {
  const void* q;
  const uint8_t *k_pages, *v_pages;
  const int *table, *lens;
  float* partials;
  int Hq, Hkv, max_pages, num_pages, shift, max_seq_len, splits, chunk;
  polar_consts_t c;
  int* status;
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit elements held by a warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); }

// Words of a lane's place in a row of codes (d / 8 bytes) and a row's scales.
template <int D>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[D / 32]) {
  if constexpr (D == 128) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x, w[1] = u.y;
  }
}
template <int D>
__device__ __forceinline__ void load_scales(const uint8_t* p, float (&s)[D / 32]) {
  if constexpr (D == 128) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    s[0] = bf16_lo(u.x), s[1] = bf16_hi(u.x), s[2] = bf16_lo(u.y), s[3] = bf16_hi(u.y);
  } else {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    s[0] = bf16_lo(u), s[1] = bf16_hi(u);
  }
}

// Term t of x's expansion in bf16 (x = t0 + t1 + t2 up to 2^-24 x).
__device__ __forceinline__ float bf16_round(float x) {
  return __bfloat162float(__float2bfloat16_rn(x));
}

// NT: bf16 terms of q and of the weights (1: bf16 queries, 3: fp32).
template <int D, int NT, typename T>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2)
    polar_decode_q4_kernel(const Q4DecodeParams p) {
  constexpr int NG = D / 32;  // groups of channels
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Q4Smem<D>& sm = *reinterpret_cast<Q4Smem<D>*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / p.Hkv, hkv = blockIdx.x % p.Hkv;
  const int split = blockIdx.y;
  const int G = p.Hq / p.Hkv;
  const int page = 1 << p.shift;
  int n = p.lens[b];
  if (n < 1 || n > p.max_seq_len) {
    if (threadIdx.x == 0 && split == 0) atomicExch(p.status, 3);
    n = n < 1 ? 0 : p.max_seq_len;
  }
  const long long first = (long long)split * p.chunk;
  const int k0 = (int)(first < n ? first : n);
  const int k1 = min(k0 + p.chunk, n);
  const int nst = (k1 - k0 + kSK - 1) / kSK;
  float* rec0 = p.partials + ((size_t)b * p.Hq + (size_t)hkv * G) * p.splits * (D + 4);
  if (nst == 0) {
    // nothing to read: an empty record (its acc is not read by the combine)
    if ((int)threadIdx.x < G) {
      float* rec = rec0 + ((size_t)threadIdx.x * p.splits + split) * (D + 4);
      rec[0] = -INFINITY, rec[1] = rec[2] = rec[3] = 0.f;
    }
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], kWarps);
    }
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  volatile int* abort_flag = &sm.abort_flag;

  if (warp == kWarps) {
    // ------------------------------------------------------------- copies --
    // lane o < 16: the stage's keys 8 o .. 8 o + 7; the first lane of a piece
    // of min(page, 128) keys issues its copies
    const int* tb = p.table + (size_t)b * p.max_pages;
    const int piece = min(page, kSK);
    const bool leader = lane < 16 && (lane * 8) % piece == 0;
    auto entry = [&](int st) -> int {
      const int key = k0 + st * kSK + lane * 8;
      return lane < 16 && key < k1 ? __ldg(tb + (key >> p.shift)) : -1;
    };
    int pg = entry(0), issued = 0;
    bool ok = true;
    for (int st = 0; st < nst && ok; ++st) {
      const int slot = st % kStages;
      const int next = st + 1 < nst ? entry(st + 1) : -1;
      if (st >= kStages)
        ok = mbar_wait_warp(&sm.empty[slot], (uint32_t)(st / kStages - 1) & 1, abort_flag, p.status);
      if (!ok) break;
      const int key = k0 + st * kSK + lane * 8;
      const bool here = lane < 16 && key < k1;
      const bool good = here && pg >= 0 && pg < p.num_pages;
      if (here && !good) atomicExch(p.status, 3);
      const uint32_t valid = __ballot_sync(0xffffffffu, good);
      // rows in whole copies of 16 bytes
      const int rows = leader && good ? min(piece, (k1 - key + 3) & ~3) : 0;
      const uint32_t bytes = __reduce_add_sync(0xffffffffu, 2u * (uint32_t)rows * q4_row_bytes(D));
      if (lane == 0) {
        sm.valid[slot] = valid;
        mbar_arrive_expect_tx(&sm.full[slot], bytes);
      }
      __syncwarp();
      if (rows > 0) {
        const int row = key & (page - 1), at = lane * 8;
        const size_t block = q4_block(pg, hkv, p.Hkv, p.shift, D);
        const size_t codes = block + (size_t)row * (D / 2);
        const size_t scales = block + ((size_t)(D / 2) << p.shift) + (size_t)row * (D / 16);
        bulk_g2s(sm.kc[slot] + at * (D / 2), p.k_pages + codes, rows * (D / 2), &sm.full[slot]);
        bulk_g2s(sm.ks[slot] + at * (D / 16), p.k_pages + scales, rows * (D / 16), &sm.full[slot]);
        bulk_g2s(sm.vc[slot] + at * (D / 2), p.v_pages + codes, rows * (D / 2), &sm.full[slot]);
        bulk_g2s(sm.vs[slot] + at * (D / 16), p.v_pages + scales, rows * (D / 16), &sm.full[slot]);
      }
      pg = next;
      issued = st + 1;
    }
    if (!ok) {
      // aborted: let the copies already issued land before the CTA exits
      volatile int never = 0;
      for (int st = issued - 1; st >= 0 && st >= issued - kStages; --st)
        mbar_wait(&sm.full[st % kStages], (uint32_t)(st / kStages) & 1, &never, p.status,
                  kWaitLimitCycles / 4);
      __syncwarp();
    }
    return;
  }

  // --------------------------------------------------------------- compute --
  // fragment coordinates; row r of a product's 16 keys (8 and more: + 8) is
  // the key (r / 2) + 4 (r % 2) of them, so that V's operand, whose columns
  // 2 c and 2 c + 1 are the keys c and c + 4, reads neighbouring rows
  const int r = lane >> 2, c = lane & 3;
  const int rk = (r >> 1) + 4 * (r & 1);
  // q as B operand: head r, channels 32 g + 8 c + (0, 4), (1, 5), (2, 6), (3, 7)
  uint32_t qb[NT][NG][4];
  {
    const T* qp = static_cast<const T*>(p.q) + ((size_t)b * p.Hq + (size_t)hkv * G + r) * D + 8 * c;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = r < G ? (float)qp[32 * g + j] : 0.f;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // 2^64 is exact in bf16: the terms are those of q
          qb[t][g][j] = pack_bf16x2(x[j] * kTwo64, x[j + 4] * kTwo64);
          if (t + 1 < NT) {
            x[j] -= bf16_round(x[j]);
            x[j + 4] -= bf16_round(x[j + 4]);
          }
        }
    }
  }
  // log2 units; the products carry 2^-65
  const float scale2 = polar_tau((float)n, p.c.log_t0) * kLog2e * rsqrtf((float)D) * kTwo65;
  float o[2 * NG][4];  // O^T tile 2 g + t: channels 32 g + 4 r + 2 t (+ 1), heads 2 c, 2 c + 1
#pragma unroll
  for (int i = 0; i < 2 * NG; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f, s0 = 0.f, s1 = 0.f;
  // selectors: half r % 2 of a word of each of two keys, as it is and with
  // the bytes of each half swapped
  const uint32_t sel_a = (r & 1) ? 0x7632u : 0x5410u, sel_b = (r & 1) ? 0x6723u : 0x4501u;

  for (int st = 0; st < nst; ++st) {
    const int slot = st % kStages;
    const bool landed = mbar_wait_warp(&sm.full[slot], (uint32_t)(st / kStages) & 1, abort_flag,
                                       p.status);
    if (!landed) break;
    const uint32_t pages_ok = sm.valid[slot];
#pragma unroll 1
    for (int sub = warp; sub < kSK / 16; sub += kWarps) {
      const int base = sub * 16, key = k0 + st * kSK + base;
      if (key >= k1) break;
      const bool whole = key + 16 <= k1 && ((pages_ok >> (2 * sub)) & 3u) == 3u;
      const bool in0 = whole || (key + rk < k1 && ((pages_ok >> (2 * sub)) & 1u));
      const bool in1 = whole || (key + 8 + rk < k1 && ((pages_ok >> (2 * sub)) & 2u));
      // ---- scores
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      {
        uint32_t ka[NG], kb[NG];
        float sa[NG], sb[NG];
        load_words<D>(sm.kc[slot] + (base + rk) * (D / 2) + c * (D / 8), ka);
        load_words<D>(sm.kc[slot] + (base + 8 + rk) * (D / 2) + c * (D / 8), kb);
        load_scales<D>(sm.ks[slot] + (base + rk) * (D / 16), sa);
        load_scales<D>(sm.ks[slot] + (base + 8 + rk) * (D / 16), sb);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
          const uint32_t za = __byte_perm(ka[g], 0, 0x2301), zb = __byte_perm(kb[g], 0, 0x2301);
          const uint32_t f0[4] = {ka[g] & kCodeMask, kb[g] & kCodeMask, (ka[g] << 4) & kCodeMask,
                                  (kb[g] << 4) & kCodeMask};
          const uint32_t f1[4] = {za & kCodeMask, zb & kCodeMask, (za << 4) & kCodeMask,
                                  (zb << 4) & kCodeMask};
          // the smallest terms first
#pragma unroll
          for (int t = NT - 1; t >= 0; --t) {
            mma16816(acc, f0, qb[t][g][0], qb[t][g][1]);
            mma16816(acc, f1, qb[t][g][2], qb[t][g][3]);
          }
          x[0] = fmaf(acc[0], sa[g], x[0]);
          x[1] = fmaf(acc[1], sa[g], x[1]);
          x[2] = fmaf(acc[2], sb[g], x[2]);
          x[3] = fmaf(acc[3], sb[g], x[3]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] *= scale2;
      }
      if (!whole) {
        // a masked row's scale may be anything
        if (!in0) x[0] = x[1] = -INFINITY;
        if (!in1) x[2] = x[3] = -INFINITY;
      }
      const float t0 = fmaxf(x[0], x[2]), t1 = fmaxf(x[1], x[3]);
      if (__any_sync(0xffffffffu, t0 > m0 + kRescale || t1 > m1 + kRescale)) {
        float u0 = t0, u1 = t1;
#pragma unroll
        for (int d = 4; d <= 16; d <<= 1) {
          u0 = fmaxf(u0, __shfl_xor_sync(0xffffffffu, u0, d));
          u1 = fmaxf(u1, __shfl_xor_sync(0xffffffffu, u1, d));
        }
        float a0 = 1.f, a1 = 1.f;
        if (u0 > m0 + kRescale) a0 = ex2_approx(m0 - u0), m0 = u0;  // 0 at the first keys
        if (u1 > m1 + kRescale) a1 = ex2_approx(m1 - u1), m1 = u1;
        l0 *= a0, l1 *= a1;
        s0 *= a0 * a0, s1 *= a1 * a1;  // squared correction factor
#pragma unroll
        for (int i = 0; i < 2 * NG; ++i) o[i][0] *= a0, o[i][2] *= a0, o[i][1] *= a1, o[i][3] *= a1;
      }
      float w[4] = {ex2_approx(x[0] - m0), ex2_approx(x[1] - m1), ex2_approx(x[2] - m0),
                    ex2_approx(x[3] - m1)};
      if (!whole) {
        if (!in0) w[0] = w[1] = 0.f;
        if (!in1) w[2] = w[3] = 0.f;
      }
      l0 += w[0] + w[2], l1 += w[1] + w[3];
      s0 = fmaf(w[0], w[0], fmaf(w[2], w[2], s0));
      s1 = fmaf(w[1], w[1], fmaf(w[3], w[3], s1));
      // ---- values
      {
        float va[NG], vb[NG];
        load_scales<D>(sm.vs[slot] + (base + rk) * (D / 16), va);
        load_scales<D>(sm.vs[slot] + (base + 8 + rk) * (D / 16), vb);
        if (!whole) {
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            if (!in0) va[g] = 0.f;
            if (!in1) vb[g] = 0.f;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] *= kTwo64;
        uint32_t y[4][NG];  // keys c, c + 4, c + 8, c + 12
#pragma unroll
        for (int i = 0; i < 4; ++i)
          load_words<D>(sm.vc[slot] + (base + c + 4 * i) * (D / 2) + (r >> 1) * (D / 8), y[i]);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const uint32_t p01 = __byte_perm(y[0][g], y[1][g], sel_a);
          const uint32_t p23 = __byte_perm(y[2][g], y[3][g], sel_a);
          const uint32_t z01 = __byte_perm(y[0][g], y[1][g], sel_b);
          const uint32_t z23 = __byte_perm(y[2][g], y[3][g], sel_b);
          const uint32_t f0[4] = {p01 & kCodeMask, (p01 << 4) & kCodeMask, p23 & kCodeMask,
                                  (p23 << 4) & kCodeMask};
          const uint32_t f1[4] = {z01 & kCodeMask, (z01 << 4) & kCodeMask, z23 & kCodeMask,
                                  (z23 << 4) & kCodeMask};
          float e[4] = {w[0] * va[g], w[1] * va[g], w[2] * vb[g], w[3] * vb[g]};
          uint32_t bl[NT], bh[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            bl[t] = transpose8(pack_bf16x2(e[0], e[1]));
            bh[t] = transpose8(pack_bf16x2(e[2], e[3]));
            if (t + 1 < NT)
#pragma unroll
              for (int i = 0; i < 4; ++i) e[i] -= bf16_round(e[i]);
          }
#pragma unroll
          for (int t = NT - 1; t >= 0; --t) {
            mma16816(o[2 * g], f0, bl[t], bh[t]);
            mma16816(o[2 * g + 1], f1, bl[t], bh[t]);
          }
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.empty[slot]);
  }

  // ------------------------------------------------- the four warps' states --
#pragma unroll
  for (int d = 4; d <= 16; d <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, d);
    l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    s0 += __shfl_xor_sync(0xffffffffu, s0, d);
    s1 += __shfl_xor_sync(0xffffffffu, s1, d);
  }
  // every warp has read its last stage, and every copy has landed: the codes'
  // buffer takes the warps' O (unless a wait ran out, which ends the call with
  // a status: then nothing is written over copies that may be in flight)
  asm volatile("bar.sync 1, 128;" ::: "memory");
  if (*abort_flag) return;
  float* join = reinterpret_cast<float*>(sm.kc);  // [warp][head][D]
  if (r == 0) {
    sm.m[warp][2 * c] = m0, sm.m[warp][2 * c + 1] = m1;
    sm.l[warp][2 * c] = l0, sm.l[warp][2 * c + 1] = l1;
    sm.q2[warp][2 * c] = s0, sm.q2[warp][2 * c + 1] = s1;
  }
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<float4*>(join + (warp * 8 + 2 * c + h) * D + 32 * g + 4 * r) =
          make_float4(o[2 * g][h], o[2 * g][2 + h], o[2 * g + 1][h], o[2 * g + 1][2 + h]);
  asm volatile("bar.sync 1, 128;" ::: "memory");
  const int t = threadIdx.x;
  for (int h = 0; h < G; ++h) {
    float M = -INFINITY;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sm.m[i][h]);
    float e[kWarps];
#pragma unroll
    for (int i = 0; i < kWarps; ++i)
      e[i] = sm.m[i][h] == -INFINITY ? 0.f : ex2_approx(sm.m[i][h] - M);
    float* rec = rec0 + ((size_t)h * p.splits + split) * (D + 4);
    if (t < D) {
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) a = fmaf(e[i], join[(i * 8 + h) * D + t], a);
      rec[4 + t] = a * kTwo65;
    }
    if (t == 0) {
      float L = 0.f, Q = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        L = fmaf(e[i], sm.l[i][h], L);
        Q = fmaf(e[i] * e[i], sm.q2[i][h], Q);
      }
      rec[0] = M == -INFINITY ? -INFINITY : M * kLn2;  // natural units
      rec[1] = L;
      rec[2] = Q;
      rec[3] = 0.f;
    }
  }
}

template <int D, int NT, typename T>
cudaError_t launch(const PagedArgs& a, cudaStream_t s) {
  Q4DecodeParams p;
  p.q = a.base.q;
  p.k_pages = static_cast<const uint8_t*>(a.k_pages);
  p.v_pages = static_cast<const uint8_t*>(a.v_pages);
  p.table = a.block_table;
  p.lens = a.base.seq_lens;
  p.partials = a.base.partials;
  p.Hq = a.base.H;
  p.Hkv = a.Hkv;
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  p.shift = a.page_shift;
  p.max_seq_len = a.base.Tkv;
  p.splits = a.base.splits;
  p.chunk = a.base.chunk;
  p.c = a.base.c;
  p.status = a.status;
  auto kern = polar_decode_q4_kernel<D, NT, T>;
  const int smem = (int)sizeof(Q4Smem<D>);
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<dim3((unsigned)(a.base.B * a.Hkv), (unsigned)a.base.splits), kThreads, smem, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_q4(const PagedArgs& a, int dtype, cudaStream_t s) {
  if (dtype == POLAR_BF16)
    return a.base.d == 64 ? launch<64, 1, __nv_bfloat16>(a, s) : launch<128, 1, __nv_bfloat16>(a, s);
  return a.base.d == 64 ? launch<64, 3, float>(a, s) : launch<128, 3, float>(a, s);
}

}  // namespace polar

using namespace polar;

namespace {

bool sizes_ok(int B, int Hq, int Hkv, int d, int max_seq_len) {
  if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return false;
  const int G = Hq / Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8) return false;
  return (d == 64 || d == 128) && max_seq_len >= 1 && max_seq_len <= (1 << 30) &&
         (long long)B * Hq <= INT_MAX;
}

// A split CTA pays about two stages' time for its start and its record:
// prefer whole waves (three CTAs a SM) of CTAs with at least two stages each.
int auto_splits_q4(int BH, int max_seq_len, int sms) {
  const int stages = (max_seq_len + kSK - 1) / kSK;
  const int slots = 3 * sms;
  int best = 1;
  double best_eff = -1.0;
  for (int s = 1; s <= 256 && s <= stages; ++s) {
    const int per = (stages + s - 1) / s;
    if (per < 2 && s > 1) break;
    const double waves = (double)BH * s / slots;
    const double eff = waves / std::ceil(waves) * per / (per + 2.0);
    if (eff > best_eff + 1e-9) {
      best_eff = eff;
      best = s;
    }
  }
  return best;
}

}  // namespace

extern "C" {

int polar_attn_decode_paged_q4_num_splits(int B, int Hkv, int max_seq_len, int d) {
  if (B < 0 || Hkv < 1 || max_seq_len < 1 || max_seq_len > (1 << 30) || (d != 64 && d != 128))
    return 0;
  int sms = 0;
  if (check_device(&sms) != POLAR_OK) sms = 148;
  const long long BH = (long long)B * Hkv;
  return auto_splits_q4((int)std::min(std::max(BH, 1LL), (long long)INT_MAX), max_seq_len, sms);
}

size_t polar_attn_decode_paged_q4_workspace_bytes(int B, int Hq, int Hkv, int max_seq_len, int d,
                                                  int num_splits) {
  if (!sizes_ok(B, Hq, Hkv, d, max_seq_len) || num_splits < 0) return 0;
  const int s =
      num_splits > 0 ? num_splits : polar_attn_decode_paged_q4_num_splits(B, Hkv, max_seq_len, d);
  return (size_t)B * Hq * s * (d + 4) * sizeof(float);
}

int polar_attn_decode_paged_q4(const void* q, const void* k_pages, const void* v_pages,
                               const int* block_table, const int* seq_lens, const void* mem,
                               const float* w_count, void* out, float* n_eff, float* conf, int B,
                               int Hq, int Hkv, int d, int page_size, int num_pages, int max_pages,
                               int max_seq_len, int dtype, const polar_consts_t* c, int num_splits,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (B < 0 || Hq < 1 || Hkv < 1 || num_splits < 0 || num_pages < 1 || max_pages < 1 ||
      max_seq_len < 1)
    return POLAR_ERR_INVALID;
  if (dtype != POLAR_F32 && dtype != POLAR_BF16) return POLAR_ERR_UNSUPPORTED;
  if (!sizes_ok(B, Hq, Hkv, d, max_seq_len) || num_splits > 65535) return POLAR_ERR_UNSUPPORTED;
  if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) != 0)
    return POLAR_ERR_UNSUPPORTED;
  if ((long long)num_pages * page_size > INT_MAX) return POLAR_ERR_UNSUPPORTED;
  if ((long long)max_pages * page_size < max_seq_len) return POLAR_ERR_INVALID;
  const polar_consts_t cc = c ? *c : defaults();
  if (!consts_ok(cc)) return POLAR_ERR_INVALID;
  if (B == 0) return POLAR_OK;
  if (!q || !k_pages || !v_pages || !block_table || !seq_lens || !mem || !w_count || !out || !n_eff)
    return POLAR_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(mem) ||
      !aligned16(w_count) || !aligned16(out) || (reinterpret_cast<uintptr_t>(block_table) & 3u) ||
      (reinterpret_cast<uintptr_t>(seq_lens) & 3u) || (reinterpret_cast<uintptr_t>(n_eff) & 3u) ||
      (reinterpret_cast<uintptr_t>(conf) & 3u))
    return POLAR_ERR_MISALIGNED;
  int sms = 0;
  int st = check_device(&sms);
  if (st != POLAR_OK) return st;
  const int splits = num_splits > 0 ? num_splits : auto_splits_q4(B * Hkv, max_seq_len, sms);
  if (!workspace || workspace_bytes < (size_t)B * Hq * splits * (d + 4) * sizeof(float))
    return POLAR_ERR_WORKSPACE;
  if (!aligned16(workspace)) return POLAR_ERR_MISALIGNED;
  PagedArgs a;
  // whole stages, which start on page pieces of 8 rows or more
  int chunk = (int)(((long long)max_seq_len + splits - 1) / splits);
  chunk = (chunk + kSK - 1) / kSK * kSK;
  a.base = DecodeArgs{q, nullptr, nullptr, mem, w_count, out, n_eff, conf, B, Hq, max_seq_len,
                      d, cc, splits, chunk, static_cast<float*>(workspace), seq_lens};
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.block_table = block_table;
  a.Hkv = Hkv;
  a.page_shift = 0;
  while ((1 << a.page_shift) < page_size) ++a.page_shift;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.status = status_word();
  if (!a.status) return cuda_status("cudaGetSymbolAddress", cudaGetLastError());
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  st = cuda_status("4-bit decode split launch", launch_decode_q4(a, dtype, s));
  if (st != POLAR_OK) return st;
  return cuda_status("4-bit decode combine launch", launch_decode_combine(a.base, dtype, s));
}

}  // extern "C"
