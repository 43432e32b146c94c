// Paged, grouped-query decode over a 4-bit cache.
//
// The mathematics is polar_decode_paged's (per query head: l = sum p, Q2 = sum
// p^2, acc = sum p v, then the epilogue of the pinned reading); the rows are
// those of polar_cache_q4.cuh.  With the codes n and the scales s of a key's
// 32-channel groups g,
//   q . k_j = sum_g sk_jg (q_g . n_jg),     acc_g = sum_j (p_j sv_jg) n_jg
// so the scales never meet the codes: a key's score is a sum of d / 32 partial
// products, and V's scales go into the weights.
//
// A row of K or V is 9 d / 16 bytes, so at the rate of DRAM about 42 codes a
// clock pass through each SM, and the instructions that unpack them are the
// other bound.  Hence warp products (m16n8k16, bf16, fp32 sums) whose A operand
// is unpacked from the packed words in registers, in at most one instruction a
// code: a code masked out of its word is the bf16 subnormal n 2^-129, exactly;
// factors 2^64 in q and 2^40 in the weights keep the sums in fp32's normal range.
// A tensor-core instruction that reads its operand from shared memory would
// need the unpacked rows written there, 4 bytes for each byte of DRAM.
//   S (16 keys x 8 heads) = K codes (A, 16 x 16 channels) . q^T (B)
//   O^T (16 channels x 8 heads) += V codes^T (A, 16 channels x 16 keys) . P'^T (B)
// P' comes from S's registers by movmatrix.  fp32 queries are split into three
// bf16 terms, whose sum is q, and so are the weights: three products each.
// The eight columns are the query heads of a KV head; with four of them half of the
// maxima, exponentials, sums and weights, with one seven eighths, are of zero rows,
// and cost what others do.
//
// Work: the stages (128 keys) of all (sequence, KV head) pairs in one row are
// cut into equal runs, a run a CTA, all resident at once: sequences of different
// lengths cost what their rows cost.  A run's part of a pair is a segment, which
// ends in a record; segments have the number (CTA + pair), which grows from one
// to the next, so there are fewer than CTAs + pairs of them.  The runs follow
// from the lengths, which every CTA sums itself.
// 160 threads: warps 0-3 compute, 32 keys of a stage each, with their own running
// maxima, sums and O, joined in shared memory at a segment's end; warp 4 copies
// (cp.async.bulk into a ring of stages; a whole page of 16 to 128 rows is one copy,
// other pieces are a copy of codes and one of scales), ahead of the segments' ends.
// Measured: 32 sequences of 32768 rows, 16 query on 4 KV heads, d = 128, pages of 64:
// 118 us, 5.1 TB/s (two copies a page: 5 more); the same copies without arithmetic 100.
// d = 64, 8 heads, 16384 rows: 76 us (two copies 7 more).  32 of up to 20000 rows, pages
// of 16: 50 us (two copies 10 more).  Records are joined eight at a time, heads and sums
// loaded together (maxima first, then the sums: 1.2 to 2 us more).
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
constexpr int kStages = 3;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;  // log2 units
constexpr float kTwo64 = 18446744073709551616.0f;
constexpr float kTwo65 = 36893488147419103232.0f;
// weights carry 2^40 into the values' products: a weight of 1 keeps 24 bits beside a
// scale down to 2^-36
constexpr float kTwo40 = 1099511627776.0f;
constexpr float kUnshiftAcc = 618970019642690137449562112.0f;  // 2^(129 - 40)
constexpr uint32_t kCodeMask = 0x80708070u;

template <int D>
struct Q4Smem {
  // a stage's rows of K and V: codes and scales of each page, as in the pages, where
  // pages of 16 to 128 rows are copied whole; else all codes, then all scales
  uint8_t k[kStages][kSK * q4_row_bytes(D)], v[kStages][kSK * q4_row_bytes(D)];
  float join[kWarps][8][D];  // the warps' O
  uint32_t valid[kStages];   // a bit for each 8 keys of the stage
  uint64_t full[kStages], empty[kStages];
  float m[kWarps][8], l[kWarps][8], q2[kWarps][8];
  int abort_flag;
};

struct Q4DecodeParams {
  const void *q, *mem;
  const float* w_count;
  void* out;
  float *n_eff, *conf;
  const uint8_t *k_pages, *v_pages;
  const int *table, *lens;
  float* records;  // [runs + B * Hkv][G][D + 4]: m (natural units), l, Q2, -, acc
  int2* spans;     // [B * Hkv] first and last record of a pair with keys
  int B, Hq, Hkv, max_pages, num_pages, shift, max_seq_len, runs;
  polar_consts_t c;
  int* status;
};

// Keys and stages of sequence b.
__device__ __forceinline__ int keys_of(const Q4DecodeParams& p, int b, bool* bad) {
  const int n = __ldg(p.lens + b);
  if (n < 1 || n > p.max_seq_len) *bad = true;
  return n < 1 ? 0 : min(n, p.max_seq_len);
}
__device__ __forceinline__ int stages_of(const Q4DecodeParams& p, int b, bool* bad) {
  return (keys_of(p, b, bad) + kSK - 1) / kSK;
}

// Sum over the warp.
__device__ __forceinline__ long long warp_total(long long v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Stages of a run, from the lengths; by a converged warp.
__device__ __forceinline__ long long stages_a_run(const Q4DecodeParams& p, bool* bad) {
  long long sum = 0;
  for (int b = threadIdx.x & 31; b < p.B; b += 32) sum += stages_of(p, b, bad);
  const long long w = warp_total(sum) * p.Hkv;
  return (w + p.runs - 1) / p.runs;
}

// Where a run is: stages [s0, s1) of the pair (b, hkv).
struct Segment {
  int b, hkv, keys;  // keys of the sequence
  int s0, s1;
  long long left;    // stages of the run after this segment
};

// The first segment of run `run`; b = B if the run is empty.  By a converged warp.
__device__ __forceinline__ Segment first_segment(const Q4DecodeParams& p, int run, long long per) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  long long at = run * per, before = 0;  // stages of the sequences before
  Segment g{p.B, 0, 0, 0, 0, 0};
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int n = b0 + lane < p.B ? stages_of(p, b0 + lane, &bad) : 0;
    long long upto = (long long)n * p.Hkv;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += u;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + upto > at);
    if (past) {
      const int l = __ffs(past) - 1;
      const int nb = __shfl_sync(0xffffffffu, n, l);
      at -= before + __shfl_sync(0xffffffffu, upto, l) - (long long)nb * p.Hkv;
      g.b = b0 + l;
      g.keys = keys_of(p, g.b, &bad);
      g.hkv = (int)(at / nb);
      g.s0 = (int)(at - (long long)g.hkv * nb);
      const long long here = per < nb - g.s0 ? per : nb - g.s0;
      g.s1 = g.s0 + (int)here;
      g.left = per - here;
      return g;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return g;
}

// The next segment of the run (left > 0): the next pair with keys, or b = B.
__device__ __forceinline__ void next_segment(const Q4DecodeParams& p, Segment& g) {
  bool bad = false;
  int nb = (g.keys + kSK - 1) / kSK;
  if (++g.hkv == p.Hkv) {
    g.hkv = 0;
    do {
      if (++g.b >= p.B) return;
      g.keys = keys_of(p, g.b, &bad);
      nb = (g.keys + kSK - 1) / kSK;
    } while (nb == 0);
  }
  g.s0 = 0;
  g.s1 = (int)(g.left < nb ? g.left : nb);
  g.left -= g.s1;
}

// Meeting of the 128 compute threads; true if `ok` holds in every one.
__device__ __forceinline__ bool compute_bar_and(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok), "n"(32 * kWarps)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same, onto zero.
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
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

// The first term of x's expansion in bf16 (x = t0 + t1 + t2 up to 2^-24 x).
__device__ __forceinline__ float bf16_round(float x) {
  return __bfloat162float(__float2bfloat16_rn(x));
}

// What a compute lane carries through a segment.
template <int D, int NT>
struct Q4State {
  static constexpr int NG = D / 32;
  uint32_t qb[NT][NG][4];  // q as B operand (terms of it)
  float o[2 * NG][4];  // O^T tile 2 g + t: channels 32 g + 4 r + 2 t (+ 1), heads 2 c, 2 c + 1
  // references of the two heads (units of x), x that moves them, sums
  float m0, m1, up0, up1, l0, l1, s0, s1;
  float scale2;  // log2 units a unit of x, the products' sum, which carries 2^-65
};

// The warp's 32 keys of a stage, their codes at kc and vc and their scales `scales`
// bytes further, as two products of 16 (the second's rows next_codes, next_scales
// bytes further), so that their chains overlap.  kWhole: every key is visible
// and on a page of the pool; else bit h of `octets` says so of the page of rows
// 8 h .., and n keys are visible.
template <int D, int NT, bool kWhole>
__device__ __forceinline__ void q4_keys(const uint8_t* kc, const uint8_t* vc, int scales,
                                        int next_codes, int next_scales, int n, uint32_t octets,
                                        Q4State<D, NT>& z) {
  constexpr int NG = D / 32, NS = 2;
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  // row r of a product's 16 keys (8 and more: + 8) is the key r / 2 of them for even
  // r, 4 + (r / 2 ^ kTurn) for odd: V's operand, whose columns 2 c and 2 c + 1 are
  // the keys c and 4 + (c ^ kTurn), reads neighbouring rows, and the lanes that read K
  // together take rows of different banks
  constexpr int kTurn = D == 128 ? 1 : 2;
  const int rk = r & 1 ? 4 + ((r >> 1) ^ kTurn) : r >> 1;
  // ---- scores: x[2 h + i] of rows 8 h + r, heads 2 c + i
  float x[4 * NS];
#pragma unroll
  for (int u = 0; u < NS; ++u) {
    const uint8_t *codes = kc + u * next_codes, *scale = kc + scales + u * next_scales;
    uint32_t ka[NG], kb[NG];
    float sa[NG], sb[NG], y[4] = {0.f, 0.f, 0.f, 0.f};
    load_words<D>(codes + rk * (D / 2) + c * (D / 8), ka);
    load_words<D>(codes + (8 + rk) * (D / 2) + c * (D / 8), kb);
    load_scales<D>(scale + rk * (D / 16), sa);
    load_scales<D>(scale + (8 + rk) * (D / 16), sb);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float acc[4];
      const uint32_t za = __byte_perm(ka[g], 0, 0x2301), zb = __byte_perm(kb[g], 0, 0x2301);
      const uint32_t f0[4] = {ka[g] & kCodeMask, kb[g] & kCodeMask, (ka[g] << 4) & kCodeMask,
                              (kb[g] << 4) & kCodeMask};
      const uint32_t f1[4] = {za & kCodeMask, zb & kCodeMask, (za << 4) & kCodeMask,
                              (zb << 4) & kCodeMask};
      // the smallest terms first
#pragma unroll
      for (int t = NT - 1; t >= 0; --t) {
        if (t == NT - 1) mma16816_first(acc, f0, z.qb[t][g][0], z.qb[t][g][1]);
        else mma16816(acc, f0, z.qb[t][g][0], z.qb[t][g][1]);
        mma16816(acc, f1, z.qb[t][g][2], z.qb[t][g][3]);
      }
      y[0] = fmaf(acc[0], sa[g], y[0]);
      y[1] = fmaf(acc[1], sa[g], y[1]);
      y[2] = fmaf(acc[2], sb[g], y[2]);
      y[3] = fmaf(acc[3], sb[g], y[3]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[4 * u + i] = y[i];
  }
  bool in[2 * NS];
  if constexpr (!kWhole) {
#pragma unroll
    for (int h = 0; h < 2 * NS; ++h) {
      in[h] = 8 * h + rk < n && ((octets >> h) & 1u);
      if (!in[h]) x[2 * h] = x[2 * h + 1] = -INFINITY;  // its scale may be anything
    }
  }
  float t0 = x[0], t1 = x[1];
#pragma unroll
  for (int h = 1; h < 2 * NS; ++h) t0 = fmaxf(t0, x[2 * h]), t1 = fmaxf(t1, x[2 * h + 1]);
  if (__any_sync(0xffffffffu, t0 > z.up0 || t1 > z.up1)) {
#pragma unroll
    for (int d = 4; d <= 16; d <<= 1) {
      t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, d));
      t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, d));
    }
    const float slack = kRescale / z.scale2;
    float a0 = 1.f, a1 = 1.f;  // 0 at the first keys
    auto correction = [&](float m, float t) {
      // of the rounded products, which the weights and the records are relative to
      return ex2_approx(__fmul_rn(m, z.scale2) - __fmul_rn(t, z.scale2));
    };
    if (t0 > z.up0) a0 = correction(z.m0, t0), z.m0 = t0, z.up0 = t0 + slack;
    if (t1 > z.up1) a1 = correction(z.m1, t1), z.m1 = t1, z.up1 = t1 + slack;
    z.l0 *= a0, z.l1 *= a1;
    z.s0 *= a0 * a0, z.s1 *= a1 * a1;  // squared correction factor
#pragma unroll
    for (int i = 0; i < 2 * NG; ++i)
      z.o[i][0] *= a0, z.o[i][2] *= a0, z.o[i][1] *= a1, z.o[i][3] *= a1;
  }
  // (the 2^40 comes after the sums: with it in the exponents these lost five bits, and
  // l, the participation ratio and the gate with them: n_eff of one key beside 1023 of
  // weight 2^-7 was off by 2.5e-6, now 1.9e-7.  Packed pairs, so that it costs no time:
  // 32 sequences of 32768 rows 118.9 us before, 120.9 with single products, 117.7)
  const float2 n01 = make_float2(-z.m0 * z.scale2, -z.m1 * z.scale2);
  const float2 scale = make_float2(z.scale2, z.scale2);
  float2 l = make_float2(z.l0, z.l1), q2 = make_float2(z.s0, z.s1);
#pragma unroll
  for (int h = 0; h < 2 * NS; ++h) {
    const float2 y = ffma2(make_float2(x[2 * h], x[2 * h + 1]), scale, n01);
    float2 w = make_float2(ex2_approx(y.x), ex2_approx(y.y));
    if constexpr (!kWhole)
      if (!in[h]) w = make_float2(0.f, 0.f);
    l = fadd2(l, w);
    q2 = ffma2(w, w, q2);
    w = fmul2(w, make_float2(kTwo40, kTwo40));
    x[2 * h] = w.x, x[2 * h + 1] = w.y;
  }
  z.l0 = l.x, z.l1 = l.y, z.s0 = q2.x, z.s1 = q2.y;
  // ---- values.  Selectors: half r % 2 of a word of each of two keys, as it is
  // and with the bytes of each half swapped.
  const uint32_t sel_a = (r & 1) ? 0x7632u : 0x5410u, sel_b = (r & 1) ? 0x6723u : 0x4501u;
#pragma unroll
  for (int u = 0; u < NS; ++u) {
    const uint8_t *codes = vc + u * next_codes, *scale = vc + scales + u * next_scales;
    float va[NG], vb[NG];
    load_scales<D>(scale + rk * (D / 16), va);
    load_scales<D>(scale + (8 + rk) * (D / 16), vb);
    if constexpr (!kWhole) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (!in[2 * u]) va[g] = 0.f;
        if (!in[2 * u + 1]) vb[g] = 0.f;
      }
    }
    uint32_t y[4][NG];  // keys c, 4 + (c ^ kTurn), and 8 more
#pragma unroll
    for (int i = 0; i < 4; ++i)
      load_words<D>(codes + (4 * i + (i & 1 ? c ^ kTurn : c)) * (D / 2) + (r >> 1) * (D / 8),
                    y[i]);
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
      float e[4] = {x[4 * u] * va[g], x[4 * u + 1] * va[g], x[4 * u + 2] * vb[g],
                    x[4 * u + 3] * vb[g]};
      uint32_t bl[NT], bh[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        bl[t] = transpose8(pack_bf16x2(e[0], e[1]));
        bh[t] = transpose8(pack_bf16x2(e[2], e[3]));
        if (t + 1 < NT)
#pragma unroll
          for (int i = 0; i < 4; ++i) e[i] -= bf16_round(e[i]);
      }
      if constexpr (NT == 1) {
        // (the tensor cores' own fp32 sums: cut to about 1e-6 over 81355 keys, far below
        // the weights' 2^-9)
        mma16816(z.o[2 * g], f0, bl[0], bh[0]);
        mma16816(z.o[2 * g + 1], f1, bl[0], bh[0]);
      } else {
        // a step's products are summed on their own and added once, in fp32's
        // rounding (the tensor cores' sums are cut: 81355 keys, error 1.0e-6)
        float d0[4], d1[4];
        mma16816_first(d0, f0, bl[NT - 1], bh[NT - 1]);
        mma16816_first(d1, f1, bl[NT - 1], bh[NT - 1]);
#pragma unroll
        for (int t = NT - 2; t >= 0; --t) {
          mma16816(d0, f0, bl[t], bh[t]);
          mma16816(d1, f1, bl[t], bh[t]);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) z.o[2 * g][i] += d0[i], z.o[2 * g + 1][i] += d1[i];
      }
    }
  }
}

// NT: bf16 terms of q and of the weights (1: bf16 queries, 3: fp32).
template <int D, int NT, typename T>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2)
    polar_decode_q4_kernel(const Q4DecodeParams p) {
  constexpr int NG = D / 32;  // groups of channels
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Q4Smem<D>& sm = *reinterpret_cast<Q4Smem<D>*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], kWarps);
    }
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  bool bad = false;
  const long long per = stages_a_run(p, &bad);
  if (blockIdx.x == 0 && warp == 0 && __any_sync(0xffffffffu, bad) && lane == 0)
    atomicExch(p.status, 3);
  Segment g = first_segment(p, (int)blockIdx.x, per);
  __syncthreads();
  volatile int* abort_flag = &sm.abort_flag;

  const int page = 1 << p.shift;
  const bool whole = page >= 16 && page <= kSK;  // pages are copied whole

  if (warp == kWarps) {
    // ------------------------------------------------------------- copies --
    // lane o < 16: the stage's keys 8 o .. 8 o + 7; the first lane of a piece
    // of min(page, 128) keys issues its copies
    const int piece = min(page, kSK);
    const bool leader = lane < 16 && (lane * 8) % piece == 0;
    int st = 0;  // stages of the run
    bool ok = true;
    for (; g.b < p.B && ok; next_segment(p, g)) {
      const int* tb = p.table + (size_t)g.b * p.max_pages;
      auto entry = [&](int s) -> int {
        const int key = s * kSK + lane * 8;
        return lane < 16 && key < g.keys ? __ldg(tb + (key >> p.shift)) : -1;
      };
      int pg = entry(g.s0);
      for (int s = g.s0; s < g.s1; ++s, ++st) {
        const int slot = st % kStages;
        const int next = s + 1 < g.s1 ? entry(s + 1) : -1;
        if (st >= kStages)
          ok = mbar_wait_warp(&sm.empty[slot], (uint32_t)(st / kStages - 1) & 1, abort_flag,
                              p.status);
        if (!ok) break;
        const int key = s * kSK + lane * 8;
        const bool here = lane < 16 && key < g.keys;
        const bool good = here && pg >= 0 && pg < p.num_pages;
        if (here && !good) atomicExch(p.status, 3);
        const uint32_t valid = __ballot_sync(0xffffffffu, good);
        // rows in whole copies of 16 bytes
        const int rows = leader && good ? min(piece, (g.keys - key + 3) & ~3) : 0;
        const uint32_t bytes =
            __reduce_add_sync(0xffffffffu, 2u * (uint32_t)rows * q4_row_bytes(D));
        if (lane == 0) {
          sm.valid[slot] = valid;
          mbar_arrive_expect_tx(&sm.full[slot], bytes);
        }
        __syncwarp();
        if (rows > 0) {
          const int row = key & (page - 1), at = lane * 8;
          const int codes_at = whole ? at * q4_row_bytes(D) : at * (D / 2);
          const int scales_at = whole ? codes_at + page * (D / 2) : kSK * (D / 2) + at * (D / 16);
          const size_t block = q4_block(pg, g.hkv, p.Hkv, p.shift, D);
          const size_t codes = block + (size_t)row * (D / 2);
          const size_t scales = block + ((size_t)(D / 2) << p.shift) + (size_t)row * (D / 16);
          uint64_t* bar = &sm.full[slot];
          if (whole && rows == page) {
            bulk_g2s(sm.k[slot] + codes_at, p.k_pages + codes, page * q4_row_bytes(D), bar);
            bulk_g2s(sm.v[slot] + codes_at, p.v_pages + codes, page * q4_row_bytes(D), bar);
          } else {
            bulk_g2s(sm.k[slot] + codes_at, p.k_pages + codes, rows * (D / 2), bar);
            bulk_g2s(sm.k[slot] + scales_at, p.k_pages + scales, rows * (D / 16), bar);
            bulk_g2s(sm.v[slot] + codes_at, p.v_pages + codes, rows * (D / 2), bar);
            bulk_g2s(sm.v[slot] + scales_at, p.v_pages + scales, rows * (D / 16), bar);
          }
        }
        pg = next;
      }
      if (g.left == 0) break;
    }
    if (!ok) {
      // aborted: let the copies already issued land before the CTA exits
      volatile int never = 0;
      for (int i = st - 1; i >= 0 && i >= st - kStages; --i)
        mbar_wait(&sm.full[i % kStages], (uint32_t)(i / kStages) & 1, &never, p.status,
                  kWaitLimitCycles / 4);
      __syncwarp();
    }
    return;
  }

  // --------------------------------------------------------------- compute --
  const int r = lane >> 2, c = lane & 3;
  // the warp's rows in a stage
  const int row = warp * 32, in_page = row & (page - 1);
  const int page_at = (row - in_page) * q4_row_bytes(D);
  const int codes_at = whole ? page_at + in_page * (D / 2) : row * (D / 2);
  const int scales_at = whole ? page_at + page * (D / 2) + in_page * (D / 16)
                              : kSK * (D / 2) + row * (D / 16);
  int st = 0;
  bool ok = true;
  for (; g.b < p.B; next_segment(p, g)) {
    Q4State<D, NT> z;
    {
      // B operand: head r, channels 32 g + 8 c + (0, 4), (1, 5), (2, 6), (3, 7)
      const T* qp = static_cast<const T*>(p.q) +
                    ((size_t)g.b * p.Hq + (size_t)g.hkv * G + r) * D + 8 * c;
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = r < G ? (float)qp[32 * i + j] : 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // 2^64 is exact in bf16: the terms are those of q
            z.qb[t][i][j] = pack_bf16x2(x[j] * kTwo64, x[j + 4] * kTwo64);
            if (t + 1 < NT) {
              x[j] -= bf16_round(x[j]);
              x[j + 4] -= bf16_round(x[j + 4]);
            }
          }
      }
    }
    z.scale2 = polar_tau((float)g.keys, p.c.log_t0) * kLog2e * rsqrtf((float)D) * kTwo65;
#pragma unroll
    for (int i = 0; i < 2 * NG; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) z.o[i][j] = 0.f;
    z.m0 = z.m1 = z.up0 = z.up1 = -INFINITY;
    z.l0 = z.l1 = z.s0 = z.s1 = 0.f;
    for (int s = g.s0; s < g.s1 && ok; ++s, ++st) {
      const int slot = st % kStages;
      ok = mbar_wait_warp(&sm.full[slot], (uint32_t)(st / kStages) & 1, abort_flag, p.status);
      if (!ok) break;
      const int n = g.keys - (s * kSK + warp * 32);  // visible keys from the warp's first on
      const uint32_t octets = (sm.valid[slot] >> (4 * warp)) & 15u;
      const uint8_t *kc = sm.k[slot] + codes_at, *vc = sm.v[slot] + codes_at;
      const int scales = scales_at - codes_at;
      const int next_codes = page == 16 ? 16 * q4_row_bytes(D) : 16 * (D / 2);
      const int next_scales = page == 16 ? 16 * q4_row_bytes(D) : 16 * (D / 16);
      if (n >= 32 && octets == 15u)
        q4_keys<D, NT, true>(kc, vc, scales, next_codes, next_scales, n, octets, z);
      else if (n > 0)
        q4_keys<D, NT, false>(kc, vc, scales, next_codes, next_scales, n, octets, z);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.empty[slot]);
    }
    // ---- the four warps' states into the segment's record
#pragma unroll
    for (int d = 4; d <= 16; d <<= 1) {
      z.l0 += __shfl_xor_sync(0xffffffffu, z.l0, d);
      z.l1 += __shfl_xor_sync(0xffffffffu, z.l1, d);
      z.s0 += __shfl_xor_sync(0xffffffffu, z.s0, d);
      z.s1 += __shfl_xor_sync(0xffffffffu, z.s1, d);
    }
    // (the reads of the last segment's join are over; a wait that ran out ends
    // the call in every warp)
    ok = compute_bar_and(ok);
    if (!ok) break;
    if (r == 0) {
      sm.m[warp][2 * c] = z.m0 * z.scale2, sm.m[warp][2 * c + 1] = z.m1 * z.scale2;
      sm.l[warp][2 * c] = z.l0, sm.l[warp][2 * c + 1] = z.l1;
      sm.q2[warp][2 * c] = z.s0, sm.q2[warp][2 * c + 1] = z.s1;
    }
#pragma unroll
    for (int i = 0; i < NG; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float4*>(&sm.join[warp][2 * c + h][32 * i + 4 * r]) = make_float4(
            z.o[2 * i][h], z.o[2 * i][2 + h], z.o[2 * i + 1][h], z.o[2 * i + 1][2 + h]);
    compute_bar_and(true);
    const int t = threadIdx.x % D, pair = g.b * p.Hkv + g.hkv;
    const int id = (int)blockIdx.x + pair;
    if (threadIdx.x == 0) {
      if (g.s0 == 0) p.spans[pair].x = id;
      if (g.s1 == (g.keys + kSK - 1) / kSK) p.spans[pair].y = id;
    }
    float* rec0 = p.records + (size_t)id * G * (D + 4);
    for (int h = threadIdx.x / D; h < G; h += 32 * kWarps / D) {
      float M = -INFINITY;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sm.m[i][h]);
      float e[kWarps];
#pragma unroll
      for (int i = 0; i < kWarps; ++i)
        e[i] = sm.m[i][h] == -INFINITY ? 0.f : ex2_approx(sm.m[i][h] - M);
      float* rec = rec0 + (size_t)h * (D + 4);
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) a = fmaf(e[i], sm.join[i][h][t], a);
      rec[4 + t] = a * kUnshiftAcc;
      if (t == 0) {
        float L = 0.f, Q = 0.f;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
          L = fmaf(e[i], sm.l[i][h], L);
          Q = fmaf(e[i] * e[i], sm.q2[i][h], Q);
        }
        *reinterpret_cast<float4*>(rec) =
            make_float4(M == -INFINITY ? -INFINITY : M * kLn2, L, Q, 0.f);
      }
    }
    if (g.left == 0) break;
  }
}

// ----------------------------------------------------------------- combine --
// One CTA a query head: D threads for the channels, times kParts groups that
// share the records of its pair.
template <int D, int kParts, typename T>
__global__ void __launch_bounds__(D* kParts)
    polar_decode_q4_combine_kernel(const Q4DecodeParams p) {
  constexpr int R = D + 4;
  const int G = p.Hq / p.Hkv, b = blockIdx.x / p.Hq, h = blockIdx.x % p.Hq;
  const int x = threadIdx.x % D, part = threadIdx.x / D;
  bool bad = false;
  const int keys = keys_of(p, b, &bad);
  const size_t row = (size_t)blockIdx.x * D + x;
  const float qx = (float)static_cast<const T*>(p.q)[row];
  const float mx = (float)static_cast<const T*>(p.mem)[row];
  const float wx = p.w_count[(size_t)h * D + x];
  // the records are written by the grid before (programmatic launch)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int2 s = keys > 0 ? p.spans[b * p.Hkv + h / G] : make_int2(0, -1);
  // (a run that gave up, recorded, leaves what the workspace held)
  if (s.x < 0 || s.y >= p.runs + p.B * p.Hkv) s = make_int2(0, -1);
  const float* rec = p.records + ((size_t)s.x * G + h % G) * R;
  const size_t step = (size_t)G * R;
  const int n = s.y - s.x + 1;
  float M = -INFINITY, a = 0.f, L = 0.f, Q = 0.f;
  if constexpr (kParts == 1) {
    // a few records: every thread reads the heads of all, eight at a time
    constexpr int kBatch = 8;
    for (int i0 = 0; i0 < n; i0 += kBatch) {
      float4 r[kBatch];
      float v[kBatch];
      float Mb = M;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const bool in = i0 + i < n;
        const float* at = rec + (i0 + i) * step;
        r[i] = in ? *reinterpret_cast<const float4*>(at) : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        v[i] = in ? at[4 + x] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) Mb = fmaxf(Mb, r[i].x);
      const float down = M == -INFINITY ? 0.f : expf(M - Mb);
      a *= down, L *= down, Q *= down * down;  // squared correction factor
      M = Mb;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        // a segment without visible keys weighs 0
        const float e = r[i].x == -INFINITY ? 0.f : expf(r[i].x - M);
        a = fmaf(e, v[i], a);
        L = fmaf(e, r[i].y, L);
        Q = fmaf(e * e, r[i].z, Q);
      }
    }
  } else {
    // many: their weights once, in shared memory, then a group's share of acc
    constexpr int N = D * kParts;
    __shared__ float weight[N], red[3][N / 32];
    __shared__ float acc[kParts][D];
    auto over_block = [&](float v, int k, auto join) {
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, o));
      if ((threadIdx.x & 31) == 0) red[k][threadIdx.x >> 5] = v;
    };
    auto larger = [](float u, float v) { return fmaxf(u, v); };
    auto sum = [](float u, float v) { return u + v; };
    for (int i = threadIdx.x; i < n; i += N) M = fmaxf(M, rec[i * step]);
    over_block(M, 0, larger);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N / 32; ++i) M = fmaxf(M, red[0][i]);
    for (int i0 = 0; i0 < n; i0 += N) {
      const int m = min(N, n - i0);
      __syncthreads();  // the last weights are read
      if ((int)threadIdx.x < m) {
        const float4 r = *reinterpret_cast<const float4*>(rec + (i0 + threadIdx.x) * step);
        const float e = r.x == -INFINITY ? 0.f : expf(r.x - M);
        weight[threadIdx.x] = e;
        L = fmaf(e, r.y, L);
        Q = fmaf(e * e, r.z, Q);
      }
      __syncthreads();
#pragma unroll 8
      for (int i = part; i < m; i += kParts) a = fmaf(weight[i], rec[(i0 + i) * step + 4 + x], a);
    }
    over_block(L, 1, sum);
    over_block(Q, 2, sum);
    acc[part][x] = a;
    __syncthreads();
    if (part != 0) return;
    a = L = Q = 0.f;
#pragma unroll
    for (int i = 0; i < kParts; ++i) a += acc[i][x];
#pragma unroll
    for (int i = 0; i < N / 32; ++i) L += red[1][i], Q += red[2][i];
  }
  // |acc|^2 in units of the power of two below L, which changes no bit (128 channels of
  // 2^52 overflowed from L = 363 on, and the direction was lost)
  const float unit =
      __uint_as_float(0x7F000000u - (__float_as_uint(L) & 0x7F800000u));  // 2^-floor(log2 L)
  const float au = a * unit;
  float acc_sq = au * au, q_sq = qx * qx;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    acc_sq += __shfl_xor_sync(0xffffffffu, acc_sq, o);
    q_sq += __shfl_xor_sync(0xffffffffu, q_sq, o);
  }
  // (D threads are left: those of group 0)
  __shared__ float2 sums[D / 32];
  if ((x & 31) == 0) sums[x >> 5] = make_float2(acc_sq, q_sq);
  asm volatile("bar.sync 1, %0;" ::"n"(D) : "memory");
  acc_sq = q_sq = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) acc_sq += sums[i].x, q_sq += sums[i].y;
  T* out = static_cast<T*>(p.out);
  if (L == 0.f) {
    // no key was visible (an invalid length or bad pages, recorded): direction
    // and count are zero, the memory stream passes
    out[row] = (T)mx;
    if (x == 0) {
      p.n_eff[blockIdx.x] = 0.f;
      if (p.conf) p.conf[blockIdx.x] = 0.f;
    }
    return;
  }
  const RowResult res =
      polar_finish_norm(M, L, Q, sqrtf(acc_sq) / (L * unit), q_sq, (float)keys, D, p.c);
  out[row] = (T)fmaf(a, res.scale_u, fmaf(res.count, wx, mx));
  if (x == 0) {
    p.n_eff[blockIdx.x] = res.n_eff;
    if (p.conf) p.conf[blockIdx.x] = res.conf;
  }
}

template <int D, int NT, typename T>
int launch(const Q4DecodeParams& p, cudaStream_t s) {
  auto kern = polar_decode_q4_kernel<D, NT, T>;
  const int smem = (int)sizeof(Q4Smem<D>);
  static_assert((NT == 1 ? 3 : 2) * (sizeof(Q4Smem<D>) + 1024) <= 233472, "CTAs a SM");
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) {
    kern<<<(unsigned)p.runs, kThreads, smem, s>>>(p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return cuda_status("4-bit decode launch", e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.B * p.Hq));
  // few pairs of many records each: eight groups share them
  const bool wide = p.runs >= 8LL * p.B * p.Hkv;
  cfg.blockDim = dim3(D * (wide ? 8 : 1));
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status("4-bit decode combine launch",
                     wide ? cudaLaunchKernelEx(&cfg, polar_decode_q4_combine_kernel<D, 8, T>, p)
                          : cudaLaunchKernelEx(&cfg, polar_decode_q4_combine_kernel<D, 1, T>, p));
}

bool sizes_ok(int B, int Hq, int Hkv, int d, int max_seq_len) {
  if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return false;
  const int G = Hq / Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8) return false;
  return (d == 64 || d == 128) && max_seq_len >= 1 && max_seq_len <= (1 << 30) &&
         (long long)B * Hq <= INT_MAX / 64;
}

// Runs: what is resident at once (three CTAs a SM, two for fp32), or the
// stages where there are fewer.
int auto_runs(int B, int Hkv, int max_seq_len, int dtype, int sms) {
  const long long stages = ((long long)max_seq_len + kSK - 1) / kSK * B * Hkv;
  const long long slots = (dtype == POLAR_BF16 ? 3LL : 2LL) * sms;
  return (int)std::max(1LL, std::min(slots, stages));
}

size_t records_bytes(int B, int Hq, int Hkv, int d, int runs) {
  return ((size_t)runs + (size_t)B * Hkv) * (Hq / Hkv) * (d + 4) * sizeof(float);
}
size_t scratch_bytes(int B, int Hq, int Hkv, int d, int runs) {
  return records_bytes(B, Hq, Hkv, d, runs) + (size_t)B * Hkv * sizeof(int2);
}

}  // namespace

}  // namespace polar

using namespace polar;

extern "C" {

int polar_attn_decode_paged_q4_num_runs(int B, int Hkv, int max_seq_len, int dtype) {
  if (B < 0 || Hkv < 1 || max_seq_len < 1 || max_seq_len > (1 << 30) ||
      (dtype != POLAR_F32 && dtype != POLAR_BF16))
    return 0;
  int sms = 0;
  if (check_device(&sms) != POLAR_OK) sms = 148;
  return auto_runs(B, Hkv, max_seq_len, dtype, sms);
}

size_t polar_attn_decode_paged_q4_workspace_bytes(int B, int Hq, int Hkv, int max_seq_len, int d,
                                                  int dtype, int num_runs) {
  if (!sizes_ok(B, Hq, Hkv, d, max_seq_len) || num_runs < 0 || num_runs > (1 << 20)) return 0;
  if (dtype != POLAR_F32 && dtype != POLAR_BF16) return 0;
  const int runs =
      num_runs > 0 ? num_runs : polar_attn_decode_paged_q4_num_runs(B, Hkv, max_seq_len, dtype);
  return scratch_bytes(B, Hq, Hkv, d, runs);
}

int polar_attn_decode_paged_q4(const void* q, const void* k_pages, const void* v_pages,
                               const int* block_table, const int* seq_lens, const void* mem,
                               const float* w_count, void* out, float* n_eff, float* conf, int B,
                               int Hq, int Hkv, int d, int page_size, int num_pages, int max_pages,
                               int max_seq_len, int dtype, const polar_consts_t* c, int num_runs,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (B < 0 || Hq < 1 || Hkv < 1 || num_runs < 0 || num_pages < 1 || max_pages < 1 ||
      max_seq_len < 1)
    return POLAR_ERR_INVALID;
  if (dtype != POLAR_F32 && dtype != POLAR_BF16) return POLAR_ERR_UNSUPPORTED;
  if (!sizes_ok(B, Hq, Hkv, d, max_seq_len) || num_runs > (1 << 20)) return POLAR_ERR_UNSUPPORTED;
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
  const int st = check_device(&sms);
  if (st != POLAR_OK) return st;
  const int runs = num_runs > 0 ? num_runs : auto_runs(B, Hkv, max_seq_len, dtype, sms);
  if (!workspace || workspace_bytes < scratch_bytes(B, Hq, Hkv, d, runs))
    return POLAR_ERR_WORKSPACE;
  if (!aligned16(workspace)) return POLAR_ERR_MISALIGNED;
  Q4DecodeParams p{q, mem, w_count, out, n_eff, conf, static_cast<const uint8_t*>(k_pages),
                   static_cast<const uint8_t*>(v_pages), block_table, seq_lens,
                   static_cast<float*>(workspace),
                   reinterpret_cast<int2*>(static_cast<char*>(workspace) +
                                           records_bytes(B, Hq, Hkv, d, runs)),
                   B, Hq, Hkv, max_pages, num_pages, 0, max_seq_len,
                   runs, cc, status_word()};
  while ((1 << p.shift) < page_size) ++p.shift;
  if (!p.status) return cuda_status("cudaGetSymbolAddress", cudaGetLastError());
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == POLAR_BF16)
    return d == 64 ? launch<64, 1, __nv_bfloat16>(p, s) : launch<128, 1, __nv_bfloat16>(p, s);
  return d == 64 ? launch<64, 3, float>(p, s) : launch<128, 3, float>(p, s);
}

}  // extern "C"
