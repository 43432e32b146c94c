// Decayed linear attention on the FP32 pipes: the single-token step, the
// states at the cuts, their scan, and the chunked outputs for fp32 tensors.
//
// Per head, S_t = g S_{t-1} + v_t k_t^T and mem_t = c S_t q_t.  Over a chunk
// of tokens with local index i and the state M before it,
//   mem_i = c [ sum_{j <= i} g^(i-j) (q_i . k_j) v_j + g^(i+1) M q_i ]
//   M'    = g^n M + sum_j g^(n-1-j) v_j k_j^T            (n tokens)
// Every power of g has an exponent >= 0, so nothing overflows for g <= 1.
// The gradients are the same sums: dq is the forward over (dmem, v, k) with
// the state transposed; dk and dv run from the last token over (v, dmem, q)
// and (k, q, dmem).  The kernels therefore take three tensors x, y, z
// (out_t sums (x_t . y_u) z_u) and a direction.  From the end, with M the
// gradient of the state after the chunk,
//   out_i = c sum_{j >= i} g^(j-i) (x_i . y_j) z_j + g^(n-1-i) M x_i
//   M'    = g^n M + c sum_j g^(j+1) z_j y_j^T
//
// fp32 tensors: the tensor cores take 24-bit values only as sums of shorter
// terms, six products for one; chunks of 64 tokens run on packed fp32 fma
// instead.  Bound: those and the shared memory reads that feed them (32 heads
// of 16384 tokens, d = 128: 1.66 ms, 38 TFLOP/s without the masked products,
// half of the FP32 pipes' nominal rate).  Each CTA holds 64 or 32 rows of the
// state: a head then spreads over as many CTAs, whose scores are computed as
// often.
//
// The 128-token tiles of all heads are dealt out to the CTAs in equal runs, so
// that few heads still fill the GPU.  A head that a run boundary cuts needs
// its state there first: one kernel sums each run's own part of the cut head,
// a scan joins the parts, and the output kernel walks all runs in parallel.
#include <type_traits>

#include "polar_device.cuh"
#include "polar_internal.h"
#include "polar_linear.cuh"

namespace polar {

namespace {

constexpr int kC = 64;        // tokens per chunk
constexpr int kZ = 32;        // z columns (rows of the state) per CTA, cut states
constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
}
// Dot products and updates run on pairs of values (fma .f32x2): half the
// instructions of scalar code, which is what bounds these kernels.
__device__ __forceinline__ float2 dot4(float4 a, float4 b, float2 c) {
  return ffma2(make_float2(a.x, a.y), make_float2(b.x, b.y),
               ffma2(make_float2(a.z, a.w), make_float2(b.z, b.w), c));
}
__device__ __forceinline__ float4 axpy4(float w, float4 y, float4 c) {
  const float2 w2 = make_float2(w, w);
  const float2 lo = ffma2(w2, make_float2(y.x, y.y), make_float2(c.x, c.y));
  const float2 hi = ffma2(w2, make_float2(y.z, y.w), make_float2(c.z, c.w));
  return make_float4(lo.x, lo.y, hi.x, hi.y);
}

// The thread's pieces of rows [t0, t0 + kC) x W of a tensor, on their way to
// shared memory: loaded while the chunk before is computed, so that a chunk
// costs one memory latency at most.  Zeros from token `end` on: what lies past
// a sequence may be anything.
template <int W>
struct Pieces {
  static constexpr int kV = W / 4, kN = kC * kV / kThreads;
  float4 v[kN];
  __device__ __forceinline__ void load(const float* src, int ld, int t0, int end) {
#pragma unroll
    for (int u = 0; u < kN; ++u) {
      const int i = threadIdx.x + u * kThreads, r = i / kV, c = (i % kV) * 4;
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (t0 + r < end) v[u] = load4<float>(src + (size_t)(t0 + r) * ld + c);
    }
  }
  template <int S>
  __device__ __forceinline__ void store(float (*dst)[S]) const {
#pragma unroll
    for (int u = 0; u < kN; ++u) {
      const int i = threadIdx.x + u * kThreads, r = i / kV, c = (i % kV) * 4;
      *reinterpret_cast<float4*>(&dst[r][c]) = v[u];
    }
  }
};

// The thread's share of a Z x D state: rows r0 .. r0 + kR - 1, four columns.
template <int D, int Z>
struct StateTile {
  static constexpr int kLanes = D / 4;
  static constexpr int kR = Z * kLanes / kThreads;
  static __device__ __forceinline__ int row0() { return (int)(threadIdx.x / kLanes) * kR; }
  static __device__ __forceinline__ int col0() { return (int)(threadIdx.x % kLanes) * 4; }
};

// acc = sum_j w_j z_j y_j^T over the rows of a chunk (zw holds w_j z_j).  The
// chunk is summed on its own and joined to what came before by the caller: the
// state is rounded once a chunk, not once a token (8192 tokens without decay:
// 1.8e-7 of the state's 2-norm instead of 1.4e-6, for 0 to 2.4 % of the time).
template <int D, int Z>
__device__ __forceinline__ void state_products(float4 (&acc)[StateTile<D, Z>::kR],
                                               const float (*y)[D + 4], const float (*zw)[Z]) {
  using S = StateTile<D, Z>;
  const int r0 = S::row0(), c0 = S::col0();
#pragma unroll
  for (int r = 0; r < S::kR; ++r) acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int j = 0; j < kC; ++j) {
    const float4 yv = *reinterpret_cast<const float4*>(&y[j][c0]);
#pragma unroll
    for (int r = 0; r < S::kR; ++r) acc[r] = axpy4(zw[j][r0 + r], yv, acc[r]);
  }
}

// ------------------------------------------------------ states at cuts --

template <int D>
struct StateSmem {
  float y[kC][D + 4];
  float zw[kC][kZ];
};

// Applications of one launch, by blockIdx.z.
struct StateBatch {
  LinearStateArgs a[2];
};
struct OutBatch {
  LinearArgs a[3];
};

// Grid (parts, D / kZ): the part of the run that reaches its cut.  Weights are
// taken from the cut, so the accumulators never need rescaling.
template <int D>
__global__ void __launch_bounds__(kThreads)
    polar_linear_state_kernel(const StateBatch batch) {
  const LinearStateArgs& a = batch.a[blockIdx.z];
  linear_let_next_start();
  using S = StateTile<D, kZ>;
  __shared__ __align__(16) StateSmem<D> sm;
  const int BH = a.B * a.H, part = blockIdx.x, z0 = blockIdx.y * kZ;
  const int i = a.reverse ? 0 : linear_portions(a.split, BH, part) - 1;
  const LinearPortion po =
      linear_portion(a.split, BH, a.H, a.T, a.lengths, a.status, part, i);
  if (!(a.reverse ? po.cut_left : po.cut_right)) return;
  const int t0 = po.row(po.first), t1 = max(t0, min(po.row(po.last), po.len));
  const float l2 = linear_log2_decay(a.log_decay, po.bh % a.H);
  const float* y = static_cast<const float*>(a.y) + (size_t)po.bh * a.T * D;
  const float* z = static_cast<const float*>(a.z) + (size_t)po.bh * a.T * D;
  float4 sum[S::kR];
#pragma unroll
  for (int r = 0; r < S::kR; ++r) sum[r] = make_float4(0.f, 0.f, 0.f, 0.f);
  Pieces<D> py;
  Pieces<kZ> pz;
  py.load(y, D, t0, t1);
  pz.load(z + z0, D, t0, t1);
  for (int c0 = t0; c0 < t1; c0 += kC) {
    __syncthreads();
    py.store(sm.y);
#pragma unroll
    for (int u = 0; u < Pieces<kZ>::kN; ++u) {
      const int t = c0 + (threadIdx.x + u * kThreads) / Pieces<kZ>::kV;
      const float w =
          t < t1 ? a.scale * linear_power(l2, a.reverse ? t - t0 + 1 : t1 - 1 - t) : 0.f;
      float4& v = pz.v[u];
      v = make_float4(v.x * w, v.y * w, v.z * w, v.w * w);
    }
    pz.store(sm.zw);
    py.load(y, D, c0 + kC, t1);
    pz.load(z + z0, D, c0 + kC, t1);
    __syncthreads();
    float4 acc[S::kR];
    state_products<D, kZ>(acc, sm.y, sm.zw);
#pragma unroll
    for (int r = 0; r < S::kR; ++r) sum[r] = axpy4(1.f, acc[r], sum[r]);
  }
  float* dst = a.cuts + ((size_t)part * D + z0) * D;
#pragma unroll
  for (int r = 0; r < S::kR; ++r)
    *reinterpret_cast<float4*>(dst + (size_t)(S::row0() + r) * D + S::col0()) = sum[r];
}

// Grid (BH, d * d / 512): four state elements a thread through the cuts of
// the head in order; a run's own sum is replaced by the state at its cut.
// Bound: latency (eight cuts' loads are in flight before the first is added;
// 6 us at 32 heads and 152 cuts, d = 128, where the bytes need 3).
constexpr int kScanThreads = 128;
__global__ void __launch_bounds__(kScanThreads) polar_linear_scan_kernel(const StateBatch batch) {
  const LinearStateArgs& a = batch.a[blockIdx.z];
  linear_let_next_start();
  linear_wait_previous();
  const int bh = blockIdx.x, dd = a.d * a.d, per = a.split.per;
  const long long h0 = (long long)bh * a.split.tiles, h1 = h0 + a.split.tiles;
  // boundaries k * per strictly inside the head
  const long long k0 = h0 / per + 1, k1 = (h1 - 1) / per;
  const int cuts = (int)(k1 - k0 + 1);
  const int e = (blockIdx.y * kScanThreads + threadIdx.x) * 4;
  if (a.init_copy)
    *reinterpret_cast<float4*>(a.init_copy + (size_t)bh * dd + e) =
        *reinterpret_cast<const float4*>(a.init + (size_t)bh * dd + e);
  if (cuts < 1) return;
  const int len = linear_length(a.lengths, bh / a.H, a.T, nullptr);
  const float ln = linear_log_decay(a.log_decay, bh % a.H);
  float4 m = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.init) m = *reinterpret_cast<const float4*>(a.init + (size_t)bh * dd + e);
  // forward: boundary k closes run k - 1; reverse: it opens run k
  auto slot = [&](int i) {
    const long long run = a.reverse ? k1 - i : k0 + i - 1;
    return reinterpret_cast<float4*>(a.cuts + (size_t)run * dd + e);
  };
  constexpr int kU = 8;
  for (int i0 = 0; i0 < cuts; i0 += kU) {
    float4 own[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u)
      own[u] = i0 + u < cuts ? __ldcg(slot(i0 + u)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (i0 + u < cuts) {
        const long long k = a.reverse ? k1 - (i0 + u) : k0 + i0 + u;  // the boundary
        const long long lo = a.reverse ? k * per : max(h0, (k - 1) * per);
        const long long hi = a.reverse ? min(h1, (k + 1) * per) : k * per;
        const int ta = (int)(lo - h0) * kLinearTile, tb = (int)(hi - h0) * kLinearTile;
        m = linear_decay(ln, max(min(len, tb) - ta, 0)).join(m, own[u]);
        *slot(i0 + u) = m;
      }
    }
  }
}

__global__ void __launch_bounds__(256) polar_linear_copy_kernel(const float* init, float* dst,
                                                                size_t n) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i < n) dst[i] = init ? init[i] : 0.f;
}

// -------------------------------------------------------------- outputs --

// A thread's dot products take the kE state rows from kE tx on: at tx, tx + 16
// .. they lie in different banks.
template <int Z>
__device__ __forceinline__ int state_slot(int r) {
  constexpr int kE = Z / 16;
  return r / kE + r % kE * 16;
}

template <int D, int Z>
struct OutSmem {
  float x[kC][D + 4];
  float y[kC][D + 4];
  float m[Z][D + 4];  // rows z0 .. of the state, row r at state_slot(r)
  float z[kC][Z];
  float zw[kC][Z];
  float p[kC][kC + 4];  // decayed scores
  float pw[kC + 1];     // powers of g
};

// Grid (parts, D / Z): the CTA walks its run's chunks with its rows of the
// state in shared memory.  Scores, the state's part and the chunk's own part
// of a row stay in one warp, so a chunk has two barriers; scores and products
// that the mask makes zero are not computed.  One CTA a SM: with the 247
// registers that this leaves, the products of a step stay apart (two CTAs,
// spilling: 818 us against 589 at 32 heads of 4096 tokens, d = 128, 32 rows).
template <int D, int Z>
__global__ void __launch_bounds__(kThreads, 1)
    polar_linear_out_kernel(const OutBatch batch) {
  const LinearArgs& a = batch.a[blockIdx.z];
  linear_let_next_start();
  linear_wait_previous();
  constexpr int kE = Z / 16;
  using S = StateTile<D, Z>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  OutSmem<D, Z>& sm = *reinterpret_cast<OutSmem<D, Z>*>(smem_raw);
  const int BH = a.B * a.H, part = blockIdx.x;
  const int z0 = blockIdx.y * Z, tid = threadIdx.x;
  // Rows 8 group .. of a chunk to a warp, which computes scores and products
  // only where they can be non-zero: the warps of one scheduler (w and w + 4)
  // get groups whose shares add up to the same.
  const int warp = tid >> 5, group = warp < 4 ? warp : 11 - warp;
  const int tx = tid & 15, ty = 2 * group + ((tid >> 4) & 1);
  const int n_po = linear_portions(a.split, BH, part);
  for (int ip = 0; ip < n_po; ++ip) {
    const LinearPortion po = linear_portion(a.split, BH, a.H, a.T, a.lengths, a.status, part,
                                            a.reverse ? n_po - 1 - ip : ip);
    const int bh = po.bh, len = po.len;
    const int t0 = po.row(po.first), t1 = min(po.row(po.last), a.T);
    const float ln = linear_log_decay(a.log_decay, bh % a.H);
    const float l2 = linear_log2_decay(a.log_decay, bh % a.H);
    const float* x = static_cast<const float*>(a.x) + (size_t)bh * a.T * D;
    const float* y = static_cast<const float*>(a.y) + (size_t)bh * a.T * D;
    const float* z = static_cast<const float*>(a.z) + (size_t)bh * a.T * D;
    float* out = static_cast<float*>(a.out) + (size_t)bh * a.T * D;
    float* fin = a.final_state && !(a.reverse ? po.cut_left : po.cut_right)
                     ? a.final_state + (size_t)bh * D * D
                     : nullptr;

    const float* st = (a.reverse ? po.cut_right : po.cut_left)
                          ? a.cuts + (size_t)(a.reverse ? part + 1 : part - 1) * D * D
                          : (a.init ? a.init + (size_t)bh * D * D : nullptr);
    __syncthreads();  // the last portion's reads are done
    for (int i = tid; i < Z * D; i += kThreads) {
      const int r = a.state_t ? i % Z : i / D, c = a.state_t ? i / Z : i % D;
      float v = 0.f;
      if (st) v = a.state_t ? st[(size_t)c * D + z0 + r] : st[(size_t)(z0 + r) * D + c];
      sm.m[state_slot<Z>(r)][c] = v;
    }
    for (int i = tid; i <= kC; i += kThreads) sm.pw[i] = linear_power(l2, i);
    // forward: the output scale applies to the state's part too; reverse: the
    // state already carries it
    const float s_in = a.reverse ? 1.f : a.scale, s_z = a.reverse ? a.scale : 1.f;
    const int n_ch = (t1 - t0 + kC - 1) / kC;
    const int end = min(len, t1);
    auto chunk = [&](int ci) { return t0 + (a.reverse ? n_ch - 1 - ci : ci) * kC; };
    Pieces<D> px, py;
    Pieces<Z> pz;
    auto fetch = [&](int c0) {
      px.load(x, D, c0, end);
      py.load(y, D, c0, end);
      pz.load(z + z0, D, c0, end);
    };
    fetch(chunk(0));
    __syncthreads();  // the powers are there
    for (int ci = 0; ci < n_ch; ++ci) {
      const int c0 = chunk(ci);
      const int n = min(max(end - c0, 0), kC);  // tokens of the chunk
      // every read of the last chunk is done: its state's update waited for them
      px.store(sm.x);
      py.store(sm.y);
      pz.store(sm.z);
#pragma unroll
      for (int u = 0; u < Pieces<Z>::kN; ++u) {
        const int r = (tid + u * kThreads) / Pieces<Z>::kV;
        const float w = r < n ? s_z * sm.pw[a.reverse ? r + 1 : n - 1 - r] : 0.f;
        float4& v = pz.v[u];
        v = make_float4(v.x * w, v.y * w, v.z * w, v.w * w);
      }
      pz.store(sm.zw);
      __syncthreads();
      const float2 zero = make_float2(0.f, 0.f);
      float o[4][kE];
#pragma unroll
      for (int ii = 0; ii < 4; ++ii)
#pragma unroll
        for (int e = 0; e < kE; ++e) o[ii][e] = 0.f;
      if (n > 0) {
        // scores: rows 4 ty .., keys tx + 16 jj of the blocks that the
        // warp's rows can see
        auto scores = [&](auto blocks, int jj0) {
          constexpr int kB = decltype(blocks)::value;
          float2 sc[4][kB];
#pragma unroll
          for (int ii = 0; ii < 4; ++ii)
#pragma unroll
            for (int jj = 0; jj < kB; ++jj) sc[ii][jj] = zero;
#pragma unroll 4
          for (int k = 0; k < D; k += 4) {
            float4 xv[4], yv[kB];
#pragma unroll
            for (int ii = 0; ii < 4; ++ii)
              xv[ii] = *reinterpret_cast<const float4*>(&sm.x[4 * ty + ii][k]);
#pragma unroll
            for (int jj = 0; jj < kB; ++jj)
              yv[jj] = *reinterpret_cast<const float4*>(&sm.y[tx + 16 * (jj0 + jj)][k]);
#pragma unroll
            for (int ii = 0; ii < 4; ++ii)
#pragma unroll
              for (int jj = 0; jj < kB; ++jj) sc[ii][jj] = dot4(xv[ii], yv[jj], sc[ii][jj]);
          }
#pragma unroll
          for (int ii = 0; ii < 4; ++ii)
#pragma unroll
            for (int jj = 0; jj < kB; ++jj) {
              const int i = 4 * ty + ii, j = tx + 16 * (jj0 + jj);
              const int dist = a.reverse ? j - i : i - j;
              sm.p[i][j] = dist >= 0 ? (sc[ii][jj].x + sc[ii][jj].y) * sm.pw[dist] : 0.f;
            }
        };
        const int half = group / 2;  // 16 rows
        const int jj0 = a.reverse ? half : 0;
        switch (a.reverse ? 4 - half : half + 1) {
          case 1: scores(std::integral_constant<int, 1>{}, jj0); break;
          case 2: scores(std::integral_constant<int, 2>{}, jj0); break;
          case 3: scores(std::integral_constant<int, 3>{}, jj0); break;
          default: scores(std::integral_constant<int, 4>{}, jj0); break;
        }
        __syncwarp();  // a warp reads its own rows of p only
        // the state's part: rows 4 ty .., state rows kE tx ..
        float2 m[4][kE], q[4][kE];
#pragma unroll
        for (int ii = 0; ii < 4; ++ii)
#pragma unroll
          for (int e = 0; e < kE; ++e) m[ii][e] = q[ii][e] = zero;
#pragma unroll 4
        for (int k = 0; k < D; k += 4) {
          float4 mv[kE];
#pragma unroll
          for (int e = 0; e < kE; ++e) mv[e] = *reinterpret_cast<const float4*>(&sm.m[tx + 16 * e][k]);
#pragma unroll
          for (int ii = 0; ii < 4; ++ii) {
            const float4 xv = *reinterpret_cast<const float4*>(&sm.x[4 * ty + ii][k]);
#pragma unroll
            for (int e = 0; e < kE; ++e) m[ii][e] = dot4(xv, mv[e], m[ii][e]);
          }
        }
        // the chunk's own part, two columns at once: q[e] of columns 2 (e / 2)
        // and the next, odd and even j apart
        const int j_lo = a.reverse ? 8 * group : 0, j_hi = a.reverse ? kC : 8 * group + 8;
#pragma unroll 2
        for (int j = j_lo; j < j_hi; j += 4) {
          float2 zv[4][kE / 2];
#pragma unroll
          for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int c = 0; c < kE / 2; ++c)
              zv[u][c] = *reinterpret_cast<const float2*>(&sm.z[j + u][kE * tx + 2 * c]);
#pragma unroll
          for (int ii = 0; ii < 4; ++ii) {
            const float4 pv = *reinterpret_cast<const float4*>(&sm.p[4 * ty + ii][j]);
#pragma unroll
            for (int c = 0; c < kE / 2; ++c) {
              q[ii][2 * c] = ffma2(make_float2(pv.x, pv.x), zv[0][c], q[ii][2 * c]);
              q[ii][2 * c + 1] = ffma2(make_float2(pv.y, pv.y), zv[1][c], q[ii][2 * c + 1]);
              q[ii][2 * c] = ffma2(make_float2(pv.z, pv.z), zv[2][c], q[ii][2 * c]);
              q[ii][2 * c + 1] = ffma2(make_float2(pv.w, pv.w), zv[3][c], q[ii][2 * c + 1]);
            }
          }
        }
#pragma unroll
        for (int ii = 0; ii < 4; ++ii) {
          const int i = 4 * ty + ii;
          const float w = i < n ? s_in * sm.pw[a.reverse ? n - 1 - i : i + 1] : 0.f;
#pragma unroll
          for (int c = 0; c < kE; c += 2) {
            o[ii][c] = fmaf(a.scale, q[ii][c].x + q[ii][c + 1].x, w * (m[ii][c].x + m[ii][c].y));
            o[ii][c + 1] =
                fmaf(a.scale, q[ii][c].y + q[ii][c + 1].y, w * (m[ii][c + 1].x + m[ii][c + 1].y));
          }
        }
      }
#pragma unroll
      for (int ii = 0; ii < 4; ++ii) {
        const int i = 4 * ty + ii;
        if (c0 + i < t1)
#pragma unroll
          for (int c = 0; c < kE; c += 2)
            *reinterpret_cast<float2*>(out + (size_t)(c0 + i) * D + z0 + kE * tx + c) =
                make_float2(i < n ? o[ii][c] : 0.f, i < n ? o[ii][c + 1] : 0.f);
      }
      // on their way while the state is updated: earlier they would hold
      // registers that the products need
      if (ci + 1 < n_ch) fetch(chunk(ci + 1));
      if (n > 0 && (ci + 1 < n_ch || fin)) {
        const LinearDecay g = linear_decay(ln, n);
        float4 acc[S::kR];
        state_products<D, Z>(acc, sm.y, sm.zw);
#pragma unroll
        for (int r = 0; r < S::kR; ++r)
          acc[r] = g.join(
              *reinterpret_cast<const float4*>(&sm.m[state_slot<Z>(S::row0() + r)][S::col0()]),
              acc[r]);
        __syncthreads();  // every read of the state and the chunk is done
#pragma unroll
        for (int r = 0; r < S::kR; ++r)
          *reinterpret_cast<float4*>(&sm.m[state_slot<Z>(S::row0() + r)][S::col0()]) = acc[r];
      }
    }
    if (fin) {
      __syncthreads();
      for (int i = tid; i < Z * D; i += kThreads)
        fin[(size_t)(z0 + i / D) * D + i % D] = sm.m[state_slot<Z>(i / D)][i % D];
    }
  }
}

// ----------------------------------------------------------------- step --

constexpr int kStepRows = 8;   // state rows per warp
constexpr int kStepWarps = 4;

// One token: the state is read and written once, which is all of the time
// (256 sequences of 16 heads, d = 128: 82 us, 6.6 TB/s, 97 % of the copy
// bandwidth).  Rows are independent, so a head's rows are spread over d / 32
// CTAs: the smallest calls then use several SMs a head (16 heads, d = 64: 3 us).
template <int D, typename T>
__global__ void __launch_bounds__(kStepWarps * 32)
    polar_linear_step_kernel(const LinearStepArgs a) {
  constexpr int kL = D / 4;      // lanes per row
  constexpr int kRW = 32 / kL;   // rows a warp holds at once
  constexpr int kN = kStepRows / kRW;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t bh = blockIdx.x / (D / (kStepRows * kStepWarps));
  const int part = blockIdx.x % (D / (kStepRows * kStepWarps));
  const int row0 = (part * kStepWarps + warp) * kStepRows + lane / kL, c0 = (lane % kL) * 4;
  float* S = a.state + bh * D * D;
  float4 s[kN];
#pragma unroll
  for (int r = 0; r < kN; ++r)
    s[r] = *reinterpret_cast<const float4*>(S + (size_t)(row0 + r * kRW) * D + c0);
  const float4 k = load4<T>(static_cast<const T*>(a.k) + bh * D + c0);
  const float4 q = load4<T>(static_cast<const T*>(a.q) + bh * D + c0);
  const LinearDecay g = linear_decay(linear_log_decay(a.log_decay, (int)(bh % a.H)), 1);
  const T* v = static_cast<const T*>(a.v) + bh * D;
  T* mem = static_cast<T*>(a.mem) + bh * D;
#pragma unroll
  for (int r = 0; r < kN; ++r) {
    const int row = row0 + r * kRW;
    const float vr = linear_load(v + row);
    s[r] = g.join(s[r], make_float4(vr * k.x, vr * k.y, vr * k.z, vr * k.w));
    *reinterpret_cast<float4*>(S + (size_t)row * D + c0) = s[r];
    const float2 o2 = dot4(s[r], q, make_float2(0.f, 0.f));
    float o = o2.x + o2.y;
#pragma unroll
    for (int w = kL / 2; w > 0; w >>= 1) o += __shfl_xor_sync(0xffffffffu, o, w);
    if (lane % kL == 0) linear_store(mem + row, a.scale * o);
  }
}

template <int D, typename T>
cudaError_t step_d(const LinearStepArgs& a, cudaStream_t s) {
  polar_linear_step_kernel<D, T>
      <<<(unsigned)a.B * a.H * (D / (kStepRows * kStepWarps)), kStepWarps * 32, 0, s>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t states_d(const StateBatch& batch, int n, cudaStream_t s) {
  polar_linear_state_kernel<D>
      <<<dim3((unsigned)batch.a[0].split.parts, D / kZ, n), kThreads, 0, s>>>(batch);
  return cudaGetLastError();
}

template <int D, int Z>
cudaError_t out_dz(const OutBatch& batch, int n, cudaStream_t s) {
  const int smem = (int)sizeof(OutSmem<D, Z>);
  cudaError_t e = cudaFuncSetAttribute(polar_linear_out_kernel<D, Z>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return linear_launch(polar_linear_out_kernel<D, Z>,
                       dim3((unsigned)batch.a[0].split.parts, D / Z, n), kThreads, smem, s,
                       batch.a[0].chained, batch);
}

// 64 state rows a CTA, so that fewer CTAs compute the same scores (294 us
// against 392 with 32 at 64 heads of 4096 tokens, d = 64; 445 against 589 at 32
// heads, d = 128), unless 32 rows a CTA find an SM each: a chunk then takes less
// time (2 heads of 100 tokens, d = 64, 16 us against 20; 8 of 300, d = 128, 34
// against 42).
template <int D>
cudaError_t out_d(const OutBatch& batch, int n, cudaStream_t s) {
  const LinearSplit& g = batch.a[0].split;
  return (long long)g.parts * (D / 32) * n <= g.sms ? out_dz<D, 32>(batch, n, s)
                                                    : out_dz<D, 64>(batch, n, s);
}

StateBatch state_batch(const LinearStateArgs* a, int n) {
  StateBatch b;
  for (int i = 0; i < 2; ++i) b.a[i] = a[i < n ? i : 0];
  return b;
}

}  // namespace

cudaError_t launch_linear_states(const LinearStateArgs* a, int n, cudaStream_t s) {
  const StateBatch b = state_batch(a, n);
  return a->d == 64 ? states_d<64>(b, n, s) : states_d<128>(b, n, s);
}

cudaError_t launch_linear_scan(const LinearStateArgs* a, int n, cudaStream_t s) {
  const StateBatch b = state_batch(a, n);
  return linear_launch(polar_linear_scan_kernel,
                       dim3((unsigned)a->B * a->H, a->d * a->d / (4 * kScanThreads), n),
                       kScanThreads, 0, s, true, b);
}

cudaError_t launch_linear_copy_state(const float* init, float* final_state, size_t n,
                                     cudaStream_t s) {
  polar_linear_copy_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(init, final_state, n);
  return cudaGetLastError();
}

cudaError_t launch_linear_out(const LinearArgs* a, int n, cudaStream_t s) {
  OutBatch b;
  for (int i = 0; i < 3; ++i) b.a[i] = a[i < n ? i : 0];
  return a->d == 64 ? out_d<64>(b, n, s) : out_d<128>(b, n, s);
}

cudaError_t launch_linear_step(const LinearStepArgs& a, int dtype, cudaStream_t s) {
  if (dtype == POLAR_BF16)
    return a.d == 64 ? step_d<64, __nv_bfloat16>(a, s) : step_d<128, __nv_bfloat16>(a, s);
  return a.d == 64 ? step_d<64, float>(a, s) : step_d<128, float>(a, s);
}

}  // namespace polar
