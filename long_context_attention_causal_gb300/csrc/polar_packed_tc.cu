// Causal Polar Attention over packed sequences with grouped heads, bf16, on the
// sm_103a tensor cores.
//
// The mathematics and the pipeline are those of the padded prefill
// (polar_prefill_tc.cu: "ATMA", §2.1 and §2.2, the participation ratio computed
// online with squared correction factors); what differs is the tile: 128 rows
// are 128 / G tokens of the G query heads of one KV head (polar_packed.cuh), so a
// K and V tile read once serves 256 rows of the group, the rows waste less of
// the diagonal (a CTA's rows span 256 / G tokens), and short prompts fill tiles
// with heads.
//
//   * a CTA owns two row tiles of one (sequence, KV head) and streams the keys
//     0 .. its last token through a ring of K and V stages filled by TMA (3-D
//     maps [token, head, channel]; a query box is {64 channels, G heads, 128 / G
//     tokens}, which is the tile's row order);
//   * S_t = Q_t K_j^T into TMEM, softmax by one warpgroup a tile (thread = row =
//     TMEM lane), P (bf16) over S, O_t += P_t V_j with A from TMEM;
//   * the last key tile of a sequence may hold the next sequence's rows: their
//     scores are masked by causality, but 0 * NaN is not 0, so two spare warps
//     zero those rows of V before the product reads them;
//   * a tile whose rows are all tokens of the sequence is stored by TMA, one
//     that the sequence ends in by its valid rows.
//
// Warp roles (384 threads): warps 0-3 softmax of tile 0, 4-7 of tile 1, warp 8
// TMA producer, 9 MMA issuer and TMEM owner, 10-11 zero V rows.  TMEM as in
// polar_prefill_tc.cu.
#include <algorithm>

#include "polar_device.cuh"
#include "polar_internal.h"
#include "polar_packed.cuh"

namespace polar {

namespace {

constexpr int kBM = 128;  // rows per tile
constexpr int kBN = 128;  // keys per tile
constexpr int kNQ = 2;    // row tiles per CTA
constexpr int kNSMax = 4;
constexpr int kThreads = 384;
constexpr int kWarpTMA = 8;
constexpr int kWarpMMA = 9;
constexpr int kWarpZero = 10;  // and 11
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

template <int D>
struct Layout {
  // Ring depths: 2 K + 2 V stages at d = 128, 4 + 4 at d = 64.  Shared memory stays above
  // half of the SM's, so one CTA per SM holds the 512 TMEM columns.
  static constexpr int kNSK = D == 128 ? 2 : 4;
  static constexpr int kNSV = kNSK;
  static constexpr int kTileBytes = kBM * D * 2;  // 128 x D bf16
  static constexpr int kHalfBytes = kBM * 128;    // one 64-column swizzle atom
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + kNQ * kTileBytes;
  static constexpr int kVOff = kKOff + kNSK * kTileBytes;
  static constexpr int kBarOff = kVOff + kNSV * kTileBytes;
  static constexpr int kSmemBytes = kBarOff + 256 + 1024;  // + align slack
  static_assert(kSmemBytes <= 232448, "shared memory");
  static_assert(kSmemBytes > 232448 / 2, "one CTA per SM (512 TMEM columns)");
  static_assert(kNSK == kNSV, "K and V stages are released together");
};

// Barriers as in the padded prefill: step j consumes V_j and K_{j+1}.  v_last and
// v_clean: the landing of the sequence's last V tile where rows of it must be
// zeroed (in place of its kv_full bytes), and that they are.
struct Bars {
  uint64_t q_full;
  uint64_t k0_full, k0_empty;
  uint64_t kv_full[kNSMax], step_done[kNSMax];
  uint64_t s_full[kNQ], p_full[kNQ], o_final[kNQ];
  uint64_t v_last, v_clean;
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  PackedTile tile;
};

struct PackedTcParams {
  const __nv_bfloat16* mem;
  const float* w_count;
  __nv_bfloat16* out;
  float* n_eff;
  float* conf;
  const int* cu;
  int* status;
  int N, B, Hq, Hkv, head_group;
  polar_consts_t c;
};

// The 128 threads of query tile t's softmax warpgroup meet at named barrier
// 1 + t; returns true iff `ok` holds in every one of them.  Every thread of
// the warpgroup reaches it, whatever its own `ok`, so an aborted warp cannot
// leave the others waiting.
__device__ __forceinline__ bool tile_bar_and(int t, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\t"
      "setp.ne.u32 pi, %2, 0;\n\t"
      "bar.red.and.pred po, %1, 128, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(r)
      : "r"(1 + t), "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}

// TMA tile store shared -> global (bulk-group completion); rows past the
// tensor's extent are not written.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* smem_src, int x,
                                             int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(smem_src)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Commit this thread's TMA stores and wait until they have read their
// shared-memory source (the buffer may be released after this returns).
__device__ __forceinline__ void tma_store_commit_wait_read() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// Order this thread's generic-proxy shared-memory writes before later
// async-proxy (TMA) reads of them.
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

template <int D, int G>
__global__ void __launch_bounds__(kThreads, 1)
    polar_packed_tc_kernel(const __grid_constant__ CUtensorMap map_q,
                           const __grid_constant__ CUtensorMap map_k,
                           const __grid_constant__ CUtensorMap map_v,
                           const __grid_constant__ CUtensorMap map_o, const PackedTcParams p) {
  using L = Layout<D>;
  constexpr int NS = L::kNSK;
  constexpr int TT = kBM / G;  // tokens of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBarOff);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 32 * kWarpTMA) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->k0_full, 1);
    mbar_init(&bars->k0_empty, 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&bars->kv_full[s], 1);
      mbar_init(&bars->step_done[s], 1);
    }
    for (int t = 0; t < kNQ; ++t) {
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t], kBM / 32);  // lane 0 of each softmax warp
      mbar_init(&bars->o_final[t], 1);
    }
    mbar_init(&bars->v_last, 1);
    mbar_init(&bars->v_clean, 2);
    mbar_init(&bars->drain, 1);
    bars->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    const PackedTile tile = packed_tile(p.cu, p.B, p.N, p.Hkv, p.head_group, kNQ * TT,
                                        (long long)blockIdx.x, p.status);
    if (lane == 0) bars->tile = tile;
  }
  if (warp == kWarpMMA) tmem_alloc(&bars->tmem_base, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort_flag = &bars->abort_flag;
  const PackedTile tile = bars->tile;
  const int hkv = tile.head;
  // tile t: tokens tok0[t] .. tok0[t] + cnt[t] - 1 of the sequence.  A tile's
  // tokens lie within one key tile (TT divides 128), its last.
  int tok0[kNQ], cnt[kNQ], nkv[kNQ];
  int nkmax = 0;
#pragma unroll
  for (int t = 0; t < kNQ; ++t) {
    tok0[t] = (tile.index * kNQ + t) * TT;
    cnt[t] = hkv < 0 ? 0 : min(max(tile.len - tok0[t], 0), TT);
    nkv[t] = cnt[t] > 0 ? tok0[t] / kBN + 1 : 0;
    nkmax = max(nkmax, nkv[t]);
  }
  // rows of the last V tile that are not the sequence's
  const int keep = tile.len - (nkmax - 1) * kBN;
  const bool dirty = nkmax > 0 && keep < kBN;

  // Registers: the softmax warpgroups take 216 a thread, the other keeps 72
  // (together the 384 x 168 that the block was launched with).
  if (hkv < 0) {
    // more CTAs than tiles: only TMEM to give back
  } else if (warp >= 4 * kNQ) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == kWarpTMA) {
      // ------------------------------------------------------ TMA producer --
      if (lane == 0) {
        tma_prefetch_desc(&map_q);
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
      }
      __syncwarp();
      const int base = tile.start;
      int nact = 0;
      for (int t = 0; t < kNQ; ++t) nact += nkv[t] > 0;
      mbar_arrive_expect_tx_warp(&bars->q_full, nact * L::kTileBytes);
      for (int t = 0; t < kNQ; ++t) {
        if (nkv[t] == 0) continue;
        for (int hh = 0; hh < D / 64; ++hh)
          tma_load_3d_warp(smem + L::kQOff + t * L::kTileBytes + hh * L::kHalfBytes, &map_q,
                           &bars->q_full, 64 * hh, hkv * G, base + tok0[t]);
      }
      mbar_arrive_expect_tx_warp(&bars->k0_full, L::kTileBytes);
      for (int hh = 0; hh < D / 64; ++hh)
        tma_load_3d_warp(smem + L::kKOff + hh * L::kHalfBytes, &map_k, &bars->k0_full, 64 * hh, hkv,
                         base);
      // step j: V_j into V stage j % NS, K_{j+1} into K stage (j + 1) % NS; both
      // were last used by step j - NS (for j = NS - 1 the K stage held K_0)
      int issued = 0;
      bool ok = true;
      for (int j = 0; j < nkmax && ok; ++j) {
        const int s = j % NS, sk = (j + 1) % NS;
        const bool k_next = j + 1 < nkmax;
        if (j == NS - 1) ok = mbar_wait_warp(&bars->k0_empty, 0, abort_flag, p.status);
        if (ok && j >= NS)
          ok = mbar_wait_warp(&bars->step_done[s], (uint32_t)(j / NS - 1) & 1, abort_flag, p.status);
        if (!ok) break;
        const bool own = dirty && !k_next;  // the tile that needs zeroing
        uint64_t* v_bar = own ? &bars->v_last : &bars->kv_full[s];
        if (own) mbar_arrive_expect_tx_warp(&bars->v_last, L::kTileBytes);
        mbar_arrive_expect_tx_warp(&bars->kv_full[s],
                                   ((own ? 0 : 1) + (k_next ? 1 : 0)) * L::kTileBytes);
        for (int hh = 0; hh < D / 64; ++hh)
          tma_load_3d_warp(smem + L::kVOff + s * L::kTileBytes + hh * L::kHalfBytes, &map_v, v_bar,
                           64 * hh, hkv, base + kBN * j);
        if (k_next)
          for (int hh = 0; hh < D / 64; ++hh)
            tma_load_3d_warp(smem + L::kKOff + sk * L::kTileBytes + hh * L::kHalfBytes, &map_k,
                             &bars->kv_full[s], 64 * hh, hkv, base + kBN * (j + 1));
        issued = j + 1;
      }
      if (!ok) {
        // aborted: let the copies already issued land before the CTA exits
        volatile int never = 0;
        const long long lim = kWaitLimitCycles / 4;
        for (int j = issued - 1; j >= 0 && j >= issued - NS; --j)
          mbar_wait(&bars->kv_full[j % NS], (uint32_t)(j / NS) & 1, &never, p.status, lim);
        if (dirty && issued == nkmax) mbar_wait(&bars->v_last, 0, &never, p.status, lim);
        mbar_wait(&bars->k0_full, 0, &never, p.status, lim);
        mbar_wait(&bars->q_full, 0, &never, p.status, lim);
        __syncwarp();
      }
    } else if (warp == kWarpMMA) {
      // ------------------------------------------------------- MMA issuer --
      // The whole warp runs the loop, one elected lane issues (polar_device.cuh).
      constexpr uint32_t kIdescS = idesc_bf16_f32(kBM, kBN, 0, 0);
      constexpr uint32_t kIdescPV = idesc_bf16_f32(kBM, D, 0, 1);
      const uint64_t desc_q = smem_desc_sw128(smem_u32(smem + L::kQOff), 16, 1024);
      const uint64_t desc_k = smem_desc_sw128(smem_u32(smem + L::kKOff), 16, 1024);
      // V: MN-major, LBO = distance between the two 64-column atoms (d = 128)
      const uint64_t desc_v =
          smem_desc_sw128(smem_u32(smem + L::kVOff), D == 128 ? L::kHalfBytes : 0, 1024);
      bool ok = mbar_wait_warp(&bars->q_full, 0, abort_flag, p.status);
      bool any_issued = false;
      auto issue_s = [&](int t, int s) {
        const uint64_t a0 = desc_q + (uint64_t)((t * L::kTileBytes) >> 4);
        const uint64_t b0 = desc_k + (uint64_t)((s * L::kTileBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint64_t off = (uint64_t)((kk >> 2) * (L::kHalfBytes >> 4) + (kk & 3) * 2);
          umma_ss_warp(tmem + 256 * t, a0 + off, b0 + off, kIdescS, kk > 0);
        }
        umma_commit_warp(&bars->s_full[t]);
      };
      auto issue_pv = [&](int t, int s, int j) {
        const uint64_t b0 = desc_v + (uint64_t)((s * L::kTileBytes) >> 4);
        const uint32_t o_tm = tmem + 256 * t + 128, p_tm = tmem + 256 * t;
        umma_ts_warp(o_tm, p_tm, b0, kIdescPV, j > 0 ? 1u : 0u);
#pragma unroll
        for (int kk = 1; kk < kBN / 16; ++kk)
          umma_ts_warp(o_tm, p_tm + kk * 8, b0 + (uint64_t)(kk * (2048 >> 4)), kIdescPV, 1u);
      };
      if (ok) ok = mbar_wait_warp(&bars->k0_full, 0, abort_flag, p.status);
      if (ok) {
        tc_fence_after();
        for (int t = 0; t < kNQ; ++t)
          if (nkv[t] > 0) issue_s(t, 0);
        umma_commit_warp(&bars->k0_empty);
        any_issued = true;
      }
      for (int j = 0; j < nkmax && ok; ++j) {
        const int s = j % NS, jn = j + 1, sn = jn % NS;
        ok = mbar_wait_warp(&bars->kv_full[s], (uint32_t)(j / NS) & 1, abort_flag, p.status);
        if (ok && dirty && jn == nkmax) ok = mbar_wait_warp(&bars->v_clean, 0, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        for (int t = 0; t < kNQ && ok; ++t) {
          if (j >= nkv[t]) continue;
          ok = mbar_wait_warp(&bars->p_full[t], (uint32_t)j & 1, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
          issue_pv(t, s, j);
          if (j == nkv[t] - 1) umma_commit_warp(&bars->o_final[t]);
          if (jn < nkv[t]) issue_s(t, sn);
        }
        if (!ok) break;
        umma_commit_warp(&bars->step_done[s]);
      }
      if (!ok && any_issued) {
        // aborted: wait for the MMAs in flight before TMEM is released
        volatile int never = 0;
        umma_commit_warp(&bars->drain);
        __syncwarp();
        mbar_wait(&bars->drain, 0, &never, p.status, kWaitLimitCycles / 4);
        __syncwarp();
      }
    } else {
      // ---------------------------------------------- rows past the sequence --
      if (dirty) {
        const bool ok = mbar_wait_warp(&bars->v_last, 0, abort_flag, p.status);
        if (ok) {
          uint8_t* v = smem + L::kVOff + ((nkmax - 1) % NS) * L::kTileBytes;
          for (int i = keep * 8 + (warp - kWarpZero) * 32 + lane; i < kBN * 8; i += 64)
#pragma unroll
            for (int hh = 0; hh < D / 64; ++hh)
              *reinterpret_cast<uint4*>(v + hh * L::kHalfBytes + i * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->v_clean);
        }
      }
    }
  } else if ((warp < 4 ? nkv[0] : nkv[1]) > 0) {
    // ------------------------------------------------- softmax + epilogue --
    asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
    const int t = warp >> 2;  // row tile of this warpgroup
    const int tk0 = t ? tok0[1] : tok0[0], tokens = t ? cnt[1] : cnt[0];
    const int steps = t ? nkv[1] : nkv[0];
    const int r = threadIdx.x & 127;
    const int token = tk0 + r / G;  // of the sequence
    const int head = hkv * G + r % G;
    const bool valid = r / G < tokens;
    const size_t at = (size_t)(tile.start + token) * p.Hq + head;  // row of the outputs
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_tm = tmem + lane_base + 256 * t;
    const uint32_t o_tm = s_tm + 128;
    bool ok = mbar_wait_warp(&bars->q_full, 0, abort_flag, p.status);
    // |q|^2 of this row: the swizzle permutes 16-byte chunks inside the row's
    // 128-byte line (chunk c ^ (r & 7) in round c: no bank conflicts)
    float q_sq = 0.f;
    if (ok) {
      for (int hh = 0; hh < D / 64; ++hh) {
        const uint4* line = reinterpret_cast<const uint4*>(smem + L::kQOff + t * L::kTileBytes +
                                                           hh * L::kHalfBytes + r * 128);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 u = line[c ^ (r & 7)];
          const uint32_t w4[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float lo = __uint_as_float(w4[e] << 16);
            const float hi = __uint_as_float(w4[e] & 0xFFFF0000u);
            q_sq = fmaf(lo, lo, q_sq);
            q_sq = fmaf(hi, hi, q_sq);
          }
        }
      }
    }
    const float n = (float)(token + 1);
    const float scale2 = polar_tau(n, p.c.log_t0) * kLog2e * rsqrtf((float)D);  // log2 units
    const int last_col = token - (steps - 1) * kBN;  // last visible key of the last tile
    float m_ref = -INFINITY, l = 0.f, q2 = 0.f;
    for (int j = 0; j < steps && ok; ++j) {
      ok = mbar_wait_warp(&bars->s_full[t], (uint32_t)j & 1, abort_flag, p.status);
      if (!ok) break;
      tc_fence_after();
      uint32_t sv[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(s_tm + 32 * c, sv[c]);
      tmem_ld_wait();
#pragma unroll
      for (int c = 0; c < 4; ++c) reg_fence32(sv[c]);
      if (j == steps - 1) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (32 * c + e > last_col) sv[c][e] = __float_as_uint(-INFINITY);
      }
      // row max: three-input max, two chains
      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          mx0 = fmax3(mx0, __uint_as_float(sv[c][e]), __uint_as_float(sv[c][e + 1]));
          mx1 = fmax3(mx1, __uint_as_float(sv[c][e + 2]), __uint_as_float(sv[c][e + 3]));
        }
      const float mt = fmaxf(mx0, mx1) * scale2;
      // tcgen05.ld/st are warp-collective: the rescale decision is taken per
      // warp; rows that do not need it use a factor of 1
      const bool need = mt > m_ref + kRescaleThreshold;
      if (__any_sync(0xffffffffu, need)) {
        const float alpha = need ? ex2_approx(m_ref - mt) : 1.0f;  // 0 on tile 0
        l *= alpha;
        q2 *= alpha * alpha;  // squared correction factor
        if (j > 0) {
          // S_j was issued after P V of the earlier tiles: they are complete
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tmem_ld32(o_tm + 32 * c, ov);
            tmem_ld_wait();
            reg_fence32(ov);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
            tmem_st32(o_tm + 32 * c, ov);
          }
        }
        if (need) m_ref = mt;
      }
      // P over S in place: keys 2c', 2c'+1 -> TMEM column c' (bf16x2)
      const float2 sc2 = make_float2(scale2, scale2);
      const float2 nm2 = make_float2(-m_ref, -m_ref);
      float2 la = make_float2(0.f, 0.f), lb = la, qa = la, qb = la;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float2 x0 = ffma2(make_float2(__uint_as_float(sv[c][e]),
                                              __uint_as_float(sv[c][e + 1])), sc2, nm2);
          const float2 x1 = ffma2(make_float2(__uint_as_float(sv[c][e + 2]),
                                              __uint_as_float(sv[c][e + 3])), sc2, nm2);
          const float2 p0 = make_float2(ex2_approx(x0.x), ex2_approx(x0.y));
          const float2 p1 = make_float2(ex2_approx(x1.x), ex2_approx(x1.y));
          la = fadd2(la, p0);
          lb = fadd2(lb, p1);
          qa = ffma2(p0, p0, qa);
          qb = ffma2(p1, p1, qb);
          pk[e / 2] = pack_bf16x2(p0.x, p0.y);
          pk[e / 2 + 1] = pack_bf16x2(p1.x, p1.y);
        }
        tmem_st16(s_tm + 16 * c, pk);
      }
      l += (la.x + la.y) + (lb.x + lb.y);
      q2 += (qa.x + qa.y) + (qb.x + qb.y);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->p_full[t]);
    }
    // the row's memory stream, loaded while the last products finish
    uint4 mrow[D / 8];
    {
      const uint4* mp = reinterpret_cast<const uint4*>(p.mem + at * D);
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        mrow[i] = ok && valid ? __ldg(mp + i) : make_uint4(0u, 0u, 0u, 0u);
    }
    if (ok) ok = mbar_wait_warp(&bars->o_final[t], 0, abort_flag, p.status);
    uint8_t* stage = smem + L::kQOff + t * L::kTileBytes;
    if (ok) {
      tc_fence_after();
      float acc_sq = 0.f;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t ov[32];
        tmem_ld32(o_tm + 32 * c, ov);
        tmem_ld_wait();
        reg_fence32(ov);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float a = __uint_as_float(ov[e]);
          acc_sq = fmaf(a, a, acc_sq);
        }
      }
      const RowResult res = polar_finish(m_ref * kLn2, l, q2, acc_sq, q_sq, n, D, p.c);
      const float* wv = p.w_count + (size_t)head * D;
      // The output tile is staged in this tile's Q buffer (its last reader, the
      // final S product, is done) in the map's 128-byte-swizzle layout: 16-byte
      // chunk ch of row r at r * 128 + ((ch ^ (r & 7)) << 4).
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t ov[32];
        tmem_ld32(o_tm + 32 * c, ov);
        tmem_ld_wait();
        reg_fence32(ov);
        const float4* wp = reinterpret_cast<const float4*>(wv + 32 * c);
        uint8_t* line = stage + (c >> 1) * L::kHalfBytes + r * 128;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint4 mu = mrow[4 * c + g];
          const float4 w0 = __ldg(wp + 2 * g), w1 = __ldg(wp + 2 * g + 1);
          const float wf[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
          const uint32_t mw[4] = {mu.x, mu.y, mu.z, mu.w};
          uint32_t o4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float m0 = __uint_as_float(mw[e] << 16);
            const float m1 = __uint_as_float(mw[e] & 0xFFFF0000u);
            const float a0 = __uint_as_float(ov[8 * g + 2 * e]);
            const float a1 = __uint_as_float(ov[8 * g + 2 * e + 1]);
            o4[e] = pack_bf16x2(fmaf(a0, res.scale_u, fmaf(res.count, wf[2 * e], m0)),
                                fmaf(a1, res.scale_u, fmaf(res.count, wf[2 * e + 1], m1)));
          }
          const int ch = (c & 1) * 4 + g;
          *reinterpret_cast<uint4*>(line + ((ch ^ (r & 7)) << 4)) =
              make_uint4(o4[0], o4[1], o4[2], o4[3]);
        }
      }
      fence_proxy_async_smem();
      if (valid) {
        p.n_eff[at] = res.n_eff;
        if (p.conf) p.conf[at] = res.conf;
      }
    }
    // the staged tile is complete once every warp of the group is
    if (tile_bar_and(t, ok)) {
      if (tokens == TT) {
        if (r == 0) {
          for (int hh = 0; hh < D / 64; ++hh)
            tma_store_3d(&map_o, stage + hh * L::kHalfBytes, 64 * hh, hkv * G,
                         tile.start + tk0);
          tma_store_commit_wait_read();
        }
      } else {
        // rows past the sequence are another's: 16 bytes a thread, valid rows
        constexpr int C = D / 8;
        const size_t row0 = (size_t)(tile.start + tk0) * p.Hq + (size_t)hkv * G;
        for (int i = r; i < tokens * G * C; i += 128) {
          const int row = i / C, ch = i % C;
          const uint4 x = *reinterpret_cast<const uint4*>(
              stage + (ch >> 3) * L::kHalfBytes + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
          __nv_bfloat16* dst = p.out + (row0 + (size_t)(row / G) * p.Hq + row % G) * D + 8 * ch;
          *reinterpret_cast<uint4*>(dst) = x;
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMMA) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D, int G>
cudaError_t launch_g(const PackedArgs& a, const CUtensorMap* m, cudaStream_t s) {
  using L = Layout<D>;
  constexpr int kTokens = kNQ * kBM / G;
  PackedTcParams p;
  p.mem = static_cast<const __nv_bfloat16*>(a.mem);
  p.w_count = a.w_count;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.n_eff = a.n_eff;
  p.conf = a.conf;
  p.cu = a.cu;
  p.status = a.status;
  p.N = a.N;
  p.B = a.B;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  // KV heads whose K and V (of all tokens) fit a third of L2
  static_assert(sizeof(Bars) <= 256, "barriers");
  p.head_group = l2_head_group(a.Hkv, 4.0 * (double)a.N * D);
  p.c = a.c;
  auto kern = polar_packed_tc_kernel<D, G>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemBytes);
  if (e != cudaSuccess) return e;
  // as many CTAs as the sequences can have tiles: each ends in at most one
  // partial tile
  const long long tiles = std::min((long long)a.N / kTokens + a.B, (long long)a.N);
  kern<<<(unsigned)(tiles * a.Hkv), kThreads, L::kSmemBytes, s>>>(m[0], m[1], m[2], m[3], p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const PackedArgs& a, const CUtensorMap* m, cudaStream_t s) {
  switch (a.Hq / a.Hkv) {
    case 1: return launch_g<D, 1>(a, m, s);
    case 2: return launch_g<D, 2>(a, m, s);
    case 4: return launch_g<D, 4>(a, m, s);
    default: return launch_g<D, 8>(a, m, s);
  }
}

}  // namespace

cudaError_t launch_packed_tc(const PackedArgs& a, const CUtensorMap* maps, cudaStream_t s) {
  return a.d == 64 ? launch_d<64>(a, maps, s) : launch_d<128>(a, maps, s);
}

}  // namespace polar
