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
//   * a CTA takes two row tiles of one (sequence, KV head) at a time (NQ; one where
//     sequences are short: launch_g) and streams the keys 0 .. their last token
//     through a ring of K and V stages filled by TMA (3-D maps [token, head,
//     channel]; a query box is {64 channels, G heads, 128 / G tokens}, which is the
//     tile's row order);
//   * S_t = Q_t K_j^T into TMEM, softmax by one warpgroup a tile (thread = row =
//     TMEM lane), P (bf16) over S, O_t += P_t V_j with A from TMEM;
//   * CTAs stay (one a SM, or two of one tile) and go from pair to pair (next_share),
//     the ring and its barriers with them: with a CTA for each pair about 9 us of
//     launch, search, first loads and last stores stood beside each pair's products
//     (16 x 1024 tokens, d = 64: 15 us a CTA for 4.5 key tiles).  The next pair's
//     first K tile follows the last V tile, its Q comes when the last scores and
//     |q|^2 are there, and its first scores are computed during the epilogue;
//   * the last key tile of a sequence may hold the next sequence's rows: their
//     scores are masked by causality, but 0 * NaN is not 0, so a spare warp
//     zeroes those rows of V before the product reads them;
//   * in the epilogue every warp works alone, and its 32 rows pass through 4 KB of
//     shared memory, so that eight lanes read a part of a row of the memory stream
//     and write one of the output together (warps that met for TMA stores of whole
//     tiles: 11500 clocks a pair from the last product on, of 20800 for two key
//     tiles).
//
// Warp roles (384 threads): warps 0-3 softmax of tile 0, 4-7 of tile 1, warp 8
// TMA producer, 9 MMA issuer and TMEM owner, 10 finds the pairs (polar_packed.cuh),
// 11 zeroes V rows and has the memory stream brought into L2; with one tile, 256
// threads and the last four from warp 4 on.  TMEM as in polar_prefill_tc.cu.
//
// Bound by the chain of a step (scores, softmax, products), 1.4 to 1.54 us for two
// tiles, and by a pair's first and last steps where prompts are short.  Measured:
// two prompts of 16384 tokens, 16 query on 4 KV heads, d = 128, 1400-1510 us
// (1456-1570 TFLOP/s); 24 prompts of 1 to 2900 tokens, 16 on 2 heads, 305-330 us;
// 200 of 1 to 190, 8 heads, d = 64, 69 us.
#include <algorithm>

#include "polar_device.cuh"
#include "polar_internal.h"
#include "polar_packed.cuh"

namespace polar {

namespace {

constexpr int kBM = 128;  // rows per tile
constexpr int kBN = 128;  // keys per tile
constexpr int kNSMax = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

// NQ: row tiles of a CTA.
template <int D, int NQ>
struct Layout {
  static constexpr int kThreads = 128 * (NQ + 1);
  static constexpr uint32_t kTmemCols = 256 * NQ;
  // Ring depths: 2 K + 2 V stages, 4 + 4 where there is room, 1 + 1 where there is
  // none (two CTAs fill each other's waits).  Shared memory allows as many CTAs a SM
  // as share its 512 TMEM columns.
  static constexpr int kNSK = NQ == 2 ? (D == 64 ? 4 : 2) : (D == 64 ? 2 : 1);
  static constexpr int kNSV = kNSK;
  static constexpr int kTileBytes = kBM * D * 2;  // 128 x D bf16
  static constexpr int kHalfBytes = kBM * 128;    // one 64-column swizzle atom
  static constexpr int kQOff = 0;
  static constexpr int kKOff = kQOff + NQ * kTileBytes;
  static constexpr int kVOff = kKOff + kNSK * kTileBytes;
  static constexpr int kStageOff = kVOff + kNSV * kTileBytes;  // 32 columns of the output rows
  static constexpr int kBarOff = kStageOff + NQ * kHalfBytes;
  static constexpr int kSlack = D == 128 && NQ == 1 ? 0 : 1024;  // to align the base
  static constexpr int kSmemBytes = kBarOff + 512 + kSlack;
  static constexpr int kCtas = 2 / NQ;  // a SM
  static_assert(kCtas * (kSmemBytes + 1024) <= 233472, "shared memory");
  static_assert((kCtas + 1) * (kSmemBytes + 1024) > 233472, "TMEM columns");
  static_assert(kNSK == kNSV, "K and V stages are released together");
};

// Steps (key tiles) are counted through all pairs of the CTA: step g consumes V_g
// and K_{g+1}, which may be the next pair's first.  kv_full: those two landed;
// step_done: step g's products are done; k0_*: K_0, before the first step.
// v_raw, v_clean: the landing of a V tile of which rows must be zeroed (in place of
// its kv_full bytes), and that they are, per V stage.  tile_*: a pair is written
// down, read by all warps, the next one is wanted.  share_full: an answer to
// next_share.
struct Bars {
  uint64_t q_full[2], q_empty[2];  // a row tile each
  uint64_t k0_full, k0_empty;
  uint64_t kv_full[kNSMax], step_done[kNSMax];
  uint64_t s_full[2], p_full[2], o_final[2];
  uint64_t v_raw[kNSMax], v_clean[kNSMax];
  uint64_t tile_full[2], tile_empty[2], tile_wanted;
  uint64_t share_full;
  uint64_t drain;
  PackedTile tile[2];
  uint4 share;  // 16-byte aligned: the answer to a request for another CTA's share
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Bars) <= 512, "barriers");

// A pair of row tiles: tokens tok0[t] .. tok0[t] + cnt[t] - 1 of the sequence are
// tile t's.  They lie within one key tile, the tile's last (TT divides 128).
template <int TT, int NQ>
struct Pair {
  int head, start;
  int tok0[NQ], cnt[NQ], nkv[NQ], steps;
  int keep;    // rows of the last V tile that are the sequence's
  bool dirty;  // not all of them
  __device__ __forceinline__ explicit Pair(const PackedTile& t) : head(t.head), start(t.start) {
    steps = 0;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      tok0[i] = (t.index * NQ + i) * TT;
      cnt[i] = head < 0 ? 0 : min(max(t.len - tok0[i], 0), TT);
      nkv[i] = cnt[i] > 0 ? tok0[i] / kBN + 1 : 0;
      steps = max(steps, nkv[i]);
    }
    keep = t.len - (steps - 1) * kBN;
    dirty = steps > 0 && keep < kBN;
  }
};

// The n-th pair of the CTA, by a converged warp; head -1 behind the last one, and
// where a wait ran out (*ok false then).
template <int TT, int NQ>
__device__ __forceinline__ Pair<TT, NQ> read_pair(Bars* bars, int n, int* status, bool* ok) {
  volatile int* abort_flag = &bars->abort_flag;
  PackedTile t{-1, 0, 0, 0};
  *ok = *ok && mbar_wait_warp(&bars->tile_full[n & 1], (uint32_t)(n >> 1) & 1, abort_flag, status);
  if (*ok) {
    t = bars->tile[n & 1];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&bars->tile_empty[n & 1]);
  }
  return Pair<TT, NQ>(t);
}

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

// Order this thread's generic-proxy shared-memory writes before later
// async-proxy (TMA) reads of them.
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Takes over the share of a CTA of this grid that has not started (cluster launch
// control): its blockIdx.x, or -1 if all have.  By a converged warp; a request
// after one that failed is not allowed.
__device__ __forceinline__ int next_share(Bars* bars, int n, int* status, bool* ok) {
  if ((threadIdx.x & 31) == 0) {
    mbar_arrive_expect_tx(&bars->share_full, 16);
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
        "[%0], [%1];" ::"r"(smem_u32(&bars->share)),
        "r"(smem_u32(&bars->share_full))
        : "memory");
  }
  __syncwarp();
  // (not given up on an abort: the answer is on its way into this CTA's memory)
  volatile int never = 0;
  if (!__all_sync(0xffffffffu,
                  mbar_wait(&bars->share_full, (uint32_t)n & 1, &never, status))) {
    bars->abort_flag = 1;
    *ok = false;
    return -1;
  }
  uint32_t got, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(smem_u32(&bars->share))
      : "memory");
  fence_proxy_async_smem();  // read before the next answer is written over it
  __syncwarp();
  return got ? (int)x : -1;
}

// A lane's pieces of its warp's rows of the memory stream: 16 bytes of each 64
// columns, or 8 of each 32.
template <int D, bool kByRow>
struct MemRows;
template <int D>
struct MemRows<D, true> {
  static constexpr int kParts = D / 64, kCols = 8;
  uint4 v[kParts][8];
  __device__ __forceinline__ void load(int c, int i, const __nv_bfloat16* src, bool there) {
    v[c][i] = there ? __ldg(reinterpret_cast<const uint4*>(src + 64 * c)) : make_uint4(0, 0, 0, 0);
  }
};
template <int D>
struct MemRows<D, false> {
  static constexpr int kParts = D / 32, kCols = 4;
  uint2 v[kParts][8];
  __device__ __forceinline__ void load(int c, int i, const __nv_bfloat16* src, bool there) {
    v[c][i] = there ? __ldg(reinterpret_cast<const uint2*>(src + 32 * c)) : make_uint2(0, 0);
  }
};

template <int D, int G, int NQ>
__global__ void __launch_bounds__(Layout<D, NQ>::kThreads, Layout<D, NQ>::kCtas)
    polar_packed_tc_kernel(const __grid_constant__ CUtensorMap map_q,
                           const __grid_constant__ CUtensorMap map_k,
                           const __grid_constant__ CUtensorMap map_v, const PackedTcParams p) {
  using L = Layout<D, NQ>;
  constexpr int NS = L::kNSK;
  constexpr int kWarpTMA = 4 * NQ, kWarpMMA = kWarpTMA + 1, kWarpNext = kWarpTMA + 2;
  constexpr int kReaders = 4 * NQ + 3;  // warps that read a pair: all but kWarpNext
  constexpr int TT = kBM / G;  // tokens of a tile
  // The epilogue: by rows, whose threads read their head's count direction (a line
  // an instruction for each head of the warp), or by pieces of rows, whose lanes
  // know one head or two but whose directions pass through shared memory in fp32.
  // Measured, rows / pieces: G = 8, 24 prompts up to 2900 tokens, 360 / 320 us; G =
  // 4, 64 up to 500, 90 / 86; G = 1, 200 up to 190, d = 64, 84 / 91.
  constexpr bool kByRow = G <= 2;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + (L::kSlack ? 1023 : 0)) & ~uintptr_t(1023));
  if (L::kSlack == 0 && smem != smem_raw) {  // not so: recorded, as a wait that ran out is
    if (threadIdx.x == 0) atomicExch(p.status, kStatusWaitTimeout);
    return;
  }
  Bars* bars = reinterpret_cast<Bars*>(smem + L::kBarOff);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 32 * kWarpTMA) {
    mbar_init(&bars->k0_full, 1);
    mbar_init(&bars->k0_empty, 1);
    for (int s = 0; s < NS; ++s) {
      mbar_init(&bars->kv_full[s], 1);
      mbar_init(&bars->step_done[s], 1);
      mbar_init(&bars->v_raw[s], 1);
      mbar_init(&bars->v_clean[s], 1);
    }
    for (int t = 0; t < NQ; ++t) {
      mbar_init(&bars->q_full[t], 1);
      mbar_init(&bars->q_empty[t], kBM / 32);  // lane 0 of each softmax warp
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t], kBM / 32);
      mbar_init(&bars->o_final[t], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->tile_full[i], 1);
      mbar_init(&bars->tile_empty[i], kReaders);
    }
    mbar_init(&bars->tile_wanted, 1);
    mbar_init(&bars->share_full, 1);
    mbar_init(&bars->drain, 1);
    bars->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kWarpMMA) tmem_alloc(&bars->tmem_base, L::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  volatile int* abort_flag = &bars->abort_flag;

  // Registers: the softmax warpgroups take 200 a thread, the other keeps 104 (together
  // the 384 x 168 that the block was launched with); with one tile 176 and 80 (256 x
  // 128).
  if (warp >= 4 * NQ) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(NQ == 2 ? 104 : 80));
    bool ok = true;
    if (warp == kWarpNext) {
      // ------------------------------------------------------- the pairs --
      // CTA i's share: the ranks i, then back and forth over the grid's CTAs.  A
      // CTA that is through takes the next share that no CTA has started on, so
      // shares go out in order, longest first, to whoever is free.
      int n = 0, asked = 0, share = (int)blockIdx.x;
      PackedTiles tiles(p.cu, p.B, p.N, p.Hkv, p.head_group, NQ * TT, p.status);
      while (ok && share >= 0) {
        for (long long k = 0; ok; ++k) {
          const long long rank =
              k * gridDim.x + ((k & 1) ? (int)gridDim.x - 1 - share : share);
          if (n >= 1)  // not earlier: the next share goes to who is nearly through
            ok = mbar_wait_warp(&bars->tile_wanted, (uint32_t)(n - 1) & 1, abort_flag, p.status);
          if (ok && n >= 2)
            ok = mbar_wait_warp(&bars->tile_empty[n & 1], (uint32_t)((n >> 1) - 1) & 1, abort_flag,
                                p.status);
          if (!ok) break;
          const PackedTile tile = tiles.find(rank);
          if (tile.head < 0) break;
          if (lane == 0) {
            bars->tile[n & 1] = tile;
            mbar_arrive(&bars->tile_full[n & 1]);
          }
          __syncwarp();
          ++n;
        }
        if (ok) share = next_share(bars, asked++, p.status, &ok);
      }
      if (ok && lane == 0) {
        // behind the last (the waits above have passed for this n)
        bars->tile[n & 1] = PackedTile{-1, 0, 0, 0};
        mbar_arrive(&bars->tile_full[n & 1]);
      }
      __syncwarp();
    } else if (warp == kWarpTMA) {
      // ---------------------------------------------------- TMA producer --
      if (lane == 0) {
        tma_prefetch_desc(&map_q);
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
      }
      __syncwarp();
      auto load_kv = [&](const CUtensorMap* map, int off, int stage, uint64_t* bar,
                         const Pair<TT, NQ>& a, int j) {
        for (int hh = 0; hh < D / 64; ++hh)
          tma_load_3d_warp(smem + off + stage * L::kTileBytes + hh * L::kHalfBytes, map, bar,
                           64 * hh, a.head, a.start + kBN * j);
      };
      int g = 0, nq[NQ] = {};
      uint32_t raw = 0;  // V stages with a zeroing load in flight or behind
      Pair<TT, NQ> cur = read_pair<TT, NQ>(bars, 0, p.status, &ok);
      for (int n = 0; ok && cur.head >= 0; ++n) {
        // the next pair is asked for when four steps, which take longer than the
        // answer does, are left to load; at once in a shorter pair, whose Q waits
        // for the last one's scores below
        if (cur.steps <= 4 && lane == 0) mbar_arrive(&bars->tile_wanted);
#pragma unroll
        for (int t = 0; t < NQ; ++t) {
          if (cur.nkv[t] == 0 || !ok) continue;
          if (nq[t] > 0)
            ok = mbar_wait_warp(&bars->q_empty[t], (uint32_t)(nq[t] - 1) & 1, abort_flag, p.status);
          if (!ok) continue;
          mbar_arrive_expect_tx_warp(&bars->q_full[t], L::kTileBytes);
          for (int hh = 0; hh < D / 64; ++hh)
            tma_load_3d_warp(smem + L::kQOff + t * L::kTileBytes + hh * L::kHalfBytes, &map_q,
                             &bars->q_full[t], 64 * hh, cur.head * G, cur.start + cur.tok0[t]);
          ++nq[t];
        }
        if (!ok) break;
        if (n == 0) {
          mbar_arrive_expect_tx_warp(&bars->k0_full, L::kTileBytes);
          load_kv(&map_k, L::kKOff, 0, &bars->k0_full, cur, 0);
        }
        Pair<TT, NQ> next(PackedTile{-1, 0, 0, 0});
        for (int j = 0; j < cur.steps; ++j) {
          const int s = g % NS;
          // V stage s and K stage (g + 1) % NS were last used by step g - NS (for g =
          // NS - 1 the K stage held K_0)
          if (g == NS - 1) ok = mbar_wait_warp(&bars->k0_empty, 0, abort_flag, p.status);
          if (ok && g >= NS)
            ok = mbar_wait_warp(&bars->step_done[s], (uint32_t)(g / NS - 1) & 1, abort_flag,
                                p.status);
          const bool last = j + 1 == cur.steps;
          if (j > 0 && j == cur.steps - 4 && lane == 0) mbar_arrive(&bars->tile_wanted);
          if (last) next = read_pair<TT, NQ>(bars, n + 1, p.status, &ok);
          if (!ok) break;
          const bool own = cur.dirty && last;  // the tile that needs zeroing
          const bool k_next = !last || next.head >= 0;
          if (own) mbar_arrive_expect_tx_warp(&bars->v_raw[s], L::kTileBytes);
          mbar_arrive_expect_tx_warp(&bars->kv_full[s],
                                     ((own ? 0 : 1) + (k_next ? 1 : 0)) * L::kTileBytes);
          load_kv(&map_v, L::kVOff, s, own ? &bars->v_raw[s] : &bars->kv_full[s], cur, j);
          if (k_next)
            load_kv(&map_k, L::kKOff, (g + 1) % NS, &bars->kv_full[s], last ? next : cur,
                    last ? 0 : j + 1);
          if (own) raw ^= 1u << s;
          ++g;
        }
        if (!ok) break;
        cur = next;
      }
      if (!ok) {
        // aborted: let the copies already issued land before the CTA exits
        volatile int never = 0;
        const long long lim = kWaitLimitCycles / 4;
        for (int i = g - 1; i >= 0 && i >= g - NS; --i)
          mbar_wait(&bars->kv_full[i % NS], (uint32_t)(i / NS) & 1, &never, p.status, lim);
        for (int s = 0; s < NS; ++s)
          if (raw >> s & 1) mbar_wait(&bars->v_raw[s], 0, &never, p.status, lim);
          else mbar_wait(&bars->v_raw[s], 1, &never, p.status, lim);
        if (nq[0] + nq[NQ - 1] > 0 && g >= 0) mbar_wait(&bars->k0_full, 0, &never, p.status, lim);
        for (int t = 0; t < NQ; ++t)
          if (nq[t] > 0)
            mbar_wait(&bars->q_full[t], (uint32_t)(nq[t] - 1) & 1, &never, p.status, lim);
        __syncwarp();
      }
    } else if (warp == kWarpMMA) {
      // ----------------------------------------------------- MMA issuer --
      // The whole warp runs the loop, one elected lane issues (polar_device.cuh).
      constexpr uint32_t kIdescS = idesc_bf16_f32(kBM, kBN, 0, 0);
      constexpr uint32_t kIdescPV = idesc_bf16_f32(kBM, D, 0, 1);
      const uint64_t desc_q = smem_desc_sw128(smem_u32(smem + L::kQOff), 16, 1024);
      const uint64_t desc_k = smem_desc_sw128(smem_u32(smem + L::kKOff), 16, 1024);
      // V: MN-major, LBO = distance between the two 64-column atoms (d = 128)
      const uint64_t desc_v =
          smem_desc_sw128(smem_u32(smem + L::kVOff), D == 128 ? L::kHalfBytes : 0, 1024);
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
      int g = 0, nq[NQ] = {}, np[NQ] = {};
      uint32_t clean = 0;  // phase of each stage's v_clean
      bool any_issued = false;
      // the first scores of a pair: its Q has landed, K stage s holds its first keys
      auto first_scores = [&](const Pair<TT, NQ>& a, int s) {
#pragma unroll
        for (int t = 0; t < NQ; ++t) {
          if (a.nkv[t] == 0 || !ok) continue;
          ok = mbar_wait_warp(&bars->q_full[t], (uint32_t)nq[t] & 1, abort_flag, p.status);
          if (!ok) continue;
          ++nq[t];
          tc_fence_after();
          issue_s(t, s);
          any_issued = true;
        }
      };
      Pair<TT, NQ> cur = read_pair<TT, NQ>(bars, 0, p.status, &ok);
      if (ok && cur.head >= 0) {
        ok = mbar_wait_warp(&bars->k0_full, 0, abort_flag, p.status);
        if (ok) first_scores(cur, 0);
        if (ok) umma_commit_warp(&bars->k0_empty);
      }
      for (int n = 0; ok && cur.head >= 0; ++n) {
        Pair<TT, NQ> next(PackedTile{-1, 0, 0, 0});
        for (int j = 0; j < cur.steps; ++j, ++g) {
          const int s = g % NS, sn = (g + 1) % NS;
          const bool last = j + 1 == cur.steps;
          ok = mbar_wait_warp(&bars->kv_full[s], (uint32_t)(g / NS) & 1, abort_flag, p.status);
          if (ok && last && cur.dirty) {
            ok = mbar_wait_warp(&bars->v_clean[s], clean >> s & 1, abort_flag, p.status);
            clean ^= 1u << s;
          }
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int t = 0; t < NQ; ++t) {
            if (j >= cur.nkv[t] || !ok) continue;
            ok = mbar_wait_warp(&bars->p_full[t], (uint32_t)np[t] & 1, abort_flag, p.status);
            if (!ok) continue;
            ++np[t];
            tc_fence_after();
            issue_pv(t, s, j);
            if (j == cur.nkv[t] - 1) umma_commit_warp(&bars->o_final[t]);
            if (j + 1 < cur.nkv[t]) issue_s(t, sn);
          }
          if (!ok) break;
          if (last) {
            next = read_pair<TT, NQ>(bars, n + 1, p.status, &ok);
            if (ok && next.head >= 0) first_scores(next, sn);
            if (!ok) break;
          }
          umma_commit_warp(&bars->step_done[s]);
        }
        if (!ok) break;
        cur = next;
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
      // ------------------------- rows past the sequence, and the memory stream --
      int g = 0;
      uint32_t raw = 0;  // phase of each stage's v_raw
      for (int n = 0; ok; ++n) {
        const Pair<TT, NQ> cur = read_pair<TT, NQ>(bars, n, p.status, &ok);
        if (!ok || cur.head < 0) break;
        // the pair's memory stream into L2: a token's heads are one piece
        const int tokens = cur.cnt[0] + (NQ == 2 ? cur.cnt[NQ - 1] : 0);
        const __nv_bfloat16* mem =
            p.mem + ((size_t)(cur.start + cur.tok0[0]) * p.Hq + (size_t)cur.head * G) * D;
        for (int i = lane; i < tokens; i += 32)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(mem +
                                                                          (size_t)i * p.Hq * D),
                       "n"(G * D * 2)
                       : "memory");
        g += cur.steps;
        if (!cur.dirty) continue;
        const int s = (g - 1) % NS;
        ok = mbar_wait_warp(&bars->v_raw[s], raw >> s & 1, abort_flag, p.status);
        if (!ok) break;
        raw ^= 1u << s;
        uint8_t* v = smem + L::kVOff + s * L::kTileBytes;
        for (int i = cur.keep * 8 + lane; i < kBN * 8; i += 32)
#pragma unroll
          for (int hh = 0; hh < D / 64; ++hh)
            *reinterpret_cast<uint4*>(v + hh * L::kHalfBytes + i * 16) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->v_clean[s]);
      }
    }
  } else {
    // ------------------------------------------------- softmax + epilogue --
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(NQ == 2 ? 200 : 176));
    const int t = warp >> 2;  // row tile of this warpgroup
    const int r = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_tm = tmem + lane_base + 256 * t;
    const uint32_t o_tm = s_tm + 128;
    uint8_t* stage = smem + L::kStageOff + t * L::kHalfBytes;  // 32 columns of the rows
    int ns = 0, no = 0;  // scores, outputs of this tile so far
    bool ok = true;
    for (int n = 0;; ++n) {
      const Pair<TT, NQ> cur = read_pair<TT, NQ>(bars, n, p.status, &ok);
      if (!ok || cur.head < 0) break;
      const int tk0 = t ? cur.tok0[NQ - 1] : cur.tok0[0];
      const int tokens = t ? cur.cnt[NQ - 1] : cur.cnt[0];
      const int steps = t ? cur.nkv[NQ - 1] : cur.nkv[0];
      if (steps == 0) continue;
      const int token = tk0 + r / G;  // of the sequence
      const int head = cur.head * G + r % G;
      const bool valid = r / G < tokens;
      const size_t at = (size_t)(cur.start + token) * p.Hq + head;  // row of the outputs
      const float nk = (float)(token + 1);
      const float scale2 = polar_tau(nk, p.c.log_t0) * kLog2e * rsqrtf((float)D);  // log2 units
      const int last_col = token - (steps - 1) * kBN;  // last visible key of the last tile
      float m_ref = -INFINITY, l = 0.f, q2 = 0.f;
      for (int j = 0; j < steps && ok; ++j) {
        ok = mbar_wait_warp(&bars->s_full[t], (uint32_t)ns & 1, abort_flag, p.status);
        if (!ok) break;
        ++ns;
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
      // The memory stream of the warp's 32 rows, while the last products finish (loads
      // between the stores below waited for those: 13000 clocks a pair at d = 128).
      // Eight lanes read, and below write, a part of a row together: row 4 i + lane /
      // 8 of the warp (a row a thread took 32 lines an instruction).
      const size_t tile_at = ((size_t)(cur.start + tk0) * p.Hq + (size_t)cur.head * G) * D;
      const int row0 = (r & 96) + (lane >> 3);
      auto row_at = [&](int i) {  // elements from the tile's first
        const uint32_t row = (uint32_t)(row0 + 4 * i);  // (128 tokens of all heads pass 2^31)
        return tile_at + ((size_t)(row / G) * (uint32_t)p.Hq + row % G) * D;
      };
      MemRows<D, kByRow> mem;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool there = ok && (row0 + 4 * i) / G < tokens;
        const __nv_bfloat16* src = p.mem + (there ? row_at(i) : 0) + mem.kCols * (lane & 7);
#pragma unroll
        for (int c = 0; c < mem.kParts; ++c) mem.load(c, i, src, there);
      }
      if (ok) ok = mbar_wait_warp(&bars->q_full[t], (uint32_t)no & 1, abort_flag, p.status);
      // |q|^2 of this row, likewise: the swizzle permutes 16-byte chunks inside the row's
      // 128-byte line (chunk c ^ (r & 7) in round c: no bank conflicts)
      float2 qa = make_float2(0.f, 0.f), qb = qa;
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
              const float2 x = make_float2(__uint_as_float(w4[e] << 16),
                                           __uint_as_float(w4[e] & 0xFFFF0000u));
              if (e & 1) qb = ffma2(x, x, qb);
              else qa = ffma2(x, x, qa);
            }
          }
        }
      }
      const float q_sq = (qa.x + qa.y) + (qb.x + qb.y);
      // Q is read, by the last scores' product too: the next pair's may come
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&bars->q_empty[t]);
      if (ok) ok = mbar_wait_warp(&bars->o_final[t], (uint32_t)no & 1, abort_flag, p.status);
      if (!ok) break;
      ++no;
      tc_fence_after();
      float acc_sq = 0.f;
#pragma unroll
      for (int c = 0; c < D / 32; c += 2) {
        uint32_t ov[2][32];
        tmem_ld32(o_tm + 32 * c, ov[0]);
        tmem_ld32(o_tm + 32 * c + 32, ov[1]);
        tmem_ld_wait();
        reg_fence32(ov[0]);
        reg_fence32(ov[1]);
        float2 sa = make_float2(0.f, 0.f), sb = sa;
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 x0 = make_float2(__uint_as_float(ov[0][e]), __uint_as_float(ov[0][e + 1]));
          const float2 x1 = make_float2(__uint_as_float(ov[1][e]), __uint_as_float(ov[1][e + 1]));
          sa = ffma2(x0, x0, sa);
          sb = ffma2(x1, x1, sb);
        }
        acc_sq += (sa.x + sa.y) + (sb.x + sb.y);
      }
      const RowResult res = polar_finish(m_ref * kLn2, l, q2, acc_sq, q_sq, nk, D, p.c);
      // Through the warp's 4 KB: 16-byte chunk ch of row r at r * 128 + ((ch ^ (r & 7))
      // << 4), no bank conflicts by rows, nor by eighths of a row.
      if constexpr (kByRow) {
        // 64 columns at a time: the memory stream to the rows' threads, outputs back
        const float* wv = p.w_count + (size_t)head * D;
#pragma unroll
        for (int hh = 0; hh < D / 64; ++hh) {
          __syncwarp();  // the last outputs are read
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = row0 + 4 * i;
            *reinterpret_cast<uint4*>(stage + row * 128 + (((lane & 7) ^ (row & 7)) << 4)) =
                mem.v[hh][i];
          }
          __syncwarp();
#pragma unroll
          for (int c = 2 * hh; c < 2 * hh + 2; ++c) {
            uint32_t ov[32];
            tmem_ld32(o_tm + 32 * c, ov);
            // (what else a chunk needs is on its way before the wait)
            const float4* wp = reinterpret_cast<const float4*>(wv + 32 * c);
            float4 w[8];
#pragma unroll
            for (int g = 0; g < 8; ++g) w[g] = __ldg(wp + g);
            tmem_ld_wait();
            reg_fence32(ov);
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              uint4* cell = reinterpret_cast<uint4*>(stage + r * 128 +
                                                     ((((c & 1) * 4 + g) ^ (r & 7)) << 4));
              const uint4 mu = *cell;
              const float wf[8] = {w[2 * g].x,     w[2 * g].y,     w[2 * g].z,     w[2 * g].w,
                                   w[2 * g + 1].x, w[2 * g + 1].y, w[2 * g + 1].z, w[2 * g + 1].w};
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
              *cell = make_uint4(o4[0], o4[1], o4[2], o4[3]);
            }
          }
          __syncwarp();
          // rows past the sequence are another's, or no one's
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = row0 + 4 * i;
            const uint4 y = *reinterpret_cast<const uint4*>(stage + row * 128 +
                                                            (((lane & 7) ^ (row & 7)) << 4));
            if (row / G < tokens)
              *reinterpret_cast<uint4*>(p.out + row_at(i) + 64 * hh + 8 * (lane & 7)) = y;
          }
        }
      } else {
        // 32 columns at a time: directions to the lanes that hold the memory stream.
        // A lane's rows belong to one head, or two where G = 8.
        constexpr int kHeads = G == 8 ? 2 : 1;
        const float* wv = p.w_count + ((size_t)cur.head * G + (lane >> 3)) * D + 4 * (lane & 7);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          tmem_ld32(o_tm + 32 * c, ov);
          float4 w[kHeads];
#pragma unroll
          for (int i = 0; i < kHeads; ++i)
            w[i] = __ldg(reinterpret_cast<const float4*>(wv + (size_t)(4 * i) * D + 32 * c));
          tmem_ld_wait();
          reg_fence32(ov);
          __syncwarp();  // the last columns are read
#pragma unroll
          for (int g = 0; g < 8; ++g)
            *reinterpret_cast<float4*>(stage + r * 128 + ((g ^ (r & 7)) << 4)) =
                make_float4(__uint_as_float(ov[4 * g]) * res.scale_u,
                            __uint_as_float(ov[4 * g + 1]) * res.scale_u,
                            __uint_as_float(ov[4 * g + 2]) * res.scale_u,
                            __uint_as_float(ov[4 * g + 3]) * res.scale_u);
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = row0 + 4 * i;
            const float count = __shfl_sync(0xffffffffu, res.count, 4 * i + (lane >> 3));
            const float4 u = *reinterpret_cast<const float4*>(stage + row * 128 +
                                                              (((lane & 7) ^ (row & 7)) << 4));
            const float4 wf = w[i % kHeads];
            const uint2 m = mem.v[c][i];
            const uint2 y = make_uint2(
                pack_bf16x2(u.x + fmaf(count, wf.x, __uint_as_float(m.x << 16)),
                            u.y + fmaf(count, wf.y, __uint_as_float(m.x & 0xFFFF0000u))),
                pack_bf16x2(u.z + fmaf(count, wf.z, __uint_as_float(m.y << 16)),
                            u.w + fmaf(count, wf.w, __uint_as_float(m.y & 0xFFFF0000u))));
            // rows past the sequence are another's, or no one's
            if (row / G < tokens)
              *reinterpret_cast<uint2*>(p.out + row_at(i) + 32 * c + 4 * (lane & 7)) = y;
          }
        }
      }
      if (valid) {
        p.n_eff[at] = res.n_eff;
        if (p.conf) p.conf[at] = res.conf;
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMMA) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

template <int D, int G, int NQ>
cudaError_t launch_n(const PackedArgs& a, const CUtensorMap* m, cudaStream_t s) {
  using L = Layout<D, NQ>;
  constexpr int kTokens = NQ * kBM / G;
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
  p.head_group = l2_head_group(a.Hkv, 4.0 * (double)a.N * D);
  p.c = a.c;
  auto kern = polar_packed_tc_kernel<D, G, NQ>;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmemBytes);
  if (e != cudaSuccess) return e;
  // Shares: as many as the sequences can have pairs of tiles (each ends in at most
  // one partial pair), but where short sequences make that a loose bound, eight a
  // SM: a share that turns out empty still costs a request.
  const long long whole = (long long)a.N / kTokens * a.Hkv;
  const long long pairs = std::min((long long)a.N / kTokens + a.B, (long long)a.N) * a.Hkv;
  const unsigned ctas = (unsigned)std::min(pairs, std::max(whole, 8LL * a.sms));
  kern<<<ctas, L::kThreads, L::kSmemBytes, s>>>(m[0], m[1], m[2], p);
  return cudaGetLastError();
}

// Two row tiles a CTA, which share K and V, or one and two CTAs a SM, whose chains
// run side by side: a short prompt leaves the second tile of a pair empty.  One where
// a sequence has on average at most 192 of a pair's 256 rows, 100 at d = 128, whose
// two rings have one stage each.  Measured, two / one, us, for prompts of random
// lengths up to the one given (the mean is half of it):
//   d = 64, G = 1:   30: 179 / 110, 190: 87 / 69, 500: 71 / 67, 1000: 68 / 73
//           G = 2:   60: 181 / 118, 190: 106 / 104, 300: 94 / 106
//           G = 4:   30: 96 / 67, 60: 101 / 93, 120: 100 / 111
//           G = 8:   30: 59 / 60, 60: 82 / 100
//   d = 128, G = 1:  30: 213 / 152, 120: 150 / 111, 190: 117 / 103, 300: 94 / 99
//            G = 2:  60: 221 / 156, 120: 162 / 167
//            G = 4:  30: 117 / 90, 60: 126 / 120, 120: 127 / 137
//            G = 8:  30: 75 / 74, 60: 106 / 119
// The lengths are on the device, so the rule knows their mean alone, with empty
// sequences and rows outside of them counted: a long prompt among many short ones may
// get the width that is slower for it.  Two / one, 8 heads unless said:
//   16384 tokens and 500 up to 30:    d = 64: 567 / 574,   d = 128: 634 / 723
//   8192 and 300 up to 60:            d = 64: 193 / 196,   d = 128: 273 / 294
//   two of 4000 and 200 up to 60:     d = 64: 116 / 108,   d = 128: 149 / 168
//   4000, 500 up to 60, 300 empty, 16 on 4 heads:  147 / 171,      179 / 213
// (all of them one tile by the rule)
template <int D, int G>
cudaError_t launch_g(const PackedArgs& a, const CUtensorMap* m, cudaStream_t s) {
  const long long few = D == 64 ? 192 : 100;
  if ((long long)a.N * G <= few * a.B) return launch_n<D, G, 1>(a, m, s);
  return launch_n<D, G, 2>(a, m, s);
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
