// Decayed linear attention of bf16 tensors on the tensor cores.
//
// The mathematics (chunks, the state before them, the two directions, the
// runs and cuts) is in polar_linear.cu; a chunk here is a tile of 128 tokens.
// Per tile, with x, y, z its rows, M the state before it (z dim x y dim) and
// w_j the powers of the decay:
//   S  = x y^T                 scores            A, B in shared memory
//   P  = S * decay, bf16                         over S in TMEM
//   O  = x M^T                 M as a bf16 operand in shared memory
//   O_i *= g^(i+1), then O += P z                A in TMEM
//   M' = g^n M + z^T (w y)
// P and the operand copy of M are rounded to bf16 once, at most 2^-8 of a value
// that the bf16 outputs round by as much again.  The state itself stays in fp32
// in TMEM: once a tile it is read, multiplied by g^n (LinearDecay) and added to
// the tile's products.  Those have an accumulator of their own, because the
// tensor core cuts off, rather than rounds, what it adds to: 16 products a tile
// straight into the state lost 1.6e-5 of it over 16K tokens of a slow decay.
// w y is not exact in bf16 and enters as a sum of bf16 terms.  Two leave at most
// 2^-17 of it (2.5e-6 of the state in the 2-norm), which no operand of x M^T
// shows; three leave 2^-25 and are taken where the caller asks for the state,
// in fp32 (kThree: 2e-7 of the state, what fp32 sums have).  The smaller terms
// are added first, so that little is cut off.  B2 H16 T16384 d128 takes 149 us
// with two terms and 175 with three.
//
// Shared memory at d = 128 is full (7 x 32 KB): two buffers of x and z, one of
// y, the state operand and one for a term of w y; see OutLayout for the other
// terms.  S, O, the tile's products and the state fill TMEM.  The outputs are
// staged in z's buffer, whose last reader makes them.
//
// Bound: HBM, closely followed by shared memory.  A tile moves 4 x 32 KB at
// d = 128, 5600 cycles at an SM's share of the measured copy bandwidth; its
// operands, two terms, the state operand and the staged outputs are about
// 576 KB of shared memory traffic, 4500 cycles at 128 bytes each (672 KB with
// three terms); the products need 2600 (3100).  Measured: 5800 cycles a tile.
// B2 H16 T16384 d128 (27 tiles a CTA) takes 98 us, 5.5 TB/s, 81 % of the copy
// bandwidth: the rest is the first loads, the last stores and the change of
// heads inside a run.
//
// Roles (one CTA per SM): warps 0-3 P and the outputs (thread = row = TMEM
// lane), the next 8 or 16 the state and the scaling of y (each group of four
// has all of its rows, and a share of the columns), then one warp each for TMA
// loads, MMA and TMEM, TMA stores.  With three terms the state's warps are the
// longest chain; 16 of them, of 80 registers a thread, take 107 us where 8 take
// 116, but none with two terms.
#include "polar_device.cuh"
#include "polar_internal.h"
#include "polar_linear.cuh"

namespace polar {

namespace {

constexpr int kTok = kLinearTile;  // tokens per tile
// Warps of the output kernel: four for P and the outputs, then these.
template <bool kThree>
struct OutRoles {
  static constexpr int kStateWarps = kThree ? 16 : 8;
  static constexpr int kStateThreads = 32 * kStateWarps;
  static constexpr int kTMA = 4 + kStateWarps, kMMA = kTMA + 1, kStore = kTMA + 2;
  static constexpr int kThreads = 32 * (kStore + 1);
};
constexpr uint32_t kColS = 0, kColO = 128, kColDS = 256, kColM = 384;  // TMEM columns

struct OutBars {
  uint64_t full_x[2], full_z[2], empty_x[2], empty_z[2];
  uint64_t full_y, empty_y;  // one phase a tile
  // outputs staged in a z buffer: one a buffer, so that the next phase needs
  // the store warp to have given that buffer back
  uint64_t staged[2];
  uint64_t s_full, p_full, o_full, o_free, m_op;  // one phase a tile
  uint64_t first, first_done, second, last, ds_full;  // one phase a state update
  uint64_t fixed;  // one phase a tile with rows past the sequence: they are zeroed
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  // by portion parity: g^31 .. g^0 (forward) or g^0 .. g^31 (reverse), read as float4
  alignas(16) float full_pw[2][32];
  float diag_pw[2][64];  // 31 zeros, then g^0 .. g^31
};

template <int D>
struct OutLayout {
  static constexpr int kTile = kTok * D * 2;
  static constexpr int kAtom = kTok * 128;  // 64 columns of a tile
  static constexpr int kXOff = 0;                  // two of x
  static constexpr int kZOff = kXOff + 2 * kTile;  // two of z, then the staged outputs
  static constexpr int kYOff = kZOff + 2 * kTile;  // one of y
  static constexpr int kMOff = kYOff + kTile;      // state operand, D rows
  static constexpr int kMAtom = D * 128;
  // Terms of scaled y, in the order of their products.  d = 64 has room for each;
  // at d = 128 the last takes the place of the state operand once x M^T has read
  // that, and the first of three makes room for the second.
  static constexpr bool kApart = D == 64;
  static constexpr int kWOff = kMOff + (kApart ? D * D * 2 : kTile);
  static constexpr int kLastOff = kApart ? kWOff + 2 * kTile : kMOff;
  static constexpr int kBarOff = kWOff + (kApart ? 3 : 1) * kTile;
  static constexpr int kSmemBytes = kBarOff + (int)sizeof(OutBars) + 1024;
  // more than half of the SM's, so one CTA holds the 512 TMEM columns
  static constexpr int kAsked = kSmemBytes > 120000 ? kSmemBytes : 120000;
  static_assert(kSmemBytes <= 232448, "shared memory");
};

struct OutMaps {
  CUtensorMap m[2][4];  // x, y, z, out of each application
};

struct OutParams {
  const float* log_decay;
  const int* lengths;
  const float *init[2], *cuts[2];  // see LinearArgs
  float* final_state[2];
  __nv_bfloat16* out[2];
  int state_t[2];
  int ops;  // applications in this launch: 1 or 2
  int BH, H, T;
  LinearSplit split;
  float scale;
  int* status;
};

// Generic-proxy accesses of shared memory come before what TMA and the tensor
// core do after it: writes are visible to them, reads are over.
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* smem_src, int x,
                                             int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(smem_src)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_store_commit_wait_read() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

__device__ __forceinline__ float2 unpack_bf16x2(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
// 16 consecutive TMEM columns of this thread's lane -> 16 registers, and by the
// size of the array.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[32]) { tmem_ld32(taddr, r); }
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[16]) {
  tmem_st16(taddr, r);
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[32]) {
  tmem_st32(taddr, r);
}
__device__ __forceinline__ void fence_regs(uint32_t (&r)[16]) { reg_fence16(r); }
__device__ __forceinline__ void fence_regs(uint32_t (&r)[32]) { reg_fence32(r); }

// w y of eight bf16 values as a sum of bf16 values: hi, the rounding of what hi
// leaves, and, if three, that of what the two leave.
template <bool kThree>
__device__ __forceinline__ void split_vec(uint4 y, float w, uint4& hi, uint4& lo, uint4& rest) {
  const uint32_t in[4] = {y.x, y.y, y.z, y.w};
  const float2 w2 = make_float2(w, w), minus = make_float2(-1.f, -1.f);
  uint32_t h[4], l[4], s[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = ffma2(unpack_bf16x2(in[e]), w2, make_float2(0.f, 0.f));
    h[e] = pack_bf16x2(f.x, f.y);
    const float2 r = ffma2(unpack_bf16x2(h[e]), minus, f);
    l[e] = pack_bf16x2(r.x, r.y);
    if constexpr (kThree) {
      const float2 t = ffma2(unpack_bf16x2(l[e]), minus, r);
      s[e] = pack_bf16x2(t.x, t.y);
    }
  }
  hi = make_uint4(h[0], h[1], h[2], h[3]);
  lo = make_uint4(l[0], l[1], l[2], l[3]);
  rest = make_uint4(s[0], s[1], s[2], s[3]);
}

// Zero rows [n, 128) of a tile in shared memory (kN threads).
template <int D, int kN>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int n, int tid) {
  for (int i = tid; i < kTok * D / 8; i += kN)
    if (((i >> 3) & (kTok - 1)) >= n) reinterpret_cast<uint4*>(tile)[i] = make_uint4(0, 0, 0, 0);
}

// One run of tiles a CTA.  kRev: from the last tile back.  kThree: terms of
// scaled y, the same number in every portion (a choice by portion in one kernel
// cost 12 us for its code).  Every role walks the same portions and tiles; it
// counts tiles (k), state updates (ku) and tiles with rows to zero (kf) for the
// phases of the barriers.
template <int D, bool kRev, bool kThree>
__global__ void __launch_bounds__(OutRoles<kThree>::kThreads, 1)
    polar_linear_out_tc_kernel(const __grid_constant__ OutMaps maps, const OutParams p) {
  using L = OutLayout<D>;
  using R = OutRoles<kThree>;
  constexpr int kStateWarps = R::kStateWarps, kStateThreads = R::kStateThreads;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  OutBars& br = *reinterpret_cast<OutBars*>(smem + L::kBarOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // two applications of one run are neighbours: they read the same tensors at
  // about the same time, the second from L2
  const int op = p.ops == 2 ? (int)(blockIdx.x & 1) : 0;
  const int part = p.ops == 2 ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;
  const CUtensorMap &map_x = maps.m[op][0], &map_y = maps.m[op][1], &map_z = maps.m[op][2],
                    &map_o = maps.m[op][3];
  float* const final_state = p.final_state[op];
  const int n_po = linear_portions(p.split, p.BH, part);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&br.full_x[i], 1);
      mbar_init(&br.full_z[i], 1);
      mbar_init(&br.empty_x[i], 1);
      mbar_init(&br.empty_z[i], 1);
      mbar_init(&br.staged[i], 4);
    }
    mbar_init(&br.full_y, 1);
    mbar_init(&br.empty_y, 1 + kStateWarps);  // the scores and the scaling have read it
    mbar_init(&br.s_full, 1);
    mbar_init(&br.p_full, 4);
    mbar_init(&br.o_full, 1);
    mbar_init(&br.o_free, 4);
    mbar_init(&br.m_op, kStateWarps);
    mbar_init(&br.first, kStateWarps);
    mbar_init(&br.second, kStateWarps);
    mbar_init(&br.ds_full, 1);
    mbar_init(&br.first_done, 1);
    mbar_init(&br.last, kStateWarps);
    mbar_init(&br.fixed, kStateWarps);
    mbar_init(&br.drain, 1);
    br.abort_flag = 0;
    fence_barrier_init();
  }
  linear_let_next_start();
  if (warp == R::kMMA) tmem_alloc(&br.tmem_base, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = br.tmem_base;
  volatile int* abort_flag = &br.abort_flag;
  auto portion = [&](int i) {
    return linear_portion(p.split, p.BH, p.H, p.T, p.lengths, p.status, part,
                          kRev ? n_po - 1 - i : i);
  };
  // the c-th live tile of a portion
  auto tile_of = [](const LinearPortion& po, int c) {
    return po.first + (kRev ? po.live - 1 - c : c);
  };
  // rows past the sequence, but inside the tensor, must be zeroed
  auto ragged = [&](int tile, int n) { return n < kTok && tile * kTok + n < p.T; };
  // the portion holds the head's last tile in walking order
  auto is_final = [&](const LinearPortion& po) {
    return final_state != nullptr && !(kRev ? po.cut_left : po.cut_right);
  };
  // the state after tile c is read by tile c + 1, or is the final one
  auto updates = [&](const LinearPortion& po, int c) { return c + 1 < po.live || is_final(po); };

  if (warp == R::kTMA) {
    // ------------------------------------------------------ TMA producer --
    if (lane == 0) {
      tma_prefetch_desc(&map_x);
      tma_prefetch_desc(&map_y);
      tma_prefetch_desc(&map_z);
    }
    __syncwarp();
    int k = 0, nz = 0, nx = 0, ny = 0;  // tiles of each issued
    bool ok = true;
    auto load = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int row, int bh) {
      mbar_arrive_expect_tx_warp(bar, L::kTile);
      for (int h = 0; h < D / 64; ++h)
        tma_load_3d_warp(dst + h * L::kAtom, map, bar, 64 * h, row, bh);
    };
    for (int ip = 0; ip < n_po && ok; ++ip) {
      const LinearPortion po = portion(ip);
      for (int c = 0; c < po.live; ++c, ++k) {
        const int st = k & 1, row = po.row(tile_of(po, c));
        const uint32_t ph = (uint32_t)(k / 2 - 1) & 1;
        // in the order in which their buffers come free
        if (k >= 2) ok = mbar_wait_warp(&br.empty_x[st], ph, abort_flag, p.status);
        if (!ok) break;
        load(smem + L::kXOff + st * L::kTile, &map_x, &br.full_x[st], row, po.bh);
        ++nx;
        if (k >= 1) ok = mbar_wait_warp(&br.empty_y, (uint32_t)(k - 1) & 1, abort_flag, p.status);
        if (!ok) break;
        load(smem + L::kYOff, &map_y, &br.full_y, row, po.bh);
        ++ny;
        if (k >= 2) ok = mbar_wait_warp(&br.empty_z[st], ph, abort_flag, p.status);
        if (!ok) break;
        load(smem + L::kZOff + st * L::kTile, &map_z, &br.full_z[st], row, po.bh);
        ++nz;
      }
    }
    if (!ok) {
      // aborted: let the copies already issued land before the CTA exits (the
      // last phase that each barrier was armed for)
      volatile int never = 0;
      const long long lim = kWaitLimitCycles / 4;
      for (int c = nz - 1; c >= 0 && c >= nz - 2; --c)
        mbar_wait(&br.full_z[c & 1], (uint32_t)(c / 2) & 1, &never, p.status, lim);
      for (int c = nx - 1; c >= 0 && c >= nx - 2; --c)
        mbar_wait(&br.full_x[c & 1], (uint32_t)(c / 2) & 1, &never, p.status, lim);
      if (ny > 0) mbar_wait(&br.full_y, (uint32_t)(ny - 1) & 1, &never, p.status, lim);
      __syncwarp();
    }
  } else if (warp == R::kMMA) {
    // ------------------------------------------------------- MMA issuer --
    // whole warp: uniform waits and descriptors, one elected lane issues
    constexpr uint32_t kIdS = idesc_bf16_f32(kTok, kTok, 0, 0);
    constexpr uint32_t kIdPV = idesc_bf16_f32(kTok, D, 0, 1);
    constexpr uint32_t kIdXM = idesc_bf16_f32(kTok, D, 0, 0);
    constexpr uint32_t kIdDS = idesc_bf16_f32(128, D, 1, 1);
    const uint32_t lbo = D == 128 ? L::kAtom : 0;
    const uint32_t base = smem_u32(smem);
    // K-major (rows of 64 columns) and MN-major (tokens as the K dim) views
    const uint64_t km = smem_desc_sw128(base, 16, 1024);
    const uint64_t mn = smem_desc_sw128(base, lbo, 1024);
    const uint64_t m_desc = smem_desc_sw128(base + L::kMOff, 16, 1024);
    auto at = [](uint32_t bytes) { return (uint64_t)(bytes >> 4); };
    auto kstep = [&](int kk, uint32_t atom) {
      return at((kk >> 2) * atom) + (uint64_t)(kk & 3) * 2;
    };
    // a term of scaled y, at `off`
    auto issue_ds = [&](int st, uint32_t off, bool add) {
      tc_fence_after();
      const uint64_t y0 = mn + at(off), z0 = mn + at(L::kZOff + st * L::kTile);
#pragma unroll
      for (int kk = 0; kk < kTok / 16; ++kk)
        umma_ss_warp(tmem + kColDS, z0 + at(kk * 2048), y0 + at(kk * 2048), kIdDS,
                     add || kk > 0);
    };
    // Order of a tile's products: S, x M^T, the terms of y, P z.  P z and the
    // next S run while the next y is scaled.  (Waiting for the next tile's
    // inputs before P z, so that S follows without a pause, measured 109 us
    // against 100: the scaling then waits for its turn.)
    int k = 0, ku = 0, kf = 0;
    bool ok = true, any = false;
    for (int ip = 0; ip < n_po && ok; ++ip) {
      const LinearPortion po = portion(ip);
      for (int c = 0; c < po.live; ++c, ++k) {
        const int st = k & 1, tile = tile_of(po, c);
        const uint32_t ph = (uint32_t)k & 1, ph2 = (uint32_t)(k / 2) & 1;
        // S: over P of the tile before, whose product is issued already
        ok = mbar_wait_warp(&br.full_x[st], ph2, abort_flag, p.status) &&
             mbar_wait_warp(&br.full_y, ph, abort_flag, p.status);
        if (ok && ragged(tile, po.tokens(tile)))
          ok = mbar_wait_warp(&br.fixed, (uint32_t)(kf++) & 1, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint64_t x0 = km + at(L::kXOff + st * L::kTile), y0 = km + at(L::kYOff);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_ss_warp(tmem + kColS, x0 + kstep(kk, L::kAtom), y0 + kstep(kk, L::kAtom), kIdS,
                       kk > 0);
        umma_commit_warp(&br.s_full);
        umma_commit_warp(&br.empty_y);
        any = true;
        // x M^T, once the state is written and the last outputs are read
        ok = mbar_wait_warp(&br.m_op, ph, abort_flag, p.status);
        if (ok && k > 0) ok = mbar_wait_warp(&br.o_free, ph ^ 1, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_ss_warp(tmem + kColO, x0 + kstep(kk, L::kAtom), m_desc + kstep(kk, L::kMAtom),
                       kIdXM, kk > 0);
        umma_commit_warp(&br.empty_x[st]);
        ok = mbar_wait_warp(&br.full_z[st], ph2, abort_flag, p.status);
        if (ok && updates(po, c)) {
          ok = mbar_wait_warp(&br.first, (uint32_t)ku & 1, abort_flag, p.status);
          if (!ok) break;
          issue_ds(st, L::kWOff, false);
          if constexpr (L::kApart) {
            if constexpr (kThree) issue_ds(st, L::kWOff + L::kTile, true);
          } else {
            if constexpr (kThree) {
              umma_commit_warp(&br.first_done);
              ok = mbar_wait_warp(&br.second, (uint32_t)ku & 1, abort_flag, p.status);
              if (!ok) break;
              issue_ds(st, L::kWOff, true);
            }
            ok = mbar_wait_warp(&br.last, (uint32_t)ku & 1, abort_flag, p.status);
            if (!ok) break;
          }
          issue_ds(st, L::kLastOff, true);
          umma_commit_warp(&br.ds_full);
          ++ku;
        }
        // P z, added to x M^T once that has its powers of the decay
        ok = ok && mbar_wait_warp(&br.p_full, ph, abort_flag, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint64_t z0 = mn + at(L::kZOff + st * L::kTile);
#pragma unroll
        for (int kk = 0; kk < kTok / 16; ++kk)
          umma_ts_warp(tmem + kColO, tmem + kColS + kk * 8, z0 + at(kk * 2048), kIdPV, 1u);
        umma_commit_warp(&br.o_full);
      }
    }
    if (!ok && any) {
      // aborted: wait for the products in flight before TMEM is released
      volatile int never = 0;
      umma_commit_warp(&br.drain);
      __syncwarp();
      mbar_wait(&br.drain, 0, &never, p.status, kWaitLimitCycles / 4);
      __syncwarp();
    }
  } else if (warp == R::kStore) {
    // ------------------------------------------------------- TMA stores --
    if (lane == 0) {
      int k = 0;
      bool ok = true;
      for (int ip = 0; ip < n_po && ok; ++ip) {
        const LinearPortion po = portion(ip);
        for (int c = 0; c < po.live; ++c, ++k) {
          const int st = k & 1;
          ok = mbar_wait(&br.staged[st], (uint32_t)(k / 2) & 1, abort_flag, p.status);
          if (!ok) break;
          for (int h = 0; h < D / 64; ++h)
            tma_store_3d(&map_o, smem + L::kZOff + st * L::kTile + h * L::kAtom, 64 * h,
                         po.row(tile_of(po, c)), po.bh);
          tma_store_commit_wait_read();
          mbar_arrive(&br.empty_z[st]);
        }
      }
    }
    __syncwarp();
  } else if (warp < 4) {
    // ------------------------------------------------- P and the outputs --
    const int r = threadIdx.x;  // row of the tile
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    const uint32_t s_tm = tmem + lane_base + kColS;
    int k = 0;
    bool go = true;  // after a failed wait a warp still joins the barriers
    for (int ip = 0; ip < n_po; ++ip) {
      const LinearPortion po = portion(ip);
      const float l2 = linear_log2_decay(p.log_decay, po.bh % p.H);
      // powers of the head's decay; two sets, so that a warp still in the last
      // portion keeps its own (every portion starts with a barrier)
      float* full_pw = br.full_pw[ip & 1];
      float* diag_pw = br.diag_pw[ip & 1];
      if (r < 32) full_pw[r] = linear_power(l2, kRev ? r : 31 - r);
      if (r < 64) diag_pw[r] = r < 31 ? 0.f : linear_power(l2, r - 31);
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (!go) continue;
      for (int c = 0; c < po.live; ++c, ++k) {
        const int st = k & 1, tile = tile_of(po, c), n = po.tokens(tile);
        const uint32_t ph = (uint32_t)k & 1;
        bool ok = __all_sync(0xffffffffu, mbar_wait(&br.s_full, ph, abort_flag, p.status));
        if (ok) {
          tc_fence_after();
          // 32-column blocks of this warp's rows: whole before the diagonal
          // one (after it in reverse), zero beyond it
#pragma unroll 1
          for (int b = 0; b < 4; ++b) {
            uint32_t pk[16];
            if (b == warp) {
              uint32_t v[32];
              tmem_ld32(s_tm + 32 * b, v);
              tmem_ld_wait();
              reg_fence32(v);
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float f[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                  const int dist = kRev ? e + u - lane : lane - e - u;
                  const float w = p.scale * diag_pw[31 + dist];
                  f[u] = dist >= 0 ? __uint_as_float(v[e + u]) * w : 0.f;
                }
                pk[e / 2] = pack_bf16x2(f[0], f[1]);
              }
            } else if (kRev ? b > warp : b < warp) {
              uint32_t v[32];
              tmem_ld32(s_tm + 32 * b, v);
              const float rf = p.scale * linear_power(l2, kRev ? 32 * b - r : r - 32 * b - 31);
              tmem_ld_wait();
              reg_fence32(v);
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 w = *reinterpret_cast<const float4*>(&full_pw[e]);
                pk[e / 2] = pack_bf16x2(__uint_as_float(v[e]) * (w.x * rf),
                                        __uint_as_float(v[e + 1]) * (w.y * rf));
                pk[e / 2 + 1] = pack_bf16x2(__uint_as_float(v[e + 2]) * (w.z * rf),
                                            __uint_as_float(v[e + 3]) * (w.w * rf));
              }
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) pk[e] = 0u;
            }
            // P block b lies over S columns 16 b .. 16 b + 15, read already
            tmem_st16(s_tm + 16 * b, pk);
          }
          tmem_st_wait();
          // x is free once x M^T is there: its rows times their powers
          ok = __all_sync(0xffffffffu, mbar_wait(&br.empty_x[st], (uint32_t)(k / 2) & 1,
                                                 abort_flag, p.status));
        }
        const bool live = r < n;
        if (ok) {
          tc_fence_after();
          const float w2 = live ? (kRev ? linear_power(l2, n - 1 - r)
                                        : p.scale * linear_power(l2, r + 1))
                                : 0.f;
#pragma unroll 1
          for (int b = 0; b < D / 32; ++b) {
            uint32_t v[32];
            tmem_ld32(tmem + lane_base + kColO + 32 * b, v);
            tmem_ld_wait();
            reg_fence32(v);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(w2 * __uint_as_float(v[e]));
            tmem_st32(tmem + lane_base + kColO + 32 * b, v);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&br.p_full);
          ok = __all_sync(0xffffffffu, mbar_wait(&br.o_full, ph, abort_flag, p.status));
        }
        if (ok) {
          tc_fence_after();
          uint8_t* line = smem + L::kZOff + st * L::kTile + r * 128;  // z's readers are done
#pragma unroll 1
          for (int b = 0; b < D / 32; ++b) {
            uint32_t o[32];
            tmem_ld32(tmem + lane_base + kColO + 32 * b, o);
            tmem_ld_wait();
            reg_fence32(o);
            if (b == D / 32 - 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&br.o_free);
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              uint32_t o4[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int i = 8 * g + 2 * e;
                o4[e] = live ? pack_bf16x2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])) : 0u;
              }
              const int ch = (b & 1) * 4 + g;
              *reinterpret_cast<uint4*>(line + (b >> 1) * L::kAtom + ((ch ^ (r & 7)) << 4)) =
                  make_uint4(o4[0], o4[1], o4[2], o4[3]);
            }
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&br.staged[st]);
        }
        if (!__all_sync(0xffffffffu, ok)) {
          go = false;
          break;
        }
      }
      // tiles past the sequence
      const int t0 = po.row(po.first + po.live), t1 = min(po.row(po.last), p.T);
      uint4* tail = reinterpret_cast<uint4*>(p.out[op] + ((size_t)po.bh * p.T + t0) * D);
      for (long long i = r; i < (long long)(t1 - t0) * (D / 8); i += 128)
        tail[i] = make_uint4(0u, 0u, 0u, 0u);
    }
  } else if (warp < 4 + kStateWarps) {
    // ------------------------------------------------ state, scaling of y --
    const int tid = threadIdx.x - 128;
    const int r = threadIdx.x & 127;   // state row (z dim) = TMEM lane
    constexpr int kCols = 128 * D / kStateThreads;
    constexpr int kB = kThree ? 16 : 32;         // columns at a time
    const int col0 = ((warp - 4) >> 2) * kCols;  // the warp's columns
    constexpr int kVecs = kTok * D / 8 / kStateThreads;  // 16-byte pieces of y a thread
    constexpr int kRows = kStateThreads / 8;
    const bool mine = r < D;           // at d = 64 lanes 64.. repeat the rows
    const uint32_t m_tm = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kColM + col0;
    const uint32_t ds_tm = m_tm - kColM + kColDS;
    // kB columns of the state: after a tile, g times the one before it plus the
    // tile's products.
    auto state_block = [&](int b, bool add, LinearDecay g, uint32_t (&v)[kB]) {
      tmem_ld(m_tm + kB * b, v);
      if (add) {
        uint32_t ds[kB];
        tmem_ld(ds_tm + kB * b, ds);
        tmem_ld_wait();
        fence_regs(v);
        fence_regs(ds);
#pragma unroll
        for (int e = 0; e < kB; e += 2) {
          const float2 m =
              g.join(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])),
                     make_float2(__uint_as_float(ds[e]), __uint_as_float(ds[e + 1])));
          v[e] = __float_as_uint(m.x);
          v[e + 1] = __float_as_uint(m.y);
        }
      } else {
        tmem_ld_wait();
        fence_regs(v);
      }
    };
    // The state to its bf16 operand for x M^T and, if new, back into TMEM.
    auto hand_over = [&](bool add, LinearDecay g) {
      int sw = r & 7;
      asm volatile("" : "+r"(sw));  // not to be kept as eight addresses across the loop
#pragma unroll
      for (int b = 0; b < kCols / kB; ++b) {
        uint32_t v[kB];
        state_block(b, add, g, v);
        if (mine) {
          const int col = col0 + kB * b;
          uint8_t* line = smem + L::kMOff + (col >> 6) * L::kMAtom + r * 128;
#pragma unroll
          for (int q = 0; q < kB / 8; ++q) {
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[e] = pack_bf16x2(__uint_as_float(v[8 * q + 2 * e]),
                                 __uint_as_float(v[8 * q + 2 * e + 1]));
            const int ch = ((col & 63) >> 3) + q;
            *reinterpret_cast<uint4*>(line + ((ch ^ sw) << 4)) =
                make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        if (add) tmem_st(m_tm + kB * b, v);
      }
      if (add) tmem_st_wait();
    };
    int k = 0, ku = 0;
    bool ok = true;
    linear_wait_previous();  // only these warps read states or write the final one
    for (int ip = 0; ip < n_po && ok; ++ip) {
      const LinearPortion po = portion(ip);
      const float ln = linear_log_decay(p.log_decay, po.bh % p.H);
      const float l2 = linear_log2_decay(p.log_decay, po.bh % p.H);
      const bool fin = is_final(po);
      if (po.live > 0 || fin) {
        // the incoming state (every reader of the last portion's is done)
        const float* src =
            (kRev ? po.cut_right : po.cut_left)
                ? p.cuts[op] + (size_t)(kRev ? part + 1 : part - 1) * D * D
                : (p.init[op] ? p.init[op] + (size_t)po.bh * D * D : nullptr);
#pragma unroll
        for (int b = 0; b < kCols / kB; ++b) {
          const int col = col0 + kB * b;
          uint32_t v[kB];
          if (!src || !mine) {
#pragma unroll
            for (int e = 0; e < kB; ++e) v[e] = 0u;
          } else if (p.state_t[op]) {
#pragma unroll
            for (int e = 0; e < kB; ++e)
              v[e] = __float_as_uint(src[(size_t)(col + e) * D + r]);
          } else {
#pragma unroll
            for (int e = 0; e < kB; e += 4) {
              const uint4 u = *reinterpret_cast<const uint4*>(src + (size_t)r * D + col + e);
              v[e] = u.x;
              v[e + 1] = u.y;
              v[e + 2] = u.z;
              v[e + 3] = u.w;
            }
          }
          __syncwarp();
          tmem_st(m_tm + kB * b, v);
        }
        tmem_st_wait();
      }
      bool wait_ds = false;  // products of the tile before are under way
      int last_n = 0;        // its tokens
      for (int c = 0; c < po.live; ++c, ++k) {
        const int st = k & 1, tile = tile_of(po, c), n = po.tokens(tile);
        const bool upd = updates(po, c);
        uint8_t* ty = smem + L::kYOff;
        ok = mbar_wait_warp(&br.full_y, (uint32_t)k & 1, abort_flag, p.status);
        if (ok && ragged(tile, n)) {
          ok = mbar_wait_warp(&br.full_z[st], (uint32_t)(k / 2) & 1, abort_flag, p.status);
          if (!ok) break;
          zero_rows<D, kStateThreads>(ty, n, tid);
          zero_rows<D, kStateThreads>(smem + L::kZOff + st * L::kTile, n, tid);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&br.fixed);
        }
        if (!ok) break;
        // y, in registers while the last products run
        const uint4* from = reinterpret_cast<const uint4*>(ty) + tid;
        uint4* to = reinterpret_cast<uint4*>(smem + L::kWOff) + tid;
        uint4 hi[kVecs];  // y, then its hi
#pragma unroll
        for (int q = 0; q < kVecs; ++q) hi[q] = from[kStateThreads * q];
        // Nothing uses y yet, so the loads may still be on their way, behind
        // slower accesses of the SM, when the arrival is seen and TMA writes the
        // next y over this one: they have to be over first.
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&br.empty_y);
        const LinearDecay g = linear_decay(ln, last_n);
        if (wait_ds) {
          ok = mbar_wait_warp(&br.ds_full, (uint32_t)(ku - 1) & 1, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
        }
        hand_over(wait_ds, g);
        last_n = n;
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&br.m_op);
        wait_ds = upd;
        if (!upd) {
          // the operand's reader, before the next portion's: x M^T of this tile.
          // Its barrier's phase before (tile k - 2) is over for sure, which a
          // wait by parity needs; that of o_full need not be.
          ok = mbar_wait_warp(&br.empty_x[st], (uint32_t)(k / 2) & 1, abort_flag, p.status);
          if (!ok) break;
          continue;
        }
        ++ku;
        // the smallest term first: the larger ones, added last, are cut off least
        uint4 lo[kVecs];
        auto write = [&](int off, const uint4 (&v)[kVecs]) {
          uint4* dst = reinterpret_cast<uint4*>(smem + off) + tid;
#pragma unroll
          for (int q = 0; q < kVecs; ++q) dst[kStateThreads * q] = v[q];
        };
        auto written = [&](uint64_t* bar) {
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar);
        };
#pragma unroll
        for (int u = 0; u < kTok / kRows; ++u) {
          const int j = (tid >> 3) + kRows * u;  // row of pieces u, u + kTok / kRows
          const float w = j >= n ? 0.f
                                 : (kRev ? p.scale * linear_power(l2, j + 1)
                                         : linear_power(l2, n - 1 - j));
#pragma unroll
          for (int q = u; q < kVecs; q += kTok / kRows) {
            uint4 rest;
            split_vec<kThree>(hi[q], w, hi[q], lo[q], rest);
            to[kStateThreads * q] = kThree ? rest : lo[q];
          }
        }
        if constexpr (L::kApart) {
          if constexpr (kThree) write(L::kWOff + L::kTile, lo);
          write(L::kLastOff, hi);
          written(&br.first);
        } else {
          written(&br.first);
          if constexpr (kThree) {
            ok = mbar_wait_warp(&br.first_done, (uint32_t)(ku - 1) & 1, abort_flag, p.status);
            if (!ok) break;
            write(L::kWOff, lo);
            written(&br.second);
          }
          // x M^T has read the state operand
          ok = mbar_wait_warp(&br.empty_x[st], (uint32_t)(k / 2) & 1, abort_flag, p.status);
          if (!ok) break;
          write(L::kLastOff, hi);
          written(&br.last);
        }
      }
      if (ok && fin) {
        if (wait_ds) {
          ok = mbar_wait_warp(&br.ds_full, (uint32_t)(ku - 1) & 1, abort_flag, p.status);
          if (!ok) break;
          tc_fence_after();
        }
        const LinearDecay g = linear_decay(ln, last_n);
        float* dst = final_state + ((size_t)po.bh * D + r) * D + col0;
#pragma unroll
        for (int b = 0; b < kCols / kB; ++b) {
          uint32_t v[kB];
          state_block(b, wait_ds, g, v);
          if (mine) {
#pragma unroll
            for (int e = 0; e < kB; e += 4)
              *reinterpret_cast<uint4*>(dst + kB * b + e) =
                  make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          }
          __syncwarp();
        }
        tc_fence_before();
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == R::kMMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------ states at cuts --

// Each run's own part of the head that its boundary cuts, y weighted by the
// distance to the cut, so nothing is ever rescaled: a tile's products (two or
// three terms, as above) go to one of two accumulators in TMEM and are added up
// in fp32 registers while the next tile's run.  The first term replaces y, the
// second goes through one buffer of its own, the third replaces the first.  The tiles are walked so that those the output kernel
// starts with come last: it then finds them in L2.  Bound: HBM (64 KB a tile at
// d = 128).  B2 H16 T16384 d128: 45 us, 5.3 TB/s, 79 % of the copy bandwidth.
// With three terms shared memory (384 KB a tile) and the scaling warps: 62 us
// with 8 of them, 56 with 16.
template <bool kThree>
struct StateRoles {
  static constexpr int kScale = kThree ? 16 : 8;  // warps that scale y and sum products
  static constexpr int kTMA = kScale, kMMA = kScale + 1;
  static constexpr int kThreads = 32 * (kScale + 2);
};

template <int D>
struct StateLayout {
  static constexpr int kNS = D == 128 ? 3 : 6;
  static constexpr int kTile = kTok * D * 2;
  static constexpr int kAtom = kTok * 128;
  static constexpr int kStage = 2 * kTile;  // y (then terms of it), z
  static constexpr int kWOff = kNS * kStage;
  static constexpr int kBarOff = kWOff + kTile;
  static constexpr int kSmemBytes = kBarOff + 512 + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory");
};

struct StateBars {
  uint64_t full[6], empty[6], first[6];
  uint64_t second, sums;       // one phase a tile
  uint64_t first_done, third;  // one phase a tile, with three terms
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};

struct StateMaps {
  CUtensorMap m[2][2];  // y, z of each application (blockIdx.y)
};

struct StateParams {
  const float* log_decay;
  const int* lengths;
  float* cuts[2];
  int reverse[2];
  float scale[2];
  int BH, H, T;
  LinearSplit split;
  int* status;
};

template <int D, bool kThree>
__global__ void __launch_bounds__(StateRoles<kThree>::kThreads, 1)
    polar_linear_state_tc_kernel(const __grid_constant__ StateMaps maps, const StateParams p) {
  using L = StateLayout<D>;
  using R = StateRoles<kThree>;
  constexpr int NS = L::kNS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  StateBars& br = *reinterpret_cast<StateBars*>(smem + L::kBarOff);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int op = blockIdx.y;
  const CUtensorMap &map_y = maps.m[op][0], &map_z = maps.m[op][1];
  const bool reverse = p.reverse[op] != 0;
  const LinearPortion po = linear_portion(
      p.split, p.BH, p.H, p.T, p.lengths, p.status, blockIdx.x,
      reverse ? 0 : linear_portions(p.split, p.BH, blockIdx.x) - 1);
  linear_let_next_start();
  if (!(reverse ? po.cut_left : po.cut_right)) return;  // the whole CTA
  const int bh = po.bh, nt = po.live;
  const int t0 = po.row(po.first), t1 = max(t0, min(po.row(po.last), po.len));
  const float l2 = linear_log2_decay(p.log_decay, bh % p.H);

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&br.full[i], 1);
      mbar_init(&br.empty[i], 1);
      mbar_init(&br.first[i], R::kScale);
    }
    mbar_init(&br.second, R::kScale);
    mbar_init(&br.sums, 1);
    mbar_init(&br.first_done, 1);
    mbar_init(&br.third, R::kScale);
    mbar_init(&br.drain, 1);
    br.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == R::kMMA) tmem_alloc(&br.tmem_base, 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = br.tmem_base;
  volatile int* abort_flag = &br.abort_flag;
  auto tile_row = [&](int c) { return t0 + (reverse ? c : nt - 1 - c) * kTok; };

  if (warp == R::kTMA) {
    if (lane == 0) {
      tma_prefetch_desc(&map_y);
      tma_prefetch_desc(&map_z);
    }
    __syncwarp();
    int issued = 0;
    bool ok = true;
    for (int c = 0; c < nt && ok; ++c) {
      const int st = c % NS;
      if (c >= NS)
        ok = mbar_wait_warp(&br.empty[st], (uint32_t)(c / NS - 1) & 1, abort_flag, p.status);
      if (!ok) break;
      uint8_t* sy = smem + st * L::kStage;
      mbar_arrive_expect_tx_warp(&br.full[st], 2 * L::kTile);
      for (int h = 0; h < D / 64; ++h) {
        tma_load_3d_warp(sy + h * L::kAtom, &map_y, &br.full[st], 64 * h, tile_row(c), bh);
        tma_load_3d_warp(sy + L::kTile + h * L::kAtom, &map_z, &br.full[st], 64 * h, tile_row(c),
                         bh);
      }
      issued = c + 1;
    }
    if (!ok) {
      volatile int never = 0;
      for (int c = issued - 1; c >= 0 && c >= issued - NS; --c)
        mbar_wait(&br.full[c % NS], (uint32_t)(c / NS) & 1, &never, p.status,
                  kWaitLimitCycles / 4);
      __syncwarp();
    }
  } else if (warp == R::kMMA) {
    constexpr uint32_t kId = idesc_bf16_f32(128, D, 1, 1);
    const uint64_t mn = smem_desc_sw128(smem_u32(smem), D == 128 ? L::kAtom : 0, 1024);
    auto at = [](uint32_t bytes) { return (uint64_t)(bytes >> 4); };
    bool ok = true, any = false;
    for (int c = 0; c < nt; ++c) {
      const int st = c % NS;
      const uint64_t y0 = mn + at(st * L::kStage), z0 = y0 + at(L::kTile), w0 = mn + at(L::kWOff);
      const uint32_t acc = tmem + (c & 1) * 128;
      auto products = [&](uint64_t term, bool add) {
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kTok / 16; ++kk)
          umma_ss_warp(acc, z0 + at(kk * 2048), term + at(kk * 2048), kId, add || kk > 0);
      };
      ok = mbar_wait_warp(&br.first[st], (uint32_t)(c / NS) & 1, abort_flag, p.status);
      if (!ok) break;
      products(y0, false);
      any = true;
      if constexpr (kThree) umma_commit_warp(&br.first_done);
      ok = mbar_wait_warp(&br.second, (uint32_t)c & 1, abort_flag, p.status);
      if (!ok) break;
      products(w0, true);
      if constexpr (kThree) {
        ok = mbar_wait_warp(&br.third, (uint32_t)c & 1, abort_flag, p.status);
        if (!ok) break;
        products(y0, true);
      }
      umma_commit_warp(&br.sums);
      umma_commit_warp(&br.empty[st]);
    }
    if (!ok && any) {
      volatile int never = 0;
      umma_commit_warp(&br.drain);
      __syncwarp();
      mbar_wait(&br.drain, 0, &never, p.status, kWaitLimitCycles / 4);
      __syncwarp();
    }
  } else {
    const int tid = threadIdx.x;
    const int r = threadIdx.x & 127;
    constexpr int kScaleThreads = 32 * R::kScale;
    constexpr int kCols = 128 * D / kScaleThreads;
    const int col = (warp >> 2) * kCols;
    float sum[kCols];  // row r of the state, columns col ..
#pragma unroll
    for (int e = 0; e < kCols; ++e) sum[e] = 0.f;
    // the products of tile c, once they are done
    auto collect = [&](int c) {
      if (!mbar_wait_warp(&br.sums, (uint32_t)c & 1, abort_flag, p.status)) return false;
      tc_fence_after();
#pragma unroll
      for (int b = 0; b < kCols / 16; ++b) {
        uint32_t v[16];
        tmem_ld16(tmem + ((uint32_t)((warp & 3) * 32) << 16) + (c & 1) * 128 + col + 16 * b, v);
        tmem_ld_wait();
        reg_fence16(v);
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[16 * b + e] += __uint_as_float(v[e]);
      }
      tc_fence_before();
      return true;
    };
    bool ok = true;
    for (int c = 0; c < nt; ++c) {
      const int st = c % NS, row = tile_row(c), n = min(kTok, t1 - row);
      ok = mbar_wait_warp(&br.full[st], (uint32_t)(c / NS) & 1, abort_flag, p.status);
      if (!ok) break;
      uint8_t* ty = smem + st * L::kStage;
      if (n < kTok) zero_rows<D, kScaleThreads>(ty + L::kTile, n, tid);
      constexpr int kVecs = kTok * D / 8 / kScaleThreads;
      constexpr int kRows = kScaleThreads / 8;  // rows of 64 columns that the warps take at once
      uint4* at = reinterpret_cast<uint4*>(ty) + tid;
      uint4 hi[kVecs], lo[kVecs];  // y, then its terms
#pragma unroll
      for (int q = 0; q < kVecs; ++q) hi[q] = at[kScaleThreads * q];
#pragma unroll
      for (int u = 0; u < kTok / kRows; ++u) {
        const int j = (tid >> 3) + kRows * u, t = row + j;  // row of pieces u, u + kTok / kRows
        const float w =
            p.scale[op] * linear_power(l2, reverse ? t - t0 + 1 : max(t1 - 1 - t, 0));
#pragma unroll
        for (int q = u; q < kVecs; q += kTok / kRows) {
          uint4 rest;
          split_vec<kThree>(hi[q], w, hi[q], lo[q], rest);
          if (j >= n) hi[q] = lo[q] = rest = make_uint4(0u, 0u, 0u, 0u);
          at[kScaleThreads * q] = kThree ? rest : lo[q];
        }
      }
      auto write = [&](uint4* to, const uint4 (&v)[kVecs], uint64_t* bar) {
#pragma unroll
        for (int q = 0; q < kVecs; ++q) to[kScaleThreads * q] = v[q];
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
      };
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&br.first[st]);
      if (c > 0) ok = collect(c - 1);  // the buffer of the second term is free then, too
      if (!ok) break;
      uint4* to = reinterpret_cast<uint4*>(smem + L::kWOff) + tid;
      if constexpr (kThree) {
        write(to, lo, &br.second);
        ok = mbar_wait_warp(&br.first_done, (uint32_t)c & 1, abort_flag, p.status);
        if (!ok) break;
        write(at, hi, &br.third);
      } else {
        write(to, hi, &br.second);
      }
    }
    if (ok && nt > 0) ok = collect(nt - 1);
    if (ok && r < D) {
      float* dst = p.cuts[op] + ((size_t)blockIdx.x * D + r) * D + col;
#pragma unroll
      for (int e = 0; e < kCols; e += 4)
        *reinterpret_cast<float4*>(dst + e) =
            make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == R::kMMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// n applications (1 or 2) that differ in tensors and states only; maps: x, y,
// z, out of each.
template <int D, bool kRev, bool kThree>
cudaError_t out_tc_t(const LinearArgs* a, int n, const CUtensorMap* maps, cudaStream_t s) {
  using L = OutLayout<D>;
  OutMaps m;
  OutParams p;
  p.log_decay = a->log_decay;
  p.lengths = a->lengths;
  for (int i = 0; i < 2; ++i) {
    const int j = i < n ? i : 0;
    for (int t = 0; t < 4; ++t) m.m[i][t] = maps[4 * j + t];
    p.init[i] = a[j].init;
    p.cuts[i] = a[j].cuts;
    p.final_state[i] = a[j].final_state;
    p.out[i] = static_cast<__nv_bfloat16*>(a[j].out);
    p.state_t[i] = a[j].state_t ? 1 : 0;
  }
  p.ops = n;
  p.BH = a->B * a->H;
  p.H = a->H;
  p.T = a->T;
  p.split = a->split;
  p.scale = a->scale;
  p.status = a->status;
  auto kern = polar_linear_out_tc_kernel<D, kRev, kThree>;
  cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAsked);
  if (e != cudaSuccess) return e;
  return linear_launch(kern, dim3((unsigned)a->split.parts * n), OutRoles<kThree>::kThreads, L::kAsked, s,
                       a->chained, m, p);
}

template <int D, bool kRev>
cudaError_t out_tc_d(const LinearArgs* a, int n, const CUtensorMap* maps, cudaStream_t s) {
  return a->exact ? out_tc_t<D, kRev, true>(a, n, maps, s) : out_tc_t<D, kRev, false>(a, n, maps, s);
}

template <int D, bool kThree>
cudaError_t state_tc_t(const LinearStateArgs* a, int n, const CUtensorMap* maps, cudaStream_t s) {
  using L = StateLayout<D>;
  StateMaps m;
  StateParams p;
  p.log_decay = a->log_decay;
  p.lengths = a->lengths;
  for (int i = 0; i < 2; ++i) {
    const int j = i < n ? i : 0;
    m.m[i][0] = maps[2 * j];
    m.m[i][1] = maps[2 * j + 1];
    p.cuts[i] = a[j].cuts;
    p.reverse[i] = a[j].reverse ? 1 : 0;
    p.scale[i] = a[j].scale;
  }
  p.BH = a->B * a->H;
  p.H = a->H;
  p.T = a->T;
  p.split = a->split;
  p.status = a->status;
  cudaError_t e = cudaFuncSetAttribute(polar_linear_state_tc_kernel<D, kThree>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       L::kSmemBytes);
  if (e != cudaSuccess) return e;
  polar_linear_state_tc_kernel<D, kThree>
      <<<dim3((unsigned)a->split.parts, n), StateRoles<kThree>::kThreads, L::kSmemBytes, s>>>(m, p);
  return cudaGetLastError();
}

template <int D>
cudaError_t state_tc_d(const LinearStateArgs* a, int n, const CUtensorMap* maps, cudaStream_t s) {
  if (n == 2 && a[0].exact != a[1].exact) {
    const cudaError_t e = state_tc_d<D>(a, 1, maps, s);
    return e != cudaSuccess ? e : state_tc_d<D>(a + 1, 1, maps + 2, s);
  }
  return a->exact ? state_tc_t<D, true>(a, n, maps, s) : state_tc_t<D, false>(a, n, maps, s);
}

}  // namespace

cudaError_t launch_linear_out_tc(const LinearArgs* a, int n, const CUtensorMap* maps,
                                 cudaStream_t s) {
  if (a->d == 64)
    return a->reverse ? out_tc_d<64, true>(a, n, maps, s) : out_tc_d<64, false>(a, n, maps, s);
  return a->reverse ? out_tc_d<128, true>(a, n, maps, s) : out_tc_d<128, false>(a, n, maps, s);
}

cudaError_t launch_linear_states_tc(const LinearStateArgs* a, int n, const CUtensorMap* maps,
                                    cudaStream_t s) {
  return a->d == 64 ? state_tc_d<64>(a, n, maps, s) : state_tc_d<128>(a, n, maps, s);
}

}  // namespace polar
