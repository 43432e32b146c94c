// Accumulated attention weights of cache rows, and eviction by them.
//
// Weights: p_j = exp(s_j - lse) needs the logsumexp over all of a sequence's
// rows, which is known only after every split has run.  The split kernels
// therefore store their logits (4 bytes per query head and row beside the
// 4 d or more bytes of K and V that the row costs), and the kernel here turns
// them into weights once the split records are there.
//
// Eviction: one CTA per (sequence, KV head) finds the keep-th largest
// (protected, weight, lower row) key by radix passes over 11, 11 and 10 bits,
// lists the evicted rows below `keep` and the kept rows past it, both
// ascending, and moves weights and positions; a second kernel copies the K
// and V rows.  The keys stay in shared memory between the passes (up to 48K
// rows; longer heads form them again).  The first pass sorts by exponent and
// two bits more, which spreads heavy-tailed weights over enough bins for
// shared-memory atomics; the later ones touch one bin's rows only.
#include <climits>
#include <cstdint>

#include "polar_device.cuh"
#include "polar_internal.h"

namespace polar {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWThreads = 256;
constexpr int kWRows = 1024;  // cache rows per CTA

// One CTA per kWRows rows of a (sequence, KV head).  Every load of a thread's
// rows is issued before the logsumexp is formed from the split records, so the
// CTA costs about one memory latency.  Bound: HBM (4 G bytes of logits and 8
// of weights a row): 20 us for 32 x 4 KV heads of 32K rows, G = 4, 100 MB,
// 5.0 TB/s.
template <int G>
__global__ void __launch_bounds__(kWThreads) polar_decode_weights_kernel(const WeightsArgs a) {
  __shared__ float s_lse[G];
  constexpr int kR = kWRows / kWThreads;
  const int parts = (a.max_seq_len + kWRows - 1) / kWRows;
  const int bh = blockIdx.x / parts, b = bh / a.Hkv, hkv = bh % a.Hkv;
  const int n = min(max(a.seq_lens[b], 0), a.max_seq_len);
  const int j0 = (int)(blockIdx.x % parts) * kWRows + threadIdx.x;
  // the logits and records come from the launches before (programmatic launch)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (j0 - (int)threadIdx.x >= n) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t head0 = (size_t)b * a.Hq + (size_t)hkv * G;
  const float* x = a.logits + head0 * a.max_seq_len;
  float* w = a.weights + (size_t)bh * a.stride;
  float xv[kR][G], wv[kR];
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const int j = j0 + r * kWThreads;
    wv[r] = j < n ? w[j] : 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g)
      xv[r][g] = j < n ? __ldcs(x + (size_t)g * a.max_seq_len + j) : -INFINITY;
  }
  if (warp < G) {
    // logsumexp of the head over its splits, log2 units
    const float* rec = a.partials + (head0 + warp) * a.splits * (a.d + 4);
    float m = -INFINITY, l = 0.f;
    for (int s = lane; s < a.splits; s += 32) {
      const float ms = rec[(size_t)s * (a.d + 4)], ls = rec[(size_t)s * (a.d + 4) + 1];
      if (ms == -INFINITY) continue;
      const float mx = fmaxf(m, ms);
      l = l * expf(m - mx) + ls * expf(ms - mx);
      m = mx;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float mo = __shfl_xor_sync(0xffffffffu, m, o);
      const float lo = __shfl_xor_sync(0xffffffffu, l, o);
      const float mx = fmaxf(m, mo);
      if (mx != -INFINITY) {
        l = l * expf(m - mx) + lo * expf(mo - mx);
        m = mx;
      }
    }
    if (lane == 0) s_lse[warp] = m == -INFINITY ? INFINITY : m * kLog2e + log2f(l);
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kR; ++r) {
    const int j = j0 + r * kWThreads;
    float p = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) p += exp2f(xv[r][g] - s_lse[g]);
    if (j < n) w[j] = wv[r] + p;
  }
}

// ------------------------------------------------------------- eviction --

constexpr int kEThreads = 1024;
constexpr int kEWarps = kEThreads / 32;
constexpr int kBins = 2048;
constexpr int kCopies = 2;           // of the histogram (fewer collisions)
constexpr int kKeysCached = 49152;   // keys that fit shared memory beside it

// Weight -> unsigned order: NaN below everything, -0 equal to 0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

struct SelectSmem {
  uint32_t hist[kCopies][kBins];
  uint32_t warp_a[kEWarps], warp_b[kEWarps];
  uint32_t prefix, need;
  int newest;
};

// Exclusive sums over the warps of two per-warp counts (in place).
__device__ __forceinline__ void scan_warps(SelectSmem& sm) {
  __syncthreads();
  if (threadIdx.x < 32) {
    uint32_t a = sm.warp_a[threadIdx.x], b = sm.warp_b[threadIdx.x];
    const uint32_t a0 = a, b0 = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t ta = __shfl_up_sync(0xffffffffu, a, o);
      const uint32_t tb = __shfl_up_sync(0xffffffffu, b, o);
      if ((int)threadIdx.x >= o) {
        a += ta;
        b += tb;
      }
    }
    sm.warp_a[threadIdx.x] = a - a0;
    sm.warp_b[threadIdx.x] = b - b0;
  }
  __syncthreads();
}

// The rows that stay and the moves of one head of n > keep rows.  kFits: the
// keys are in shared memory.  One CTA a head leaves the walks bound by issue and
// by latency, so every walk takes kRows rows a thread at a time, all loaded
// before the first is used, and steps whose rows lie on one side of the cut
// count and list only what that side has: 52 -> 32 us at 128 heads of 32K rows
// (reading weights and positions once would take 5).
template <bool kFits>
__device__ __forceinline__ void select_rows(const EvictArgs& a, SelectSmem& sm, uint32_t* s_keys,
                                            int n) {
  constexpr int kRows = 8;
  const int bh = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float* w = a.weights + (size_t)bh * a.stride;
  int* pos = a.positions + (size_t)bh * a.stride;
  int newest = INT_MIN;
#pragma unroll kRows
  for (int j = tid; j < n; j += kEThreads) newest = max(newest, pos[j]);
  newest = __reduce_max_sync(0xffffffffu, newest);
  if (lane == 0) atomicMax(&sm.newest, newest);
  __syncthreads();
  const long long guard = (long long)sm.newest - a.recent;  // positions above stay
  // keys of rows j0, j0 + step, .. below `end`; 0 past it
  auto make_keys = [&](int j0, int step, int end, uint32_t (&key)[kRows]) {
    int p[kRows];
    float x[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int j = j0 + u * step;
      p[u] = j < end ? pos[j] : INT_MIN;
      x[u] = j < end ? w[j] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) key[u] = p[u] > guard ? 0xFFFFFFFFu : order_key(x[u]);
  };
  auto get_keys = [&](int j0, int step, int end, uint32_t (&key)[kRows]) {
    if constexpr (kFits) {
#pragma unroll
      for (int u = 0; u < kRows; ++u) key[u] = j0 + u * step < end ? s_keys[j0 + u * step] : 0u;
    } else {
      make_keys(j0, step, end, key);
    }
  };
  constexpr int kStep = kRows * kEThreads;
  if constexpr (kFits) {
    for (int j0 = tid; j0 < n; j0 += kStep) {
      uint32_t key[kRows];
      make_keys(j0, kEThreads, n, key);
#pragma unroll
      for (int u = 0; u < kRows; ++u)
        if (j0 + u * kEThreads < n) s_keys[j0 + u * kEThreads] = key[u];
    }
  }
  // key of the keep-th largest row, from the top bits down
  uint32_t prefix = 0, need = (uint32_t)a.keep;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10, shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
    for (int i = tid; i < kCopies * kBins; i += kEThreads) (&sm.hist[0][0])[i] = 0;
    __syncthreads();
    for (int j0 = tid; j0 < n; j0 += kStep) {
      uint32_t key[kRows];
      get_keys(j0, kEThreads, n, key);
#pragma unroll
      for (int u = 0; u < kRows; ++u)
        if (j0 + u * kEThreads < n && (pass == 0 || (key[u] >> (shift + bits)) == prefix))
          atomicAdd(&sm.hist[warp % kCopies][(key[u] >> shift) & ((1u << bits) - 1u)], 1u);
    }
    __syncthreads();
    // bin that holds the need-th largest: two bins a thread, from the top
    const int top = kBins - 1 - 2 * tid;
    uint32_t c0 = 0, c1 = 0;
#pragma unroll
    for (int k = 0; k < kCopies; ++k) {
      c0 += sm.hist[k][top];
      c1 += sm.hist[k][top - 1];
    }
    uint32_t before = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += t;
    }
    if (lane == 31) {
      sm.warp_a[warp] = before;
      sm.warp_b[warp] = 0;
    }
    scan_warps(sm);
    before += sm.warp_a[warp] - (c0 + c1);  // rows in larger bins
    if (before < need && need <= before + c0 + c1) {
      const bool first = need <= before + c0;
      sm.prefix = (prefix << bits) | (uint32_t)(first ? top : top - 1);
      sm.need = need - before - (first ? 0u : c0);
    }
    __syncthreads();
    prefix = sm.prefix;
    need = sm.need;
    __syncthreads();
  }
  // Rows above the threshold stay, and the first `need` equal to it.  Each
  // warp owns a run of rows.  One walk counts rows above and equal on both
  // sides of the cut: the equal rows that stay are the first ones, so their
  // numbers follow from a scan, and with them the ranks of the rows that move.
  const int span = (n + kEThreads - 1) / kEThreads * 32;
  const int w0 = min(warp * span, n), w1 = min(w0 + span, n);
  // all of a step's rows are the warp's, on one side of the cut
  auto one_side = [&](int j0) {
    return j0 + 32 * kRows <= w1 && (j0 + 32 * kRows <= a.keep || j0 >= a.keep);
  };
  uint32_t above_lo = 0, above_hi = 0, eq_lo = 0, eq_hi = 0;
  for (int j0 = w0; j0 < w1; j0 += 32 * kRows) {
    uint32_t key[kRows];
    get_keys(j0 + lane, 32, w1, key);
    if (one_side(j0)) {
      uint32_t up = 0, eq = 0;
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        up += key[u] > prefix;
        eq += key[u] == prefix;
      }
      if (j0 < a.keep) {
        above_lo += up;
        eq_lo += eq;
      } else {
        above_hi += up;
        eq_hi += eq;
      }
      continue;
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int j = j0 + 32 * u + lane;
      if (j >= w1) continue;
      const bool up = key[u] > prefix, eq = key[u] == prefix;
      if (j < a.keep) {
        above_lo += up;
        eq_lo += eq;
      } else {
        above_hi += up;
        eq_hi += eq;
      }
    }
  }
  above_lo = __reduce_add_sync(0xffffffffu, above_lo);
  above_hi = __reduce_add_sync(0xffffffffu, above_hi);
  eq_lo = __reduce_add_sync(0xffffffffu, eq_lo);
  eq_hi = __reduce_add_sync(0xffffffffu, eq_hi);
  if (lane == 0) {
    sm.warp_a[warp] = eq_lo + eq_hi;
    sm.warp_b[warp] = 0;
  }
  scan_warps(sm);
  uint32_t rank = sm.warp_a[warp];  // equal rows before this warp's
  __syncthreads();
  const uint32_t stay = min(need > rank ? need - rank : 0u, eq_lo + eq_hi);
  const uint32_t stay_lo = min(stay, eq_lo);
  const uint32_t rows_lo = (uint32_t)(min(w1, a.keep) - min(w0, a.keep));
  const uint32_t holes = rows_lo - above_lo - stay_lo;
  if (lane == 0) {
    sm.warp_a[warp] = holes;
    sm.warp_b[warp] = above_hi + stay - stay_lo;
  }
  scan_warps(sm);
  uint32_t hole_at = sm.warp_a[warp], mover_at = sm.warp_b[warp];
  if (warp == kEWarps - 1 && lane == 0) {
    a.counts[bh] = (int)(hole_at + holes);
    a.counts[gridDim.x + bh] = n;
    sm.need = hole_at + holes;
  }
  const uint32_t below = (1u << lane) - 1u;
  int2* mv = a.moves + (size_t)bh * a.max_moves;
  // only the warp that holds the last equal row that stays ranks equal rows
  const bool ranked = stay > 0 && stay < eq_lo + eq_hi;
  for (int j0 = w0; j0 < w1; j0 += 32 * kRows) {
    uint32_t key[kRows];
    get_keys(j0 + lane, 32, w1, key);
    if (!ranked && one_side(j0)) {
      const bool lo = j0 < a.keep;
      uint32_t at = lo ? hole_at : mover_at;
      int* list = lo ? &mv->y : &mv->x;
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const bool kept = key[u] > prefix || (stay > 0 && key[u] == prefix);
        const uint32_t m = __ballot_sync(0xffffffffu, kept != lo);
        if (kept != lo) list[2 * (size_t)(at + __popc(m & below))] = j0 + 32 * u + lane;
        at += __popc(m);
      }
      if (lo)
        hole_at = at;
      else
        mover_at = at;
      continue;
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int j = j0 + 32 * u + lane;
      const bool is_eq = j < w1 && key[u] == prefix;
      const uint32_t m_eq = __ballot_sync(0xffffffffu, is_eq);
      const bool kept =
          j < w1 && (key[u] > prefix || (is_eq && rank + __popc(m_eq & below) < need));
      rank += __popc(m_eq);
      const bool hole = j < w1 && !kept && j < a.keep, mover = kept && j >= a.keep;
      const uint32_t m_h = __ballot_sync(0xffffffffu, hole);
      const uint32_t m_m = __ballot_sync(0xffffffffu, mover);
      if (hole) mv[hole_at + __popc(m_h & below)].y = j;
      if (mover) mv[mover_at + __popc(m_m & below)].x = j;
      hole_at += __popc(m_h);
      mover_at += __popc(m_m);
    }
  }
  __syncthreads();
  const int total = (int)sm.need;
  // sources lie past the cut and targets before it: all loads may go first
  for (int i0 = tid; i0 < total; i0 += kStep) {
    int2 m[kRows];
    float wv[kRows];
    int pv[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u)
      m[u] = i0 + u * kEThreads < total ? mv[i0 + u * kEThreads] : make_int2(0, -1);
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      wv[u] = w[m[u].x];
      pv[u] = pos[m[u].x];
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u)
      if (m[u].y >= 0) {
        w[m[u].y] = wv[u];
        pos[m[u].y] = pv[u];
      }
  }
  __syncthreads();
  for (int j = a.keep + tid; j < n; j += kEThreads) w[j] = 0.f;
}

__global__ void __launch_bounds__(kEThreads) polar_evict_select_kernel(const EvictArgs a,
                                                                        int cached) {
  __shared__ SelectSmem sm;
  extern __shared__ uint32_t s_keys[];
  // the move kernel may be launched; it waits for this one
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int bh = blockIdx.x;
  int n = a.seq_lens[bh / a.Hkv];
  if (n < 0 || n > a.max_seq_len) {
    if (threadIdx.x == 0) atomicExch(a.status, 3);
    n = min(max(n, 0), a.max_seq_len);
  }
  if (n <= a.keep) {
    if (threadIdx.x == 0) {
      a.counts[bh] = 0;
      a.counts[gridDim.x + bh] = n;
    }
    return;
  }
  if (threadIdx.x == 0) sm.newest = INT_MIN;
  __syncthreads();
  if (n <= cached)
    select_rows<true>(a, sm, s_keys, n);
  else
    select_rows<false>(a, sm, s_keys, n);
}

// Grid (parts, B * Hkv): the listed rows of K and V, 16 bytes a thread, four
// pieces in flight.  Sources lie past the cut and targets before it, so loads
// may run ahead of stores.  Bound: HBM.  128 heads of 32K rows, d = 128 bf16,
// cut to a quarter: 146 us for 403 MB read and written, 5.5 TB/s, 82 % of the
// copy bandwidth (single rows of 256 bytes).  Eight pieces in flight: 229 us;
// 16 CTAs a head instead of 64: 170 us; streaming loads and stores: 150 us.
constexpr int kMThreads = 256, kMUnroll = 4;
__global__ void __launch_bounds__(kMThreads) polar_evict_move_kernel(const EvictArgs a) {
  const int bh = blockIdx.y, b = bh / a.Hkv, h = bh % a.Hkv;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int total = a.counts[bh], n = a.counts[gridDim.y + bh];
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) a.new_lens[b] = min(n, a.keep);
  const int vecs = a.row_bytes >> 4;            // 16-byte pieces of a row (a power of two)
  const int shift = 31 - __clz(vecs) + 1;       // of a K and a V row
  const int* table = a.block_table + (size_t)b * a.max_pages;
  const int2* mv = a.moves + (size_t)bh * a.max_moves;
  const int page = 1 << a.page_shift;
  const long long pieces = (long long)total << shift, step = (long long)gridDim.x * kMThreads;
  for (long long i0 = (long long)blockIdx.x * kMThreads + threadIdx.x; i0 < pieces;
       i0 += kMUnroll * step) {
    uint4 v[kMUnroll];
    uint4* to[kMUnroll];
#pragma unroll
    for (int u = 0; u < kMUnroll; ++u) {
      const long long i = i0 + u * step;
      to[u] = nullptr;
      if (i >= pieces) continue;
      const int2 m = mv[i >> shift];
      const int piece = (int)(i & ((1 << shift) - 1));
      const int p_from = table[m.x >> a.page_shift], p_to = table[m.y >> a.page_shift];
      if (p_from < 0 || p_from >= a.num_pages || p_to < 0 || p_to >= a.num_pages) {
        atomicExch(a.status, 3);
        continue;
      }
      const size_t from = ((size_t)p_from * a.Hkv + h) * page + (m.x & (page - 1));
      const size_t dst = ((size_t)p_to * a.Hkv + h) * page + (m.y & (page - 1));
      uint8_t* pool = static_cast<uint8_t*>(piece < vecs ? a.k_pages : a.v_pages);
      const size_t off = (size_t)(piece & (vecs - 1)) * 16;
      v[u] = *reinterpret_cast<const uint4*>(pool + from * a.row_bytes + off);
      to[u] = reinterpret_cast<uint4*>(pool + dst * a.row_bytes + off);
    }
#pragma unroll
    for (int u = 0; u < kMUnroll; ++u)
      if (to[u]) *to[u] = v[u];
  }
}

}  // namespace

cudaError_t launch_decode_weights(const WeightsArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.max_seq_len + kWRows - 1) / kWRows) * a.B * a.Hkv);
  cfg.blockDim = dim3(kWThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  switch (a.Hq / a.Hkv) {
    case 1: return cudaLaunchKernelEx(&cfg, polar_decode_weights_kernel<1>, a);
    case 2: return cudaLaunchKernelEx(&cfg, polar_decode_weights_kernel<2>, a);
    case 4: return cudaLaunchKernelEx(&cfg, polar_decode_weights_kernel<4>, a);
    default: return cudaLaunchKernelEx(&cfg, polar_decode_weights_kernel<8>, a);
  }
}

cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t s) {
  const int heads = a.B * a.Hkv;
  const int cached = a.max_seq_len < kKeysCached ? a.max_seq_len : kKeysCached;
  const int smem = cached * (int)sizeof(uint32_t);
  // the attribute belongs to the function, not to the call: one value for all,
  // or a call of another thread could lower it before this one's launch
  cudaError_t e = cudaFuncSetAttribute(polar_evict_select_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kKeysCached * (int)sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  polar_evict_select_kernel<<<heads, kEThreads, smem, s>>>(a, cached);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long pieces = (long long)a.max_moves * 2 * (a.row_bytes >> 4);
  const long long each = 2 * kMThreads * kMUnroll;  // pieces a CTA should have
  long long parts = (pieces + each - 1) / each;
  parts = parts < 1 ? 1 : (parts > 64 ? 64 : parts);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)parts, heads);
  cfg.blockDim = dim3(kMThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, polar_evict_move_kernel, a);
}

}  // namespace polar

using namespace polar;

// Rows one head may have to move: as many as both sides of the cut hold.
static int evict_max_moves(int max_seq_len, int keep) {
  const int past = max_seq_len > keep ? max_seq_len - keep : 0;
  return past < keep ? past : keep;
}

extern "C" {

size_t polar_cache_evict_workspace_bytes(int B, int Hkv, int max_seq_len, int keep) {
  if (B < 0 || Hkv < 1 || max_seq_len < 1 || keep < 1 || (long long)B * Hkv > 65535) return 0;
  const size_t heads = (size_t)B * Hkv;
  return heads * evict_max_moves(max_seq_len, keep) * sizeof(int2) + heads * 2 * sizeof(int);
}

int polar_cache_evict(void* k_pages, void* v_pages, const int* block_table,
                      const int* seq_lens, float* weights, int* positions, int* new_lens,
                      int B, int Hkv, int d, int page_size, int num_pages, int max_pages,
                      int max_seq_len, int stride, int dtype, int keep, int recent,
                      void* workspace, size_t workspace_bytes, void* stream) {
  if (B < 0 || Hkv < 1 || num_pages < 1 || max_pages < 1 || max_seq_len < 1 || keep < 1 ||
      recent < 0 || recent > keep || stride < max_seq_len)
    return POLAR_ERR_INVALID;
  if (dtype != POLAR_F32 && dtype != POLAR_BF16) return POLAR_ERR_UNSUPPORTED;
  if ((d != 64 && d != 128) || max_seq_len > (1 << 30) || (long long)B * Hkv > 65535)
    return POLAR_ERR_UNSUPPORTED;
  if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) != 0)
    return POLAR_ERR_UNSUPPORTED;
  if ((long long)max_pages * page_size < max_seq_len) return POLAR_ERR_INVALID;
  if (B == 0) return POLAR_OK;
  if (!k_pages || !v_pages || !block_table || !seq_lens || !weights || !positions || !new_lens)
    return POLAR_ERR_INVALID;
  const void* words[] = {block_table, seq_lens, weights, positions, new_lens};
  for (const void* p : words)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return POLAR_ERR_MISALIGNED;
  if (!aligned16(k_pages) || !aligned16(v_pages)) return POLAR_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < polar_cache_evict_workspace_bytes(B, Hkv, max_seq_len, keep))
    return POLAR_ERR_WORKSPACE;
  if (!aligned16(workspace)) return POLAR_ERR_MISALIGNED;
  int st = check_device(nullptr);
  if (st != POLAR_OK) return st;
  int* status = status_word();
  if (!status) return cuda_status("cudaGetSymbolAddress", cudaGetLastError());
  EvictArgs a{};
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.weights = weights;
  a.positions = positions;
  a.new_lens = new_lens;
  a.B = B;
  a.Hkv = Hkv;
  a.d = d;
  while ((1 << a.page_shift) < page_size) ++a.page_shift;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.max_seq_len = max_seq_len;
  a.stride = stride;
  a.row_bytes = d * (dtype == POLAR_BF16 ? 2 : 4);
  a.keep = keep;
  a.recent = recent;
  a.max_moves = evict_max_moves(max_seq_len, keep);
  a.moves = static_cast<int2*>(workspace);
  a.counts = reinterpret_cast<int*>(a.moves + (size_t)B * Hkv * a.max_moves);
  a.status = status;
  return cuda_status("cache eviction launch",
                     launch_cache_evict(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
