// Pages of a paged cache handed out and taken back on the device: block
// tables, slot maps, positions and packed offsets from sequence lengths.
// (No counterpart on the pages: a service next to the paged decode.)
//
// With P rows a page, a sequence of len rows that gets `new` more needs
//   need_b = ceil((len_b + new_b) / P) - ceil(len_b / P)
// pages; it gets them from the top of a stack of free pages, in the order of
// the sequences, if its own and all earlier needs fit what the stack holds.
// Both sums over b are scans, made together.  The work is a few bytes a sequence
// and a token and is bound by launch and load latency, so a small call is one
// launch of one block, which scans and then fills, its offsets in shared memory;
// a large one adds a grid that fills (a programmatic launch; a token's sequence
// is found by a search in the offsets).  Measured: release and extension of 256
// sequences by a token each 10 us on the device, of 96 by 1 to 8000 tokens 12 us.
#include <algorithm>
#include <climits>
#include <cstdint>

#include "polar_device.cuh"
#include "polar_internal.h"
#include "polar_span.h"

namespace polar {

namespace {

constexpr int kScan = 1024;  // threads of the scan, at most
constexpr int kFill = 256;
constexpr int kHeld = 2048;  // sequences whose offsets fit shared memory

struct PagesArgs {
  int* table;        // [B, max_pages]
  const int* lens;   // [B] rows held
  const int* next;   // [B] extend: new tokens; release: rows to keep
  int* free_pages;   // [capacity] stack
  const int* count;  // [1] pages on the stack
  int *lens_out, *count_out;
  int *cu, *positions, *slots;  // extend: [B + 1], [tokens], [tokens]
  int2* plan;  // [B + 1]: extend (first new row or -1, stack index of the first
               // new page); release (first table entry, entries before); [B]: the
               // total of what is filled, and the stack's height before
  int B, max_pages, shift, num_pages, capacity, tokens;
  int* status;
};

struct Two {
  long long x, y;
};

// Inclusive scans of x and y over the block, `total` their last values.
__device__ __forceinline__ Two block_scan(Two v, Two* part, Two& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
    if (lane >= o) v.x += x, v.y += y;
  }
  __syncthreads();  // the previous scan's reads of part are over
  if (lane == 31) part[warp] = v;
  __syncthreads();
  total = Two{0, 0};
  Two before{0, 0};
  for (int w = 0; w < warps; ++w) {
    if (w == warp) before = total;
    total.x += part[w].x, total.y += part[w].y;
  }
  return Two{before.x + v.x, before.y + v.y};
}

__device__ __forceinline__ void flag(const PagesArgs& a) { atomicExch(a.status, 3); }

// Sequence whose part of [0, total) holds i: the last b with start(b) <= i.
template <typename F>
__device__ __forceinline__ int find(int B, int i, F start) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start(mid) <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// cu, plan: the arguments' arrays, or copies of them in shared memory
__device__ __forceinline__ void fill_token(const PagesArgs& a, const int* cu, const int2* plans,
                                           int t, int total) {
  int slot = -1, pos = 0;
  if (t < total) {
    const int b = find(a.B, t, [&](int x) { return cu[x]; });
    const int2 plan = plans[b];
    if (plan.x >= 0) {
      pos = plan.x + (t - cu[b]);
      const int page = pos >> a.shift, mask = (1 << a.shift) - 1;
      const int held = (plan.x + mask) >> a.shift;  // pages before this call
      int id;
      if (page < held) {
        id = a.table[(size_t)b * a.max_pages + page];
      } else {
        id = a.free_pages[plan.y - (page - held)];
        // a new page's first row is a new token's
        if ((pos & mask) == 0) a.table[(size_t)b * a.max_pages + page] = id;
      }
      if (id >= 0 && id < a.num_pages) {
        slot = (id << a.shift) + (pos & mask);
      } else {
        flag(a);
      }
    }
  }
  a.positions[t] = pos;
  a.slots[t] = slot;
}

__device__ __forceinline__ void fill_freed(const PagesArgs& a, const int2* plans, int top, int i) {
  const int b = find(a.B, i, [&](int x) { return plans[x].y; });
  const int2 plan = plans[b];
  int id = a.table[(size_t)b * a.max_pages + plan.x + i - plan.y];
  if (id < 0 || id >= a.num_pages) {
    flag(a);
    id = -1;
  }
  const long long at = (long long)top + i;  // (both near 2^31 at most)
  if (at < a.capacity) a.free_pages[at] = id;
}

// kAlone: the block fills too (its sequences fit kHeld)
template <bool kExtend, bool kAlone>
__global__ void __launch_bounds__(kScan) pages_scan_kernel(const PagesArgs a) {
  __shared__ Two part[32];
  __shared__ int cu_held[kAlone && kExtend ? kHeld : 1];
  __shared__ int2 plan_held[kAlone ? kHeld : 1];
  if (!kAlone) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int mask = (1 << a.shift) - 1;
  int count = *a.count;
  if (count < 0 || count > a.capacity) {
    if (threadIdx.x == 0) flag(a);
    count = count < 0 ? 0 : a.capacity;
  }
  auto pages_of = [&](long long rows) { return (rows + mask) >> a.shift; };
  Two run{0, 0};        // extend: tokens, pages; release: -, pages of the sequences so far
  long long taken = 0;  // pages of this thread's sequences that got them
  if (kExtend && threadIdx.x == 0) a.cu[0] = 0;
  for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
    const int b = b0 + (int)threadIdx.x;
    const bool in = b < a.B;
    int len = in ? a.lens[b] : 0, next = in ? a.next[b] : 0;
    const long long most = (long long)a.max_pages << a.shift;
    const bool bad = len < 0 || len > most || next < 0 || (!kExtend && next > len);
    if (bad) {
      flag(a);
      next = kExtend ? 0 : len;  // such a sequence is left as it is
    }
    Two total;
    if (kExtend) {
      const bool room = !bad && (long long)len + next <= most;
      long long need = room ? pages_of((long long)len + next) - pages_of(len) : 0;
      Two upto = block_scan(Two{next, need}, part, total);
      upto.x += run.x;
      bool fits = room && upto.x <= a.tokens;
      if (run.x + total.x > a.tokens) {
        // sequences past max_tokens need no pages: their sums once more
        if (!fits) need = 0;
        Two again;
        upto.y = block_scan(Two{0, need}, part, again).y;
        total.y = again.y;
      }
      upto.y += run.y;
      if (!bad && !fits) flag(a);
      const bool ok = fits && (need == 0 || upto.y <= count);
      if (ok) taken += need;
      if (in) {
        const int end = (int)min(upto.x, (long long)a.tokens);
        const int2 plan = make_int2(ok ? len : -1, (int)(count - 1 - (upto.y - need)));
        a.cu[b + 1] = end;
        a.lens_out[b] = ok ? len + next : len;
        if (kAlone) {
          plan_held[b] = plan;
          if (b + 1 < a.B) cu_held[b + 1] = end;
          if (b == 0) cu_held[0] = 0;
        } else {
          a.plan[b] = plan;
        }
      }
    } else {
      const long long keep = pages_of(next), give = bad ? 0 : pages_of(len) - keep;
      const long long upto = run.y + block_scan(Two{0, give}, part, total).y;
      if (in) {
        const int2 plan = make_int2((int)keep, (int)(upto - give));
        a.lens_out[b] = next;
        if (kAlone) plan_held[b] = plan;
        else a.plan[b] = plan;
      }
    }
    run.x += total.x, run.y += total.y;
  }
  if (kExtend) {
    Two total;
    block_scan(Two{0, taken}, part, total);
    taken = total.y;
  }
  const int fill = kExtend ? (int)min(run.x, (long long)a.tokens) : (int)run.y;
  if (threadIdx.x == 0) {
    if (!kAlone) a.plan[a.B] = make_int2(fill, count);
    if (!kExtend && count + run.y > a.capacity) flag(a);
    *a.count_out =
        kExtend ? (int)(count - taken) : (int)min(count + run.y, (long long)a.capacity);
  }
  if (kAlone) {
    __syncthreads();  // plans and offsets
    if (kExtend) {
      for (int t = threadIdx.x; t < a.tokens; t += blockDim.x)
        fill_token(a, cu_held, plan_held, t, fill);
    } else {
      for (int i = threadIdx.x; i < fill; i += blockDim.x) fill_freed(a, plan_held, count, i);
    }
  }
}

template <bool kExtend>
__global__ void __launch_bounds__(kFill) pages_fill_kernel(const PagesArgs a) {
  __shared__ int cu_held[kExtend ? kHeld : 1];
  __shared__ int2 plan_held[kHeld];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 all = a.plan[a.B];
  const int total = all.x, end = kExtend ? a.tokens : total;
  const bool held = a.B <= kHeld;
  if (held) {
    for (int b = threadIdx.x; b < a.B; b += kFill) {
      plan_held[b] = a.plan[b];
      if (kExtend) cu_held[b] = a.cu[b];
    }
    __syncthreads();
  }
  const int2* plan = held ? plan_held : a.plan;
  const int* cu = held && kExtend ? cu_held : a.cu;
  const long long step = (long long)gridDim.x * kFill;
  for (long long i = (long long)blockIdx.x * kFill + threadIdx.x; i < end; i += step) {
    if (kExtend) fill_token(a, cu, plan, (int)i, total);
    else fill_freed(a, plan, all.y, (int)i);
  }
}

template <bool kExtend>
cudaError_t launch(const PagesArgs& a, long long items, int sms, cudaStream_t s) {
  // One block fills some thousand items in the time of a second launch (and
  // releases are a few of the entries that `items` allows for).
  const bool alone = a.B <= kHeld && items <= (kExtend ? 4096 : 16384);
  const long long width = alone ? std::max((long long)a.B, std::min(items, (long long)kScan)) : a.B;
  const int threads = (int)std::min((width + 31) / 32 * 32, (long long)kScan);
  if (alone) {
    pages_scan_kernel<kExtend, true><<<1, threads, 0, s>>>(a);
    return cudaGetLastError();
  }
  pages_scan_kernel<kExtend, false><<<1, threads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || items == 0) return e;  // (no tokens: nothing to fill)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min((items + kFill - 1) / kFill, 6LL * sms));
  cfg.blockDim = dim3(kFill);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pages_fill_kernel<kExtend>, a);
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

size_t plan_bytes(int B) { return ((size_t)B + 1) * sizeof(int2); }

// Checks that both calls share.  POLAR_OK with *shift set, or the refusal.
int check(const PagesArgs& a, int page_size, const void* workspace, size_t workspace_bytes,
          int* shift) {
  if (a.B < 0 || a.max_pages < 1 || a.num_pages < 1 || a.capacity < 0 || a.tokens < 0)
    return POLAR_ERR_INVALID;
  if (page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) != 0)
    return POLAR_ERR_UNSUPPORTED;
  if ((long long)a.num_pages * page_size > INT_MAX || (long long)a.max_pages * page_size > INT_MAX ||
      (long long)a.B * a.max_pages > INT_MAX || a.B > (1 << 24))
    return POLAR_ERR_UNSUPPORTED;
  *shift = 0;
  while ((1 << *shift) < page_size) ++*shift;
  if (a.B == 0) return POLAR_OK;
  if (!a.table || !a.lens || !a.next || (a.capacity && !a.free_pages) || !a.count || !a.lens_out ||
      !a.count_out)
    return POLAR_ERR_INVALID;
  if (!aligned4(a.table) || !aligned4(a.lens) || !aligned4(a.next) || !aligned4(a.free_pages) ||
      !aligned4(a.count) || !aligned4(a.lens_out) || !aligned4(a.count_out) || !aligned4(a.cu) ||
      !aligned4(a.positions) || !aligned4(a.slots))
    return POLAR_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < plan_bytes(a.B)) return POLAR_ERR_WORKSPACE;
  if (!aligned16(workspace)) return POLAR_ERR_MISALIGNED;
  return POLAR_OK;
}

// The written tensors must not meet others; lens_out and count_out may be
// lens and count.
bool clash(const PagesArgs& a) {
  const size_t n = (size_t)a.B * 4;
  const Strided outs[] = {span(a.table, n * a.max_pages), span(a.free_pages, (size_t)a.capacity * 4),
                          span(a.lens_out, n),            span(a.count_out, 4),
                          span(a.cu, n + 4),              span(a.positions, (size_t)a.tokens * 4),
                          span(a.slots, (size_t)a.tokens * 4), span(a.plan, plan_bytes(a.B))};
  const Strided ins[] = {span(a.lens, n), span(a.next, n), span(a.count, 4)};
  for (const Strided& o : outs) {
    for (const Strided& other : outs)
      if (&other != &o && meet(o, other)) return true;
    for (const Strided& i : ins) {
      const bool same = (o.p == a.lens_out && i.p == a.lens) || (o.p == a.count_out && i.p == a.count);
      if (!same && meet(o, i)) return true;
    }
  }
  return false;
}

}  // namespace

}  // namespace polar

using namespace polar;

extern "C" {

size_t polar_pages_workspace_bytes(int B) { return B >= 0 ? plan_bytes(B) : 0; }

int polar_pages_extend(int* block_table, const int* seq_lens, const int* new_tokens,
                       const int* free_pages, const int* free_count, int* lens_out,
                       int* count_out, int* cu_seqlens, int* positions, int* slots, int B,
                       int max_pages, int page_size, int num_pages, int free_capacity,
                       int max_tokens, void* workspace, size_t workspace_bytes, void* stream) {
  PagesArgs a{block_table, seq_lens,   new_tokens, const_cast<int*>(free_pages), free_count,
              lens_out,    count_out,  cu_seqlens, positions,                    slots,
              static_cast<int2*>(workspace), B, max_pages, 0, num_pages, free_capacity, max_tokens,
              nullptr};
  int st = check(a, page_size, workspace, workspace_bytes, &a.shift);
  if (st != POLAR_OK || B == 0) return st;
  if (!cu_seqlens || (max_tokens > 0 && (!positions || !slots))) return POLAR_ERR_INVALID;
  if (clash(a)) return POLAR_ERR_INVALID;
  int sms = 0;
  st = check_device(&sms);
  if (st != POLAR_OK) return st;
  a.status = status_word();
  if (!a.status) return cuda_status("cudaGetSymbolAddress", cudaGetLastError());
  return cuda_status("page extension launch",
                     launch<true>(a, max_tokens, sms, static_cast<cudaStream_t>(stream)));
}

int polar_pages_release(const int* block_table, const int* seq_lens, const int* keep_lens,
                        int* free_pages, const int* free_count, int* lens_out, int* count_out,
                        int B, int max_pages, int page_size, int num_pages, int free_capacity,
                        void* workspace, size_t workspace_bytes, void* stream) {
  PagesArgs a{const_cast<int*>(block_table), seq_lens, keep_lens, free_pages, free_count, lens_out,
              count_out, nullptr, nullptr, nullptr, static_cast<int2*>(workspace), B, max_pages, 0,
              num_pages, free_capacity, 0, nullptr};
  int st = check(a, page_size, workspace, workspace_bytes, &a.shift);
  if (st != POLAR_OK || B == 0) return st;
  if (clash(a)) return POLAR_ERR_INVALID;
  int sms = 0;
  st = check_device(&sms);
  if (st != POLAR_OK) return st;
  a.status = status_word();
  if (!a.status) return cuda_status("cudaGetSymbolAddress", cudaGetLastError());
  return cuda_status("page release launch",
                     launch<false>(a, (long long)B * max_pages, sms,
                                   static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
