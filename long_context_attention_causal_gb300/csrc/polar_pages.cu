// Pages of a paged cache handed out and taken back on the device: block
// tables, slot maps, positions and packed offsets from sequence lengths.
// (No counterpart on the pages: a service next to the paged decode.)
//
// With P rows a page, a sequence of len rows that gets `new` more needs
//   need_b = ceil((len_b + new_b) / P) - ceil(len_b / P)
// pages; it gets them from the top of a stack of free pages, in the order of
// the sequences, if its own and all earlier needs fit what the stack holds.
// Both sums over b are scans.  The work is a few bytes a sequence and a token
// and is bound by launch and load latency, so a small call is one launch of
// one block, which scans and then fills; a large one adds a grid that fills
// (a programmatic launch, its tokens found by a search in the offsets).
#include <algorithm>
#include <climits>
#include <cstdint>

#include "polar_device.cuh"
#include "polar_internal.h"
#include "polar_span.h"

namespace polar {

namespace {

constexpr int kScan = 1024;  // threads of the scan
constexpr int kFill = 256;

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

__device__ __forceinline__ long long warp_scan(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Inclusive scan over the block, `total` its last value.
__device__ __forceinline__ long long block_scan(long long v, long long* part, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long own = warp_scan(v, lane);
  __syncthreads();  // the previous scan's reads of part are over
  if (lane == 31) part[warp] = own;
  __syncthreads();
  if (warp == 0) part[lane] = warp_scan(part[lane], lane);
  __syncthreads();
  total = part[31];
  return own + (warp ? part[warp - 1] : 0);
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

__device__ __forceinline__ void fill_token(const PagesArgs& a, int t, int total) {
  int slot = -1, pos = 0;
  if (t < total) {
    const int b = find(a.B, t, [&](int x) { return a.cu[x]; });
    const int2 plan = a.plan[b];
    if (plan.x >= 0) {
      pos = plan.x + t - a.cu[b];
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

__device__ __forceinline__ void fill_freed(const PagesArgs& a, int i) {
  const int b = find(a.B, i, [&](int x) { return a.plan[x].y; });
  const int2 plan = a.plan[b];
  const int at = a.plan[a.B].y + i;
  int id = a.table[(size_t)b * a.max_pages + plan.x + i - plan.y];
  if (id < 0 || id >= a.num_pages) {
    flag(a);
    id = -1;
  }
  if (at < a.capacity) a.free_pages[at] = id;
}

template <bool kExtend, bool kAlone>
__global__ void __launch_bounds__(kScan) pages_scan_kernel(const PagesArgs a) {
  __shared__ long long part[32];
  if (!kAlone) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int mask = (1 << a.shift) - 1;
  int count = *a.count;
  if (count < 0 || count > a.capacity) {
    if (threadIdx.x == 0) flag(a);
    count = count < 0 ? 0 : a.capacity;
  }
  long long tokens = 0, pages = 0, taken = 0;  // sums over the sequences so far
  if (kExtend && threadIdx.x == 0) a.cu[0] = 0;
  for (int b0 = 0; b0 < a.B; b0 += kScan) {
    const int b = b0 + (int)threadIdx.x;
    const bool in = b < a.B;
    int len = in ? a.lens[b] : 0, next = in ? a.next[b] : 0;
    const long long most = (long long)a.max_pages << a.shift;
    const bool bad = len < 0 || len > most || next < 0 || (!kExtend && next > len);
    if (bad) {
      flag(a);
      next = kExtend ? 0 : len;  // such a sequence is left as it is
    }
    long long total;
    if (kExtend) {
      const long long end = tokens + block_scan(next, part, total);
      const bool fits = !bad && (long long)len + next <= most && end <= a.tokens;
      if (!bad && !fits) flag(a);
      if (in) a.cu[b + 1] = (int)min(end, (long long)a.tokens);
      tokens += total;
      const long long need = fits ? ((len + (long long)next + mask) >> a.shift) -
                                        (((long long)len + mask) >> a.shift)
                                  : 0;
      const long long upto = pages + block_scan(need, part, total);
      const bool ok = fits && (need == 0 || upto <= count);
      pages += total;
      if (in) {
        a.plan[b] = make_int2(ok ? len : -1, (int)(count - 1 - (upto - need)));
        a.lens_out[b] = ok ? len + next : len;
      }
      block_scan(ok ? need : 0, part, total);
      taken += total;
    } else {
      const long long keep = ((long long)next + mask) >> a.shift;
      const long long give = bad ? 0 : (((long long)len + mask) >> a.shift) - keep;
      const long long upto = pages + block_scan(give, part, total);
      pages += total;
      if (in) {
        a.plan[b] = make_int2((int)keep, (int)(upto - give));
        a.lens_out[b] = next;
      }
    }
  }
  const int fill = kExtend ? (int)min(tokens, (long long)a.tokens) : (int)pages;
  if (threadIdx.x == 0) {
    a.plan[a.B] = make_int2(fill, count);
    if (!kExtend && count + pages > a.capacity) flag(a);
    *a.count_out = kExtend ? (int)(count - taken)
                           : (int)min(count + pages, (long long)a.capacity);
  }
  if (kAlone) {
    __syncthreads();  // the block's own plan and offsets
    if (kExtend) {
      for (int t = threadIdx.x; t < a.tokens; t += kScan) fill_token(a, t, fill);
    } else {
      for (int i = threadIdx.x; i < fill; i += kScan) fill_freed(a, i);
    }
  }
}

template <bool kExtend>
__global__ void __launch_bounds__(kFill) pages_fill_kernel(const PagesArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int total = a.plan[a.B].x;
  const int end = kExtend ? a.tokens : total;
  const long long step = (long long)gridDim.x * kFill;
  for (long long i = (long long)blockIdx.x * kFill + threadIdx.x; i < end; i += step) {
    if (kExtend) fill_token(a, (int)i, total);
    else fill_freed(a, (int)i);
  }
}

template <bool kExtend>
cudaError_t launch(const PagesArgs& a, long long items, int sms, cudaStream_t s) {
  // One block fills about 1000 items a microsecond; a second launch costs
  // less from a few thousand on.
  if (items <= 4096) {
    pages_scan_kernel<kExtend, true><<<1, kScan, 0, s>>>(a);
    return cudaGetLastError();
  }
  pages_scan_kernel<kExtend, false><<<1, kScan, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min((items + kFill - 1) / kFill, 8LL * sms));
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
  if (!a.table || !a.lens || !a.next || !a.free_pages || !a.count || !a.lens_out || !a.count_out)
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
