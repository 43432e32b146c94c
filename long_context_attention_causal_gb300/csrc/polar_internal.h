// Internal launch interface between the C ABI (polar_api.cu) and the kernel
// translation units.  Arguments here are already validated.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "polar_attn.h"

namespace polar {

struct FwdArgs {
  const void *q, *k, *v, *mem;
  const float* w_count;
  void* out;
  float* n_eff;
  float* conf;  // may be null
  int B, H, T, d;
  polar_consts_t c;
  int* status;  // device address of the library's status word
  float* stats = nullptr;  // optional [B, H, T, 2]: logsumexp, |a| (bf16 path)
  // Backward mode of the bf16 kernel (dout != null): instead of out, n_eff
  // and conf it writes dA, the per-row gradient record and the count * g
  // partials (polar_grad.cuh).
  const void* dout = nullptr;
  void* da = nullptr;
  float* grad_rows = nullptr;
  float* dw_part = nullptr;
};

struct DecodeArgs {
  const void *q, *k, *v, *mem;
  const float* w_count;
  void* out;
  float* n_eff;
  float* conf;  // may be null
  int B, H, Tkv, d;
  polar_consts_t c;
  int splits;      // >= 1
  int chunk;       // keys per split
  float* partials; // [B, H, splits, d + 4]
  const int* seq_lens = nullptr;  // [B] per-sequence key counts (paged), else Tkv
};

struct PagedArgs {
  DecodeArgs base;  // q, mem, out, n_eff, conf, w_count, partials; H = Hq, Tkv = max_seq_len
  const void *k_pages, *v_pages;  // [num_pages, Hkv, page, d]
  const int* block_table;         // [B, max_pages]
  int Hkv, page_shift, num_pages, max_pages;
  int* status;
  float* logits = nullptr;  // optional [B, Hq, Tkv]: every row's logit, log2 units
};

// weights[b][hkv][j] += sum over the group's heads of exp2(logit) / l, from the
// logits and the split records that a paged split kernel wrote.
struct WeightsArgs {
  const float *logits, *partials;
  const int* seq_lens;
  float* weights;
  int B, Hq, Hkv, d, splits, max_seq_len, stride;
};

struct EvictArgs {
  void *k_pages, *v_pages;
  const int *block_table, *seq_lens;
  float* weights;
  int *positions, *new_lens;
  int B, Hkv, d, page_shift, num_pages, max_pages, max_seq_len, stride, row_bytes;
  int keep, recent;
  int* counts;   // [B * Hkv] rows to move, then [B * Hkv] lengths
  int2* moves;   // [B * Hkv][max_moves] (from, to)
  int max_moves;
  int* status;
};

// How the decayed linear recurrence is spread over CTAs: the tiles of all
// (b, h), head by head, in `parts` runs of `per` tiles.  A head that a run
// boundary cuts is continued from a state handed over (LinearStateArgs).
constexpr int kLinearTile = 128;
struct LinearSplit {
  int tiles;  // of one head
  int per, parts;
  bool cut;   // some boundary lies inside a head
  int sms;
};

// One application of the recurrence over all (b, h):
//   forward: out_t = s * (sum_{u <= t} g^(t-u) (x_t . y_u) z_u + g^(t+1) M x_t)
//   reverse: out_t = s * sum_{u >= t} g^(u-t) (x_t . y_u) z_u + g^(L-1-t) M x_t
// with M the state at the sequence's start (forward) or end (reverse).  The
// stored states are [z dim][y dim], transposed if state_t.
struct LinearArgs {
  const void *x, *y, *z;  // [B, H, T, d]
  void* out;              // [B, H, T, d]
  const float* log_decay;
  const int* lengths;     // may be null
  int B, H, T, d;
  float scale;
  bool reverse, state_t;
  LinearSplit split;
  const float* init;      // [B, H, d, d] state at the start (end), or null (zero)
  const float* cuts;      // states at the cuts (LinearStateArgs), null without cuts
  float* final_state;     // [B, H, d, d] state at the other end, or null (not with state_t)
  int* status;
  bool exact;             // the caller asks for the state at the other end
  bool chained = false;   // follows a kernel of the same call (programmatic launch)
};

// States at the cuts.  Forward: slot i is the state at the end of run i,
// reverse: at its start.  The state kernels sum each run's own part of the
// cut head; the scan joins them in place, from init.
struct LinearStateArgs {
  const void *y, *z;
  const float* log_decay;
  const int* lengths;
  int B, H, T, d;
  float scale;  // factor of the state's products
  bool reverse;
  LinearSplit split;
  const float* init;  // may be null
  float* cuts;        // [parts][d][d]
  int* status;
  float* init_copy;   // [B, H, d, d]: where the scan copies init, or null
  bool exact;         // the caller asks for the final state
};
// Each launch takes n applications that differ in tensors, states, direction
// and scale only: states and scans 1 or 2, outputs in fp32 1 to 3.
// fp32 on the FP32 pipes.
cudaError_t launch_linear_states(const LinearStateArgs* a, int n, cudaStream_t s);
cudaError_t launch_linear_scan(const LinearStateArgs* a, int n, cudaStream_t s);
cudaError_t launch_linear_out(const LinearArgs* a, int n, cudaStream_t s);
// bf16 on the tensor cores: outputs 1, or 2 of one direction.  maps: x, y, z,
// out of each / y, z of each (128-row boxes).
cudaError_t launch_linear_out_tc(const LinearArgs* a, int n, const CUtensorMap* maps,
                                 cudaStream_t s);
cudaError_t launch_linear_states_tc(const LinearStateArgs* a, int n, const CUtensorMap* maps,
                                    cudaStream_t s);
// final = init (or zero) for prompts without tokens.
cudaError_t launch_linear_copy_state(const float* init, float* final_state, size_t n,
                                     cudaStream_t s);

struct LinearStepArgs {
  float* state;
  const void *q, *k, *v;
  const float* log_decay;
  void* mem;
  int B, H, d;
  float scale;
};
cudaError_t launch_linear_step(const LinearStepArgs& a, int dtype, cudaStream_t s);

cudaError_t launch_decode_weights(const WeightsArgs& a, cudaStream_t s);
cudaError_t launch_cache_evict(const EvictArgs& a, cudaStream_t s);

struct MemoryArgs {
  float* state;                   // [B, H, d, d] fp32, updated in place
  const void *q, *k, *v;          // [B, H, T, d]
  const float *alpha, *beta;      // [B, H, T]
  void* mem;                      // [B, H, T, d]
  int B, H, T, d;
  float eps;
};

struct BwdArgs {
  const void *q, *k, *v, *dout;  // [B, H, T, d] of dtype
  const float* w_count;          // [H, d]
  float *dq, *dk, *dv;           // [B, H, T, d] fp32
  float* dw;                     // [H, d] fp32
  int B, H, T, d;
  polar_consts_t c;
  float* workspace;              // bwd_workspace_floats(...) floats
  int* status = nullptr;         // device status word (tensor-core path)
};

// Backward of the causal prefill, fp32 inputs (FP32 pipes).
size_t bwd_workspace_floats(int B, int H, int T, int d);
cudaError_t launch_bwd(const BwdArgs& a, int dtype, cudaStream_t s);

// Backward of the causal prefill, bf16 inputs (tensor cores).  The forward
// kernel in backward mode fills the workspace (dA, row records, count * g
// partials); the tile kernels then write dQ, dK, dV and dw.
struct BwdTcLayout {
  void* da;        // [BH, T, d] bf16
  float* rows;     // row records, pair blocks (polar_grad.cuh)
  float* dw_part;  // [BH, ceil(T / 32), d]
  size_t bytes;
};
BwdTcLayout bwd_tc_layout(void* workspace, int B, int H, int T, int d);
// Row pass of the backward from the forward's saved outputs (bf16): fills
// the same workspace as the forward kernel's backward mode.
struct SavedRows {
  const void *out, *mem;  // [B, H, T, d] bf16
  const float *n_eff, *conf, *stats;
};
cudaError_t launch_bwd_rows_saved(const BwdArgs& a, const SavedRows& sv, const BwdTcLayout& w,
                                  cudaStream_t s);
// maps: q, k, v, dA (128-row boxes)
cudaError_t launch_bwd_tc(const BwdArgs& a, const BwdTcLayout& w, const CUtensorMap* maps,
                          cudaStream_t s);

// Gated-delta memory steps over T tokens, state updated in place.
cudaError_t launch_memory_step(const MemoryArgs& a, int dtype, cudaStream_t s);

// Paged, grouped-query split kernel (combine: launch_decode_combine).
cudaError_t launch_decode_paged_split(const PagedArgs& a, int dtype, cudaStream_t s);
// The same split on the tensor cores (bf16; cache rows num_pages * Hkv * page
// addressable as int32).  mk, mv: 2-D maps [rows, d] with a {64, min(page,
// kPagedTcStageKeys)} box and 128-byte swizzle.
constexpr int kPagedTcStageKeys = 64;
cudaError_t launch_decode_paged_tc(const PagedArgs& a, const CUtensorMap& mk,
                                   const CUtensorMap& mv, cudaStream_t s);

// Heads per group in the multi-wave CTA orders of the tensor-core kernels
// (each group's streamed operands kept in L2): the largest divisor of BH
// whose heads' per_head_bytes fit a third of the current device's L2 (a
// short search below that bound; a near miss keeps the bound), at least 1.
int l2_head_group(int BH, double per_head_bytes);

// bf16 causal prefill on the tensor cores (tcgen05 + TMEM + TMA).
// map_o: the output [BH, T, d] with the same 128-row boxes (the forward
// epilogue's TMA store; unused in backward mode).
cudaError_t launch_fwd_tc(const FwdArgs& a, const CUtensorMap& map_q,
                          const CUtensorMap& map_k, const CUtensorMap& map_v,
                          const CUtensorMap& map_o, cudaStream_t s);

// fp32 causal prefill on the FP32 pipes.
cudaError_t launch_fwd_f32(const FwdArgs& a, cudaStream_t s);

// Split-KV decode: partial states per (b, h, split), then the combine.
cudaError_t launch_decode_split(const DecodeArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_decode_combine(const DecodeArgs& a, int dtype, cudaStream_t s);

// Host helpers shared by the entry points (defined in polar_api.cu).
bool aligned16(const void* p);
bool consts_ok(const polar_consts_t& c);
polar_consts_t defaults();
int check_device(int* num_sms);
int auto_splits(int BH, int Tkv, int num_sms);
bool decode_sizes_ok(int B, int H, int Tkv, int d);
void set_last_error(const char* msg);
int cuda_status(const char* what, cudaError_t e);
int* status_word();  // device address of the current device's status word, or null
// 3-D map over a [BH, T, d] bf16 tensor with a {64, rows, 1} box and 128-byte
// swizzle; out-of-range rows read as zeros.
bool make_map(CUtensorMap* map, const void* base, int BH, int T, int d, int rows = 128);

// Bounded-wait self test (one thread, a barrier nothing completes).
cudaError_t launch_selftest_wait(long long limit_cycles, int* status, cudaStream_t s);

}  // namespace polar
