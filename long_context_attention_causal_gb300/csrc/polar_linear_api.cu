// C ABI of the decayed linear attention: argument validation, the split of a
// sequence into segments, and the launches.  The contract of every entry
// point is in include/polar_attn.h, the mathematics in polar_linear.cu.
#include <climits>
#include <cmath>
#include <cstdint>

#include "polar_device.cuh"
#include "polar_internal.h"

namespace polar {

namespace {

struct Segments {
  int nseg, seg_tokens;
};

// Segments per sequence.  One segment per head needs no state pass but leaves
// SMs idle when heads are few; with n > 1 every CTA walks 1/n of the tiles at
// one and a half times the cost a tile (the state pass reads y and z once
// more), plus a tile's time for the start and about four for the two extra
// launches.  The count with the least cost over whole waves is taken.
Segments segments(int BH, int T, int d, int dtype, int sms) {
  const int tiles = (T + kLinearTile - 1) / kLinearTile;
  if (tiles < 1) return {0, kLinearTile};
  const long long per_seg = dtype == POLAR_BF16 ? 1 : d / 32;  // CTAs per segment
  const long long slots = dtype == POLAR_BF16 ? sms : 2ll * sms;
  long long best = 1;
  double best_cost = 1e300;
  for (long long n = 1; n <= tiles && n <= 1024; ++n) {
    const long long per = (tiles + n - 1) / n;
    const long long real = (tiles + per - 1) / per;
    const double waves = (double)((BH * real * per_seg + slots - 1) / slots);
    const double cost = n == 1 ? waves * (per + 1) : waves * 1.5 * (per + 1) + 4;
    if (cost < best_cost - 1e-9) {
      best_cost = cost;
      best = n;
    }
  }
  const int per = (int)((tiles + best - 1) / best);
  return {(tiles + per - 1) / per, per * kLinearTile};
}

bool sizes_ok(int B, int H, int T, int d, int dtype) {
  return B >= 0 && H >= 0 && T >= 0 && (d == 64 || d == 128) &&
         (dtype == POLAR_F32 || dtype == POLAR_BF16) && (long long)B * H <= (1 << 20) &&
         T <= (1 << 28);
}

int check_sizes(int B, int H, int T, int d, int dtype, float scale) {
  if (B < 0 || H < 0 || T < 0 || !std::isfinite(scale)) return POLAR_ERR_INVALID;
  return sizes_ok(B, H, T, d, dtype) ? POLAR_OK : POLAR_ERR_UNSUPPORTED;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

size_t state_bytes(int B, int H, int T, int d, int dtype) {
  int sms = 0;
  if (check_device(&sms) != POLAR_OK) sms = 148;
  const Segments g = segments(B * H, T, d, dtype, sms);
  return (size_t)B * H * g.nseg * d * d * sizeof(float);
}

// bf16 runs on the tensor cores, fp32 on the FP32 pipes.
int run_states(const LinearStateArgs& a, int dtype, cudaStream_t s) {
  int st;
  if (dtype == POLAR_BF16) {
    CUtensorMap maps[2];
    if (!make_map(&maps[0], a.y, a.B * a.H, a.T, a.d) ||
        !make_map(&maps[1], a.z, a.B * a.H, a.T, a.d))
      return POLAR_ERR_CUDA;
    st = cuda_status("linear state launch", launch_linear_states_tc(a, maps, s));
  } else {
    st = cuda_status("linear state launch", launch_linear_states(a, s));
  }
  if (st != POLAR_OK) return st;
  return cuda_status("linear scan launch", launch_linear_scan(a, s));
}

int run_out(const LinearArgs& a, int dtype, cudaStream_t s) {
  if (dtype != POLAR_BF16) return cuda_status("linear output launch", launch_linear_out(a, s));
  CUtensorMap maps[4];
  const void* bases[4] = {a.x, a.y, a.z, a.out};
  for (int i = 0; i < 4; ++i)
    if (!make_map(&maps[i], bases[i], a.B * a.H, a.T, a.d)) return POLAR_ERR_CUDA;
  return cuda_status("linear output launch", launch_linear_out_tc(a, maps, s));
}

}  // namespace

}  // namespace polar

using namespace polar;

extern "C" {

size_t polar_linear_workspace_bytes(int B, int H, int T, int d, int dtype) {
  if (!sizes_ok(B, H, T, d, dtype)) return 0;
  return state_bytes(B, H, T, d, dtype);
}

size_t polar_linear_bwd_workspace_bytes(int B, int H, int T, int d, int dtype) {
  if (!sizes_ok(B, H, T, d, dtype)) return 0;
  return 2 * state_bytes(B, H, T, d, dtype);
}

int polar_linear_fwd(const void* q, const void* k, const void* v, const float* log_decay,
                     const int* lengths, const float* state_in, void* mem, float* state_out,
                     int B, int H, int T, int d, int dtype, float scale, void* workspace,
                     size_t workspace_bytes, void* stream) {
  int st = check_sizes(B, H, T, d, dtype, scale);
  if (st != POLAR_OK) return st;
  if (B == 0 || H == 0 || (T == 0 && !state_out)) return POLAR_OK;
  if (!log_decay || (T > 0 && (!q || !k || !v || !mem))) return POLAR_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(mem) ||
      !aligned16(state_in) || !aligned16(state_out) || !aligned4(log_decay) || !aligned4(lengths))
    return POLAR_ERR_MISALIGNED;
  int sms = 0;
  st = check_device(&sms);
  if (st != POLAR_OK) return st;
  const Segments g = segments(B * H, T, d, dtype, sms);
  const size_t need = (size_t)B * H * g.nseg * d * d * sizeof(float);
  if (need && (!workspace || workspace_bytes < need)) return POLAR_ERR_WORKSPACE;
  if (!aligned16(workspace)) return POLAR_ERR_MISALIGNED;
  int* status = status_word();
  if (!status) return cuda_status("cudaGetSymbolAddress", cudaGetLastError());
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* seg = static_cast<float*>(workspace);
  // The tensor-core kernel writes the state of a whole sequence itself.
  const bool tc = dtype == POLAR_BF16;
  const bool walked = g.nseg > 1 || (state_out && !(tc && g.nseg == 1));
  if (walked) {
    const LinearStateArgs a{k, v, log_decay, lengths, B, H, T, d, 1.f, false,
                            g.nseg, g.seg_tokens, state_in, seg, state_out, status};
    st = T > 0 ? run_states(a, dtype, s) : cuda_status("linear scan launch", launch_linear_scan(a, s));
    if (st != POLAR_OK) return st;
  }
  if (T == 0) return POLAR_OK;
  const LinearArgs a{q, k, v, mem, log_decay, lengths, B, H, T, d, scale, false, false,
                     g.nseg, g.seg_tokens, state_in, walked ? seg : nullptr, status,
                     walked ? nullptr : state_out};
  return run_out(a, dtype, s);
}

int polar_linear_step(float* state, const void* q, const void* k, const void* v,
                      const float* log_decay, void* mem, int B, int H, int d, int dtype,
                      float scale, void* stream) {
  int st = check_sizes(B, H, 1, d, dtype, scale);
  if (st != POLAR_OK) return st;
  if (B == 0 || H == 0) return POLAR_OK;
  if (!state || !q || !k || !v || !log_decay || !mem) return POLAR_ERR_INVALID;
  if (!aligned16(state) || !aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(mem) ||
      !aligned4(log_decay))
    return POLAR_ERR_MISALIGNED;
  st = check_device(nullptr);
  if (st != POLAR_OK) return st;
  const LinearStepArgs a{state, q, k, v, log_decay, mem, B, H, d, scale};
  return cuda_status("linear step launch",
                     launch_linear_step(a, dtype, static_cast<cudaStream_t>(stream)));
}

int polar_linear_bwd(const void* q, const void* k, const void* v, const float* log_decay,
                     const int* lengths, const float* state_in, const void* dmem,
                     const float* dstate_out, void* dq, void* dk, void* dv, float* dstate_in,
                     int B, int H, int T, int d, int dtype, float scale, void* workspace,
                     size_t workspace_bytes, void* stream) {
  int st = check_sizes(B, H, T, d, dtype, scale);
  if (st != POLAR_OK) return st;
  if (B == 0 || H == 0 || (T == 0 && !dstate_in)) return POLAR_OK;
  if (!log_decay || (T > 0 && (!q || !k || !v || !dmem || !dq || !dk || !dv)))
    return POLAR_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(dmem) || !aligned16(dq) ||
      !aligned16(dk) || !aligned16(dv) || !aligned16(state_in) || !aligned16(dstate_out) ||
      !aligned16(dstate_in) || !aligned4(log_decay) || !aligned4(lengths))
    return POLAR_ERR_MISALIGNED;
  int sms = 0;
  st = check_device(&sms);
  if (st != POLAR_OK) return st;
  const Segments g = segments(B * H, T, d, dtype, sms);
  const size_t one = (size_t)B * H * g.nseg * d * d;
  const size_t need = 2 * one * sizeof(float);
  if (need && (!workspace || workspace_bytes < need)) return POLAR_ERR_WORKSPACE;
  if (!aligned16(workspace)) return POLAR_ERR_MISALIGNED;
  int* status = status_word();
  if (!status) return cuda_status("cudaGetSymbolAddress", cudaGetLastError());
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* seg_s = static_cast<float*>(workspace);
  float* seg_r = seg_s + one;
  const bool tc = dtype == POLAR_BF16;
  if (g.nseg > 1) {
    const LinearStateArgs a{k, v, log_decay, lengths, B, H, T, d, 1.f, false,
                            g.nseg, g.seg_tokens, state_in, seg_s, nullptr, status};
    st = run_states(a, dtype, s);
    if (st != POLAR_OK) return st;
  }
  const bool walked = g.nseg > 1 || (dstate_in && !(tc && g.nseg == 1));
  if (walked) {
    const LinearStateArgs a{q, dmem, log_decay, lengths, B, H, T, d, scale, true,
                            g.nseg, g.seg_tokens, dstate_out, seg_r, dstate_in, status};
    st = T > 0 ? run_states(a, dtype, s) : cuda_status("linear scan launch", launch_linear_scan(a, s));
    if (st != POLAR_OK) return st;
  }
  if (T == 0) return POLAR_OK;
  const float* before_r = walked ? seg_r : nullptr;
  const LinearArgs aq{dmem, v, k, dq, log_decay, lengths, B, H, T, d, scale, false, true,
                      g.nseg, g.seg_tokens, state_in, g.nseg > 1 ? seg_s : nullptr, status};
  const LinearArgs ak{v, dmem, q, dk, log_decay, lengths, B, H, T, d, scale, true, true,
                      g.nseg, g.seg_tokens, dstate_out, before_r, status};
  // last: it may write dstate_in over dstate_out, which dk's kernel reads
  const LinearArgs av{k, q, dmem, dv, log_decay, lengths, B, H, T, d, scale, true, false,
                      g.nseg, g.seg_tokens, dstate_out, before_r, status,
                      walked ? nullptr : dstate_in};
  for (const LinearArgs* a : {&aq, &ak, &av}) {
    st = run_out(*a, dtype, s);
    if (st != POLAR_OK) return st;
  }
  return POLAR_OK;
}

}  // extern "C"
