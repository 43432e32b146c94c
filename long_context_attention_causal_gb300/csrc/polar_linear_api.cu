// C ABI of the decayed linear attention: argument validation, the split of a
// sequence into segments, and the launches.  The contract of every entry
// point is in include/polar_attn.h, the mathematics in polar_linear.cu.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "polar_device.cuh"
#include "polar_internal.h"

namespace polar {

namespace {

// Runs of tiles.  Whole heads to a CTA need one launch and read every row
// once, but leave SMs idle when heads are few.  Equal runs over all slots
// cut heads: y and z of what lies before a cut are read a second time, and a
// state and a scan launch come first.  The cheaper of the two is taken.  In
// tiles of an SM's time, equal runs of `even` tiles cost about 1.6 even + 5 for
// bf16 (d = 128, states of two terms, whole / cut: 64 heads of 2048 tokens 55 /
// 65 us, 100 of 2048 57 / 85, 200 of 4096 191 / 220, 160 of 8192 358 / 333, 32 of
// 16384 354 / 159).
// fp32 tiles take longer than the launches do: about 1.05 even + 0.9 (d = 64,
// whole / cut: 2 heads of 256 tokens 29 / 26 us, 8 of 512 47 / 26, 76 of 1024 90
// / 95, 24 of 2048 172 / 75, 64 of 4096 338 / 290, 200 of 2048 444 / 400; d =
// 128: 20 of 512 74 / 79, 40 of 2048 363 / 290).  The backward's three outputs
// share a launch there, so whole heads fill the SMs sooner (200 heads of 2048,
// d = 64, 874 / 1031; 20 of 512, d = 128, 94 / 124).
LinearSplit split(int BH, int T, int d, int dtype, int sms, bool backward) {
  LinearSplit r;
  r.sms = sms;
  r.tiles = (T + kLinearTile - 1) / kLinearTile;
  // CTAs at once: one a SM, in fp32 d / 64 to a run
  const long long slots = dtype == POLAR_BF16 ? sms : std::max(1, sms / (d / 64));
  auto whole = [&](long long heads) { return r.tiles * ((heads + slots - 1) / slots); };
  auto even = [&](long long heads) { return (heads * r.tiles + slots - 1) / slots; };
  const long long heads = dtype == POLAR_F32 && backward ? 3LL * BH : BH;
  const bool uncut = dtype == POLAR_BF16 ? whole(heads) <= 1.6 * even(heads) + 5.0
                                         : whole(heads) <= 1.05 * even(heads) + 0.9;
  r.per = (int)std::max(1LL, uncut ? whole(BH) : even(BH));
  r.parts = (int)(((long long)BH * r.tiles + r.per - 1) / r.per);
  r.cut = r.per % std::max(r.tiles, 1) != 0;
  return r;
}

bool sizes_ok(int B, int H, int T, int d, int dtype) {
  return B >= 0 && H >= 0 && T >= 0 && (d == 64 || d == 128) &&
         (dtype == POLAR_F32 || dtype == POLAR_BF16) && (long long)B * H <= (1 << 20) &&
         T <= (1 << 28) &&
         (long long)B * H * ((T + kLinearTile - 1) / kLinearTile) <= INT_MAX;
}

int check_sizes(int B, int H, int T, int d, int dtype, float scale) {
  if (B < 0 || H < 0 || T < 0 || !std::isfinite(scale)) return POLAR_ERR_INVALID;
  return sizes_ok(B, H, T, d, dtype) ? POLAR_OK : POLAR_ERR_UNSUPPORTED;
}

// Bytes of a tensor; an output that meets another tensor is refused, and the
// workspace, which is written too, where it meets any.
struct Span {
  const void* p;
  size_t bytes;
};
bool meet(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x && y && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}
bool any_meet(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
  for (const Span& o : outs) {
    for (const Span& i : ins)
      if (meet(o, i)) return true;
    for (const Span& other : outs)
      if (&other != &o && meet(o, other)) return true;
  }
  return false;
}
// The spans of a [B, H, T, d] tensor, of the states, the decay and the
// lengths; `same` is left out of the states where an output may be that input
// itself.
struct Sizes {
  size_t rows, states, heads, batch;
  Sizes(int B, int H, int T, int d, int dtype)
      : rows((size_t)B * H * T * d * (dtype == POLAR_BF16 ? 2 : 4)),
        states((size_t)B * H * d * d * 4),
        heads((size_t)H * 4),
        batch((size_t)B * 4) {}
  Span row(const void* p) const { return {p, rows}; }
  Span decay(const void* p) const { return {p, heads}; }
  Span lengths(const void* p) const { return {p, batch}; }
  Span state(const void* p, const void* same = nullptr) const {
    return {p == same ? nullptr : p, states};
  }
};

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A state a cut, and one a head for a copy of the incoming states: the CTA
// that ends a cut head may write state_out over the state_in that the CTA of
// its start has yet to read.
size_t cut_floats(const LinearSplit& g, int d) { return (size_t)g.parts * d * d; }
size_t cut_bytes(const LinearSplit& g, int BH, int d) {
  return g.cut ? (cut_floats(g, d) + (size_t)BH * d * d) * sizeof(float) : 0;
}

// check_device with an assumed SM count where there is no device: sizes and
// refusals do not need one.
int device_or_assumed(int* sms) {
  const int st = check_device(sms);
  if (st != POLAR_OK) *sms = 148;
  return st;
}

size_t workspace_bytes_of(int B, int H, int T, int d, int dtype, bool backward) {
  int sms = 0;
  device_or_assumed(&sms);
  return B * H > 0 && T > 0 ? cut_bytes(split(B * H, T, d, dtype, sms, backward), B * H, d) : 0;
}

// bf16 runs on the tensor cores, fp32 on the FP32 pipes.  n applications that
// differ in tensors, states, direction and scale.
int run_states(const LinearStateArgs* a, int n, int dtype, cudaStream_t s) {
  int st;
  if (dtype == POLAR_BF16) {
    CUtensorMap maps[4];
    for (int i = 0; i < n; ++i)
      if (!make_map(&maps[2 * i], a[i].y, a[i].B * a[i].H, a[i].T, a[i].d) ||
          !make_map(&maps[2 * i + 1], a[i].z, a[i].B * a[i].H, a[i].T, a[i].d))
        return POLAR_ERR_CUDA;
    st = cuda_status("linear state launch", launch_linear_states_tc(a, n, maps, s));
  } else {
    st = cuda_status("linear state launch", launch_linear_states(a, n, s));
  }
  if (st != POLAR_OK) return st;
  return cuda_status("linear scan launch", launch_linear_scan(a, n, s));
}

int run_out(LinearArgs* a, int n, int dtype, cudaStream_t s) {
  if (dtype != POLAR_BF16) return cuda_status("linear output launch", launch_linear_out(a, n, s));
  // one direction and one number of terms a launch
  for (int i = 0; i < n;) {
    const int m =
        i + 1 < n && a[i + 1].reverse == a[i].reverse && a[i + 1].exact == a[i].exact ? 2 : 1;
    if (i > 0) a[i].chained = true;
    CUtensorMap maps[8];
    for (int j = 0; j < m; ++j) {
      const void* bases[4] = {a[i + j].x, a[i + j].y, a[i + j].z, a[i + j].out};
      for (int t = 0; t < 4; ++t)
        if (!make_map(&maps[4 * j + t], bases[t], a->B * a->H, a->T, a->d)) return POLAR_ERR_CUDA;
    }
    const int st = cuda_status("linear output launch", launch_linear_out_tc(a + i, m, maps, s));
    if (st != POLAR_OK) return st;
    i += m;
  }
  return POLAR_OK;
}

}  // namespace

}  // namespace polar

using namespace polar;

extern "C" {

size_t polar_linear_workspace_bytes(int B, int H, int T, int d, int dtype) {
  if (!sizes_ok(B, H, T, d, dtype)) return 0;
  return workspace_bytes_of(B, H, T, d, dtype, false);
}

size_t polar_linear_bwd_workspace_bytes(int B, int H, int T, int d, int dtype) {
  if (!sizes_ok(B, H, T, d, dtype)) return 0;
  return 2 * workspace_bytes_of(B, H, T, d, dtype, true);
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
  const int device = device_or_assumed(&sms);
  const LinearSplit g = split(B * H, T, d, dtype, sms, false);
  const size_t need = cut_bytes(g, B * H, d);
  const Sizes z(B, H, T, d, dtype);
  const Span scratch{workspace, std::min(need, workspace_bytes)};  // what may be written of it
  if (any_meet({z.row(mem), z.state(state_out), scratch},
               {z.row(q), z.row(k), z.row(v), z.state(state_in, state_out), z.decay(log_decay),
                z.lengths(lengths)}))
    return POLAR_ERR_INVALID;
  if (device != POLAR_OK) return device;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0)
    return cuda_status("linear state copy", launch_linear_copy_state(
                                                state_in, state_out, (size_t)B * H * d * d, s));
  if (need && (!workspace || workspace_bytes < need)) return POLAR_ERR_WORKSPACE;
  if (!aligned16(workspace)) return POLAR_ERR_MISALIGNED;
  int* status = status_word();
  if (!status) return cuda_status("cudaGetSymbolAddress", cudaGetLastError());
  float* cuts = static_cast<float*>(workspace);
  float* copy = g.cut && state_in && state_in == state_out ? cuts + cut_floats(g, d) : nullptr;
  if (g.cut) {
    const LinearStateArgs a{k, v, log_decay, lengths, B, H, T, d, 1.f, false,
                            g, state_in, cuts, status, copy, state_out != nullptr};
    st = run_states(&a, 1, dtype, s);
    if (st != POLAR_OK) return st;
  }
  LinearArgs a{q, k, v, mem, log_decay, lengths, B, H, T, d, scale, false, false,
               g, copy ? copy : state_in, cuts, state_out, status, state_out != nullptr,
               g.cut};
  return run_out(&a, 1, dtype, s);
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
  const Sizes z(B, H, 1, d, dtype);
  if (any_meet({z.row(mem), z.state(state)},
               {z.row(q), z.row(k), z.row(v), z.decay(log_decay)}))
    return POLAR_ERR_INVALID;
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
  const int device = device_or_assumed(&sms);
  const LinearSplit g = split(B * H, T, d, dtype, sms, true);
  const size_t one = cut_bytes(g, B * H, d), need = 2 * one;
  const Sizes z(B, H, T, d, dtype);
  const Span scratch{workspace, std::min(need, workspace_bytes)};  // what may be written of it
  if (any_meet({z.row(dq), z.row(dk), z.row(dv), z.state(dstate_in), scratch},
               {z.row(q), z.row(k), z.row(v), z.row(dmem), z.state(state_in),
                z.state(dstate_out, dstate_in), z.decay(log_decay), z.lengths(lengths)}))
    return POLAR_ERR_INVALID;
  if (device != POLAR_OK) return device;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0)
    return cuda_status("linear state copy",
                       launch_linear_copy_state(dstate_out, dstate_in, (size_t)B * H * d * d, s));
  if (need && (!workspace || workspace_bytes < need)) return POLAR_ERR_WORKSPACE;
  if (!aligned16(workspace)) return POLAR_ERR_MISALIGNED;
  int* status = status_word();
  if (!status) return cuda_status("cudaGetSymbolAddress", cudaGetLastError());
  float* cuts_s = static_cast<float*>(workspace);
  float* cuts_r = cuts_s + one / sizeof(float);
  float* copy =
      g.cut && dstate_out && dstate_out == dstate_in ? cuts_r + cut_floats(g, d) : nullptr;
  if (g.cut) {
    // dq's states last: its kernel then starts on tiles that are still in L2
    const LinearStateArgs a[2] = {{q, dmem, log_decay, lengths, B, H, T, d, scale, true,
                                   g, dstate_out, cuts_r, status, copy, dstate_in != nullptr},
                                  {k, v, log_decay, lengths, B, H, T, d, 1.f, false,
                                   g, state_in, cuts_s, status, nullptr, false}};
    st = run_states(a, 2, dtype, s);
    if (st != POLAR_OK) return st;
  }
  // dk and dv share a launch where they share their terms.  dk needs no more
  // than two, and the two launches that follow from that take less time (B2 H16
  // T16384 d128: 424 us, 444 in one), unless one leaves half of the SMs idle (B8
  // H8 T1111 d64: 84, 55 in one).
  const float* r_init = copy ? copy : dstate_out;
  LinearArgs a[3] = {{dmem, v, k, dq, log_decay, lengths, B, H, T, d, scale, false, true,
                      g, state_in, cuts_s, nullptr, status, false, g.cut},
                     {v, dmem, q, dk, log_decay, lengths, B, H, T, d, scale, true, true,
                      g, r_init, cuts_r, nullptr, status, dstate_in && 2LL * g.parts <= sms},
                     {k, q, dmem, dv, log_decay, lengths, B, H, T, d, scale, true, false,
                      g, r_init, cuts_r, dstate_in, status, dstate_in != nullptr}};
  // dv's CTA would write dstate_in over the dstate_out that dk's has yet to
  // read: in place and uncopied, dv goes after the others
  if (!dstate_in || r_init != dstate_in) return run_out(a, 3, dtype, s);
  st = run_out(a, 2, dtype, s);
  return st == POLAR_OK ? run_out(a + 2, 1, dtype, s) : st;
}

}  // extern "C"
