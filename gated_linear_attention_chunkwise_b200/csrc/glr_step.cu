// glr_step.cu -- one token of the gated linear recurrence for every running sequence
// (include/dig_gla.h, glr_step).
//
// Bound: memory, and for few rows the latency of one load after another (slot, then state).
// A block takes one row, or with few rows a part of its channels; a thread takes four
// channels at a time.  The rows of one slot are its successive tokens: the block of the first
// of them applies them all in row order and the others leave, so no two blocks touch a
// state, whatever the slots hold (4.3 us for one row of 1152 channels, 6.3 us for 256 rows of
// 4096, 21 us for 4096 rows of 2048).  Finding that out is one pass over the slots by the block's
// threads while the row's own loads are under way: hidden behind them up to a few thousand
// rows, then quadratic (2048 channels, with slots / without: 16384 rows 134 / 78 us, 65535 rows
// 1659 / 292).
#include <algorithm>

#include "glr.cuh"

namespace dig {

namespace {

constexpr int kThreads = 128;

template <typename T, int kKind, bool kComp>
__global__ void __launch_bounds__(kThreads) glr_step_k(GlrStepArgs a, int parts) {
  using G = GateT<T, kKind>;
  const T* const x = static_cast<const T*>(a.x);
  const G* const gate = static_cast<const G*>(a.gate);
  T* const out = static_cast<T*>(a.out);
  const int i = blockIdx.x / parts, part = blockIdx.x - i * parts;
  const int slot = a.slots ? a.slots[i] : i;
  const int c0 = (part * kThreads + threadIdx.x) * 4, step = parts * kThreads * 4;
  if (slot < 0 || slot >= a.nslots) {
    if (slot >= a.nslots && threadIdx.x == 0) report_status(GLA_ERR_INVALID_ARG);
    if (a.fill)
      for (int c = c0; c < a.C; c += step) store4(out + (int64_t)i * a.C + c, all4(0.f));
    return;
  }
  const float inv_norm = 1.f / a.gate_norm;
  const float* const from = a.state + (int64_t)slot * a.C;
  float* const to = a.state_out + (int64_t)slot * a.C;
  // The first four channels' loads go out before the search for other rows of the slot.
  F4 h = all4(0.f), u = all4(0.f), g = all4(0.f);
  if (c0 < a.C) {
    h = load4(from + c0);
    u = load4(x + i * a.x_stride + c0);
    g = load4(gate + i * a.gate_stride + c0);
  }
  bool before = false, behind = false;
  if (a.slots) {
    for (int j = threadIdx.x; j < a.N; j += kThreads) {
      const bool same = a.slots[j] == slot;
      before |= same && j < i;
      behind |= same && j > i;
    }
    if (__syncthreads_or(before)) return;
    behind = __syncthreads_or(behind);
  }
  for (int c = c0; c < a.C; c += step) {
    if (c != c0) {
      h = load4(from + c);
      u = load4(x + i * a.x_stride + c);
      g = load4(gate + i * a.gate_stride + c);
    }
    for (int j = i;;) {
      const Gates4 k = make_gates4<T, kKind, kComp>(g, inv_norm);
      h = fma4(k.alpha, h, kComp ? mul4(k.rest, u) : u);
      store4(out + (int64_t)j * a.C + c, h);
      if (!behind) break;
      do ++j;
      while (j < a.N && a.slots[j] != slot);
      if (j >= a.N) break;
      u = load4(x + j * a.x_stride + c);
      g = load4(gate + j * a.gate_stride + c);
    }
    store4(to + c, h);
  }
}

template <typename T, int kKind>
cudaError_t launch(const GlrStepArgs& a, cudaStream_t st) {
  // A row is shared between blocks while there are fewer than 8 blocks an SM; a block that
  // takes a whole row searches the slots once for all its channels.
  const int chunks = (a.C + 4 * kThreads - 1) / (4 * kThreads);
  const int parts = std::max(1, std::min(chunks, 148 * 8 / a.N));
  const unsigned grid = (unsigned)parts * a.N;
  if (a.complement)
    glr_step_k<T, kKind, true><<<grid, kThreads, 0, st>>>(a, parts);
  else
    glr_step_k<T, kKind, false><<<grid, kThreads, 0, st>>>(a, parts);
  return cudaGetLastError();
}

template <typename T>
cudaError_t by_gate(const GlrStepArgs& a, cudaStream_t st) {
  switch (gate_kind(a.gate_norm)) {
    case kGateLog: return launch<T, kGateLog>(a, st);
    case kGateSigmoid: return launch<T, kGateSigmoid>(a, st);
    default: return launch<T, kGateLogit>(a, st);
  }
}

}  // namespace

cudaError_t glr_step_launch(const GlrStepArgs& a, cudaStream_t st) {
  return a.bf16 ? by_gate<__nv_bfloat16>(a, st) : by_gate<float>(a, st);
}

}  // namespace dig
