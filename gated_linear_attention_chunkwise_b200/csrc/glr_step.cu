// glr_step.cu -- one token of the gated linear recurrence for every running sequence
// (include/dig_gla.h, glr_step).
#include "glr.cuh"

namespace dig {

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float load_f32(const float* p) { return *p; }
__device__ __forceinline__ float load_f32(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_f32(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f32(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// One thread per (row, channel).  Rows that name the same state belong together: the
// first of them applies all, in row order, the others do nothing.
template <typename T, int kKind>
__global__ void __launch_bounds__(kThreads) glr_step_k(GlrStepArgs a, int cblocks) {
  using G = GateT<T, kKind>;
  const T* x = static_cast<const T*>(a.x);
  const G* gate = static_cast<const G*>(a.gate);
  T* out = static_cast<T*>(a.out);
  const int i = blockIdx.x / cblocks;
  const int c = (blockIdx.x - i * cblocks) * kThreads + threadIdx.x;
  if (c >= a.C) return;
  const int slot = a.slots ? a.slots[i] : i;
  if (slot < 0 || slot >= a.nslots) {
    if (slot >= a.nslots) report_status(GLA_ERR_INVALID_ARG);
    if (a.fill) store_f32(out + (int64_t)i * a.C + c, 0.f);
    return;
  }
  const float inv_norm = 1.f / a.gate_norm;
  if (a.slots)
    for (int j = 0; j < i; ++j)
      if (a.slots[j] == slot) return;
  float h = a.state[(int64_t)slot * a.C + c];
  for (int j = i; j < a.N; ++j) {
    if (j != i && (!a.slots || a.slots[j] != slot)) continue;
    const Gates k = make_gates<kKind>(both(load_f32(gate + j * a.gate_stride + c)), inv_norm);
    const float u = load_f32(x + j * a.x_stride + c);
    h = fmaf(k.alpha.x, h, a.complement ? k.rest.x * u : u);
    store_f32(out + (int64_t)j * a.C + c, h);
  }
  a.state_out[(int64_t)slot * a.C + c] = h;
}

template <typename T, int kKind>
cudaError_t launch(const GlrStepArgs& a, cudaStream_t st) {
  const int cblocks = (a.C + kThreads - 1) / kThreads;
  glr_step_k<T, kKind><<<(unsigned)cblocks * a.N, kThreads, 0, st>>>(a, cblocks);
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
