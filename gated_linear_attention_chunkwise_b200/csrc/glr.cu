// glr.cu -- the gated linear recurrence over a token grid in scan order or over packed
// sequences, and its backward pass (include/dig_gla.h, glr_fwd and glr_bwd).
#include <float.h>

#include "glr.cuh"

namespace dig {

namespace {

constexpr int kThreads = 128;

// One thread per (sequence, channel), walking the sequence token by token.
struct Seq {
  int64_t row0;
  int len;
};
__device__ __forceinline__ Seq sequence(const GlrArgs& a, int n, int T) {
  if (!a.cu) return Seq{(int64_t)n * T, T};
  const int s = min(max(a.cu[n], 0), T), e = min(max(a.cu[n + 1], s), T);
  return Seq{s, e - s};
}
__device__ __forceinline__ int token(const GlrArgs& a, const ScanGeom& g, int len, int p) {
  if (a.cu) return a.dir ? len - 1 - p : p;
  return scan_pos_to_token(g, p);
}

// Records sequence lengths that are not ascending or leave the rows.
__device__ __forceinline__ void check_lengths(const GlrArgs& a, int T) {
  for (int n = threadIdx.x; n <= a.nseq; n += kThreads) {
    const int s = a.cu[n];
    if (s < 0 || s > T || (n && s < a.cu[n - 1])) report_status(GLA_ERR_INVALID_ARG);
  }
}

template <typename T, int kKind>
__global__ void __launch_bounds__(kThreads) glr_fwd_k(GlrArgs a, ScanGeom g, int cblocks) {
  using G = GateT<T, kKind>;
  const T* x = static_cast<const T*>(a.x);
  const G* gate = static_cast<const G*>(a.gate);
  T* out = static_cast<T*>(a.out);
  const int n = blockIdx.x / cblocks;
  const int c = (blockIdx.x - n * cblocks) * kThreads + threadIdx.x;
  if (a.cu && blockIdx.x == 0) check_lengths(a, g.T);
  if (c >= a.C) return;
  if (n == a.nseq) {
    if (a.cu && a.fill)
      for (int64_t r = 0; r < g.T; ++r)
        if (r < a.cu[0] || r >= a.cu[a.nseq]) store_f32(out + r * a.C + c, 0.f);
    return;
  }
  const Seq s = sequence(a, n, g.T);
  const float inv_norm = 1.f / a.gate_norm;
  float h = a.h0 ? a.h0[(int64_t)n * a.C + c] : 0.f;
  for (int p = 0; p < s.len; ++p) {
    const int64_t row = s.row0 + token(a, g, s.len, p);
    const Gate k = make_gate<kKind>(load_f32(gate + row * a.gate_stride + c), inv_norm);
    const float u = load_f32(x + row * a.x_stride + c);
    if (k.alpha > FLT_MAX) report_status(GLA_ERR_RANGE);
    h = fmaf(k.alpha, h, a.complement ? k.rest * u : u);
    store_f32(out + row * a.C + c, h);
  }
  if (a.h_last) a.h_last[(int64_t)n * a.C + c] = h;
}

template <typename T, int kKind>
__global__ void __launch_bounds__(kThreads) glr_bwd_k(GlrArgs a, ScanGeom g, int cblocks) {
  using G = GateT<T, kKind>;
  const T* x = static_cast<const T*>(a.x);
  const G* gate = static_cast<const G*>(a.gate);
  const T* hs = static_cast<const T*>(a.h);
  const T* dout = static_cast<const T*>(a.dout);
  T* dx = static_cast<T*>(a.dx);
  G* dgate = static_cast<G*>(a.dgate);
  const int n = blockIdx.x / cblocks;
  const int c = (blockIdx.x - n * cblocks) * kThreads + threadIdx.x;
  if (a.cu && blockIdx.x == 0) check_lengths(a, g.T);
  if (c >= a.C) return;
  if (n == a.nseq) {
    if (a.cu && a.fill)
      for (int64_t r = 0; r < g.T; ++r)
        if (r < a.cu[0] || r >= a.cu[a.nseq]) {
          store_f32(dx + r * a.C + c, 0.f);
          store_f32(dgate + r * a.C + c, 0.f);
        }
    return;
  }
  const Seq s = sequence(a, n, g.T);
  const float inv_norm = 1.f / a.gate_norm;
  float r = a.dh_last ? a.dh_last[(int64_t)n * a.C + c] : 0.f;
  for (int p = s.len - 1; p >= 0; --p) {
    const int64_t row = s.row0 + token(a, g, s.len, p);
    const Gate k = make_gate<kKind>(load_f32(gate + row * a.gate_stride + c), inv_norm);
    if (k.alpha > FLT_MAX) report_status(GLA_ERR_RANGE);
    float before = 0.f;
    if (p > 0)
      before = load_f32(hs + (s.row0 + token(a, g, s.len, p - 1)) * a.C + c);
    else if (a.h0)
      before = a.h0[(int64_t)n * a.C + c];
    const float d = load_f32(dout + row * a.C + c) + r;
    r = k.alpha * d;
    if (a.complement) before -= load_f32(x + row * a.x_stride + c);
    store_f32(dx + row * a.C + c, a.complement ? k.rest * d : d);
    store_f32(dgate + row * a.C + c, r * before * k.slope);
  }
  if (a.dh0) a.dh0[(int64_t)n * a.C + c] = r;
}

template <typename T, int kKind>
cudaError_t launch(const GlrArgs& a, bool bwd, cudaStream_t st) {
  const ScanGeom g = make_geom(a.Hg, a.Wg, a.cu ? 0 : a.dir);
  const int cblocks = (a.C + kThreads - 1) / kThreads;
  const unsigned grid = (unsigned)cblocks * (a.nseq + (a.cu ? 1 : 0));
  if (bwd)
    glr_bwd_k<T, kKind><<<grid, kThreads, 0, st>>>(a, g, cblocks);
  else
    glr_fwd_k<T, kKind><<<grid, kThreads, 0, st>>>(a, g, cblocks);
  return cudaGetLastError();
}

template <typename T>
cudaError_t by_gate(const GlrArgs& a, bool bwd, cudaStream_t st) {
  switch (gate_kind(a.gate_norm)) {
    case kGateLog: return launch<T, kGateLog>(a, bwd, st);
    case kGateSigmoid: return launch<T, kGateSigmoid>(a, bwd, st);
    default: return launch<T, kGateLogit>(a, bwd, st);
  }
}

}  // namespace

cudaError_t glr_fwd_launch(const GlrArgs& a, cudaStream_t st) {
  return a.bf16 ? by_gate<__nv_bfloat16>(a, false, st) : by_gate<float>(a, false, st);
}
cudaError_t glr_bwd_launch(const GlrArgs& a, cudaStream_t st) {
  return a.bf16 ? by_gate<__nv_bfloat16>(a, true, st) : by_gate<float>(a, true, st);
}

}  // namespace dig
