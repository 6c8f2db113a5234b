// glr.cuh -- what the kernels of the gated linear recurrence share: gates, element
// types and the arguments of a launch.
#pragma once

#include <math.h>

#include "dev_common.cuh"
#include "internal.h"

namespace dig {

// How the forget gate is given: fp32 log_alpha, or logits g in the element type with
// log_alpha = logsigmoid(g) / gate_norm (gate_norm 1 is the plain sigmoid).
enum GateKind { kGateLog = 0, kGateSigmoid = 1, kGateLogit = 2 };

inline GateKind gate_kind(float gate_norm) {
  return gate_norm == 0.f ? kGateLog : gate_norm == 1.f ? kGateSigmoid : kGateLogit;
}

// One gate: alpha, 1 - alpha (formed without the cancellation of a subtraction, so that
// gates near 1 keep their relative accuracy), and d log_alpha / d gate.
struct Gate {
  float alpha, rest, slope;
};

// inv_norm = 1 / gate_norm (kGateLogit).  The unused fields cost nothing once inlined.
template <int kKind>
__device__ __forceinline__ Gate make_gate(float g, float inv_norm) {
  Gate r;
  if constexpr (kKind == kGateLog) {
    r.alpha = expf(g);
    r.rest = -expm1f(g);
    r.slope = 1.f;
  } else {
    // e^{-|g|} never overflows; sigmoid(|g|) = 1 / (1 + e), sigmoid(-|g|) = e / (1 + e).
    const float e = expf(-fabsf(g));
    const float big = 1.f / (1.f + e), small = e * big;
    const float sig = g < 0.f ? small : big, sigm = g < 0.f ? big : small;
    if constexpr (kKind == kGateSigmoid) {
      r.alpha = sig;
      r.rest = sigm;
      r.slope = sigm;
    } else {
      const float la = (fminf(g, 0.f) - log1pf(e)) * inv_norm;
      r.alpha = expf(la);
      r.rest = -expm1f(la);
      r.slope = sigm * inv_norm;
    }
    if (g != g) r.alpha = r.rest = r.slope = g;  // fminf would drop a NaN
  }
  return r;
}

__device__ __forceinline__ float load_f32(const float* p) { return *p; }
__device__ __forceinline__ float load_f32(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_f32(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f32(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Element type of the gate tensor.
template <typename T, int kKind>
using GateT = std::conditional_t<kKind == kGateLog, float, T>;

}  // namespace dig
