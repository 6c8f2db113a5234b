// glr.cuh -- what the kernels of the gated linear recurrence share: gates, four channels
// at a time, spans of tokens and their exchange inside a cluster, sequences in packed rows.
#pragma once

#include <float.h>
#include <math.h>

#include <type_traits>

#include "four.cuh"
#include "internal.h"

namespace dig {

// ---- gates ------------------------------------------------------------------------------

// How the forget gate is given: fp32 log_alpha, or logits g in the element type with
// log_alpha = logsigmoid(g) / gate_norm (gate_norm 1 is the plain sigmoid).
enum GateKind { kGateLog = 0, kGateSigmoid = 1, kGateLogit = 2 };

inline GateKind gate_kind(float gate_norm) {
  return gate_norm == 0.f ? kGateLog : gate_norm == 1.f ? kGateSigmoid : kGateLogit;
}

// Element type of the gate tensor.
template <typename T, int kKind>
using GateT = std::conditional_t<kKind == kGateLog, float, T>;

// 2^x and 1 / x in hardware: relative error at most 2^-22.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// 1 - e^x from x and e^x, without the cancellation of the subtraction near 0: the Taylor
// polynomial within |x| < 0.15 (remainder 3e-9 of it), where 1 - e^x would lose more than
// three of the 24 bits.
__device__ __forceinline__ float2 one_minus_exp(float2 x, float2 ex) {
  float2 p = __ffma2_rn(x, both(1.f / 720.f), both(1.f / 120.f));
  p = __ffma2_rn(x, p, both(1.f / 24.f));
  p = __ffma2_rn(x, p, both(1.f / 6.f));
  p = __ffma2_rn(x, p, both(0.5f));
  p = __ffma2_rn(x, p, both(1.f));
  return make_float2(fabsf(x.x) < 0.15f ? -x.x * p.x : 1.f - ex.x, fabsf(x.y) < 0.15f ? -x.y * p.y : 1.f - ex.y);
}

// log(1 + e) for e in [0, 1], relative error 2e-7: e times the polynomial that interpolates
// log(1 + e) / e at the nine Chebyshev nodes of [0, 1].  (A hardware logarithm of 1 + e keeps
// no relative accuracy for small e, that is for gates that hardly forget.)
__device__ __forceinline__ float2 log_one_plus(float2 e) {
  float2 p = __ffma2_rn(e, both(0.0051261018961668015f), both(-0.029074065387248993f));
  p = __ffma2_rn(e, p, both(0.0775160863995552f));
  p = __ffma2_rn(e, p, both(-0.13602247834205627f));
  p = __ffma2_rn(e, p, both(0.19076880812644958f));
  p = __ffma2_rn(e, p, both(-0.2483539879322052f));
  p = __ffma2_rn(e, p, both(0.3331812024116516f));
  p = __ffma2_rn(e, p, both(-0.4999944567680359f));
  p = __ffma2_rn(e, p, both(0.9999999403953552f));
  return __fmul2_rn(e, p);
}

// Two gates: alpha; 1 - alpha with its own relative accuracy; d log_alpha / d gate.  The
// fields a caller does not use cost nothing once inlined.
struct Gates {
  float2 alpha, rest, slope;
};
template <int kKind>
__device__ __forceinline__ Gates make_gates(float2 g, float inv_norm) {
  Gates r;
  if constexpr (kKind == kGateLog) {
    r.alpha = make_float2(exp2_fast(g.x * kLog2e), exp2_fast(g.y * kLog2e));
    r.rest = one_minus_exp(g, r.alpha);
    r.slope = both(1.f);
  } else {
    // e = e^{-|g|} never overflows; sigmoid(|g|) = 1 / (1 + e), sigmoid(-|g|) = e / (1 + e).
    const float2 e = make_float2(exp2_fast(-fabsf(g.x) * kLog2e), exp2_fast(-fabsf(g.y) * kLog2e));
    const float2 w = __fadd2_rn(e, both(1.f));
    const float2 big = make_float2(rcp_fast(w.x), rcp_fast(w.y)), small = __fmul2_rn(e, big);
    const float2 off = make_float2(g.x < 0.f ? big.x : small.x, g.y < 0.f ? big.y : small.y);
    if constexpr (kKind == kGateSigmoid) {
      r.alpha = make_float2(g.x < 0.f ? small.x : big.x, g.y < 0.f ? small.y : big.y);
      r.rest = r.slope = off;
    } else {
      const float2 l = log_one_plus(e);  // carries a NaN that fminf drops
      const float2 la = make_float2((fminf(g.x, 0.f) - l.x) * inv_norm, (fminf(g.y, 0.f) - l.y) * inv_norm);
      r.alpha = make_float2(exp2_fast(la.x * kLog2e), exp2_fast(la.y * kLog2e));
      r.rest = one_minus_exp(la, r.alpha);
      r.slope = __fmul2_rn(off, both(inv_norm));
    }
  }
  return r;
}

// ---- four gates ---------------------------------------------------------------------------

struct Gates4 {
  F4 alpha, rest, slope;
};
template <int kKind>
__device__ __forceinline__ Gates4 make_gates4(F4 g, float inv_norm) {
  const Gates p = make_gates<kKind>(g.a, inv_norm), q = make_gates<kKind>(g.b, inv_norm);
  return Gates4{F4{p.alpha, q.alpha}, F4{p.rest, q.rest}, F4{p.slope, q.slope}};
}

}  // namespace dig
