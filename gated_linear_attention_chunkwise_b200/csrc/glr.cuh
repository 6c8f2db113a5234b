// glr.cuh -- the gates of the gated linear recurrence, four channels at a time, for the walk
// over sequences (glr_scan.cuh) and the single token (glr_step.cu).
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

// The exponential behind the logits: 1 - alpha and the gradient inherit its relative error, so
// calls in fp32 (kFine) take expf; calls in bf16 the hardware's, far below half a step of 2^-9.
template <bool kFine>
__device__ __forceinline__ float2 exp_of(float2 x) {
  if constexpr (kFine) return make_float2(expf(x.x), expf(x.y));
  const float2 t = __fmul2_rn(x, both(kLog2e));
  return make_float2(exp2_fast(t.x), exp2_fast(t.y));
}

// alpha = e^x and, where kRest, 1 - alpha.  Near 0 both come from the Taylor polynomial of
// e^x - 1: a subtraction would lose the leading bits of 1 - alpha, and the hardware's e^x is off
// by up to 2^-22 just below 1, an error of the decay that acts again at every token (1.9 units of
// 2^-24 measured, 0.6 from the polynomial: one rounding).  alpha alone needs three powers within
// |x| < 1/16 (remainder 8e-9): behind that a state is gone in 16 tokens.  1 - alpha needs five
// within 0.15 (3e-9 of it); in fp32, where the subtraction would still cost 10 units there, seven
// within 1/2 (1e-8 of it).
template <bool kFine, bool kRest>
__device__ __forceinline__ void decay(float2 x, float2& alpha, float2& rest) {
  constexpr bool kLong = kFine && kRest;
  constexpr float kNear = kLong ? 0.5f : kRest ? 0.15f : 0.0625f;
  const float2 ex = exp_of<false>(x);
  float2 p = both(kLong ? 1.f / 40320.f : kRest ? 1.f / 720.f : 1.f / 24.f);
  if constexpr (kLong) {
    p = __ffma2_rn(x, p, both(1.f / 5040.f));
    p = __ffma2_rn(x, p, both(1.f / 720.f));
  }
  if constexpr (kRest) {
    p = __ffma2_rn(x, p, both(1.f / 120.f));
    p = __ffma2_rn(x, p, both(1.f / 24.f));
  }
  p = __ffma2_rn(x, p, both(1.f / 6.f));
  p = __ffma2_rn(x, p, both(0.5f));
  p = __ffma2_rn(x, p, both(1.f));
  const bool near_x = fabsf(x.x) < kNear, near_y = fabsf(x.y) < kNear;
  float2 close;
  if constexpr (kRest) {
    const float2 less = __fmul2_rn(x, p);
    rest = make_float2(near_x ? -less.x : 1.f - ex.x, near_y ? -less.y : 1.f - ex.y);
    close = make_float2(1.f - rest.x, 1.f - rest.y);
  } else {
    close = __ffma2_rn(x, p, both(1.f));
  }
  alpha = make_float2(near_x ? close.x : ex.x, near_y ? close.y : ex.y);
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
  float2 alpha{}, rest{}, slope{};
};
template <int kKind, bool kFine, bool kRest>
__device__ __forceinline__ Gates make_gates(float2 g, float inv_norm) {
  Gates r;
  if constexpr (kKind == kGateLog) {
    decay<kFine, kRest>(g, r.alpha, r.rest);
    r.slope = both(1.f);
  } else {
    // e = e^{-|g|} never overflows; sigmoid(-|g|) = e / (1 + e), sigmoid(|g|) = 1 - that.
    const float2 e = exp_of<kFine>(make_float2(-fabsf(g.x), -fabsf(g.y)));
    const float2 w = __fadd2_rn(e, both(1.f));
    const float2 inv = make_float2(rcp_fast(w.x), rcp_fast(w.y));
    const float2 small = __fmul2_rn(e, inv), big = __ffma2_rn(small, both(-1.f), both(1.f));
    const float2 off = make_float2(g.x < 0.f ? big.x : small.x, g.y < 0.f ? big.y : small.y);
    if constexpr (kKind == kGateSigmoid) {
      r.alpha = make_float2(g.x < 0.f ? small.x : big.x, g.y < 0.f ? small.y : big.y);
      r.rest = r.slope = off;
    } else {
      // (the logarithm carries a NaN that fminf drops)
      const float2 l = log_one_plus(e);
      const float2 la = __fmul2_rn(__ffma2_rn(l, both(-1.f), make_float2(fminf(g.x, 0.f), fminf(g.y, 0.f))), both(inv_norm));
      decay<kFine, kRest>(la, r.alpha, r.rest);
      r.slope = __fmul2_rn(off, both(inv_norm));
    }
  }
  return r;
}

// ---- four gates ---------------------------------------------------------------------------

struct Gates4 {
  F4 alpha, rest, slope;
};
template <typename T, int kKind, bool kRest>
__device__ __forceinline__ Gates4 make_gates4(F4 g, float inv_norm) {
  constexpr bool kFine = sizeof(T) == 4;
  const Gates p = make_gates<kKind, kFine, kRest>(g.a, inv_norm), q = make_gates<kKind, kFine, kRest>(g.b, inv_norm);
  return Gates4{F4{p.alpha, q.alpha}, F4{p.rest, q.rest}, F4{p.slope, q.slope}};
}

}  // namespace dig
