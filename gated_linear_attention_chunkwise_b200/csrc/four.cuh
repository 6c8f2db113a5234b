// four.cuh -- four channels of a row at a time: packed fp32 arithmetic (two channels an
// instruction) and the vector loads and stores of both element types.
#pragma once

#include "dev_common.cuh"

namespace dig {

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// ---- four channels ------------------------------------------------------------------------

struct F4 {
  float2 a, b;
};
__device__ __forceinline__ F4 all4(float v) { return F4{both(v), both(v)}; }
__device__ __forceinline__ F4 fma4(F4 x, F4 y, F4 z) { return F4{__ffma2_rn(x.a, y.a, z.a), __ffma2_rn(x.b, y.b, z.b)}; }
__device__ __forceinline__ F4 mul4(F4 x, F4 y) { return F4{__fmul2_rn(x.a, y.a), __fmul2_rn(x.b, y.b)}; }
__device__ __forceinline__ F4 add4(F4 x, F4 y) { return F4{__fadd2_rn(x.a, y.a), __fadd2_rn(x.b, y.b)}; }
__device__ __forceinline__ F4 sub4(F4 x, F4 y) { return fma4(y, all4(-1.f), x); }

// Four consecutive channels of a row as they lie in memory, and as fp32.
template <typename T>
struct Four;
template <>
struct Four<__nv_bfloat16> {
  using Raw = uint2;
  static __device__ __forceinline__ F4 get(Raw r) { return F4{unpack_bf16x2(r.x), unpack_bf16x2(r.y)}; }
  static __device__ __forceinline__ Raw put(F4 f) { return make_uint2(pack_bf16x2(f.a.x, f.a.y), pack_bf16x2(f.b.x, f.b.y)); }
};
template <>
struct Four<float> {
  using Raw = float4;
  static __device__ __forceinline__ F4 get(Raw r) { return F4{make_float2(r.x, r.y), make_float2(r.z, r.w)}; }
  static __device__ __forceinline__ Raw put(F4 f) { return make_float4(f.a.x, f.a.y, f.b.x, f.b.y); }
};
template <typename T>
__device__ __forceinline__ F4 load4(const T* p) {
  return Four<T>::get(*reinterpret_cast<const typename Four<T>::Raw*>(p));
}
template <typename T>
__device__ __forceinline__ void store4(T* p, F4 f) {
  *reinterpret_cast<typename Four<T>::Raw*>(p) = Four<T>::put(f);
}

}  // namespace dig
