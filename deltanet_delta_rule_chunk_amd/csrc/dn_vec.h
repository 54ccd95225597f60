// dn_vec.h -- pieces of rows as fp32 vectors, and the layer's scalar maps, for
// the short convolution, the selective scan and the norm with addition.
#pragma once

#include "dn_common.h"
#include "dn_mfma.h"

namespace dn {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Four elements as they lie in memory.
template <typename T> struct Raw4;
template <> struct Raw4<float> { f32x4 v; };
template <> struct Raw4<bf16> { uint2 v; };

template <typename T>
__device__ __forceinline__ Raw4<T> raw4(const T* p) { return *reinterpret_cast<const Raw4<T>*>(p); }
__device__ __forceinline__ f32x4 wide(Raw4<float> r) { return r.v; }
__device__ __forceinline__ f32x4 wide(Raw4<bf16> r) {
  return f32x4{__uint_as_float(r.v.x << 16), __uint_as_float(r.v.x & 0xffff0000u),
               __uint_as_float(r.v.y << 16), __uint_as_float(r.v.y & 0xffff0000u)};
}
template <typename T> __device__ __forceinline__ Raw4<T> narrow(f32x4 x);
template <> __device__ __forceinline__ Raw4<float> narrow<float>(f32x4 x) { return {x}; }
template <> __device__ __forceinline__ Raw4<bf16> narrow<bf16>(f32x4 x) {
  return {make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]))};
}
template <typename T>
__device__ __forceinline__ void put4(T* p, f32x4 x) { *reinterpret_cast<Raw4<T>*>(p) = narrow<T>(x); }

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_fast(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ float sigmoid(float x) { return rcp_fast(1.f + exp2_fast(-kLog2e * x)); }

// log(1 + e^x) = max(x, 0) + log1p(e), e = e^-|x| in (0, 1].  log1p(e) = 2 atanh(s) =
// s f(s^2), s = e / (2 + e) <= 1/3; f(q) = 2 + 2 q / 3 + 2 q^2 / 5 + ... by the polynomial of degree
// 4 that is nearest to it on [0, 1/9] in relative error (2^-26.9; equal ripples,
// found by exchange).  So a small e keeps all of its bits, which log(1 + e) would lose.
__device__ __forceinline__ float softplus(float x) {
  const float e = exp2_fast(-kLog2e * fabsf(x));
  const float s = e * rcp_fast(2.f + e), q = s * s;
  float p = 0.28178334f;
  p = fmaf(p, q, 0.27960601f);
  p = fmaf(p, q, 0.40024909f);
  p = fmaf(p, q, 0.66666317f);
  p = fmaf(p, q, 2.f);
  return fmaf(s, p, fmaxf(x, 0.f));
}

}  // namespace dn
