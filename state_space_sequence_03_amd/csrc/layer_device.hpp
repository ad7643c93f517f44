// layer_device.hpp -- what the kernels around the scan share: vectors of io
// elements as fp32, the SiLU gate and its derivative, operands with strides.
#pragma once
#include "ssd_device.hpp"

namespace ssd {

// A [batch, token, channel] operand: element strides of the two outer axes.
// Offsets are 64-bit, so rows may lie past 2^31 elements.
struct Strides {
  int64_t batch, token;
};

// V consecutive io elements <-> fp32.  V is the elements of 16 bytes, and
// p 16-byte aligned; or V is 1.
template <int V> __device__ __forceinline__ void load_v(const bf16* p, float* v) {
  if constexpr (V == 8) {
    const bf16x8 w = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = static_cast<float>(w[e]);
  } else {
    static_assert(V == 1, "one element or 16 bytes");
    v[0] = static_cast<float>(*p);
  }
}
template <int V> __device__ __forceinline__ void load_v(const float* p, float* v) {
  if constexpr (V == 4) {
    const floatx4 w = *reinterpret_cast<const floatx4*>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = w[e];
  } else {
    static_assert(V == 1, "one element or 16 bytes");
    v[0] = *p;
  }
}
template <int V> __device__ __forceinline__ void store_v(bf16* p, const float* v) {
  if constexpr (V == 8) {
    bf16x8 w;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = static_cast<bf16>(v[e]);
    *reinterpret_cast<bf16x8*>(p) = w;
  } else {
    *p = static_cast<bf16>(v[0]);
  }
}
template <int V> __device__ __forceinline__ void store_v(float* p, const float* v) {
  if constexpr (V == 4) {
    *reinterpret_cast<floatx4*>(p) = floatx4{v[0], v[1], v[2], v[3]};
  } else {
    *p = v[0];
  }
}
// The same 16 bytes (or one element) held unconverted, so that rows loaded
// ahead cost the registers of their io type only.
template <typename T, int V> struct RawV { typedef T type; };
template <> struct RawV<bf16, 8> { typedef bf16x8 type; };
template <> struct RawV<float, 4> { typedef floatx4 type; };
template <typename T, int V>
__device__ __forceinline__ typename RawV<T, V>::type load_raw(const T* p) {
  return *reinterpret_cast<const typename RawV<T, V>::type*>(p);
}
template <typename T, int V>
__device__ __forceinline__ typename RawV<T, V>::type zero_raw() {
  typename RawV<T, V>::type r;
  if constexpr (V == 1) {
    r = T(0.0f);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) r[e] = T(0.0f);
  }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void widen(const typename RawV<T, V>::type& r, float* v) {
  if constexpr (V == 1) {
    v[0] = static_cast<float>(r);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = static_cast<float>(r[e]);
  }
}

// 1 / (1 + e^-v) on the hardware exp2 and reciprocal (1 ulp each); v far below
// zero gives e^-v = inf and the reciprocal 0.
__device__ __forceinline__ float sigmoid_f32(float v) {
  return __builtin_amdgcn_rcpf(1.0f + fast_exp2(-kLog2e * v));
}
// d silu(v) / dv for silu(v) = v s, s = sigmoid(v)
__device__ __forceinline__ float silu_slope(float v, float s) {
  return s * fmaf(v, 1.0f - s, 1.0f);
}

}  // namespace ssd
