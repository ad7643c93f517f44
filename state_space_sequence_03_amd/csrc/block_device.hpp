// block_device.hpp -- what the kernels of a residual block share: eight elements at
// any alignment, 8-bit values with their block's scale.
#pragma once
#include "layer_device.hpp"

namespace ssd {

constexpr int kBlock8 = 128;   // elements of one scale
constexpr float kMost8 = 448.0f;                    // the largest e4m3 value
constexpr float kLeast8 = 7.888609052210118e-31f;   // 2^-100: a block's least magnitude, so that 448 / it is finite

// Eight elements, aligned to one of them only: a slice may start anywhere, and rows of
// an odd width do.  The memory system takes such accesses whole.
typedef bf16 bf16x8_any __attribute__((ext_vector_type(8), aligned(2)));
typedef float floatx4_any __attribute__((ext_vector_type(4), aligned(4)));

// The same held unconverted, for rows loaded ahead.
template <typename T> struct Raw8;
template <> struct Raw8<bf16> {
  bf16x8 v;
  __device__ __forceinline__ float operator[](int e) const { return static_cast<float>(v[e]); }
};
template <> struct Raw8<float> {
  floatx4 a, b;
  __device__ __forceinline__ float operator[](int e) const { return e < 4 ? a[e] : b[e - 4]; }
};
__device__ __forceinline__ Raw8<bf16> raw8(const bf16* p, int n) {
  Raw8<bf16> r;
  if (n >= 8) {
    r.v = *reinterpret_cast<const bf16x8_any*>(p);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e] = e < n ? p[e] : static_cast<bf16>(0.0f);
  }
  return r;
}
__device__ __forceinline__ Raw8<float> raw8(const float* p, int n) {
  Raw8<float> r;
  if (n >= 8) {
    r.a = *reinterpret_cast<const floatx4_any*>(p);
    r.b = *reinterpret_cast<const floatx4_any*>(p + 4);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      r.a[e] = e < n ? p[e] : 0.0f;
      r.b[e] = e + 4 < n ? p[e + 4] : 0.0f;
    }
  }
  return r;
}

// The first `n` of the eight elements at p (all of them where n >= 8), zeros behind them.
__device__ __forceinline__ void load8(const bf16* p, int n, float (&v)[8]) {
  if (n >= 8) {
    const bf16x8_any w = *reinterpret_cast<const bf16x8_any*>(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = static_cast<float>(w[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < n ? static_cast<float>(p[e]) : 0.0f;
  }
}
__device__ __forceinline__ void load8(const float* p, int n, float (&v)[8]) {
  if (n >= 8) {
    const floatx4_any a = *reinterpret_cast<const floatx4_any*>(p);
    const floatx4_any b = *reinterpret_cast<const floatx4_any*>(p + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = a[e];
      v[4 + e] = b[e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = e < n ? p[e] : 0.0f;
  }
}
__device__ __forceinline__ void store8(bf16* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    bf16x8_any w;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = static_cast<bf16>(v[e]);
    *reinterpret_cast<bf16x8_any*>(p) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[e] = static_cast<bf16>(v[e]);
  }
}
__device__ __forceinline__ void store8(float* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    floatx4_any a, b;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = v[e];
      b[e] = v[4 + e];
    }
    *reinterpret_cast<floatx4_any*>(p) = a;
    *reinterpret_cast<floatx4_any*>(p + 4) = b;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[e] = v[e];
  }
}

// The offset of a row of a strided operand; fewer than 2^31 rows.
__device__ __forceinline__ int64_t row_at(const Strides& s, int64_t row, int64_t L) {
  const uint32_t b = (uint32_t)row / (uint32_t)L;
  return (int64_t)b * s.batch + (int64_t)((uint32_t)row - b * (uint32_t)L) * s.token;
}

// max |v|, leaving NaN out (fmaxf takes the other operand).
__device__ __forceinline__ float most_of(const float (&v)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));
  return m;
}
// The largest over the lanes that share `lane / 16`, in all of them: a block of 128 in pieces of eight.
// Rotations of the 16 lanes ride on the max itself; numbers >= 0 are in the order of their bits.
__device__ __forceinline__ uint32_t most_of_16(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x128, 0xf, 0xf, true));   // by 8
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x124, 0xf, 0xf, true));
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x122, 0xf, 0xf, true));
  m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x121, 0xf, 0xf, true));   // by 1
  return m;
}
__device__ __forceinline__ float most_of_16(float m) {
  return __builtin_bit_cast(float, most_of_16(__builtin_bit_cast(uint32_t, m)));
}

// m / 448 for 2^-100 <= m, correctly rounded: the quotient by the reciprocal, and what it leaves of m joined to it.
__device__ __forceinline__ float scale_of(float m) {
  const float s = m * (1.0f / kMost8), left = fmaf(-s, kMost8, m);
  return m < __builtin_inff() ? fmaf(left, 1.0f / kMost8, s) : m;
}

// 448 / m in two parts, to about 2^-44 of it: the hardware reciprocal (of m / 448, which stays normal) and
// what it leaves of 448.  An infinite m gives 0.
struct Inverse8 {
  float hi, lo;
};
__device__ __forceinline__ Inverse8 inverse8(float m) {
  Inverse8 by;
  by.hi = __builtin_amdgcn_rcpf(m * (1.0f / kMost8));
  const float lo = fmaf(-by.hi, m, kMost8) * (by.hi * (1.0f / kMost8));
  by.lo = by.hi == 0.0f ? 0.0f : lo;
  return by;
}

// v 448 / m as e4m3, to nearest even, for eight values: at most 448 (1 + 2^-23), which rounds to 448, so
// nothing has to be cut off.  What the second part adds goes into the fma with the first, so the sum is
// rounded once, to fp32, in front of the conversion, and a value falls on the wrong side of the middle between
// two e4m3 values only within half a step of fp32 of it.  (Written as a product and additions of what it lost, the
// compiler contracts the last of them with the product, and the loss counts twice.)
__device__ __forceinline__ uint2 convert8(const float (&p)[8]) {
  auto four = [&](int i) {   // the first pair's registers take the other half of the word: any value will do
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(p[i], p[i + 1], __builtin_bit_cast(int, p[i]), false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(p[i + 2], p[i + 3], w, true);
  };
  return make_uint2(four(0), four(4));
}
__device__ __forceinline__ uint2 pack8(const float (&v)[8], Inverse8 by) {
  float p[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) p[e] = fmaf(v[e], by.hi, v[e] * by.lo);
  return convert8(p);
}
__device__ __forceinline__ uint2 pack8(const float (&v)[8], float m) { return pack8(v, inverse8(m)); }
// The same of values with roundings of their own: by 448 / m in fp32, which adds half a step or less to them.
__device__ __forceinline__ uint2 pack8_once(const float (&v)[8], float m) {
  const Inverse8 by = inverse8(m);
  const float one = by.hi + by.lo;
  float p[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) p[e] = v[e] * one;
  return convert8(p);
}
// The same of values v + rest.
__device__ __forceinline__ uint2 pack8(const float (&v)[8], const float (&rest)[8], float m) {
  const Inverse8 by = inverse8(m);
  float p[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) p[e] = fmaf(v[e], by.hi, fmaf(rest[e], by.hi, v[e] * by.lo));
  return convert8(p);
}

}  // namespace ssd
