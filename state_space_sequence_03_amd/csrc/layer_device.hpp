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

// V consecutive io elements <-> fp32, p aligned to all of them.
template <typename T, int V> struct RawV { typedef T type; };
template <> struct RawV<bf16, 8> { typedef bf16x8 type; };
template <> struct RawV<bf16, 4> { typedef bf16x4 type; };
template <> struct RawV<float, 4> { typedef floatx4 type; };
typedef float floatx2 __attribute__((ext_vector_type(2)));
template <> struct RawV<float, 2> { typedef floatx2 type; };
template <int V> __device__ __forceinline__ void load_v(const bf16* p, float* v) {
  const typename RawV<bf16, V>::type w = *reinterpret_cast<const typename RawV<bf16, V>::type*>(p);
  if constexpr (V == 1) {
    v[0] = static_cast<float>(w);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = static_cast<float>(w[e]);
  }
}
template <int V> __device__ __forceinline__ void load_v(const float* p, float* v) {
  const typename RawV<float, V>::type w = *reinterpret_cast<const typename RawV<float, V>::type*>(p);
  if constexpr (V == 1) {
    v[0] = w;
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = w[e];
  }
}
template <int V> __device__ __forceinline__ void store_v(bf16* p, const float* v) {
  typename RawV<bf16, V>::type w;
  if constexpr (V == 1) {
    w = static_cast<bf16>(v[0]);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] = static_cast<bf16>(v[e]);
  }
  *reinterpret_cast<typename RawV<bf16, V>::type*>(p) = w;
}
template <int V> __device__ __forceinline__ void store_v(float* p, const float* v) {
  typename RawV<float, V>::type w;
  if constexpr (V == 1) {
    w = v[0];
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) w[e] = v[e];
  }
  *reinterpret_cast<typename RawV<float, V>::type*>(p) = w;
}
// The same held unconverted, so that rows loaded ahead cost the registers of
// their io type only.
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

// Sums over the rows of a [n][ld] array of part sums, one column per 8 threads of
// a 256-thread workgroup (32 columns of 128 bytes, every eighth row each, four
// loads in flight), in 64 bits and in a fixed order.  The first 32 threads get the
// sums; `p` points to the thread's column, or is null past the last one.
__device__ __forceinline__ float column_sum(const float* p, int64_t n, int64_t ld) {
  __shared__ double sums[8][32];
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  if (p) {
    int64_t r = threadIdx.x / 32;
    for (; r + 24 < n; r += 32) {
      float v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = p[(r + 8 * u) * ld];
#pragma unroll
      for (int u = 0; u < 4; ++u) s[u] += (double)v[u];
    }
    for (; r < n; r += 8) s[0] += (double)p[r * ld];
  }
  sums[threadIdx.x / 32][threadIdx.x % 32] = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  double v = 0.0;
  if (threadIdx.x < 32)
    for (int q = 0; q < 8; ++q) v += sums[q][threadIdx.x];
  return (float)v;
}

// Sums of K values over the TG threads of a group, in every one of them: shuffles
// inside a wave (TG a power of two up to a wave, or whole waves), then the waves'
// sums through LDS.
template <int K>
__device__ __forceinline__ void group_sum(float (&v)[K], int tg, float* lds) {
  const int in_wave = tg < kWave ? tg : kWave;
  for (int off = in_wave / 2; off >= 1; off >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor(v[k], off, kWave);
  if (tg > kWave) {
    const int waves = tg / kWave, wave = threadIdx.x / kWave;
    __syncthreads();   // the last row's sums have been read
    if (threadIdx.x % kWave == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) lds[wave * K + k] = v[k];
    __syncthreads();
    const int first = wave / waves * waves;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.0f;
    for (int q = 0; q < waves; ++q)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += lds[(first + q) * K + k];
  }
}

}  // namespace ssd
