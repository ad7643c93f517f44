// selscan_device.hpp -- lane layout and cross-lane sums of the selective-scan
// kernels.
//
// A wave holds a tile of channels x states: RN neighbouring lanes share the
// states, padded with zero B and C to NP of them, and the 64 / RN lane groups hold
// consecutive channels, two per lane.  The forward kernels give a lane up to 8 states
// (RN = 2, 4 or 8), which keeps the sum over states (y) short; the backward kernel
// 4 (RN = NP / 4), because it sums over channels (dB, dC) as well and holds the
// states of 8 tokens.  What belongs to a channel alone (step size, gate) is prepared
// once per channel, by one lane of its group, and read by the others as a DPP
// broadcast.
#pragma once
#include "layer_device.hpp"

namespace ssd {

template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
  return __builtin_bit_cast(float,
                            __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
// Lane J of each group of four lanes, as a register of its own: folded into the
// four products that use it, the DPP operand would halve the rate of each of them.
template <int J> __device__ __forceinline__ float quad_bcast(float v) {
  float r = dpp_move<J * 0x55>(v);
  __asm__("" : "+v"(r));
  return r;
}

// Lane J (0 or 1) of each pair of lanes.
template <int J> __device__ __forceinline__ float pair_bcast(float v) {
  float r = dpp_move<J ? 0xF5 : 0xA0>(v);   // quad_perm [1,1,3,3] or [0,0,2,2]
  __asm__("" : "+v"(r));
  return r;
}

// A few rows of a [token][channel] operand through a buffer resource: a lane's
// byte offsets from the first row stay in registers, moving on by some rows costs
// scalar work only, and the resource ends after the last valid row, so that loads
// past it give zero and stores past it are dropped, as at kOutside for lanes
// without a channel.  With no valid row it is empty.
typedef __amdgpu_buffer_rsrc_t Rows;
constexpr unsigned kOutside = 0x80000000u;   // eight rows end before it, and it plus them below 2^32
__device__ __forceinline__ unsigned fresh(unsigned v) {
  __asm__ volatile("" : "+v"(v));   // sums with it are formed where they are used, not kept across a loop
  return v;
}
template <typename T> __device__ __forceinline__ Rows rows_bytes(const T* first, unsigned bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(first), (short)0, (int)bytes, 0x00020000);
}
template <typename T>
__device__ __forceinline__ Rows rows_at(const T* first, int valid, int64_t stride, int64_t width) {
  const unsigned bytes =
      valid > 0 ? (unsigned)(valid - 1) * (unsigned)(stride * sizeof(T)) + (unsigned)(width * sizeof(T)) : 0u;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(first), (short)0, (int)bytes, 0x00020000);
}
template <typename T> __device__ __forceinline__ T row_load(Rows r, unsigned bytes) {
  if constexpr (sizeof(T) == 2)
    return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(r, (int)bytes, 0, 0));
  else
    return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(r, (int)bytes, 0, 0));
}
__device__ __forceinline__ void row_load4(Rows r, unsigned bytes, float* v) {
  const floatx4 w = __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(r, (int)bytes, 0, 0));
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = w[e];
}
__device__ __forceinline__ void row_store4(Rows r, unsigned bytes, const float* v) {
  typedef unsigned uintx4 __attribute__((ext_vector_type(4)));
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(uintx4, floatx4{v[0], v[1], v[2], v[3]}), r,
                                         (int)bytes, 0, 0);
}
template <typename T> __device__ __forceinline__ void row_store(Rows r, unsigned bytes, T v) {
  if constexpr (sizeof(T) == 2)
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, v), r, (int)bytes, 0, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, v), r, (int)bytes, 0, 0);
}

// Two values summed over pairs of lanes: even lanes get v0's sums, odd lanes v1's.
__device__ __forceinline__ float pair_fold(float v0, float v1, int lane) {
  const bool b0 = lane & 1;
  return (b0 ? v1 : v0) + dpp_move<0xB1>(b0 ? v0 : v1);   // lane ^ 1
}
// The rest of a sum over RN lanes, after pair_fold.
template <int RN> __device__ __forceinline__ float pairs_sum(float v) {
  if constexpr (RN >= 4) v += dpp_move<0x4E>(v);          // lane ^ 2
  if constexpr (RN >= 8) v += __shfl_xor(v, 4, kWave);
  return v;
}

// Four values summed over the four lanes of a quad: lane q gets the sum of v[q].
__device__ __forceinline__ float quad_fold(const float (&v)[4], int lane) {
  const bool b0 = lane & 1, b1 = lane & 2;
  const float w0 = (b0 ? v[1] : v[0]) + dpp_move<0xB1>(b0 ? v[0] : v[1]);   // lane ^ 1
  const float w1 = (b0 ? v[3] : v[2]) + dpp_move<0xB1>(b0 ? v[2] : v[3]);
  return (b1 ? w1 : w0) + dpp_move<0x4E>(b1 ? w0 : w1);                     // lane ^ 2
}
// The rest of a sum over RN lanes, after quad_fold.
template <int RN> __device__ __forceinline__ float quads_sum(float v) {
#pragma unroll
  for (int off = 4; off < RN; off *= 2) v += __shfl_xor(v, off, kWave);
  return v;
}

// v0 and v1 each summed over the lane pairs 32 apart: the lower half of the
// wave gets v0's sums, the upper half v1's.
__device__ __forceinline__ float halves_fold(float v0, float v1) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, v0),
                                                  __builtin_bit_cast(unsigned, v1), false, false);
  const unsigned lo = r[0], hi = r[1];
  return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
}
// The same between neighbouring rows of 16: even rows get v0's sums, odd rows v1's.
__device__ __forceinline__ float rows_fold(float v0, float v1) {
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, v0),
                                                  __builtin_bit_cast(unsigned, v1), false, false);
  const unsigned lo = r[0], hi = r[1];
  return __builtin_bit_cast(float, lo) + __builtin_bit_cast(float, hi);
}

// The step sizes of one channel at M tokens: bias, softplus and clamp as
// dt_prepare, and with SLOPE the derivative by the raw value: the logistic of it
// where softplus is on, zero where the clamp holds (its ends pass the
// gradient).  The uniform branch is taken once for all M, whose independent
// chains of exp2, log and reciprocal then overlap.
//
// softplus(v) = max(v, 0) + log1p(w) with w = e^-|v| <= 1.  For u = 1 + w as
// rounded, c = w - (u - 1) is exact and log1p(w) = log(u) + log(1 + c / u); c is at
// most half a step of u, so c for the second term is off by less than 2^-24
// (u - 1) < 1.5 2^-24 log(u).  The logistic is 1 / u or w / u.
struct DtLane {
  float bias, lo, hi;
  int softplus;
};
__device__ __forceinline__ DtLane dt_lane(const DtXform& f, int64_t c) {
  return {f.bias ? f.bias[c] : 0.0f, f.lo, f.hi, f.softplus};
}
template <int M, bool SLOPE>
__device__ __forceinline__ void dt_values(const DtLane& f, float (&v)[M], float (&slope)[SLOPE ? M : 1]) {
#pragma unroll
  for (int u = 0; u < M; ++u) v[u] += f.bias;
  if (f.softplus) {
#pragma unroll
    for (int u = 0; u < M; ++u) {
      const float w = fast_exp2(-fabsf(v[u]) * kLog2e);
      const float s = 1.0f + w;
      if constexpr (SLOPE) slope[u] = (v[u] >= 0.0f ? 1.0f : w) * __builtin_amdgcn_rcpf(s);
      const float c = w - (s - 1.0f);
      v[u] = fmaxf(v[u], 0.0f) + fmaf(__builtin_amdgcn_logf(s), 0.6931471805599453f, c);
    }
  } else if constexpr (SLOPE) {
#pragma unroll
    for (int u = 0; u < M; ++u) slope[u] = 1.0f;
  }
#pragma unroll
  for (int u = 0; u < M; ++u) {
    if constexpr (SLOPE)
      if (!(v[u] >= f.lo && v[u] <= f.hi)) slope[u] = 0.0f;
    v[u] = __builtin_amdgcn_fmed3f(v[u], f.lo, f.hi);
  }
}

// Workspace rows of the chunked passes: [batch][chunks][channels][NP] fp32
// states and [batch][chunks][channels] step-size sums.
constexpr int kSub = 8;     // tokens whose states the backward pass holds in registers
struct ScanShape {
  int64_t L, D, N, G, Dg;   // Dg = channels per group
  int64_t K, T;             // chunks and tokens per chunk
  int64_t tiles;            // workgroups per group of channels
};

// Padded states, and what the two source files of the scan share on
// the host: chained start states and end gradients of every chunk, checkpoints, sizes.
inline int selscan_np(int64_t N) { return N <= 16 ? 16 : N <= 32 ? 32 : 64; }
// The forward pass alone pads less: 2, 4 or 8 lanes of 4, 6 or 8 states.
inline int selscan_fwd_np(int64_t N) {
  return N <= 8 ? 8 : N <= 16 ? 16 : N <= 24 ? 24 : N <= 32 ? 32 : N <= 48 ? 48 : 64;
}
struct ScanArgs;
hipError_t launch_selscan_both(const ScanArgs& a, const ScanShape& s, float* H, float* R,
                               float* sumdt, float* ckpt, float* sumsub, hipStream_t stream);
size_t selscan_state_bytes(int64_t batch, const ScanShape& s, int np);
size_t selscan_sum_bytes(int64_t batch, const ScanShape& s);

}  // namespace ssd
