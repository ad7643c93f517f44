// selscan_device.hpp -- lane layout and cross-lane sums of the selective-scan
// kernels.
//
// A wave holds a tile of channels x states: RN neighbouring lanes share the
// states, padded with zero B and C to NP of them, and the 64 / RN lane groups hold
// consecutive channels, two per lane.  The forward kernels give a lane 8 states
// (RN = NP / 8), which keeps the sum over states (y) short; the backward kernel
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

// An element of a row: the row's pointer is uniform (a pair of scalar registers),
// the lane's place in it a 32-bit byte offset, so that no lane adds 64-bit
// addresses.  The empty statement keeps the compiler from adding the offset first.
template <typename T> struct GlobalPtr {
  typedef __attribute__((address_space(1))) T* type;
};
__device__ __forceinline__ unsigned here_offset(unsigned bytes) {
  __asm__("" : "+v"(bytes));   // the same for the offset: its widening stays beside the accesses
  return bytes;
}
template <typename T> __device__ __forceinline__ T row_load(const T* row, unsigned bytes) {
  uint64_t base = reinterpret_cast<uint64_t>(row);
  __asm__("" : "+s"(base));
  typedef typename GlobalPtr<const T>::type Ptr;
  typedef typename GlobalPtr<const char>::type Bytes;
  return *reinterpret_cast<Ptr>(reinterpret_cast<Bytes>(base) + bytes);
}
template <typename T> __device__ __forceinline__ void row_store(T* row, unsigned bytes, T v) {
  uint64_t base = reinterpret_cast<uint64_t>(row);
  __asm__("" : "+s"(base));
  typedef typename GlobalPtr<T>::type Ptr;
  typedef typename GlobalPtr<char>::type Bytes;
  *reinterpret_cast<Ptr>(reinterpret_cast<Bytes>(base) + bytes) = v;
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
      if constexpr (SLOPE) slope[u] = sigmoid_f32(v[u]);
      v[u] = softplus_f32(v[u]);
    }
  } else if constexpr (SLOPE) {
#pragma unroll
    for (int u = 0; u < M; ++u) slope[u] = 1.0f;
  }
#pragma unroll
  for (int u = 0; u < M; ++u) {
    if constexpr (SLOPE)
      if (!(v[u] >= f.lo && v[u] <= f.hi)) slope[u] = 0.0f;
    v[u] = fminf(fmaxf(v[u], f.lo), f.hi);
  }
}

// Workspace rows of the chunked passes: [batch][chunks][channels][NP] fp32
// states and [batch][chunks][channels] step-size sums.
struct ScanShape {
  int64_t L, D, N, G, Dg;   // Dg = channels per group
  int64_t K, T;             // chunks and tokens per chunk
  int64_t tiles;            // workgroups per group of channels
};

// Padded states, and what the two source files of the scan share on
// the host: chained start states and end gradients of every chunk, workspace sizes.
inline int selscan_np(int64_t N) { return N <= 16 ? 16 : N <= 32 ? 32 : 64; }
struct ScanArgs;
hipError_t launch_selscan_both(const ScanArgs& a, const ScanShape& s, float* H, float* R,
                               float* sumdt, hipStream_t stream);
size_t selscan_state_bytes(int64_t batch, const ScanShape& s);
size_t selscan_sum_bytes(int64_t batch, const ScanShape& s);

}  // namespace ssd
